"""Oracle of the root-mean-square norm with a residual (test infrastructure
only): float64 torch operations, gradients by autograd.
    h = x + residual,  y = h / sqrt(mean(h^2) + eps) * gamma
"""
import torch


def forward(x, gamma, residual, eps):
    """x [N,C] -> (y [N,C], h [N,C], rstd [N]) in float64."""
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if gamma is None else y * gamma.double()), h, rstd


def grads(total, gamma, eps, dy, dtotal=None):
    """Gradients of <dy, y> + <dtotal, h> for h = total: (dx, dgamma) in float64."""
    h = total.double().detach().clone().requires_grad_(True)
    g = torch.ones(total.shape[1], dtype=torch.float64, device=total.device) if gamma is None else gamma.double().detach().clone()
    g.requires_grad_(True)
    y, _, _ = forward(h, g, None, eps)
    loss = (y * dy.double()).sum()
    if dtotal is not None:
        loss = loss + (h * dtotal.double()).sum()
    return torch.autograd.grad(loss, [h, g])


def e4m3_values():
    """The numbers that 8 bits of e4m3 stand for, by code 0 .. 255 (NaN at 127 and 255)."""
    out = []
    for code in range(256):
        sign, exponent, mantissa = (-1.0 if code & 128 else 1.0), (code >> 3) & 15, code & 7
        if exponent == 15 and mantissa == 7:
            out.append(float("nan"))
        else:
            out.append(sign * (mantissa / 8 * 2.0 ** -6 if exponent == 0 else (1 + mantissa / 8) * 2.0 ** (exponent - 7)))
    return torch.tensor(out, dtype=torch.float64)

"""Oracle of the group norm with an activation, channels last (test
infrastructure only): float64 torch operations, gradients by autograd.
    y = act((x - mean) / sqrt(var + eps) * gamma + beta)
with mean and biased variance over the L positions and C/G channels of a
sample's group.
"""
import torch


def forward(x, gamma, beta, G, eps, activation):
    """x [N,L,C] -> (y [N,L,C], mean [N,G], rstd [N,G]) in float64."""
    N, L, C = x.shape
    xg = x.double().reshape(N, L, G, C // G)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    z = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, L, C)
    if gamma is not None:
        z = z * gamma.double()
    if beta is not None:
        z = z + beta.double()
    if activation == "silu":
        z = z * torch.sigmoid(z)
    elif activation == "relu":
        z = torch.relu(z)
    return z, mean, rstd


def grads(x, gamma, beta, G, eps, activation, dy):
    """(dx, dgamma, dbeta) of <dy, y> in float64; zeros for a NULL gamma or beta's place are not made (None)."""
    xs = x.double().detach().clone().requires_grad_(True)
    g = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if gamma is None else gamma.double().detach().clone()
    b = torch.zeros_like(g) if beta is None else beta.double().detach().clone()
    g.requires_grad_(True)
    b.requires_grad_(True)
    y, _, _ = forward(xs, g, b, G, eps, activation)
    return torch.autograd.grad((y * dy.double()).sum(), [xs, g, b])

"""Oracle of the short causal convolution (test infrastructure only): float64
torch operations, gradients by autograd.
    y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j})
Inputs before the first token are the state's W - 1 rows (or 0); the state that
goes out is the last W - 1 rows of the state and the valid tokens.
"""
import torch


def forward(x, weight, bias, activation, state=None, lengths=None):
    """x [B,T,D] -> (y [B,T,D], state_final [B,W-1,D]) in float64; rows at and past the length give zeros."""
    B, T, D = x.shape
    W = weight.shape[1]
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths]
    out, last = [], []
    for b in range(B):
        first = torch.zeros(W - 1, D, dtype=torch.float64, device=x.device) if state is None else state[b].double()
        full = torch.cat([first, x[b, :n[b]].double()])
        p = torch.stack([sum(full[t + j] * weight[:, j].double() for j in range(W)) for t in range(n[b])]) if n[b] else full[:0]
        if bias is not None:
            p = p + bias.double()
        y = p * torch.sigmoid(p) if activation == "silu" else p
        out.append(torch.cat([y, torch.zeros(T - n[b], D, dtype=torch.float64, device=x.device)]))
        last.append(full[n[b]:])
    return torch.stack(out), torch.stack(last)


def grads(x, weight, bias, activation, dy, state=None, lengths=None, dstate=None):
    """Gradients of <dy, y> + <dstate, state_final>: (dx, dweight, dbias, dstate_init) in float64."""
    B, T, D = x.shape
    W = weight.shape[1]
    leaf = lambda v: v.double().detach().clone().requires_grad_(True)  # noqa: E731
    z = torch.zeros(1, dtype=torch.float64, device=x.device)
    args = [leaf(x), leaf(weight), leaf(z.expand(D) if bias is None else bias),
            leaf(z.expand(B, W - 1, D) if state is None else state)]
    y, last = forward(args[0], args[1], args[2], activation, args[3], lengths)
    keep = torch.ones(B, T, 1, dtype=torch.bool, device=x.device)
    if lengths is not None:
        keep = (torch.arange(T, device=x.device) < lengths.to(x.device).view(B, 1)).unsqueeze(-1)
    loss = (y * torch.where(keep, dy.double(), 0.0)).sum()
    if dstate is not None:
        loss = loss + (last * dstate.double()).sum()
    got = torch.autograd.grad(loss, args, allow_unused=True)
    return tuple(torch.zeros_like(a) if g is None else g for g, a in zip(got, args))

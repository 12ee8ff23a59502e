"""Oracle of the linear attention with a decay per head (test infrastructure only).

The definition token by token in float64 torch operations, on whatever device
the inputs are on; gradients by autograd through it.  Per sequence b and head
h, g = exp(log_decay[h]):
    S_t = g S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   t = 1 .. lengths[b]
Rows at and past a sequence's length give zeros and leave S as it is.
"""
import torch


def forward(q, k, v, log_decay, scale, S_init=None, lengths=None):
    """q, k, v [B,T,H,d]; returns (o [B,T,H,d], S_final [B,H,d,d]) in float64."""
    B, T, H, d = q.shape
    n = torch.full((B,), T, device=q.device) if lengths is None else lengths.to(q.device).clamp(0, T)
    valid = (torch.arange(T, device=q.device) < n[:, None])[:, :, None, None]
    q, k, v = (torch.where(valid, x.double(), 0.0) for x in (q, k, v))
    g = torch.exp(log_decay.double().clamp(max=0)).view(1, H, 1, 1)
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if S_init is None else S_init.double()
    out = []
    for t in range(T):
        new = g * S + k[:, t].unsqueeze(-1) * v[:, t].unsqueeze(-2)
        S = torch.where(valid[:, t].unsqueeze(-1), new, S)
        out.append(scale * (q[:, t].unsqueeze(-2) @ S).squeeze(-2))
    o = torch.stack(out, 1) if T else torch.zeros_like(q)
    return torch.where(valid, o, 0.0), S


def sizes(q, k, v, log_decay, scale, S_init=None, lengths=None):
    """The same sums over magnitudes: what an entry's rounding errors are relative to."""
    return forward(q.abs(), k.abs(), v.abs(), log_decay, abs(scale), None if S_init is None else S_init.abs(), lengths)


def grads(q, k, v, log_decay, scale, do, S_init=None, lengths=None, dS_final=None):
    """Gradients of <do, o> + <dS_final, S_final>: (dq, dk, dv, dS_init) in float64."""
    B, T, H, d = q.shape
    xs = [x.double().detach().clone().requires_grad_(True) for x in (q, k, v)]
    S0 = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if S_init is None else S_init.double()
    S0 = S0.detach().clone().requires_grad_(True)
    o, S = forward(*xs, log_decay, scale, S0, lengths)
    valid = torch.ones_like(o, dtype=torch.bool)
    if lengths is not None:
        n = lengths.to(q.device).clamp(0, T)
        valid = (torch.arange(T, device=q.device) < n[:, None])[:, :, None, None].expand_as(o)
    loss = (o * torch.where(valid, do.double(), 0.0)).sum()
    if dS_final is not None:
        loss = loss + (S * dS_final.double()).sum()
    got = torch.autograd.grad(loss, xs + [S0], allow_unused=True)
    return tuple(torch.zeros_like(x) if gx is None else gx for gx, x in zip(got, xs + [S0]))


def grad_sizes(q, k, v, log_decay, scale, do, S_init=None, lengths=None, dS_final=None):
    """grads() over magnitudes."""
    return grads(q.abs(), k.abs(), v.abs(), log_decay, abs(scale), do.abs(), None if S_init is None else S_init.abs(),
                 lengths, None if dS_final is None else dS_final.abs())

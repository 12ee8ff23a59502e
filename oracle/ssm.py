"""Oracle of the selective state space scan (test infrastructure only).

The definition token by token in float64 torch operations, on whatever device
the inputs are on; gradients by autograd through it.  With s = softplus(dt +
dt_bias) (or dt + dt_bias) and the group of a channel understood:
    h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,   y_t = (C_t . h_t + skip u_t) silu(z_t)
Rows at and past a sequence's length give zeros and leave h as it is.
"""
import torch


def _valid(u, lengths):
    B, T = u.shape[:2]
    n = torch.full((B,), T, device=u.device) if lengths is None else lengths.to(u.device).clamp(0, T)
    return (torch.arange(T, device=u.device) < n[:, None])[:, :, None]


def _step(raw, softplus):
    return torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw


def forward(u, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, softplus=True, h_init=None, lengths=None):
    """u, dt, z [B,T,D], A [D,N], Bt, Ct [B,T,G,N]; returns (y [B,T,D], h_final [B,D,N]) in float64."""
    B, T, D = u.shape
    G, N = Bt.shape[2:]
    valid = _valid(u, lengths)
    u, dt, z = (None if v is None else torch.where(valid, v.double(), 0.0) for v in (u, dt, z))
    Bt, Ct = (torch.where(valid[..., None], v.double(), 0.0).repeat_interleave(D // G, 2) for v in (Bt, Ct))
    s = torch.where(valid, _step(dt if dt_bias is None else dt + dt_bias.double(), softplus), 0.0)
    h = torch.zeros(B, D, N, dtype=torch.float64, device=u.device) if h_init is None else h_init.double()
    out = []
    for t in range(T):
        h = torch.exp(s[:, t, :, None] * A.double()) * h + (s[:, t] * u[:, t])[..., None] * Bt[:, t]
        out.append((Ct[:, t] * h).sum(-1))
    y = torch.stack(out, 1) if T else torch.zeros_like(u)
    if skip is not None:
        y = y + skip.double() * u
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    return torch.where(valid, y, 0.0), h


NAMES = ("u", "dt", "A", "Bt", "Ct", "skip", "z", "dt_bias", "h_init")


def grads(dy, args, softplus=True, lengths=None, dh_final=None):
    """Gradients of <dy, y> + <dh_final, h_final> by the arguments that are given: a dict of NAMES in float64."""
    leaves = {k: v.double().detach().clone().requires_grad_(True) for k, v in args.items() if v is not None}
    y, h = forward(**leaves, softplus=softplus, lengths=lengths)
    loss = (y * torch.where(_valid(dy, lengths), dy.double(), 0.0)).sum()
    if dh_final is not None:
        loss = loss + (h * dh_final.double()).sum()
    got = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g for (k, v), g in zip(leaves.items(), got)}


class Near:
    """A sum of terms as the sum of their magnitudes m and a bound w on its error, both sums over the terms; the unit
    of w is one rounding, 2^-24.  Products add relative errors, sums add errors; both round once."""

    def __init__(self, m, w=0.0):
        self.m, self.w = m, w + torch.zeros_like(m)

    def __mul__(self, o):
        return Near(self.m * o.m, self.m * o.w + self.w * o.m + self.m * o.m)

    def __add__(self, o):
        m = self.m + o.m
        return Near(m, self.w + o.w + m)

    def total(self, dims):
        m = self.m.sum(dims)
        n = 1
        for k in dims if isinstance(dims, tuple) else (dims,):
            n *= self.m.shape[k]
        return Near(m, self.w.sum(dims) + n * m)

    def __getitem__(self, i):
        return Near(self.m[i], self.w[i])


STEP = 32.0     # roundings of a step: see _steps
GATE = 40.0     # of silu(z) and its slope


def errors(dy, args, softplus=True, lengths=None, dh_final=None):
    """Bounds on the error of a computation in 32 bits, in units of 2^-24, entry by entry: (y, h_final, a dict of the
    gradients' as in grads; None for these where dy is None).  They hold for any order of the sums.

    A step's relative error: the exponential of an argument whose rounding is carried (2^-22, its approximation's
    bound, 4 units), a reciprocal (2), and about ten roundings of a series whose terms fall by 9: under 20 units; the
    sum dt + dt_bias rounds by |v| units at most, which softplus' slope turns into |v| units of the step at most.  A
    decay exp(s A): |s A| times the step's and the two products' errors, and 4 units of its own."""
    f = {k: v.double().abs() if v is not None and k not in ("dt", "A", "z", "dt_bias") else None if v is None else v.double()
         for k, v in args.items()}
    B, T, D = args["u"].shape
    G, N = args["Bt"].shape[2:]
    valid = _valid(args["u"], lengths)
    clean = lambda v: torch.where(valid.view(*valid.shape[:2], *[1] * (v.dim() - 2)), v, 0.0)  # noqa: E731
    raw = clean(f["dt"]) if f.get("dt_bias") is None else clean(f["dt"]) + f["dt_bias"]
    s = clean(_step(raw, softplus).abs())
    step = Near(s, (STEP + raw.abs()) * s if softplus else clean(raw.abs() + (f["dt"].abs() + (0 if f.get("dt_bias") is None else f["dt_bias"].abs()))))
    wide = lambda v: Near(clean(v).repeat_interleave(D // G, 2))  # noqa: E731
    u, Bt, Ct = Near(clean(f["u"])), wide(f["Bt"]), wide(f["Ct"])
    x = step * u
    rel = torch.where(s > 0, step.w / s, 0.0)
    sA = clean(_step(raw, softplus))[..., None] * f["A"]
    a = Near(torch.exp(sA), torch.exp(sA) * (4 + sA.abs() * (rel[..., None] + 3)))
    h = Near(torch.zeros(B, D, N, dtype=torch.float64, device=s.device) if f.get("h_init") is None else f["h_init"])
    hs, out = [h], []
    for t in range(T):
        h = a[:, t] * h + Near(x.m[:, t, :, None], x.w[:, t, :, None]) * Bt[:, t]
        hs.append(h)
        out.append((Ct[:, t] * h).total(-1))
    stack = lambda v: Near(torch.stack([o.m for o in v], 1), torch.stack([o.w for o in v], 1))  # noqa: E731
    y = stack(out) if T else Near(torch.zeros_like(s))
    if f.get("skip") is not None:
        y = y + Near(f["skip"].expand_as(s)) * u
    plain = y
    if f.get("z") is not None:
        z = clean(f["z"])
        e = torch.sigmoid(z)
        gate = Near((z * e).abs(), (z * e).abs() * (GATE + z.abs()))
        y = y * gate
    if dy is None:
        return y.w, h.w, None
    d = Near(clean(dy.double().abs()))
    up = d if f.get("z") is None else d * gate
    got = {}
    if f.get("z") is not None:
        slope = e * (1 + z.abs() * (1 - e))
        got["z"] = (d * plain * Near(slope, slope * (GATE + z.abs()))).w
    g = Near(torch.zeros(B, D, N, dtype=torch.float64, device=s.device) if dh_final is None else dh_final.double().abs())
    absA = Near(f["A"].abs().expand(B, D, N))
    parts = {k: [] for k in ("du", "ddt", "dA", "dB", "dC")}
    for t in range(T - 1, -1, -1):
        p = Near(up.m[:, t, :, None].expand(B, D, N), up.w[:, t, :, None].expand(B, D, N))
        here = g + p * Ct[:, t]
        g = a[:, t] * here
        q = g * hs[t]
        st = Near(step.m[:, t, :, None].expand(B, D, N), step.w[:, t, :, None].expand(B, D, N))
        through = (here * Bt[:, t]).total(-1)
        parts["dA"].append(q * st)
        parts["ddt"].append((q * absA).total(-1) + through * u[:, t])
        parts["du"].append(through * step[:, t])
        groups = lambda v: Near(v.m.unflatten(1, (G, D // G)), v.w.unflatten(1, (G, D // G))).total(2)  # noqa: E731
        parts["dB"].append(groups(here * Near(x.m[:, t, :, None].expand(B, D, N), x.w[:, t, :, None].expand(B, D, N))))
        parts["dC"].append(groups(p * hs[t + 1]))
    ordered = {k: stack(v[::-1]) for k, v in parts.items()} if T else None
    if T:
        got["A"] = ordered["dA"].total((0, 1)).w
        slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
        ddt = ordered["ddt"] * Near(clean(slope), clean(slope) * (GATE + raw.abs()))
        du = ordered["du"]
        if f.get("skip") is not None:
            du = du + Near(f["skip"].expand_as(s)) * up
            got["skip"] = (up * u).total((0, 1)).w
        got.update(u=du.w, dt=ddt.w, Bt=ordered["dB"].w, Ct=ordered["dC"].w)
        if f.get("dt_bias") is not None:
            got["dt_bias"] = ddt.total((0, 1)).w
    else:
        got.update({k: torch.zeros_like(f[k]) for k in ("A", "skip", "dt_bias", "u", "dt", "Bt", "Ct") if f.get(k) is not None})
    if f.get("h_init") is not None:
        got["h_init"] = g.w
    return y.w, h.w, got

"""A selective state space scan (prompt, single token, gradients), the short causal convolution in front of it
(the same three) and the root-mean-square norm with the residual's addition (outputs in the input's type or in
8 bits with scales, and gradients): the cases they are timed on, their plain forms in elementary torch
operations, and their values in 64 bits from the definitions.

Scan, per sequence b, channel c (of group c // (D / G)) and state n, s = softplus(dt + dt_bias):
    h_t[c,n] = exp(s_t[c] A[c,n]) h_{t-1}[c,n] + s_t[c] u_t[c] B_t[n]        (h_0 = h_init or 0)
    y_t[c]   = (sum_n C_t[n] h_t[c,n] + skip[c] u_t[c]) * silu(z_t[c])
Convolution over the last W tokens of a channel (inputs before the first token from a state, or 0):
    y_t[c] = silu(bias[c] + sum_j weight[c,j] x_{t-W+1+j}[c])
Norm of a row: with h = x + residual, y = h / sqrt(mean(h^2) + eps) * gamma; in 8 bits (e4m3) each block of
channels is divided by its scale, its largest magnitude over 448.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5
E4M3_MAX = 448.0
RANK = 32        # columns of a packed projection in front of B and C


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a training batch's or a prompt batch's forward; z, B and C are slices of packed projections
        dict(name="scan_mid_bf16", op="scan", B=64, T=1024, D=1024, N=16, G=1, dtype="bf16", gate=True, ragged=False,
             state=False, packed=True),
        # two long contexts, far fewer streams than the GPU holds, states carried in and out
        dict(name="scan_long_fp32", op="scan", B=2, T=8192, D=1024, N=16, G=1, dtype="fp32", gate=False, ragged=False,
             state=True, packed=False),
        # rollouts of uneven lengths, padded to one length, some empty, state carried in and out, two groups
        dict(name="scan_rl_ragged_bf16", op="scan", B=512, T=512, D=256, N=32, G=2, dtype="bf16", gate=True, ragged=True,
             state=True, packed=True),
        # one new token for a full serving batch: every state is read and written
        dict(name="scan_token_bf16", op="scan_token", B=512, D=1024, N=64, G=1, dtype="bf16", gate=True),
        # gradients of the training batch
        dict(name="scan_grad_mid_bf16", op="scan_grad", B=64, T=1024, D=1024, N=16, G=1, dtype="bf16", gate=True,
             ragged=False, state=False, packed=True),
        # gradients of a few-shot episode's short prompt: many short sequences
        dict(name="scan_grad_fewshot_fp32", op="scan_grad", B=128, T=26, D=256, N=16, G=1, dtype="fp32", gate=True,
             ragged=False, state=True, packed=False),
        # the convolution in front of the training batch's scan, on a slice of the packed projection
        dict(name="conv_mid_bf16", op="conv", B=64, T=1024, D=1024, W=4, dtype="bf16", ragged=False, state=False, packed=True),
        # one new token for a handful of sequences: latency
        dict(name="conv_token_few_fp32", op="conv_token", B=4, D=1024, W=4, dtype="fp32"),
        # gradients on the rollouts
        dict(name="conv_grad_rl_fp32", op="conv_grad", B=512, T=512, D=256, W=4, dtype="fp32", ragged=True, state=True,
             packed=False),
        # the norm in front of a product in 8 bits, the residual stream updated beside it
        dict(name="norm8_mid_bf16", op="norm8", N=65536, C=1024, block=128, dtype="bf16"),
        # the norm of a serving batch's single tokens
        dict(name="norm_token_fp16", op="norm", N=96, C=4096, dtype="fp16"),
        # gradients of the training batch's norms, the residual stream's own gradient added
        dict(name="norm_grad_mid_bf16", op="norm_grad", N=65536, C=512, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "scan_token", "conv", "conv_grad", "conv_token", "norm", "norm8",
                     "norm_grad"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    if op in ("scan", "scan_grad"):
        while True:
            G = rng.choice([1, 1, 2, 4])
            case = dict(op=op, B=_log_int(rng, 1, 512), T=_log_int(rng, 1, 8192), D=8 * G * _log_int(rng, 1, 2048 // (8 * G)),
                        N=rng.choice([16, 16, 32, 64]), G=G, dtype=dtype, gate=rng.random() < 0.6, ragged=rng.random() < 0.4,
                        state=rng.random() < 0.5, packed=rng.random() < 0.4)
            states = case["B"] * case["T"] * case["D"] * case["N"]
            if 1 << 16 <= states <= 1 << 29 and sum(_lengths(case)) > 0:
                return case
    if op == "scan_token":
        G = rng.choice([1, 1, 2, 4])
        return dict(op=op, B=_log_int(rng, 1, 512), D=8 * G * _log_int(rng, 1, 1024 // (8 * G)), N=rng.choice([16, 32, 64]), G=G,
                    dtype=dtype, gate=rng.random() < 0.6)
    if op in ("conv", "conv_grad"):
        while True:
            case = dict(op=op, B=_log_int(rng, 1, 512), T=_log_int(rng, 1, 8192), D=8 * _log_int(rng, 1, 512),
                        W=rng.choice([2, 3, 4]), dtype=dtype, ragged=rng.random() < 0.4, state=rng.random() < 0.5,
                        packed=rng.random() < 0.4)
            if 1 << 12 <= case["B"] * case["T"] * case["D"] <= 1 << 25 and sum(_lengths(case)) > 0:
                return case
    if op == "conv_token":
        return dict(op=op, B=_log_int(rng, 1, 512), D=8 * _log_int(rng, 1, 512), W=rng.choice([2, 3, 4]), dtype=dtype)
    while True:
        C = 128 * _log_int(rng, 1, 64) if op == "norm8" else 8 * _log_int(rng, 2, 1024)
        case = dict(op=op, N=_log_int(rng, 1, 200000), C=C, dtype=dtype)
        if op == "norm8":
            case["block"] = rng.choice([0, 128])
        if 1 << 10 <= case["N"] * C <= 1 << 26:
            return case


def _lengths(case):
    """Valid tokens of each sequence, in no order: spread evenly over 0 .. T (the whole T where not ragged)."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [(T * i) // max(1, B - 1) if B > 1 else (T + 1) // 2 for i in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case)
    op = case["op"]
    if op.startswith("norm"):
        N, C = case["N"], case["C"]
        x, residual = normal(N, C), normal(N, C) * (0.5 + 2 * torch.rand(C, generator=g, device=dev))
        s["gamma"] = 1 + 0.2 * normal(C)
        if op == "norm_grad":          # what the forward pass left behind: the sum in its type, the norm's factor
            s["total"] = (x + residual).to(dt)
            s["rstd"] = torch.rsqrt(s["total"].double().square().mean(1) + EPS).float()
            s["dy"], s["dtotal"] = normal(N, C, dtype=dt), normal(N, C, dtype=dt)
        else:
            s["x"], s["residual"] = x.to(dt), residual.to(dt)
        return s
    B, D = case["B"], case["D"]
    tokens = (B,) if op.endswith("token") else (B, case["T"])
    s["lengths"] = None
    if case.get("ragged"):
        n = torch.tensor(_lengths(case), device=dev, dtype=torch.int32)
        s["lengths"] = n[torch.randperm(B, generator=g, device=dev)].contiguous()
    state = case.get("state", True)
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = normal(*tokens, 2 * D, dtype=dt)[..., :D] if case.get("packed") else normal(*tokens, D, dtype=dt)
        s["weight"], s["bias"] = normal(D, W) * W ** -0.5, 0.2 * normal(D)
        s["state_in"] = normal(B, W - 1, D, dtype=dt) if state else None
        if op == "conv_grad":
            s["dy"] = normal(*tokens, D, dtype=dt)
            s["dstate"] = normal(B, W - 1, D, dtype=dt) if state else None
        return s
    N, G = case["N"], case["G"]
    u = 1.2 * normal(*tokens, D)
    s["u"] = (u * torch.sigmoid(u)).to(dt)                    # what a convolution with SiLU gives
    s["dt"] = normal(*tokens, D, dtype=dt) * 0.5
    start = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=g, device=dev, dtype=torch.float64))
    s["dt_bias"] = torch.log(torch.expm1(start)).float()      # softplus(dt_bias) between 0.001 and 0.1
    s["A"] = -torch.arange(1, N + 1, device=dev) * torch.exp(0.1 * normal(D, N))
    s["skip"] = 1 + 0.2 * normal(D)
    if case.get("packed"):
        s["z"] = normal(*tokens, 2 * D, dtype=dt)[..., D:] if case["gate"] else None
        p = normal(*tokens, RANK + 2 * G * N, dtype=dt)[..., RANK:]
        s["Bt"], s["Ct"] = p[..., :G * N].unflatten(-1, (G, N)), p[..., G * N:].unflatten(-1, (G, N))
    else:
        s["z"] = normal(*tokens, D, dtype=dt) if case["gate"] else None
        s["Bt"], s["Ct"] = normal(*tokens, G, N, dtype=dt), normal(*tokens, G, N, dtype=dt)
    s["h_in"] = normal(B, D, N) * 0.2 if state else None
    if op == "scan_grad":
        s["dy"] = normal(*tokens, D, dtype=dt)
        s["dh"] = normal(B, D, N) * 0.2 if state else None
    return s


# ------------------------------------------------------------------ plain forms
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _valid(s):
    """[B, T, 1]: whether a token is before its sequence's end."""
    B, T = s["B"], s["T"]
    t = torch.arange(T, device="cuda").view(1, T, 1)
    return t < (T if s["lengths"] is None else s["lengths"].view(B, 1, 1))


def _clean(valid, v):
    return torch.where(valid.view(*valid.shape[:2], *[1] * (v.dim() - 2)), v.float(), torch.zeros((), device=v.device))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by halves: pairs of steps are one step of half as many."""
    T = a.shape[1]
    if T == 1:
        return b
    m, rest = T // 2, (T - 1) // 2
    odd = _scan(a[:, 1::2] * a[:, 0:2 * m:2], a[:, 1::2] * b[:, 0:2 * m:2] + b[:, 1::2])
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :rest] + b[:, 2::2]
    return h


def _of_channels(v, D):
    """[B, T, G, N] -> [B, T, D, N] (a view): a group's values for each of its channels."""
    B, T, G, N = v.shape
    return v.unsqueeze(3).expand(B, T, G, D // G, N).reshape(B, T, D, N)


def _scan_parts(s):
    valid = _valid(s)
    u, Bt, Ct = _clean(valid, s["u"]), _clean(valid, s["Bt"]), _clean(valid, s["Ct"])
    raw = s["dt"].float() + s["dt_bias"]
    step = _clean(valid, _softplus(raw))          # 0 past the end: the state stays as it is
    a = torch.exp(step.unsqueeze(-1) * s["A"])
    b = (step * u).unsqueeze(-1) * _of_channels(Bt, s["D"])
    if s["h_in"] is not None:
        b[:, 0] += a[:, 0] * s["h_in"]
    return valid, u, Bt, Ct, raw, step, a, _scan(a, b)


def _plain_scan(s):
    valid, u, _, Ct, _, _, _, h = _scan_parts(s)
    y = (_of_channels(Ct, s["D"]) * h).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        z = _clean(valid, s["z"])
        y = y * (z * torch.sigmoid(z))
    return y.to(s["u"].dtype), h[:, -1].contiguous()


def _plain_scan_token(s):
    u, Bt, Ct = s["u"].float(), s["Bt"].float(), s["Ct"].float()
    B, D, N, G = s["B"], s["D"], s["N"], s["G"]
    of = lambda v: v.unsqueeze(2).expand(B, G, D // G, N).reshape(B, D, N)  # noqa: E731
    step = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(step.unsqueeze(-1) * s["A"]) * s["h_in"] + (step * u).unsqueeze(-1) * of(Bt)
    y = (of(Ct) * h).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["u"].dtype), h


def _plain_scan_grad(s):
    valid, u, Bt, Ct, raw, step, a, h = _scan_parts(s)
    B, T, D, N, G = s["B"], s["T"], s["D"], s["N"], s["G"]
    dy, dt = _clean(valid, s["dy"]), s["u"].dtype
    dz = None
    if s["z"] is not None:
        z = _clean(valid, s["z"])
        e = torch.sigmoid(z)
        y = (_of_channels(Ct, D) * h).sum(-1) + s["skip"] * u
        dz = (dy * y * e * (1 + z * (1 - e))).to(dt)
        dy = dy * (z * e)
    b = dy.unsqueeze(-1) * _of_channels(Ct, D)                       # dL/dh_t = C_t dy_t + a_{t+1} dL/dh_{t+1}
    if s["dh"] is not None:
        b[:, -1] += s["dh"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = torch.flip(_scan(torch.flip(after, (1,)), torch.flip(b, (1,))), (1,))
    del after, b
    before = torch.zeros_like(a[:, :1]) if s["h_in"] is None else s["h_in"].unsqueeze(1)
    q = g * a * torch.cat([before, h[:, :-1]], 1)                    # dL/d(s_t A)
    gx = (g * _of_channels(Bt, D)).sum(-1)
    du = gx * step + s["skip"] * dy
    draw = _clean(valid, ((q * s["A"]).sum(-1) + gx * u) * torch.sigmoid(raw))
    dA = (q * step.unsqueeze(-1)).sum((0, 1))
    groups = lambda v: v.view(B, T, G, D // G, N).sum(3).to(dt)  # noqa: E731
    dB, dC = groups(g * (step * u).unsqueeze(-1)), groups(dy.unsqueeze(-1) * h)
    return (du.to(dt), draw.to(dt), dA, dB, dC, (dy * u).sum((0, 1)), dz, draw.sum((0, 1)),
            None if s["h_in"] is None else a[:, 0] * g[:, 0])


def _conv_window(s):
    """fp32 inputs with the W - 1 before them, [B, T + W - 1, D] (zeros past the end)."""
    x = _clean(_valid(s), s["x"])
    first = torch.zeros(s["B"], s["W"] - 1, s["D"], device=x.device) if s["state_in"] is None else s["state_in"].float()
    return torch.cat([first, x], 1)


def _conv_taps(full, weight, T):
    """sum_j weight[c,j] full[t+j,c]"""
    return (full.unfold(1, weight.shape[1], 1)[:, :T] * weight).sum(-1)


def _last_inputs(s):
    """Rows lengths .. lengths + W - 2 of the inputs with those before them: the state at each sequence's end."""
    B, T, W, D = s["B"], s["T"], s["W"], s["D"]
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    return (n.view(B, 1) + torch.arange(W - 1, device="cuda")).unsqueeze(-1).expand(B, W - 1, D)


def _plain_conv(s):
    full = _conv_window(s)
    y = _conv_taps(full, s["weight"], s["T"]) + s["bias"]
    y = _clean(_valid(s), y * torch.sigmoid(y))
    dt = s["x"].dtype
    return y.to(dt), torch.gather(full, 1, _last_inputs(s)).to(dt)


def _plain_conv_token(s):
    full = torch.cat([s["state_in"].float(), s["x"].float().unsqueeze(1)], 1)
    y = (full.transpose(1, 2) * s["weight"]).sum(-1) + s["bias"]
    dt = s["x"].dtype
    return (y * torch.sigmoid(y)).to(dt), full[:, 1:].to(dt)


def _plain_conv_grad(s):
    full, W, T, dt = _conv_window(s), s["W"], s["T"], s["x"].dtype
    y = _conv_taps(full, s["weight"], T) + s["bias"]
    e = torch.sigmoid(y)
    d = _clean(_valid(s), s["dy"]) * e * (1 + y * (1 - e))
    dw = torch.einsum("btdw,btd->dw", full.unfold(1, W, 1)[:, :T], d)
    pad = torch.zeros(s["B"], W - 1, s["D"], device=d.device)
    dfull = _conv_taps(torch.cat([pad, d, pad], 1), torch.flip(s["weight"], (1,)), T + W - 1)
    if s["dstate"] is not None:
        dfull = dfull.scatter_add(1, _last_inputs(s), s["dstate"].float())
    dx = _clean(_valid(s), dfull[:, W - 1:])
    return dx.to(dt), dw, d.sum((0, 1)), None if s["state_in"] is None else dfull[:, :W - 1].to(dt)


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y, dt = h * rstd.unsqueeze(1) * s["gamma"], s["x"].dtype
    if s["op"] == "norm":
        return y.to(dt), h.to(dt), rstd
    N, C = y.shape
    blocks = y.view(N, -1, s["block"] or C)
    scale = blocks.abs().amax(-1) / E4M3_MAX
    q = blocks / torch.where(scale > 0, scale, torch.ones((), device=y.device)).unsqueeze(-1)
    return q.view(N, C).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale, h.to(dt), rstd


def _plain_norm_grad(s):
    rstd, dy = s["rstd"].unsqueeze(1), s["dy"].float()
    xh = s["total"].float() * rstd
    d = dy * s["gamma"]
    dx = rstd * (d - xh * (d * xh).mean(1, keepdim=True)) + s["dtotal"].float()
    return dx.to(s["total"].dtype), (dy * xh).sum(0)


def run(state):
    s = state
    op = s["op"]
    if own:
        from self_referential_weight_gb300 import binding
        if op == "scan":
            return binding.srwm_ssm_forward(s["u"], s["dt"], s["A"], s["Bt"], s["Ct"], skip=s["skip"], z=s["z"],
                                            dt_bias=s["dt_bias"], h_init=s["h_in"], lengths=s["lengths"])
        if op == "scan_token":
            return binding.srwm_ssm_step(s["u"], s["dt"], s["A"], s["Bt"], s["Ct"], s["h_in"], skip=s["skip"], z_t=s["z"],
                                         dt_bias=s["dt_bias"])
        if op == "scan_grad":
            return binding.srwm_ssm_backward(s["u"], s["dt"], s["A"], s["Bt"], s["Ct"], s["dy"], skip=s["skip"], z=s["z"],
                                             dt_bias=s["dt_bias"], h_init=s["h_in"], lengths=s["lengths"], dh_final=s["dh"])
        if op == "conv":
            return binding.srwm_conv_forward(s["x"], s["weight"], s["bias"], state_init=s["state_in"], lengths=s["lengths"],
                                             activation="silu")
        if op == "conv_token":
            return binding.srwm_conv_step(s["x"], s["weight"], s["bias"], s["state_in"], activation="silu")
        if op == "conv_grad":
            return binding.srwm_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], state_init=s["state_in"],
                                              lengths=s["lengths"], dstate_final=s["dstate"], activation="silu")
        if op == "norm":
            y, _, total, rstd = binding.srwm_rmsnorm_forward(s["x"], s["gamma"], residual=s["residual"], eps=EPS)
            return y, total, rstd
        if op == "norm8":
            return binding.srwm_rmsnorm_forward(s["x"], s["gamma"], residual=s["residual"], eps=EPS, out="e4m3",
                                                block=s["block"])
        return binding.srwm_rmsnorm_backward(s["total"], s["gamma"], s["rstd"], s["dy"], dtotal=s["dtotal"])
    plain = dict(scan=_plain_scan, scan_token=_plain_scan_token, scan_grad=_plain_scan_grad, conv=_plain_conv,
                 conv_token=_plain_conv_token, conv_grad=_plain_conv_grad, norm=_plain_norm, norm8=_plain_norm,
                 norm_grad=_plain_norm_grad)
    return plain[op](s)


# ------------------------------------------------------------------ floors
def work(case):
    e, op = DTYPES[case["dtype"]].itemsize, case["op"]
    if op.startswith("norm"):
        n, N, C = case["N"] * case["C"], case["N"], case["C"]
        if op == "norm":
            return {"bytes": 4 * n * e + 4 * N + 4 * C, "flops": 5 * n}
        if op == "norm8":
            return {"bytes": 3 * n * e + n + 4 * N + 4 * C + 4 * N * (C // case["block"] if case["block"] else 1), "flops": 8 * n}
        return {"bytes": 4 * n * e + 4 * N + 8 * C, "flops": 10 * n}
    B, D, T = case["B"], case["D"], case.get("T", 1)
    full = B * T
    rows = full if op.endswith("token") else sum(_lengths(case))
    if op.startswith("conv"):
        W = case["W"]
        state, taps = B * (W - 1) * D * e, D * (W + 1) * 4
        if op == "conv":
            return {"bytes": (rows + full) * D * e + state * (2 if case["state"] else 1) + taps, "flops": rows * D * (2 * W + 5)}
        if op == "conv_token":
            return {"bytes": 2 * B * D * e + 2 * state + taps, "flops": B * D * (2 * W + 5)}
        return {"bytes": (2 * rows + full) * D * e + state * (3 if case["state"] else 0) + 2 * taps,
                "flops": rows * D * (6 * W + 10)}
    N, G = case["N"], case["G"]
    states, gate, bc = B * D * N * 4, int(case["gate"]), 2 * G * N
    params = D * (N + 2) * 4
    if op == "scan":
        return {"bytes": (rows * ((2 + gate) * D + bc) + full * D) * e + states * (2 if case["state"] else 1) + params,
                "flops": rows * D * (7 * N + 20)}
    if op == "scan_token":
        return {"bytes": B * ((3 + gate) * D + bc) * e + 2 * states + params, "flops": B * D * (7 * N + 20)}
    return {"bytes": (rows * ((3 + gate) * D + bc) + full * ((2 + gate) * D + bc)) * e + states * (3 if case["state"] else 0) + 2 * params,
            "flops": rows * D * (25 * N + 50)}


# ------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    f = lambda v: v.double()  # noqa: E731
    op = case["op"]
    if op.startswith("norm"):
        gamma = f(s["gamma"])
        if op == "norm_grad":          # by the Jacobian of h -> h * rstd at the rstd that is given
            h, r, up = f(s["total"]), f(s["rstd"])[:, None], f(s["dy"])
            w = torch.einsum("nc,nc->n", up * gamma, h)[:, None] * r ** 3 / case["C"]
            return up * gamma * r - w * h + f(s["dtotal"]), torch.einsum("nc,nc->c", up, h * r)
        h = f(s["x"]) + f(s["residual"])
        r = (h.square().mean(-1) + EPS).rsqrt()
        y = torch.einsum("nc,n,c->nc", h, r, gamma)
        if op == "norm":
            return y, h, r
        width = case["block"] or case["C"]
        top = torch.linalg.vector_norm(y.unflatten(1, (-1, width)), ord=math.inf, dim=-1) / E4M3_MAX
        return y / top.repeat_interleave(width, 1), top, h, r
    B, D = case["B"], case["D"]
    dev = torch.device("cuda")
    if op.startswith("conv"):
        W = case["W"]
        T = case.get("T", 1)
        x = f(s["x"]).reshape(B, T, D)
        n = torch.full((B,), T, device=dev) if s["lengths"] is None else s["lengths"].long()
        keep = (torch.arange(T, device=dev) < n[:, None])[:, :, None]
        x = torch.where(keep, x, 0.0).requires_grad_(True)
        first = torch.zeros(B, W - 1, D, device=dev, dtype=torch.float64) if s["state_in"] is None else f(s["state_in"])
        first = first.detach().requires_grad_(True)
        weight, bias = f(s["weight"]).requires_grad_(True), f(s["bias"]).requires_grad_(True)
        full = torch.cat([first, x], 1)
        pre = torch.nn.functional.conv1d(full.transpose(1, 2), weight.unsqueeze(1), bias, groups=D).transpose(1, 2)
        y = torch.where(keep, torch.nn.functional.silu(pre), 0.0)
        last = torch.stack([full[b, m:m + W - 1] for b, m in enumerate(n.tolist())])
        if op == "conv":
            return y.detach(), last.detach()
        if op == "conv_token":
            return y.detach().view(B, D), last.detach()
        loss = (y * f(s["dy"])).sum()
        if s["dstate"] is not None:
            loss = loss + (last * f(s["dstate"])).sum()
        dx, dw, db, d0 = torch.autograd.grad(loss, [x, weight, bias, first])
        return torch.where(keep, dx, 0.0), dw, db, None if s["state_in"] is None else d0
    N, G, T = case["N"], case["G"], case.get("T", 1)
    if B * T * D * N > 1 << 31:        # every state in 64 bits, and its gradient
        return None
    tok = (lambda v: v.unsqueeze(1)) if op == "scan_token" else (lambda v: v)
    u, raw, Bt, Ct, A, skip = (f(v) for v in (tok(s["u"]), tok(s["dt"]), tok(s["Bt"]), tok(s["Ct"]), s["A"], s["skip"]))
    z = None if s["z"] is None else f(tok(s["z"]))
    raw = raw + f(s["dt_bias"])
    step = torch.nn.functional.softplus(raw, threshold=100)
    n = torch.full((B,), T, device=dev) if s["lengths"] is None else s["lengths"]
    h0 = torch.zeros(B, D, N, device=dev, dtype=torch.float64) if s["h_in"] is None else f(s["h_in"])
    wide = lambda v, t: v[:, t].repeat_interleave(D // G, 1)  # noqa: E731   [B, G, N] -> [B, D, N]
    grad = op == "scan_grad"
    h, y, kept = h0, torch.zeros(B, T, D, device=dev, dtype=torch.float64), []
    for t in range(T):
        live = (t < n)[:, None]
        if grad:
            kept.append(h)
        new = torch.exp(step[:, t, :, None] * A) * h + (step[:, t] * u[:, t])[..., None] * wide(Bt, t)
        h = torch.where(live[..., None], new, h)
        y[:, t] = torch.where(live, torch.einsum("bdn,bdn->bd", wide(Ct, t), h) + skip * u[:, t], 0.0)
    gate = 1.0 if z is None else torch.nn.functional.silu(z)
    if op == "scan":
        return torch.where((torch.arange(T, device=dev) < n[:, None])[..., None], y * gate, 0.0), h
    if op == "scan_token":
        return (y * gate)[:, 0], h
    dy, g = f(s["dy"]), torch.zeros_like(h0) if s["dh"] is None else f(s["dh"])
    du, draw = torch.zeros_like(y), torch.zeros_like(y)
    dz = None if z is None else torch.zeros_like(y)
    dB, dC, dA = torch.zeros_like(Bt), torch.zeros_like(Ct), torch.zeros_like(A)
    dskip, dbias = torch.zeros_like(skip), torch.zeros_like(skip)
    for t in range(T - 1, -1, -1):
        live = (t < n)[:, None]
        up = torch.where(live, dy[:, t], 0.0)
        if z is not None:
            e = 1 / (1 + torch.exp(-z[:, t]))
            dz[:, t] = up * y[:, t] * (e + z[:, t] * e * (1 - e))
            up = up * z[:, t] * e
        d, x, before = torch.where(live, step[:, t], 0.0), torch.where(live, u[:, t], 0.0), kept.pop()
        a = torch.exp(d[..., None] * A)
        now = a * before + (d * x)[..., None] * wide(Bt, t)
        here = g + up[..., None] * wide(Ct, t)
        through = torch.einsum("bdn,bdn->bd", here, wide(Bt, t))
        da = here * a * before
        dd = torch.where(live, (torch.einsum("bdn,dn->bd", da, A) + through * x) * torch.sigmoid(raw[:, t]), 0.0)
        du[:, t], draw[:, t] = torch.where(live, through * d, 0.0) + skip * up, dd
        dA += torch.einsum("bdn,bd->dn", da, d)
        dB[:, t] = (here * (d * x)[..., None]).unflatten(1, (G, D // G)).sum(2)
        dC[:, t] = (now * up[..., None]).unflatten(1, (G, D // G)).sum(2)
        dskip, dbias = dskip + (up * x).sum(0), dbias + dd.sum(0)
        g = torch.where(live[..., None], a * here, g)
    return du, draw, dA, dB, dC, dskip, dz, dbias, None if s["h_in"] is None else g

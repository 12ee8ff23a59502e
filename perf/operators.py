"""Linear attention with a per-head decay (prompt, single token, gradients) and group norm with an
activation (channels last, and its gradients): the cases they are timed on, their plain forms in
elementary torch operations, and their values in 64 bits from the definitions.

Linear attention, per sequence b and head h, decay g = exp(log_decay[h]):
    S_t = g S_{t-1} + k_t v_t^T        (S_0 = S_init or 0)
    o_t = scale * S_t^T q_t
Group norm of x [N, L, C] over G groups of C/G neighbouring channels and all L positions:
    y = act((x - mean) * rstd * gamma + beta),  rstd = 1 / sqrt(var + eps)
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5
CHUNK = 64   # tokens per block of the plain form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few-shot episode's short prompt: many short sequences, latency and launch bound
        dict(name="prompt_fewshot_fp32", op="prompt", B=128, T=26, H=16, d=16, dtype="fp32", decay="slow",
             ragged=False, state=False, packed=False),
        # a training batch's or a prompt batch's forward, q, k, v as views of one packed projection
        dict(name="prompt_mid_bf16", op="prompt", B=64, T=1024, H=8, d=64, dtype="bf16", decay="slow",
             ragged=False, state=False, packed=True),
        # long contexts, fewer streams than the GPU holds: the long axis is split
        dict(name="prompt_long_fp32", op="prompt", B=16, T=8192, H=8, d=64, dtype="fp32", decay="slow",
             ragged=False, state=True, packed=False),
        # rollouts of uneven lengths, padded to one length, some empty, state carried in and out
        dict(name="prompt_rl_ragged_bf16", op="prompt", B=512, T=512, H=4, d=32, dtype="bf16", decay="slopes",
             ragged=True, state=True, packed=False),
        # one new token for a handful of sequences: latency
        dict(name="token_few_bf16", op="token", B=4, H=8, d=64, dtype="bf16", decay="slow"),
        # one new token for a full serving batch: every state is read and written
        dict(name="token_many_bf16", op="token", B=512, H=16, d=64, dtype="bf16", decay="slow"),
        # gradients of the few-shot episode
        dict(name="grad_fewshot_fp32", op="grad", B=128, T=26, H=16, d=16, dtype="fp32", decay="slow",
             ragged=False, state=True, packed=False),
        # gradients of the training batch
        dict(name="grad_mid_bf16", op="grad", B=64, T=1024, H=8, d=64, dtype="bf16", decay="slow",
             ragged=False, state=False, packed=True),
        # the norm of each head's output, a group per head and token (L = 1)
        dict(name="norm_heads_bf16", op="norm", N=65536, L=1, C=512, G=8, dtype="bf16", act="silu"),
        # its gradients on the rollouts' shape
        dict(name="norm_grad_heads_fp32", op="norm_grad", N=262144, L=1, C=128, G=4, dtype="fp32", act="silu"),
        # feature maps of an image encoder in front of the model
        dict(name="norm_maps_fp32", op="norm", N=208, L=1764, C=64, G=8, dtype="fp32", act="relu"),
        # gradients on the next stage's smaller maps
        dict(name="norm_grad_maps_bf16", op="norm_grad", N=101, L=441, C=64, G=16, dtype="bf16", act="silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "grad", "token", "norm", "norm_grad"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    if op in ("prompt", "grad"):
        while True:
            case = dict(op=op, B=_log_int(rng, 1, 512), T=_log_int(rng, 1, 8192), H=rng.randint(1, 16),
                        d=rng.choice([16, 32, 64]), dtype=dtype, decay=rng.choice(["slow", "slopes"]),
                        ragged=rng.random() < 0.4, state=rng.random() < 0.5, packed=rng.random() < 0.4)
            size = case["B"] * case["T"] * case["H"] * case["d"]
            if 1 << 12 <= size <= 1 << 25 and sum(_lengths(case)) > 0 and work(case)["bytes"] <= 1e9:
                return case
    if op == "token":
        return dict(op=op, B=_log_int(rng, 1, 512), H=rng.randint(1, 16), d=rng.choice([16, 32, 64]), dtype=dtype,
                    decay=rng.choice(["slow", "slopes"]))
    while True:
        G = rng.choice([1, 2, 4, 8, 16, 32])
        C = G * rng.choice([1, 2, 3, 4, 8, 16, 32, 64])
        heads = rng.random() < 0.4
        L = 1 if heads else _log_int(rng, 2, 10000)
        N = _log_int(rng, 1, 200000 if heads else 300)
        # groups of a few values are left out: their gradients all but cancel, and 32 bits hold nothing of them
        if C % 8 == 0 and C <= 1024 and L * (C // G) >= 8 and 1 << 12 <= N * L * C <= 1 << 26:
            break
    return dict(op=op, N=N, L=L, C=C, G=G, dtype=dtype, act=rng.choice(["none", "silu", "relu"]))


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
    if case["op"] in ("prompt", "grad", "token"):
        B, H, d = case["B"], case["H"], case["d"]
        h = torch.arange(H, device=dev, dtype=torch.float64)
        if case["decay"] == "slow":     # memories of 32 to 4096 tokens, a factor apart
            s["log_decay"] = torch.log1p(-(2.0 ** (-5 - 7 * h / max(1, H - 1)))).float()
        else:                           # slopes from about 1/2 down to 1/256 per token
            s["log_decay"] = (-(2.0 ** (-8 * (h + 1) / H))).float()
        s["scale"] = d ** -0.5
        if case["op"] == "token":
            s["q"], s["k"], s["v"] = (normal(B, H, d, dtype=dt) for _ in range(3))
            s["S_in"] = normal(B, H, d, d) * 4
            return s
        T = case["T"]
        if case["packed"]:
            s["q"], s["k"], s["v"] = normal(B, T, 3, H, d, dtype=dt).unbind(2)
        else:
            s["q"], s["k"], s["v"] = (normal(B, T, H, d, dtype=dt) for _ in range(3))
        s["lengths"] = None
        if case["ragged"]:
            n = torch.tensor(_lengths(case), device=dev, dtype=torch.int32)
            s["lengths"] = n[torch.randperm(B, generator=g, device=dev)].contiguous()
        s["S_init"] = normal(B, H, d, d) * 4 if case["state"] else None
        if case["op"] == "grad":
            s["do"] = normal(B, T, H, d, dtype=dt)
            s["dS_final"] = normal(B, H, d, d) if case["state"] else None
        return s
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    s["x"] = (normal(N, L, C) * (0.5 + torch.rand(C, generator=g, device=dev)) + 0.7 * normal(C)).to(dt)
    s["gamma"], s["beta"] = 1 + 0.2 * normal(C), 0.2 * normal(C)
    if case["op"] == "norm_grad":
        s["dy"] = normal(N, L, C, dtype=dt)
        x = s["x"].double().view(N, L, G, C // G)
        mean, var = x.mean((1, 3)), x.var((1, 3), unbiased=False)   # what the forward pass left behind
        s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + EPS).float()
    return s


# ------------------------------------------------------------------ plain forms
def _causal(a, b, c, log_decay, scale):
    """out_t = scale * sum_{s <= t} exp(log_decay (t - s)) (a_t . b_s) c_s over [B, T, H, d], in blocks of CHUNK
    tokens: inside a block by its masked matrix, from earlier blocks by their decayed sums of b c^T."""
    B, T, H, d = a.shape
    n = -(-T // CHUNK)

    def blocks(x):
        full = torch.zeros(B, n * CHUNK, H, d, device=x.device, dtype=torch.float32)
        full[:, :T] = x
        return full.view(B, n, CHUNK, H, d).permute(0, 3, 1, 2, 4)      # [B, H, n, CHUNK, d]

    a, b, c = blocks(a), blocks(b), blocks(c)
    i = torch.arange(CHUNK, device=a.device)
    lg = log_decay.float().view(H, 1, 1)
    gap = (i[:, None] - i[None, :])
    inside = torch.where(gap >= 0, torch.exp(lg * gap.clamp(min=0)), torch.zeros((), device=a.device))   # [H, CHUNK, CHUNK]
    out = ((a @ b.transpose(-1, -2)) * inside.view(1, H, 1, CHUNK, CHUNK)) @ c
    left = torch.exp(lg * (CHUNK - 1 - i).view(1, CHUNK, 1)).view(1, H, 1, CHUNK, 1)
    sums = (b * left).transpose(-1, -2) @ c                              # [B, H, n, d, d]
    m = torch.arange(n, device=a.device)
    before = m[:, None] - 1 - m[None, :]
    carry = torch.where(before >= 0, torch.exp(lg * CHUNK * before.clamp(min=0)), torch.zeros((), device=a.device))  # [H, n, n]
    start = (carry.view(1, H, n, n) @ sums.reshape(B, H, n, d * d)).view(B, H, n, d, d)
    since = torch.exp(lg * (i + 1).view(1, CHUNK, 1)).view(1, H, 1, CHUNK, 1)
    out = (out + (a * since) @ start) * scale
    return out.permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, d)[:, :T]


def _powers(log_decay, n):
    """exp(log_decay n) [B, T, H, 1] for exponents n [B, T], 0 where n is negative."""
    lg = log_decay.float().view(1, 1, -1)
    n = n.unsqueeze(-1)
    return torch.where(n >= 0, torch.exp(lg * n.clamp(min=0)), torch.zeros((), device=n.device)).unsqueeze(-1)


def _sum_outer(a, b):
    """sum_t a_t b_t^T over [B, T, H, d] -> [B, H, d, d]"""
    return a.permute(0, 2, 3, 1) @ b.permute(0, 2, 1, 3)


def _times_state(a, S):
    """a_t^T S over [B, T, H, d]"""
    return (a.permute(0, 2, 1, 3) @ S).permute(0, 2, 1, 3)


def _masked(s):
    B, T = s["B"], s["T"]
    t = torch.arange(T, device=s["q"].device).view(1, T)
    n = torch.full((B, 1), T, device=t.device) if s["lengths"] is None else s["lengths"].view(B, 1)
    valid = (t < n).view(B, T, 1, 1)
    clean = lambda x: torch.where(valid, x.float(), torch.zeros((), device=x.device))  # noqa: E731
    return t.expand(B, T), n.expand(B, T), valid, clean


def _plain_prompt(s):
    t, n, valid, clean = _masked(s)
    q, k, v, lg = clean(s["q"]), clean(s["k"]), clean(s["v"]), s["log_decay"]
    o = _causal(q, k, v, lg, s["scale"])
    S = _sum_outer(k * _powers(lg, n - 1 - t), v)
    if s["S_init"] is not None:
        o = o + s["scale"] * _times_state(q * _powers(lg, t + 1), s["S_init"])
        S = S + _powers(lg, n[:, :1]).view(s["B"], s["H"], 1, 1) * s["S_init"]
    return torch.where(valid, o, torch.zeros((), device=o.device)).to(s["q"].dtype), S


def _plain_grad(s):
    t, n, valid, clean = _masked(s)
    q, k, v, do, lg = clean(s["q"]), clean(s["k"]), clean(s["v"]), clean(s["do"]), s["log_decay"]
    back = lambda x: torch.flip(x, (1,))  # noqa: E731
    dq = _causal(do, v, k, lg, s["scale"])
    dk = back(_causal(back(v), back(do), back(q), lg, s["scale"]))
    dv = back(_causal(back(k), back(q), back(do), lg, s["scale"]))
    dS = s["scale"] * _sum_outer(q * _powers(lg, torch.where(t < n, t + 1, -1)), do)
    if s["S_init"] is not None:
        dq = dq + s["scale"] * _times_state(do * _powers(lg, t + 1), s["S_init"].transpose(-1, -2))
    if s["dS_final"] is not None:
        w = _powers(lg, n - 1 - t)
        dk = dk + _times_state(v * w, s["dS_final"].transpose(-1, -2))
        dv = dv + _times_state(k * w, s["dS_final"])
        dS = dS + _powers(lg, n[:, :1]).view(s["B"], s["H"], 1, 1) * s["dS_final"]
    zero, dt = torch.zeros((), device=q.device), s["q"].dtype
    return tuple(torch.where(valid, x, zero).to(dt) for x in (dq, dk, dv)) + (dS,)


def _plain_token(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S = torch.exp(s["log_decay"]).view(1, -1, 1, 1) * s["S_in"] + k.unsqueeze(-1) * v.unsqueeze(-2)
    o = s["scale"] * (q.unsqueeze(-1) * S).sum(-2)
    return o.to(s["q"].dtype), S


def _act(z, act):
    return z * torch.sigmoid(z) if act == "silu" else torch.clamp(z, min=0) if act == "relu" else z


def _silu_slope(z):
    e = torch.sigmoid(z)
    return e * (1 + z * (1 - e))


def _plain_norm(s):
    N, L, C, G = s["N"], s["L"], s["C"], s["G"]
    x = s["x"].float().view(N, L, G, C // G)
    mean = x.mean((1, 3))
    dev = x - mean.view(N, 1, G, 1)
    rstd = 1 / torch.sqrt((dev * dev).mean((1, 3)) + EPS)
    z = (dev * rstd.view(N, 1, G, 1)).view(N, L, C) * s["gamma"] + s["beta"]
    return _act(z, s["act"]).to(s["x"].dtype), mean, rstd


def _plain_norm_grad(s):
    N, L, C, G = s["N"], s["L"], s["C"], s["G"]
    rstd = s["rstd"].view(N, 1, G, 1)
    xh = ((s["x"].float().view(N, L, G, C // G) - s["mean"].view(N, 1, G, 1)) * rstd).view(N, L, C)
    dz = s["dy"].float()
    if s["act"] == "silu":
        dz = dz * _silu_slope(xh * s["gamma"] + s["beta"])
    elif s["act"] == "relu":   # the side of the border in 64 bits: a value next to it changes its gradient whole
        x64 = s["x"].double().view(N, L, G, C // G) - s["mean"].double().view(N, 1, G, 1)
        dz = dz * ((x64 * rstd.double()).view(N, L, C) * s["gamma"].double() + s["beta"].double() > 0)
    dgamma, dbeta = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    dh = (dz * s["gamma"]).view(N, L, G, C // G)
    xg = xh.view(N, L, G, C // G)
    m1, m2 = dh.mean((1, 3), keepdim=True), (dh * xg).mean((1, 3), keepdim=True)
    dx = (rstd * (dh - m1 - xg * m2)).view(N, L, C)
    return dx.to(s["x"].dtype), dgamma, dbeta


def run(state):
    s = state
    if own:
        from self_referential_weight_gb300 import binding
        if s["op"] == "prompt":
            return binding.srwm_linattn_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                                S_init=s["S_init"], lengths=s["lengths"])
        if s["op"] == "grad":
            return binding.srwm_linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                                 S_init=s["S_init"], lengths=s["lengths"], dS_final=s["dS_final"])
        if s["op"] == "token":
            return binding.srwm_linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["S_in"], scale=s["scale"])
        if s["op"] == "norm":
            return binding.srwm_groupnorm_forward(s["x"], s["gamma"], s["beta"], s["G"], eps=EPS,
                                                  activation=s["act"])
        return binding.srwm_groupnorm_backward(s["x"], s["gamma"], s["beta"], s["G"], s["mean"], s["rstd"], s["dy"],
                                               activation=s["act"])
    plain = dict(prompt=_plain_prompt, grad=_plain_grad, token=_plain_token, norm=_plain_norm,
                 norm_grad=_plain_norm_grad)
    return plain[s["op"]](s)


# ------------------------------------------------------------------ floors
def work(case):
    e = DTYPES[case["dtype"]].itemsize
    if case["op"] in ("prompt", "grad", "token"):
        H, d = case["H"], case["d"]
        if case["op"] == "token":
            rows = case["B"] * H
            return {"bytes": rows * (8 * d * d + 4 * d * e), "flops": rows * 5 * d * d}
        rows, states = sum(_lengths(case)) * H, case["B"] * H * 4 * d * d
        full = case["B"] * case["T"] * H
        if case["op"] == "prompt":
            return {"bytes": (3 * rows + full) * d * e + states * (2 if case["state"] else 1),
                    "flops": rows * 4 * d * d}
        return {"bytes": (4 * rows + 3 * full) * d * e + states * (3 if case["state"] else 1),
                "flops": rows * 10 * d * d}
    n = case["N"] * case["L"] * case["C"]
    stats = 8 * case["N"] * case["G"]
    if case["op"] == "norm":
        return {"bytes": 2 * n * e + stats + 8 * case["C"], "flops": 8 * n}
    return {"bytes": 3 * n * e + stats + 16 * case["C"], "flops": 18 * n}


# ------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    f = lambda x: x.double()  # noqa: E731
    if case["op"] in ("prompt", "grad", "token"):
        g = torch.exp(f(s["log_decay"])).view(1, -1, 1, 1)
        B, H, d, scale = case["B"], case["H"], case["d"], s["scale"]
        if case["op"] == "token":
            S = g * f(s["S_in"]) + torch.einsum("bhi,bhj->bhij", f(s["k"]), f(s["v"]))
            return torch.einsum("bhi,bhij->bhj", f(s["q"]), S) * scale, S
        T = case["T"]
        n = torch.full((B,), T, device=g.device) if s["lengths"] is None else s["lengths"]
        S = torch.zeros(B, H, d, d, device=g.device, dtype=torch.float64) if s["S_init"] is None else f(s["S_init"])
        lasts = n.view(B, 1, 1, 1)
        row = lambda x, t: torch.where(t < n.view(B, 1, 1), f(x[:, t]), 0.0)  # noqa: E731
        if case["op"] == "prompt":
            o = torch.zeros(B, T, H, d, device=g.device, dtype=torch.float64)
            for t in range(T):
                new = g * S + row(s["k"], t).unsqueeze(-1) * row(s["v"], t).unsqueeze(-2)
                S = torch.where(t < lasts, new, S)
                o[:, t] = scale * (row(s["q"], t).unsqueeze(-2) @ S).squeeze(-2)
            return o, S
        dq, dk, dv = (torch.zeros(B, T, H, d, device=g.device, dtype=torch.float64) for _ in range(3))
        for t in range(T):
            new = g * S + row(s["k"], t).unsqueeze(-1) * row(s["v"], t).unsqueeze(-2)
            S = torch.where(t < lasts, new, S)
            dq[:, t] = scale * (S @ row(s["do"], t).unsqueeze(-1)).squeeze(-1)
        D = torch.zeros_like(S) if s["dS_final"] is None else f(s["dS_final"])   # dL/dS_t
        for t in range(T - 1, -1, -1):
            here = D + scale * row(s["q"], t).unsqueeze(-1) * row(s["do"], t).unsqueeze(-2)
            dk[:, t] = (here @ row(s["v"], t).unsqueeze(-1)).squeeze(-1)
            dv[:, t] = (row(s["k"], t).unsqueeze(-2) @ here).squeeze(-2)
            D = torch.where(t < lasts, g * here, D)
        return dq, dk, dv, D
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    x, gamma, beta = f(s["x"]).reshape(N, L, G, -1), f(s["gamma"]), f(s["beta"])
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, (1, 3), correction=0)
        rstd = (var + EPS).rsqrt()
        z = ((x - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, L, C) * gamma + beta
        y = z if case["act"] == "none" else torch.where(z > 0, z, 0.0) if case["act"] == "relu" else z / (1 + torch.exp(-z))
        return y, mean, rstd
    # by the Jacobian of x -> (x - mean) * rstd at the mean and rstd that are given
    mean, r = f(s["mean"])[:, None, :, None], f(s["rstd"])[:, None, :, None]
    u = (x - mean) * r
    z = u.reshape(N, L, C) * gamma + beta
    e = 1 / (1 + torch.exp(-z))
    slope = torch.ones_like(z) if case["act"] == "none" else (z > 0).double() if case["act"] == "relu" else e + z * e * (1 - e)
    dz = f(s["dy"]) * slope
    du = (dz * gamma).reshape(N, L, G, -1)
    size = L * (C // G)
    dx = r * (du - du.sum((1, 3), keepdim=True) / size - u * ((du * u).sum((1, 3), keepdim=True) / size))
    return dx.reshape(N, L, C), (dz * u.reshape(N, L, C)).sum((0, 1)), dz.sum((0, 1))

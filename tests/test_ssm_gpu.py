"""The selective state space scan on the GPU, against its definition token by
token in float64 (oracle/ssm.py).

Tolerances: oracle.ssm.errors bounds, entry by entry, what fp32 arithmetic can
lose, in roundings (2^-24) of the magnitudes that take part; it derives the
bounds of a step, a decay and a gate.  The kernels' own choices stay inside
them: approximate exponentials (2^-22) and reciprocals (2^-23), and a split
axis, which adds two roundings and a decay's error for each of at most 64
segments (`joins`).  A result in 16 bits rounds once more: 2^-8 (bf16) or
2^-11 (fp16) of itself, half the smallest subnormal step of fp16, 2^-25.
Exponentials and products below fp32's smallest normal number, 2^-126, may be
flushed to 0: `tiny` covers what a few thousand of them sum up to.
"""
import pytest
import torch

from oracle import ssm as oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TINY = 2.0 ** -100
GRADS = (("u", "dt"), ("A",), ("Bt", "Ct"), ("skip", "z", "dt_bias", "h_init"))


def near(got, ref, units, what, joins=0):
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    tol = units * 2.0 ** -24 * (1 + joins / 8) + TINY
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * ref.abs()
    elif got.dtype == F16:
        tol = tol + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    over = (got.double() - ref).abs() - tol
    assert over.numel() == 0 or float(over.max()) <= 0, (
        f"{what}: off by {float((got.double() - ref).abs().flatten()[int(over.argmax())]):.3e} at {int(over.argmax())}, "
        f"allowed {float(tol.flatten()[int(over.argmax())]):.3e}")


def make(seed, B, T, D, N, G, dtype, gate=True, packed=False, state=True, top=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    a = dict(u=n(B, T, D).to(dtype), dt=n(B, T, D).to(dtype), A=-torch.exp(1.5 * n(D, N)))
    if packed:
        p = n(B, T, 32 + 2 * G * N).to(dtype)[..., 32:]
        a["Bt"], a["Ct"] = p[..., :G * N].unflatten(-1, (G, N)), p[..., G * N:].unflatten(-1, (G, N))
    else:
        a["Bt"], a["Ct"] = n(B, T, G, N).to(dtype), n(B, T, G, N).to(dtype)
    a["skip"] = n(D)
    a["z"] = None if not gate else n(B, T, 2 * D).to(dtype)[..., D:] if packed else n(B, T, D).to(dtype)
    a["dt_bias"] = n(D) - 3 + top
    a["h_init"] = n(B, D, N) if state else None
    return a, n(B, T, D).to(dtype), n(B, D, N)


def clean(a):
    return {k: v if v is None else torch.nan_to_num(v, 0.0, 0.0, 0.0) for k, v in a.items()}


def check_forward(a, lengths=None, softplus=True, joins=0, **kw):
    y, h = binding.srwm_ssm_forward(**a, softplus=softplus, lengths=lengths, **kw)
    ry, rh = oracle.forward(**clean(a), softplus=softplus, lengths=lengths)
    ey, eh, _ = oracle.errors(None, clean(a), softplus, lengths)
    assert y.dtype == a["u"].dtype and h.dtype == F32
    near(y, ry, ey, "y", joins)
    near(h, rh, eh, "h_final", joins)
    return y, h


def check_backward(a, dy, lengths=None, dh=None, softplus=True, joins=0, **kw):
    rest = {k: v for k, v in a.items() if k not in ("u", "dt", "A", "Bt", "Ct")}
    got = binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, **rest, softplus=softplus, lengths=lengths,
                                    dh_final=dh, **kw)
    ref = oracle.grads(torch.nan_to_num(dy, 0.0, 0.0, 0.0), clean(a), softplus, lengths, dh)
    _, _, err = oracle.errors(torch.nan_to_num(dy, 0.0, 0.0, 0.0), clean(a), softplus, lengths, dh)
    assert len(got) == len(oracle.NAMES)
    for name, x in zip(oracle.NAMES, got):
        assert (x is None) == (a.get(name) is None), name
        if x is not None:
            assert x.dtype == (F32 if name in ("A", "skip", "dt_bias", "h_init") else a["u"].dtype), name
            near(x, ref[name], err[name], "d" + name, joins)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 33, 100])
def test_forward_lengths_and_types(T, N, dtype):
    a, _, _ = make(T + N, 3, T, 40, N, 1, dtype)
    check_forward(a)
    a, _, _ = make(T + N, 2, T, 144, N, 2, dtype, gate=False, state=False)
    check_forward(a)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 17, 50])
def test_backward_lengths_and_types(T, N, dtype):
    a, dy, dh = make(T + N, 3, T, 40, N, 1, dtype)
    check_backward(a, dy, None, dh)
    a, dy, _ = make(T + N, 2, T, 144, N, 2, dtype, gate=False, state=False)
    check_backward(a, dy)


@pytest.mark.parametrize("D,G", [(8, 1), (16, 2), (24, 1), (136, 1), (128, 1), (264, 1), (96, 4), (520, 5)])
@pytest.mark.parametrize("N", [16, 32, 64])
def test_widths_and_groups(D, G, N):
    a, dy, dh = make(D + N, 2, 19, D, N, G, BF16, packed=True)
    check_forward(a)
    check_backward(a, dy, None, dh)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 64])
def test_ragged_batches(N, dtype):
    """Lengths below 0, 0, 1, inside and at the end of a tile, T and above; NaN and infinity behind them."""
    T = 45
    lengths = torch.tensor([-3, 0, 1, 7, 8, 16, 17, 44, 45, 46, 1000], device=DEV, dtype=torch.int32)
    B = lengths.numel()
    a, dy, dh = make(N, B, T, 40, N, 1, dtype)
    past = torch.arange(T, device=DEV)[None, :] >= lengths.clamp(0, T)[:, None]
    for i, k in enumerate(("u", "dt", "Bt", "Ct", "z")):
        a[k][past] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    dy[past] = float("nan")
    y, h = check_forward(a, lengths)
    assert (y[past] == 0).all() and torch.equal(h[0], a["h_init"][0]) and torch.equal(h[1], a["h_init"][1])
    got = check_backward(a, dy, lengths, dh)
    for k in (0, 1, 3, 4, 6):
        assert (got[k][past] == 0).all()
    assert torch.equal(got[8][:2], dh[:2])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,N,G", [(1, 1500, 64, 16, 1), (2, 1031, 24, 32, 1), (1, 700, 72, 64, 3), (3, 517, 128, 16, 2)])
def test_few_long_sequences(B, T, D, N, G, dtype):
    """The axis is split here; ragged ends inside, at and before the last segment."""
    a, dy, dh = make(T, B, T, D, N, G, dtype)
    assert binding.srwm_ssm_workspace_bytes(B, T, D, N, G) > 256
    check_forward(a, joins=64)
    check_backward(a, dy, None, dh, joins=64)
    lengths = torch.tensor([T // 3, T - 1, 2][:B], device=DEV, dtype=torch.int32)
    check_forward(a, lengths, joins=64)
    check_backward(a, dy, lengths, dh, joins=64)


@pytest.mark.parametrize("top", [-12.0, 3.0, 20.0])
def test_steps_small_and_large(top):
    """Steps down to e^-15, where softplus is its argument's exponential, and far above 1, where decays vanish."""
    a, dy, dh = make(3, 2, 40, 64, 16, 1, F32, top=top)
    check_forward(a)
    check_backward(a, dy, None, dh)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_without_softplus_and_parts_left_out(dtype):
    a, dy, dh = make(5, 2, 30, 48, 16, 1, dtype)
    a["dt"] = (a["dt"].float().abs() * 0.2).to(dtype)
    a["dt_bias"] = a["dt_bias"].abs() * 0.01
    check_forward(a, softplus=False)
    check_backward(a, dy, None, dh, softplus=False)
    for k in ("skip", "z", "dt_bias", "h_init"):
        b = dict(a)
        b[k] = None
        check_forward(b, softplus=k == "z")
        check_backward(b, dy, None, None, softplus=k == "z")


def test_strong_decays_keep_their_gradients():
    """Decays down to e^-40 a token: what is left of a state, and its gradient, keep their relative precision."""
    a, dy, dh = make(6, 2, 24, 32, 16, 1, F32, top=2.0)
    a["A"] = -torch.linspace(0.5, 20, 16, device=DEV).expand(32, 16).contiguous()
    check_forward(a)
    check_backward(a, dy, None, dh)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("B,D,G", [(1, 8, 1), (3, 40, 1), (70, 264, 3), (301, 1032, 3)])
def test_step(B, D, G, N, dtype):
    for packed in (False, True):
        a, _, _ = make(B + N, B, 1, D, N, G, dtype, packed=packed)
        one = {k: v[:, 0] if k in ("u", "dt", "Bt", "Ct", "z") else v for k, v in a.items()}
        call = lambda **kw: binding.srwm_ssm_step(one["u"], one["dt"], one["A"], one["Bt"], one["Ct"], skip=one["skip"],  # noqa: E731
                                                  z_t=one["z"], dt_bias=one["dt_bias"], **kw)
        y, h = call(h_in=one["h_init"])
        ry, rh = oracle.forward(**a)
        ey, eh, _ = oracle.errors(None, a)
        near(y, ry[:, 0], ey[:, 0], "y")
        near(h, rh, eh, "h_out")
        state = one["h_init"].clone()
        y2, h2 = call(h_in=state, h_out=state)
        assert h2.data_ptr() == state.data_ptr() and torch.equal(y2, y) and torch.equal(state, h)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 64])
def test_windows_and_single_tokens_continue_a_prompt(N, dtype):
    T = 41
    a, _, _ = make(N, 3, T, 72, N, 1, dtype)
    _, h = check_forward(a)
    part = lambda lo, hi: {k: v[:, lo:hi].contiguous() if k in ("u", "dt", "Bt", "Ct", "z") else v for k, v in a.items()}  # noqa: E731
    y1, h1 = binding.srwm_ssm_forward(**part(0, 19))
    y2, h2 = binding.srwm_ssm_forward(**{**part(19, 37), "h_init": h1})
    outs = [y1, y2]
    for t in range(37, T):
        y, h2 = binding.srwm_ssm_step(a["u"][:, t], a["dt"][:, t], a["A"], a["Bt"][:, t], a["Ct"][:, t], h2, skip=a["skip"],
                                      z_t=a["z"][:, t], dt_bias=a["dt_bias"])
        outs.append(y[:, None])
    ry, rh = oracle.forward(**a)
    ey, eh, _ = oracle.errors(None, a)
    near(torch.cat(outs, 1), ry, ey, "y")
    near(h2, rh, eh, "h")


def test_gradients_against_differences():
    """The kernels' own forward pass, in fp32, along random directions: the loss' second difference is below h^2, its
    rounding about 1e-5 / h."""
    a, dy, dh = make(9, 2, 12, 24, 16, 1, F32)
    got = dict(zip(oracle.NAMES, check_backward(a, dy, None, dh)))

    def loss(args):
        y, h = binding.srwm_ssm_forward(**args)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    step = 2.0 ** -7
    for name in oracle.NAMES:
        g = torch.Generator(device=DEV).manual_seed(len(name))
        d = torch.randn(a[name].shape, generator=g, device=DEV)
        d = d * step / d.norm()
        up, down = (loss({**a, name: a[name] + k * d}) for k in (1, -1))
        want = float((got[name].double() * d.double()).sum())
        size = float(got[name].double().norm()) * step
        assert abs((up - down) / 2 - want) <= 0.02 * size + 1e-4, name


def test_not_finite_inputs_stay_in_their_channel():
    for k, at in (("u", (1, 5, 9)), ("dt", (1, 20, 3)), ("z", (0, 2, 30))):
        a, dy, _ = make(11, 2, 30, 40, 16, 1, F32)
        y0, h0 = binding.srwm_ssm_forward(**a)
        for bad in (float("nan"), float("inf")):
            b = dict(a)
            b[k] = a[k].clone()
            b[k][at] = bad
            y, h = binding.srwm_ssm_forward(**b)
            other = torch.ones_like(y, dtype=torch.bool)
            other[at[0], at[1]:, at[2]] = False
            assert torch.equal(y[other], y0[other])
            if bad != bad:
                assert torch.isnan(y[at])
                if k != "z":
                    assert torch.isnan(h[at[0], at[2]]).all()
            keep = torch.ones(2, 40, dtype=torch.bool, device=DEV)
            keep[at[0], at[2]] = False
            assert torch.equal(h[keep], h0[keep])


def test_zero_tokens():
    a, dy, dh = make(1, 2, 0, 24, 16, 1, F32)
    y, h = binding.srwm_ssm_forward(**a)
    assert y.shape == (2, 0, 24) and torch.equal(h, a["h_init"])
    rest = {k: v for k, v in a.items() if k not in ("u", "dt", "A", "Bt", "Ct")}
    got = binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, **rest, dh_final=dh)
    assert torch.equal(got[8], dh)
    for k in (2, 5, 7):
        assert (got[k] == 0).all()


@pytest.mark.parametrize("B,T", [(3, 50), (1, 900)])
def test_same_bits_streams_and_graphs(B, T):
    """Repeats, another stream, two streams at once with workspaces of their own, and replays of a captured run give the same bits."""
    a, dy, dh = make(2, B, T, 64, 16, 1, BF16)
    rest = {k: v for k, v in a.items() if k not in ("u", "dt", "A", "Bt", "Ct")}

    def both(**kw):
        return (*binding.srwm_ssm_forward(**a, **kw),
                *binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, **rest, dh_final=dh, **kw))

    first = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    runs = [both(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for run in runs + [kept]:
        for x, r in zip(run, first):
            assert torch.equal(x, r)


def test_gradients_into_packed_arrays():
    a, dy, dh = make(4, 2, 21, 40, 32, 1, BF16, packed=True)
    plain = check_backward(a, dy, None, dh)
    pbc = torch.full((2, 21, 32 + 64), 7.0, device=DEV, dtype=BF16)
    pz = torch.full((2, 21, 80), 7.0, device=DEV, dtype=BF16)
    got = check_backward(a, dy, None, dh, dB=pbc[..., 32:64].unflatten(-1, (1, 32)), dC=pbc[..., 64:].unflatten(-1, (1, 32)),
                         dz=pz[..., 40:])
    assert (pbc[..., :32] == 7).all() and (pz[..., :40] == 7).all()
    for x, r in zip(got, plain):
        assert torch.equal(x, r)


def test_many_streams():
    """More CTAs than the GPU holds, of uneven lengths: a sample of sequences against the oracle."""
    B, T, D, N = 900, 37, 136, 16
    a, dy, dh = make(8, B, T, D, N, 1, BF16)
    lengths = torch.arange(B, device=DEV, dtype=torch.int32) % (T + 1)
    y, h = binding.srwm_ssm_forward(**a, lengths=lengths)
    rest = {k: v for k, v in a.items() if k not in ("u", "dt", "A", "Bt", "Ct")}
    got = binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, **rest, lengths=lengths, dh_final=dh)
    pick = torch.tensor([0, 1, 300, 511, 898, 899], device=DEV)
    sub = {k: v[pick] if k in ("u", "dt", "Bt", "Ct", "z", "h_init") else v for k, v in a.items()}
    ry, rh = oracle.forward(**sub, lengths=lengths[pick])
    ref = oracle.grads(dy[pick], sub, True, lengths[pick], dh[pick])
    ey, eh, err = oracle.errors(dy[pick], sub, True, lengths[pick], dh[pick])
    near(y[pick], ry, ey, "y")
    near(h[pick], rh, eh, "h")
    for name, x in zip(oracle.NAMES, got):
        if name not in ("A", "skip", "dt_bias"):
            near(x[pick], ref[name], err[name], "d" + name)


def test_gradients_in_slices():
    """More sequences than the workspace holds states for, the last two of them cut: single sequences against the oracle,
    and the parameters' gradients against those of the two halves (a slice left out would miss a third)."""
    B, T, D, N = 66, 300, 2048, 64
    a, dy, dh = make(8, B, T, D, N, 1, BF16)
    lengths = (torch.arange(B, device=DEV, dtype=torch.int32) * 37) % (T + 1)
    lengths[[0, 33, 65]] = torch.tensor([300, 41, 299], device=DEV, dtype=torch.int32)
    assert binding.srwm_ssm_backward_workspace_bytes(B, T, D, N, 1) < 0.8 * B * T * D * N

    def run(part):
        one = {k: v[part].contiguous() if k in ("u", "dt", "Bt", "Ct", "z", "h_init") else v for k, v in a.items()}
        rest = {k: v for k, v in one.items() if k not in ("u", "dt", "A", "Bt", "Ct")}
        return binding.srwm_ssm_backward(one["u"], one["dt"], one["A"], one["Bt"], one["Ct"], dy[part].contiguous(), **rest,
                                         lengths=lengths[part].contiguous(), dh_final=dh[part].contiguous())

    got, first, second = run(slice(0, B)), run(slice(0, 33)), run(slice(33, B))
    pick = torch.tensor([0, 33, 65], device=DEV)
    sub = {k: v[pick] if k in ("u", "dt", "Bt", "Ct", "z", "h_init") else v for k, v in a.items()}
    ref = oracle.grads(dy[pick], sub, True, lengths[pick], dh[pick])
    _, _, err = oracle.errors(dy[pick], sub, True, lengths[pick], dh[pick])
    for name, x, p, q in zip(oracle.NAMES, got, first, second):
        if name in ("A", "skip", "dt_bias"):
            assert float((x - p - q).norm()) <= 1e-4 * float(x.norm()), name
        else:
            near(x[pick], ref[name], err[name], "d" + name, joins=64)
            part = torch.cat([p, q])
            assert float((x.float() - part.float()).norm()) <= 2.0 ** -8 * float(part.float().norm()), name


def param_grads(a, dy, lengths, **kw):
    rest = {k: v for k, v in a.items() if k not in ("u", "dt", "A", "Bt", "Ct")}
    return dict(zip(oracle.NAMES, binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, **rest, lengths=lengths, **kw)))


@pytest.mark.parametrize("T", [255, 256, 257, 600])
def test_parameter_gradients_of_whole_sequences(T):
    """Blocks of 256 tokens have partial sums of their own: inside, at and behind a block's end, and ragged lengths that leave
    the last ones empty.  The 640 CTAs of 40 sequences are more than half of a wave of 912: nothing is cut."""
    B, D, N = 40, 1024, 16
    a, dy, dh = make(T, B, T, D, N, 1, BF16)
    lengths = torch.tensor([T, 1, 0, 256, 255, 257, T - 1, 300], device=DEV, dtype=torch.int32).repeat(5)
    for n in (None, lengths):
        check_backward(a, dy, n, dh)


def test_parameter_gradients_of_segments_of_several_blocks():
    """448 CTAs of 7 sequences: two segments of 312 tokens each, with two blocks of partial sums; ragged ends in either."""
    a, dy, dh = make(3, 7, 620, 4096, 16, 1, BF16)
    lengths = torch.tensor([620, 600, 312, 313, 200, 0, 570], device=DEV, dtype=torch.int32)
    for n in (None, lengths):
        check_backward(a, dy, n, dh, joins=64)


def test_parameter_gradients_of_whole_and_cut_sequences():
    """fp32: 38 of 40 sequences fill a wave of 608 CTAs, the other two are cut; partial sums of both kinds beside each other."""
    a, dy, dh = make(4, 40, 300, 1024, 16, 1, F32)
    lengths = torch.arange(40, device=DEV, dtype=torch.int32) * 7 + 27
    for n in (None, lengths):
        check_backward(a, dy, n, dh, joins=64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,N", [(1, 1500, 64, 16), (2, 1031, 24, 32), (1, 700, 72, 64)])
def test_growth_past_fp32_leaves_zeros(B, T, D, N, dtype):
    """A cut axis, and half of the channels growing by e^100 and more over a segment: states that are 0 until the last token
    and gradients that are 0 from the second token on stay so, as token by token."""
    a, dy, _ = make(T + 1, B, T, D, N, 1, dtype, state=False, top=3.5)
    assert binding.srwm_ssm_workspace_bytes(B, T, D, N, 1) > 256
    a["A"][::2] = 3 + torch.rand(D // 2, N, device=DEV)
    a["dt"] = a["dt"].clamp(-1, 1)
    a["dt_bias"] = a["dt_bias"].clamp(0, 3)       # steps of 0.3 to 4: a decay of e^16 at most
    a["u"][:, :-1, ::2] = 0
    dy[:, 1:, ::2] = 0
    check_forward(a, joins=64)
    check_backward(a, dy, joins=64)


@pytest.mark.parametrize("D,N,T,copies", [(1024, 16, 8, 640), (512, 64, 26, 100)])
def test_parameter_gradients_of_large_batches(D, N, T, copies):
    """Copies of 64 sequences, more than the workspace holds: the parameters' gradients are as many times the 64 sequences',
    and each copy's own gradients are theirs.  What adding up the copies costs beside the 64 sequences' own bound: partial
    sums in chains of at most a 32nd of the sequences, 5 joins and a few slices, each addition rounding by 2^-24 of the sum of
    magnitudes, which that bound holds 64 T times."""
    B = 64 * copies
    a, dy, _ = make(T, 64, T, D, N, 1, BF16, state=False)
    lengths = torch.arange(64, device=DEV, dtype=torch.int32) * 5 % (T + 1)
    many = {k: v.repeat(copies, *[1] * (v.dim() - 1)) if k in ("u", "dt", "Bt", "Ct", "z") else v for k, v in a.items()}
    each = T / 8 * D * N * 4 + T * -(-D // (1024 // N)) * 8 * N + D * (N + 2) * 4
    assert B * each > 2.2e9 and binding.srwm_ssm_backward_workspace_bytes(B, T, D, N, 1) < 2.1e9
    got = param_grads(many, dy.repeat(copies, 1, 1), lengths.repeat(copies))
    ref = oracle.grads(dy, a, True, lengths)
    _, _, err = oracle.errors(dy, a, True, lengths)
    for name, x in got.items():
        if name in ("A", "skip", "dt_bias"):
            near(x, copies * ref[name], copies * err[name] * (1 + (B / 32 + 64) / (64 * T)), "d" + name)
        elif x is not None:
            assert torch.equal(x, x[:64].repeat(copies, *[1] * (x.dim() - 1))), "d" + name
            near(x[:64], ref[name], err[name], "d" + name)


def test_binding_refuses():
    a, dy, _ = make(1, 2, 5, 24, 16, 1, F32)
    call = lambda **kw: binding.srwm_ssm_forward(**{**a, **kw})  # noqa: E731
    for bad in (dict(dt=a["dt"].double()), dict(dt=a["dt"][:, :4]), dict(A=a["A"].half()), dict(A=a["A"][:, :8]),
                dict(Ct=a["Ct"].cpu()), dict(skip=a["skip"][:8]), dict(h_init=a["h_init"][:1]), dict(z=a["z"].half()),
                dict(lengths=torch.tensor([1, 2])), dict(lengths=torch.tensor([1, 2], device=DEV)),
                dict(u=a["u"].transpose(0, 1).contiguous().transpose(0, 1)), dict(y=torch.empty(2, 5, 24, device=DEV, dtype=BF16))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(u=None)
    with pytest.raises(binding.SrwmError):
        call(y=a["u"])
    with pytest.raises(binding.SrwmError):      # 8 states
        call(A=a["A"][:, :8].contiguous(), Bt=a["Bt"][..., :8].contiguous(), Ct=a["Ct"][..., :8].contiguous(), h_init=None)
    with pytest.raises(ValueError):
        binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, dskip=torch.empty(24, device=DEV))
    with pytest.raises(ValueError):
        binding.srwm_ssm_backward(a["u"], a["dt"], a["A"], a["Bt"], a["Ct"], dy, dB=torch.empty_like(a["Bt"]))

"""The short causal convolution on the GPU, against its definition in float64
(oracle/conv.py).

Tolerances, per entry: p = bias + sum of W products rounds W + 1 times, each by
at most 2^-24 of the sum A of the magnitudes; silu(p) adds its slope (at most
1.1) times that, an approximate exponential (2^-22 and |p| 2^-23 of its
argument's rounding) and reciprocal (2^-23): (W + 4 + 20 + |p|) 2^-24 of A and
of the result cover it.  A gradient g = dy act'(p) has the same, relative to
|dy| (1.1 + A), and sums of it over n terms round n times more.  16-bit results
round once: 2^-8 (bf16) or 2^-11 (fp16, at least 2^-25).
"""
import pytest
import torch

from oracle import conv as oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def near(got, ref, tol, what):
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * ref.abs()
    elif got.dtype == F16:
        tol = tol + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    over = (got.double() - ref).abs() - tol
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3e}"


def make(seed, B, T, D, W, dtype, packed=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = n(B, T, 2 * D).to(dtype)[..., D:] if packed else n(B, T, D).to(dtype)
    return x, n(D, W), n(D), n(B, W - 1, D).to(dtype), n(B, T, D).to(dtype), n(B, W - 1, D).to(dtype)


def sizes(x, weight, bias, state, lengths):
    A, _ = oracle.forward(x.abs(), weight.abs(), None if bias is None else bias.abs(), "none", None if state is None else state.abs(), lengths)
    return A


def check_forward(x, weight, bias, act="silu", state=None, lengths=None, **kw):
    y, last = binding.srwm_conv_forward(x, weight, bias, act, state_init=state, lengths=lengths, **kw)
    ry, rl = oracle.forward(x, weight, bias, act, state, lengths)
    A = sizes(torch.nan_to_num(x.float(), 0.0, 0.0, 0.0), weight, bias, state, lengths)
    W = weight.shape[1]
    assert y.dtype == x.dtype and last.dtype == x.dtype
    near(y, ry, (1.1 * (W + 4) + 20 + A) * 2.0 ** -24 * A, "y")
    assert torch.equal(last.double(), rl), "state_final"
    return y, last


def check_backward(x, weight, bias, dy, act="silu", state=None, lengths=None, dstate=None, **kw):
    got = binding.srwm_conv_backward(x, weight, bias, dy, act, state_init=state, lengths=lengths, dstate_final=dstate, **kw)
    ref = oracle.grads(x, weight, bias, act, torch.nan_to_num(dy, 0.0, 0.0, 0.0), state, lengths, dstate)
    clean = torch.nan_to_num(x.float(), 0.0, 0.0, 0.0)
    A = sizes(clean, weight, bias, state, lengths)
    W, (B, T, D) = weight.shape[1], x.shape
    gsize = torch.nan_to_num(dy.double().abs(), 0.0, 0.0, 0.0) * (1.1 + A) if act == "silu" else torch.nan_to_num(dy.double().abs(), 0.0, 0.0, 0.0)
    unit = (gsize * (W + 30 + 2 * A), gsize)        # errors of g in roundings, and its magnitude

    def through(v):                                  # by magnitudes, as the gradients themselves
        return oracle.grads(clean.abs(), weight.abs(), None if bias is None else bias.abs(), "none", v,
                            None if state is None else state.abs(), lengths, None if dstate is None else dstate.abs())

    err, mag = through(unit[0]), through(unit[1])
    terms = (W + 1, B * T, B * T, W + 1)
    for name, x_, r, e, m, n in zip(("dx", "dweight", "dbias", "dstate_init"), got, ref, err, mag, terms):
        given = name in ("dx", "dweight") or (bias if name == "dbias" else state) is not None
        assert (x_ is not None) == given, name
        if given:
            assert x_.dtype == (x.dtype if name in ("dx", "dstate_init") else F32)
            near(x_, r, (e + (n + 2) * m) * 2.0 ** -24, name)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 31, 32, 33, 70])
def test_lengths_and_types(T, W, dtype):
    x, w, b, s, dy, ds = make(T + W, 3, T, 40, W, dtype)
    check_forward(x, w, b, "silu", s)
    check_forward(x, w, None, "none")
    check_backward(x, w, b, dy, "silu", s, None, ds)
    check_backward(x, w, None, dy, "none")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [8, 24, 128, 136, 264, 1000])
def test_widths_and_packed_slices(D, dtype):
    x, w, b, s, dy, ds = make(D, 2, 37, D, 4, dtype, packed=True)
    check_forward(x, w, b, "silu", s)
    packed = torch.full((2, 37, 2 * D), 7.0, device=DEV, dtype=dtype)
    got = check_backward(x, w, b, dy, "silu", s, None, ds, dx=packed[..., :D])
    assert (packed[..., D:] == 7).all() and got[0].data_ptr() == packed.data_ptr()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 4])
def test_ragged_batches(W, dtype):
    T = 70
    lengths = torch.tensor([-3, 0, 1, 2, 3, 31, 32, 33, 64, 69, 70, 71, 1 << 30], device=DEV, dtype=torch.int32)
    x, w, b, s, dy, ds = make(W, lengths.numel(), T, 24, W, dtype)
    past = torch.arange(T, device=DEV)[None, :] >= lengths.clamp(0, T)[:, None]
    x[past], dy[past] = float("nan"), float("inf")
    y, last = check_forward(x, w, b, "silu", s, lengths)
    assert (y[past] == 0).all() and torch.equal(last[:2], s[:2])
    got = check_backward(x, w, b, dy, "silu", s, lengths, ds)
    assert (got[0][past] == 0).all()
    check_forward(x, w, b, "silu", None, lengths)
    check_backward(x, w, b, dy, "silu", None, lengths, ds)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,D", [(1, 8), (5, 264), (300, 128)])
def test_step(B, D, W, dtype):
    x, w, b, s, _, _ = make(B + W, B, 1, D, W, dtype, packed=True)
    y, last = binding.srwm_conv_step(x[:, 0], w, b, s)
    ry, rl = oracle.forward(x, w, b, "silu", s)
    A = sizes(x, w, b, s, None)
    near(y, ry[:, 0], ((1.1 * (W + 4) + 20 + A) * 2.0 ** -24 * A)[:, 0], "y")
    assert torch.equal(last.double(), rl)
    state = s.clone()
    y2, s2 = binding.srwm_conv_step(x[:, 0], w, b, state, state_out=state)
    assert s2.data_ptr() == state.data_ptr() and torch.equal(y2, y) and torch.equal(state, last)
    y3, _ = binding.srwm_conv_step(x[:, 0], w, None, s, activation="none")
    r3, _ = oracle.forward(x, w, None, "none", s)
    near(y3, r3[:, 0], (W + 1) * 2.0 ** -24 * sizes(x, w, None, s, None)[:, 0], "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_windows_and_single_tokens_are_one_prompt(dtype):
    x, w, b, s, _, _ = make(3, 2, 50, 40, 4, dtype)
    y, last = binding.srwm_conv_forward(x, w, b, state_init=s)
    y1, s1 = binding.srwm_conv_forward(x[:, :1].contiguous(), w, b, state_init=s)
    y2, s2 = binding.srwm_conv_forward(x[:, 1:40].contiguous(), w, b, state_init=s1)
    outs = [y1, y2]
    for t in range(40, 50):
        o, s2 = binding.srwm_conv_step(x[:, t], w, b, s2)
        outs.append(o[:, None])
    assert torch.equal(torch.cat(outs, 1), y) and torch.equal(s2, last)


def test_gradients_against_differences():
    x, w, b, s, dy, ds = make(5, 2, 9, 24, 4, F32)
    got = check_backward(x, w, b, dy, "silu", s, None, ds)

    def loss(a):
        y, last = binding.srwm_conv_forward(a[0], a[1], a[2], state_init=a[3])
        return float((y.double() * dy.double()).sum() + (last.double() * ds.double()).sum())

    base, h = [x, w, b, s], 2.0 ** -7      # second differences below h^2, the loss' rounding about 1e-5
    for i, g in enumerate(got):
        d = torch.randn(base[i].shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV)
        d = d * h / d.norm()
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + d, base[i] - d
        assert abs((loss(up) - loss(down)) / 2 - float((g.double() * d.double()).sum())) <= 0.01 * float(g.double().norm()) * h + 1e-4


def test_zero_tokens_and_empty_outputs():
    x, w, b, s, dy, ds = make(1, 2, 0, 24, 4, F32)
    y, last = binding.srwm_conv_forward(x, w, b, state_init=s)
    assert y.shape == (2, 0, 24) and torch.equal(last, s)
    got = binding.srwm_conv_backward(x, w, b, dy, state_init=s, dstate_final=ds)
    assert torch.equal(got[3], ds) and (got[1] == 0).all() and (got[2] == 0).all()


def test_same_bits_streams_and_graphs():
    x, w, b, s, dy, ds = make(2, 40, 130, 136, 4, BF16)

    def both(**kw):
        return (*binding.srwm_conv_forward(x, w, b, state_init=s, **kw),
                *binding.srwm_conv_backward(x, w, b, dy, state_init=s, dstate_final=ds, **kw))

    first = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [both(stream=q) for _ in range(3) for q in streams]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for run in runs + [kept]:
        assert all(torch.equal(p, r) for p, r in zip(run, first))


def test_binding_refuses():
    x, w, b, s, dy, _ = make(1, 2, 5, 24, 4, F32)
    for bad in (dict(x=x.double()), dict(weight=w.half()), dict(weight=w[:8]), dict(bias=b[:8]), dict(state_init=s[:1]),
                dict(state_init=s.half()), dict(activation="gelu"), dict(lengths=torch.tensor([1, 2], device=DEV)),
                dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(y=torch.empty(2, 5, 16, device=DEV))):
        with pytest.raises(ValueError):
            binding.srwm_conv_forward(**{**dict(x=x, weight=w, bias=b), **bad})
    for bad in (dict(activation="relu"), dict(weight=torch.randn(24, 5, device=DEV)), dict(weight=torch.randn(24, 1, device=DEV)), dict(y=x)):
        with pytest.raises(binding.SrwmError):
            binding.srwm_conv_forward(**{**dict(x=x, weight=w, bias=b), **bad})
    with pytest.raises(ValueError):
        binding.srwm_conv_backward(x, w, None, dy, dbias=torch.empty(24, device=DEV))

"""The root-mean-square norm on the GPU, against its definition in float64
(oracle/rmsnorm.py).

Tolerances, per entry: h = x + residual rounds once; the sum of C squares
rounds C times (2^-24 each of a sum of positive terms, so of itself), its root
halves that; two products and a division follow: (C / 2 + 8) 2^-24 of |y|.  The
rounding of h is relative to h itself.  Results in 16 bits round once more,
2^-8 (bf16) or 2^-11 (fp16, at least 2^-25).  In 8 bits a value is within half
a step of y / scale, 2^-4 of itself or 2^-10 (half the smallest step), plus
what y and scale are off by, relative to it.  Gradients: the mean over C
products rounds C times, relative to the sum of its terms' magnitudes.
"""
import pytest
import torch

from oracle import rmsnorm as oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


def near(got, ref, tol, what):
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * ref.abs()
    elif got.dtype == F16:
        tol = tol + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    over = (got.double() - ref).abs() - tol - 2.0 ** -140
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3e}"


def make(seed, N, C, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return n(N, C).to(dtype), (2 * n(N, C)).to(dtype), n(C), n(N, C).to(dtype), n(N, C).to(dtype)


def check_forward(x, gamma, residual=None, eps=EPS, **kw):
    y, scale, total, rstd = binding.srwm_rmsnorm_forward(x, gamma, residual=residual, eps=eps, **kw)
    ry, rh, rr = oracle.forward(x, gamma, residual, eps)
    unit = (x.shape[1] / 2 + 8) * 2.0 ** -24
    assert scale is None and (total is None) == (residual is None) and y.dtype == x.dtype and rstd.dtype == F32
    near(y, ry, unit * ry.abs(), "y")
    near(rstd, rr, unit * rr, "rstd")
    if total is not None:
        near(total, rh, 2.0 ** -24 * rh.abs(), "total")
    return y, total, rstd


def check_8bit(x, gamma, residual=None, block=0, eps=EPS):
    y, scale, total, rstd = binding.srwm_rmsnorm_forward(x, gamma, residual=residual, eps=eps, out="e4m3", block=block)
    N, C = x.shape
    ry, rh, rr = oracle.forward(x, gamma, residual, eps)
    unit = (C / 2 + 12) * 2.0 ** -24
    rs = ry.view(N, -1, block or C).abs().amax(-1) / 448
    assert y.dtype == torch.float8_e4m3fn and scale.shape == rs.shape and scale.dtype == F32
    near(scale, rs, unit * rs, "scale")
    near(rstd, rr, unit * rr, "rstd")
    values = oracle.e4m3_values().to(DEV)[y.view(torch.uint8).long()]
    q = (ry.view(N, -1, block or C) / torch.where(rs > 0, rs, 1.0)[..., None]).view(N, C)
    near(values, q, 2.0 ** -4 * q.abs() * (1 + unit) + 2.0 ** -10 + 2 * unit * q.abs(), "y8")
    return y, scale


def check_backward(total, gamma, dy, dtotal=None, **kw):
    _, _, r = oracle.forward(total, gamma, None, EPS)
    rstd = r.float()
    dx, dg = binding.srwm_rmsnorm_backward(total, gamma, rstd, dy, dtotal=dtotal, **kw)
    rx, rg = oracle.grads(total, gamma, EPS, dy, dtotal)
    N, C = total.shape
    d = dy.double().abs() * (1 if gamma is None else gamma.double().abs())
    xh = total.double().abs() * r[:, None]
    mean = (d * xh).mean(1, keepdim=True)
    size = r[:, None] * (d + xh * mean) + (0 if dtotal is None else dtotal.double().abs())
    near(dx, rx, (C + 12) * 2.0 ** -24 * size, "dx")
    assert (dg is None) == (gamma is None)
    if dg is not None:
        near(dg, rg, (N + 4) * 2.0 ** -24 * (dy.double().abs() * xh).sum(0), "dgamma")
    return dx, dg


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("C", [8, 24, 64, 256, 264, 512, 1000, 1024, 1032, 2048, 4104, 8192])
@pytest.mark.parametrize("N", [1, 5])
def test_widths_and_types(N, C, dtype):
    x, r, g, dy, dt = make(N + C, N, C, dtype)
    check_forward(x, g, r)
    check_forward(x, None)
    check_backward(x, g, dy, dt)
    check_backward(x, None, dy)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,C", [(3000, 128), (700, 264), (1500, 1024), (650, 4096), (610, 8192), (5001, 8)])
def test_many_rows(N, C, dtype):
    x, r, g, dy, dt = make(C, N, C, dtype)
    check_forward(x, g, r)
    check_backward(x, g, dy, dt)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("N,C", [(1, 128), (7, 256), (3, 1152), (2, 8192), (900, 1024), (700, 4096)])
def test_8_bits(N, C, block, dtype):
    x, r, g, _, _ = make(N + C, N, C, dtype)
    check_8bit(x, g, r, block)
    check_8bit(x, None, None, block)


@pytest.mark.parametrize("C", [8, 24, 264, 1000])
def test_8_bits_by_rows_of_odd_widths(C):
    x, r, g, _, _ = make(C, 9, C, BF16)
    check_8bit(x, g, r, 0)


def test_8_bits_at_the_borders():
    """A row and a block of zeros, magnitudes down to fp32's smallest, ties, and values that are not finite."""
    x = torch.randn(6, 256, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    x[0] = 0
    x[1, :128] = 0
    x[2] = 0
    x[2, 5] = 1e-44
    x[3] *= 1e-42
    x[4] *= 1e-30
    for block in (0, 128):
        y, scale = check_8bit(x, None, None, block)
        assert (y[0].float() == 0).all() and (scale[0] == 0).all()
        if block:
            assert scale[1, 0] == 0 and (y[1, :128].float() == 0).all()
        assert (y.float().abs().amax(1)[3:] == 448).all()
    bad = x.clone()
    bad[5, 200] = float("nan")
    y, scale, _, rstd = binding.srwm_rmsnorm_forward(bad, None, out="e4m3", block=128)
    assert torch.isnan(y[5].float()).all() and torch.isnan(scale[5]).all() and torch.isnan(rstd[5])
    y0, s0, _, _ = binding.srwm_rmsnorm_forward(x, None, out="e4m3", block=128)
    assert torch.equal(y[:5].view(torch.uint8), y0[:5].view(torch.uint8)) and torch.equal(scale[:5], s0[:5])


def test_codes_are_the_nearest():
    """With a row whose largest value is 448 times a power of two, y / scale is exact: codes round to nearest, ties to even."""
    codes = oracle.e4m3_values()[:127].to(DEV)
    mids = (codes[:-1] + codes[1:]) / 2
    row = torch.cat([codes, mids, torch.zeros(256 - 253, device=DEV, dtype=torch.float64)])
    row[-1] = 448.0
    gamma = row.float()
    x = torch.ones(1, 256, device=DEV)
    y, scale, _, rstd = binding.srwm_rmsnorm_forward(x, gamma, eps=2.0 ** -40, out="e4m3")
    assert float(rstd) == 1.0 and float(scale) == 1.0
    got = y[0, :253].view(torch.uint8).long().cpu()
    assert torch.equal(got[:127], torch.arange(127))
    low = torch.arange(126)
    assert torch.equal(got[127:], torch.where(low % 2 == 0, low, low + 1))


def nearest_code(y, scale):
    """Codes of positive y / scale to the nearest, ties to even, in whole fp64 arithmetic: a border between two codes has at
    most 5 significant bits and a scale 24, so their product and its comparison with y are exact."""
    codes = oracle.e4m3_values()[:127].to(DEV)
    borders = (codes[:-1] + codes[1:]) / 2 * scale.double()
    low = torch.searchsorted(borders, y.double())               # borders below y
    tie = (low < 126) & (borders[low.clamp(max=125)] == y.double())
    return torch.where(tie & (low % 2 == 1), low + 1, low)


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("power", [0, 90, -40, -55, -70, -95, -110])
def test_codes_are_the_nearest_at_any_scale(power, block):
    """Results on the borders between two codes and one step of fp32 beside them, at scales that are no powers of two: with
    rows of ones and a factor of 1 the results are gamma itself, so every code is known exactly."""
    g = torch.Generator().manual_seed(power + 200)
    short = [int(v) * 2 + 1 for v in torch.randint(1 << 7, 1 << 8, (12,), generator=g)]        # scales whose borders are exact
    long = [int(v) * 2 + 1 for v in torch.randint(1 << 22, 1 << 23, (12,), generator=g)]       # and of 24 bits
    codes = oracle.e4m3_values()[:127].to(DEV)
    mids = (codes[:-1] + codes[1:]) / 2
    x = torch.ones(2, 384, device=DEV)
    for m in short + long:
        top = torch.tensor(448.0 * m / 2 ** m.bit_length() * 2.0 ** power, dtype=torch.float64).float()
        top, scale = top.to(DEV), (top / 448).to(DEV)            # fp32's own division, on the CPU
        at = (mids * scale.double()).float()
        rows = torch.stack([at, torch.nextafter(at, top), torch.nextafter(at, -top)]).T.reshape(-1)     # 378 results
        gamma = torch.cat([rows[:127], top[None], rows[127:254], top[None], rows[254:], rows[:3], top[None]])
        y, s, _, rstd = binding.srwm_rmsnorm_forward(x, gamma, eps=2.0 ** -40, out="e4m3", block=block)
        assert (rstd == 1).all() and (s == scale).all(), m
        want = nearest_code(gamma, scale)
        for row in y.view(torch.uint8).long():
            assert torch.equal(row, want), (m, int((row != want).sum()))


def test_residual_stream_in_place():
    x, r, g, _, _ = make(7, 300, 512, BF16)
    y, total, _ = check_forward(x, g, r)
    stream = r.clone()
    y2, _, t2, _ = binding.srwm_rmsnorm_forward(x, g, residual=stream, total=stream)
    assert t2.data_ptr() == stream.data_ptr() and torch.equal(t2, total) and torch.equal(y2, y)


def test_gradients_against_differences():
    x, r, g, dy, _ = make(4, 6, 64, F32)
    total = (x + r)
    dx, dg = check_backward(total, g, dy)
    h = 2.0 ** -8
    for base, grad, at in (([total, g], dx, 0), ([total, g], dg, 1)):
        d = torch.randn(base[at].shape, generator=torch.Generator(device=DEV).manual_seed(at), device=DEV)
        d = d * h / d.norm()
        loss = lambda k: float((binding.srwm_rmsnorm_forward(*[v + k * d if i == at else v for i, v in enumerate(base)])[0].double()  # noqa: E731
                                * dy.double()).sum())
        assert abs((loss(1) - loss(-1)) / 2 - float((grad.double() * d.double()).sum())) <= 0.01 * float(grad.double().norm()) * h + 1e-4


def test_no_rows():
    x, r, g, dy, dt = make(1, 0, 64, F32)
    y, _, total, rstd = binding.srwm_rmsnorm_forward(x, g, residual=r)
    assert y.shape == total.shape == (0, 64) and rstd.shape == (0,)
    y, scale, _, _ = binding.srwm_rmsnorm_forward(x, g, out="e4m3")
    assert y.shape == (0, 64) and scale.shape == (0, 1)
    dx, dg = binding.srwm_rmsnorm_backward(x, g, rstd, dy)
    assert dx.shape == (0, 64) and (dg == 0).all()


def test_same_bits_streams_and_graphs():
    x, r, g, dy, dt = make(2, 3000, 520, BF16)

    def both(**kw):
        y, _, total, rstd = binding.srwm_rmsnorm_forward(x, g, residual=r, **kw)
        return (y, total, rstd, *binding.srwm_rmsnorm_backward(total, g, rstd, dy, dtotal=dt, **kw))

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
        assert all(torch.equal(p, q) for p, q in zip(run, first))


def test_binding_refuses():
    x, r, g, dy, _ = make(1, 4, 64, F32)
    for bad in (dict(x=x.double()), dict(x=x[:, ::2]), dict(gamma=g[:8]), dict(residual=r.half()), dict(out="int8"),
                dict(total=torch.empty_like(x)), dict(scale=torch.empty(4, 1, device=DEV)), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            binding.srwm_rmsnorm_forward(**{**dict(x=x, gamma=g), **bad})
    with pytest.raises(TypeError):
        binding.srwm_rmsnorm_forward(x, g, eps=None)
    for bad in (dict(eps=0.0), dict(block=128), dict(out="e4m3", block=64), dict(out="e4m3", block=128), dict(y=x)):
        with pytest.raises(binding.SrwmError):
            binding.srwm_rmsnorm_forward(**{**dict(x=x, gamma=g), **bad})
    with pytest.raises(binding.SrwmError):
        binding.srwm_rmsnorm_backward(x, g, torch.ones(4, device=DEV), dy, workspace=torch.empty(16, device=DEV, dtype=torch.uint8))


@pytest.mark.parametrize("block", [-1, -128, 128 - 2 ** 32, -2 ** 32, 2 ** 31, 2 ** 32 + 128, 2 ** 63 - 1, -2 ** 63])
def test_binding_refuses_blocks_that_do_not_fit(block):
    """Among them numbers whose lower 32 bits are a block that there is: for it the scales would need more room."""
    x, _, g, _, _ = make(1, 4, 512, F32)
    with pytest.raises(binding.SrwmError):
        binding.srwm_rmsnorm_forward(x, g, out="e4m3", block=block)


def test_8_bits_of_infinite_results():
    """A result past fp32's largest number: its block's scale is infinite, its own code NaN, the block's others 0."""
    x = torch.ones(3, 256, device=DEV)
    x[1] = -1
    gamma = torch.ones(256, device=DEV)
    gamma[200] = float("inf")
    for block, at in ((128, slice(128, 256)), (0, slice(0, 256))):
        y, scale, _, _ = binding.srwm_rmsnorm_forward(x, gamma, out="e4m3", block=block)
        want = torch.zeros(256, device=DEV)
        want[200] = float("nan")
        assert torch.isinf(scale[:, -1]).all()
        assert torch.equal(torch.isnan(y.float())[:, at], torch.isnan(want).expand(3, 256)[:, at])
        assert (torch.nan_to_num(y.float())[:, at] == 0).all()
        if block:
            assert torch.isfinite(scale[:, 0]).all() and (y.float()[:, :128].abs() == 448).all()

"""Group norm with an activation, channels last, on the GPU against float64
(oracle/groupnorm.py).

Tolerances.  A group of m values: its mean and variance are fp32 sums of m
terms in a tree of depth below 64 (runs of at most 32 terms per thread and
log2 steps after), so each is off by at most 64 * 2^-24 of its sum of
magnitudes.  With x = mean + dev, an error of 2^-18 |x|max on the mean moves
xh by that times rstd.  So xh is good to 2^-17 (1 + rstd |x|max) and outputs
take that times |gamma|, and the type's half step of themselves.
"""
import pytest
import torch

from oracle import groupnorm as oracle
from oracle import linattn as la_oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
ACTS = ["none", "silu", "relu"]
# (N, L, C, G): one token's heads; odd sample and position counts; groups of 1, 2, 3 and many channels; one group;
# groups that straddle 16-byte pieces; samples of one position, of a few thousand, and beyond a CTA cluster's memory
SHAPES = [(1, 1, 8, 1), (7, 1, 64, 4), (1001, 1, 128, 4), (333, 1, 512, 8), (65, 1, 1024, 16), (5, 1, 24, 1),
          (3, 2, 16, 8), (13, 5, 24, 8), (4, 49, 40, 5), (9, 441, 64, 16), (2, 1764, 64, 8), (3, 7, 8, 8),
          (2, 33, 96, 32), (1, 7057, 64, 4), (2, 3, 8192, 32), (1, 1, 8192, 1), (17, 1, 4096, 8), (1, 300, 8192, 1),
          (1, 40001, 128, 2), (1, 120001, 64, 1), (600, 9, 256, 32), (50, 25, 72, 3)]


def make(seed, N, L, C, dtype, offset=0.7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = (n(N, L, C) * (0.5 + torch.rand(C, generator=g, device=DEV)) + offset * n(C)).to(dtype)
    return x, 1 + 0.2 * n(C), 0.2 * n(C), n(N, L, C).to(dtype)


def loss_of_stats(x, rstd, G):
    """2^-17 (1 + rstd |x|max) per sample and group, spread to [N, 1, C]."""
    N, L, C = x.shape
    top = x.double().abs().reshape(N, L, G, C // G).amax((1, 3))
    return (2.0 ** -17 * (1 + rstd * top)).repeat_interleave(C // G, 1).unsqueeze(1)


def check_forward(x, gamma, beta, G, act, eps=1e-5):
    N, L, C = x.shape
    y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, G, eps=eps, activation=act)
    ry, rm, rr = oracle.forward(x, gamma, beta, G, eps, act)
    assert y.dtype == x.dtype and torch.isfinite(y.float()).all()
    lost = loss_of_stats(x, rr, G)
    ga = 1.0 if gamma is None else gamma.double().abs()
    be = 0.0 if beta is None else beta.double().abs()
    z = oracle.forward(x, None, None, G, eps, "none")[0].abs()
    tol = 1.1 * lost * ga * (1 + z) + 2.0 ** -20 * be + HALF_STEP[x.dtype] * ry.abs() + 2.0 ** -25   # |act'| <= 1.1
    assert ((y.double() - ry).abs() <= tol).all(), float(((y.double() - ry).abs() - tol).max())
    top = x.double().abs().reshape(N, L, G, C // G).amax((1, 3))
    assert ((mean.double() - rm).abs() <= 2.0 ** -18 * top).all()
    assert ((rstd.double() - rr).abs() <= rr * 2.0 ** -17 * (1 + rr * top)).all()
    return y, mean, rstd


def check_backward(x, gamma, beta, G, act, dy, eps=1e-5):
    """dx = rstd (dh - mean(dh) - xh mean(dh xh)): each of the three terms is
    good to the loss of the statistics relative to its magnitudes; dgamma and
    dbeta are sums of N L terms in runs of at most 2^10 and a tree: 2^10 *
    2^-24 of the sum of magnitudes, besides each term's own error."""
    N, L, C = x.shape
    _, rm, rr = oracle.forward(x, gamma, beta, G, eps, act)
    mean, rstd = rm.float(), rr.float()
    dx, dg, db = binding.srwm_groupnorm_backward(x, gamma, beta, G, mean, rstd, dy, activation=act)
    rdx, rdg, rdb = oracle.grads(x, gamma, beta, G, eps, act, dy)
    if act == "relu":
        # the oracle's own border is at its fp64 statistics, the call's at the fp32 ones it is given: leave no value between
        z = oracle.forward(x, gamma, beta, G, eps, "none")[0]
        m64, r64 = mean.double(), rstd.double()
        zz = ((x.double().reshape(N, L, G, -1) - m64[:, None, :, None]) * r64[:, None, :, None]).reshape(N, L, C)
        zz = zz * (1.0 if gamma is None else gamma.double()) + (0.0 if beta is None else beta.double())
        assert ((z > 0) == (zz > 0)).all(), "the inputs of this test put a value between the two borders"
    xh = oracle.forward(x, None, None, G, eps, "none")[0]
    ga = 1.0 if gamma is None else gamma.double().abs()
    lost = loss_of_stats(x, rr, G)
    dh = 1.1 * dy.double().abs() * ga
    grp = lambda t: t.reshape(N, L, G, -1).mean((1, 3)).repeat_interleave(C // G, 1).unsqueeze(1)  # noqa: E731
    r = rr.repeat_interleave(C // G, 1).unsqueeze(1)
    # SiLU's slope changes by at most 0.5 per unit of z
    size = r * (dh * (1 + ga * (1 + xh.abs())) + grp(dh * (1 + ga)) + xh.abs() * grp(dh * (1 + ga) * (1 + xh.abs())))
    tol = 3 * lost * size + HALF_STEP[x.dtype] * rdx.abs() + 2.0 ** -25
    assert torch.isfinite(dx.float()).all()
    assert ((dx.double() - rdx).abs() <= tol).all(), float(((dx.double() - rdx).abs() - tol).max())
    term = 1.1 * dy.double().abs() * (1 + ga) * (1 + xh.abs()) ** 2
    allow = (2.0 ** -14 * term + lost * term).sum((0, 1)) + 1e-30
    assert ((dg.double() - rdg).abs() <= allow).all() and ((db.double() - rdb).abs() <= allow).all()
    return dx, dg, db


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    N, L, C, G = shape
    x, gamma, beta, _ = make(N + L + C, N, L, C, dtype)
    check_forward(x, gamma, beta, G, ACTS[(N + L + C // 8) % 3])
    check_forward(x, None, beta if N % 2 else None, G, "none")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype):
    N, L, C, G = shape
    x, gamma, beta, dy = make(N + L + C, N, L, C, dtype)
    check_backward(x, gamma, beta, G, "silu", dy)
    check_backward(x, None, None, G, "none", dy)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(200, 1, 128, 4), (6, 81, 48, 6)], ids=str)
def test_activations(shape, act):
    N, L, C, G = shape
    x, gamma, beta, dy = make(5, N, L, C, F32)
    check_forward(x, gamma, beta, G, act)
    check_backward(x, gamma, beta, G, act, dy)


@pytest.mark.parametrize("shape", [(64, 1, 64, 2), (3, 500, 64, 4), (1, 9000, 64, 1), (1, 120001, 64, 2)], ids=str)
def test_mean_far_above_the_spread(shape):
    """A mean 1000 times the deviation: sums of squares would lose the variance."""
    N, L, C, G = shape
    x, gamma, beta, _ = make(9, N, L, C, F32, offset=0.0)
    x = x + 1000.0
    check_forward(x, gamma, beta, G, "none")


def test_equal_values_and_wide_eps():
    """A group of one value throughout: variance 0, y = act(beta) exactly, and finite gradients."""
    x = torch.full((3, 17, 32), 5.0, device=DEV)
    _, gamma, beta, dy = make(3, 3, 17, 32, F32)
    y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, 4, eps=1e-3)
    assert torch.equal(y, beta.expand_as(y)) and (mean == 5).all()
    assert ((rstd.double() - 1e-3 ** -0.5).abs() <= 2.0 ** -20 * 32).all()
    dx, _, _ = binding.srwm_groupnorm_backward(x, gamma, beta, 4, mean, rstd, dy)
    assert torch.isfinite(dx).all()
    check_forward(make(3, 3, 17, 32, BF16)[0], gamma, beta, 4, "silu", eps=0.5)


def test_relu_slope_next_to_its_border():
    """Arguments within a rounding of 0: the side is the exact one's."""
    N, C = 4096, 64
    x, gamma, _, dy = make(12, N, 1, C, F32)
    _, rm, rr = oracle.forward(x, gamma, None, 1, 1e-5, "none")
    mean, rstd = rm.float(), rr.float()
    beta = -((x[0, 0] - mean[0]) * rstd[0] * gamma)                     # sample 0's arguments are all about 1e-8
    z = ((x.double() - mean.double()[:, :, None]) * rstd.double()[:, :, None]) * gamma.double() + beta.double()
    dx, dg, db = binding.srwm_groupnorm_backward(x, gamma, beta, 1, mean, rstd, dy, activation="relu")
    dz = dy.double() * (z > 0)
    xh = (x.double() - mean.double()[:, :, None]) * rstd.double()[:, :, None]
    dh = dz * gamma.double()
    want = rstd.double()[:, :, None] * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    assert ((dx.double() - want).abs() <= 2.0 ** -16 * rstd.double()[:, :, None] * (1 + want.abs().amax())).all()
    assert ((db.double() - dz.sum((0, 1))).abs() <= 2.0 ** -14 * dz.abs().sum((0, 1))).all()


def test_gradients_against_differences():
    """A central difference of the forward pass along a direction, step h: the
    forward's rounding over h, and h^2 times a third derivative of order one
    per value."""
    N, L, C, G, h = 4, 30, 48, 6, 2.0 ** -6
    x, gamma, beta, dy = make(21, N, L, C, F32)
    _, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, G, activation="silu")
    grads = binding.srwm_groupnorm_backward(x, gamma, beta, G, mean, rstd, dy, activation="silu")

    def loss(x, gamma, beta):
        return float((binding.srwm_groupnorm_forward(x, gamma, beta, G, activation="silu")[0].double() * dy.double()).sum())

    base = [x, gamma, beta]
    for i in range(3):
        u = torch.randn_like(base[i])
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * u, base[i] - h * u
        got = (loss(*up) - loss(*dn)) / (2 * h)
        want = float((grads[i].double() * u.double()).sum())
        n = x.numel()
        assert abs(got - want) <= 8 * (2.0 ** -20 / h + h * h) * n ** 0.5 * 4, i


def test_no_samples():
    x, gamma, beta, dy = make(1, 0, 3, 16, F32)
    y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, 4)
    dx, dg, db = binding.srwm_groupnorm_backward(x, gamma, beta, 4, mean, rstd, dy)
    assert y.shape == dx.shape == x.shape and (dg == 0).all() and (db == 0).all()


def test_not_finite_inputs_stay_in_their_group():
    x, gamma, beta, dy = make(8, 6, 50, 32, F32)
    y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, 4)
    x[2, 7, 9] = float("nan")
    x[4, 1, 0] = float("inf")
    y2, _, _ = binding.srwm_groupnorm_forward(x, gamma, beta, 4)
    hit = torch.zeros(6, 32, dtype=torch.bool, device=DEV)
    hit[2, 8:16] = hit[4, 0:8] = True
    hit = hit.unsqueeze(1).expand_as(y)
    assert torch.equal(y[~hit], y2[~hit]) and torch.isnan(y2[hit]).all()


@pytest.mark.parametrize("shape", [(700, 1, 128, 4), (5, 441, 64, 16), (1, 120001, 64, 2)], ids=str)
def test_same_bits_streams_and_graphs(shape):
    N, L, C, G = shape
    x, gamma, beta, dy = make(14, N, L, C, BF16)

    def both(x, gamma, beta, dy):
        y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, G, activation="silu")
        return (y, mean, rstd) + binding.srwm_groupnorm_backward(x, gamma, beta, G, mean, rstd, dy, activation="silu")

    want = both(x, gamma, beta, dy)
    for a, b in zip(want, both(x, gamma, beta, dy)):
        assert torch.equal(a, b)
    ins = [torch.zeros_like(t) for t in (x, gamma, beta, dy)]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both(*ins)
    for a, b in zip(ins, (x, gamma, beta, dy)):
        a.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    N, L, C, G = 5, 1 << 20, 512, 8
    assert N * L * C > 1 << 31
    x = torch.randn(N, L, C, device=DEV, dtype=BF16)
    y, mean, rstd = binding.srwm_groupnorm_forward(x, None, None, G)
    one = x[-1:].contiguous()
    y1, m1, r1 = binding.srwm_groupnorm_forward(one, None, None, G)
    assert ((mean[-1:] - m1).abs() <= 2.0 ** -16).all() and ((rstd[-1:] - r1).abs() <= 2.0 ** -16).all()
    assert ((y[-1:, -1000:].float() - y1[:, -1000:].float()).abs() <= 2.0 ** -7 * (y1[:, -1000:].float().abs() + 0.01)).all()
    dx, _, _ = binding.srwm_groupnorm_backward(x, None, None, G, mean, rstd, x)
    dx1, _, _ = binding.srwm_groupnorm_backward(one, None, None, G, m1, r1, one)
    assert ((dx[-1:, -1000:].float() - dx1[:, -1000:].float()).abs() <= 2.0 ** -6 * (1 + dx1[:, -1000:].float().abs())).all()


def test_binding_refuses():
    x, gamma, beta, dy = make(1, 3, 5, 16, F32)
    f = binding.srwm_groupnorm_forward
    for bad in (lambda: f(x.double(), gamma, beta, 4), lambda: f(x.transpose(0, 1), gamma, beta, 4),
                lambda: f(x, gamma[:8], beta, 4), lambda: f(x, gamma, beta, 4, activation="gelu"),
                lambda: f(x.cpu(), gamma, beta, 4)):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: f(x, gamma, beta, 3), 2), (lambda: f(x, gamma, beta, 4, eps=0.0), 3),
                        (lambda: f(x, gamma, beta, 4, y=x), 5),
                        (lambda: f(x[..., :12].contiguous(), gamma[:12].contiguous(), None, 4), 3)):
        with pytest.raises(binding.SrwmError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_attention_with_its_head_norm(dtype):
    """The two together, as a layer has them: linear attention, then the norm of
    each head's output with SiLU, and back; against autograd in float64.  Each
    operator's own error is bounded in its tests; here the norm of the
    difference is held to the intermediate's and the outputs' half steps with
    their amplification by the norm (of order one), 8 in all, on top of 2^-16."""
    B, T, H, d = 3, 100, 4, 32
    g = torch.Generator(device=DEV).manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v, dz = (n(B, T, H, d).to(dtype) for _ in range(4))
    lg = torch.tensor([-0.02, -0.1, -0.005, -0.5], device=DEV)
    gamma, beta = 1 + 0.2 * n(H * d), 0.2 * n(H * d)
    o, S = binding.srwm_linattn_forward(q, k, v, lg)
    x = o.view(B * T, 1, H * d)
    z, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, H, activation="silu")
    do, dg, db = binding.srwm_groupnorm_backward(x, gamma, beta, H, mean, rstd, dz.view(B * T, 1, H * d), activation="silu")
    grads = binding.srwm_linattn_backward(q, k, v, lg, do.view(B, T, H, d))
    leaves = [t.double().requires_grad_(True) for t in (q, k, v, gamma, beta)]
    ro, _ = la_oracle.forward(*leaves[:3], lg, d ** -0.5)
    rz, _, _ = oracle.forward(ro.reshape(B * T, 1, H * d), leaves[3], leaves[4], H, 1e-5, "silu")
    want = (rz,) + torch.autograd.grad((rz * dz.double().view_as(rz)).sum(), leaves)
    for name, a, b in zip(("z", "dq", "dk", "dv", "dgamma", "dbeta"), (z,) + grads[:3] + (dg, db), want):
        off = float((a.double() - b.detach().view_as(a)).norm() / b.detach().norm())
        assert off <= 8 * HALF_STEP[dtype] + 2.0 ** -16, (name, off)


@pytest.mark.parametrize("shape", [(700, 1, 128, 4), (101, 441, 64, 16), (5, 1764, 64, 8), (3, 40001, 64, 4), (50, 25, 72, 3)],
                         ids=str)
def test_repeats_beside_another_stream_give_the_same_bits(shape):
    N, L, C, G = shape
    sets = [make(s, N, L, C, BF16) for s in (3, 4)]

    def run(x, gamma, beta, dy):
        y, mean, rstd = binding.srwm_groupnorm_forward(x, gamma, beta, G, activation="silu")
        return (y, mean, rstd) + binding.srwm_groupnorm_backward(x, gamma, beta, G, mean, rstd, dy, activation="silu")

    first = [run(*s) for s in sets]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = []
        for s, st in zip(sets, side):
            with torch.cuda.stream(st):
                got.append(run(*s))
        torch.cuda.synchronize()
        for a, b in zip(first, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_relu_border_over_positions():
    """As for rows: one position's arguments within a rounding of 0, groups over positions."""
    N, L, C = 128, 6, 64
    x, gamma, _, dy = make(15, N, L, C, F32)
    _, rm, rr = oracle.forward(x, gamma, None, 1, 1e-5, "none")
    mean, rstd = rm.float(), rr.float()
    beta = -((x[0, 0] - mean[0]) * rstd[0] * gamma)
    wide = [v.double()[:, :, None] for v in (mean, rstd)]
    xh = (x.double() - wide[0]) * wide[1]
    dx, dg, db = binding.srwm_groupnorm_backward(x, gamma, beta, 1, mean, rstd, dy, activation="relu")
    dz = dy.double() * (xh * gamma.double() + beta.double() > 0)
    dh = dz * gamma.double()
    want = wide[1] * (dh - dh.mean((1, 2), keepdim=True) - xh * (dh * xh).mean((1, 2), keepdim=True))
    assert ((dx.double() - want).abs() <= 2.0 ** -16 * wide[1] * (1 + want.abs().amax())).all()
    assert ((db.double() - dz.sum((0, 1))).abs() <= 2.0 ** -14 * dz.abs().sum((0, 1))).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(70000, 1, 64, 2), (9000, 1, 96, 3), (9001, 1, 520, 1), (301, 1, 24, 8), (300, 50, 64, 8),
                                   (1000, 7, 64, 64), (5, 900, 512, 16), (1, 120001, 64, 1), (3, 40000, 256, 8)], ids=str)
def test_parameter_gradients_count_every_position_once(shape, dtype):
    """Whole numbers, mean 0 and rstd 1: every product is at most 32 and every
    partial sum below 2^24, so the sums are exact in any order, and one
    position or range left out or taken twice changes them."""
    N, L, C, G = shape
    assert 32 * N * L < 1 << 24
    g = torch.Generator(device=DEV).manual_seed(N + L)
    x = torch.randint(-4, 5, (N, L, C), generator=g, device=DEV).to(dtype)
    dy = torch.randint(-8, 9, (N, L, C), generator=g, device=DEV).to(dtype)
    mean, rstd = torch.zeros(N, G, device=DEV), torch.ones(N, G, device=DEV)
    _, dg, db = binding.srwm_groupnorm_backward(x, None, None, G, mean, rstd, dy)
    assert torch.equal(db.double(), dy.double().sum((0, 1)))
    assert torch.equal(dg.double(), (dy.double() * x.double()).sum((0, 1)))

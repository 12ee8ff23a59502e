"""Linear attention with a decay per head on the GPU, against its definition
token by token in float64 (oracle/linattn.py).

Tolerances, per entry, with A the same sums over magnitudes (every rounding is
relative to a partial sum, and no partial sum exceeds A):
  * fp32: inputs as fp16 pairs after a power-of-two scaling hold 2^-22 of a
    value, each of the three factors of a term once, dropped low-by-low
    products 2^-22 twice, the intermediate score and state once more each:
    under 8 * 2^-22 = 32 * 2^-24.  fp32 accumulation: at most (d + 64) / 8
    tensor steps inside a chunk and two roundings per chunk on the state, each
    2^-23 (the tensor cores truncate): (d + 64 + 2 * chunks) * 2^-23 covers it.
  * pairs are scaled to the largest value among 16 tokens: a floor of 2^-30 of
    the largest A of the stream covers entries far below their neighbours.
    Where tokens of zeros follow others under a strong decay, A itself falls
    below that: a term g^i x y is an fp16 pair whose scale is set by its 16
    tokens' largest values at the nearest of the 16 positions, and at most 31
    rows away, so its error is up to half the pair's smallest step, 2^-25, of
    2^14: 2^-39 of max|x| max|y| (times d for a score), whatever g^i is.  At
    most 2 * 128 of them meet in a chunk's sums and what older chunks left
    decays no slower than their terms: 2^-31 max|x| max|y| (`floor`).
  * bf16: the score and the state enter their products as one fp16 number,
    2^-11 each, or (d = 64, T >= 128) the score as one bf16, 2^-8 of each term
    and so of A; the output rounds by 2^-8 of itself.  fp16: they enter as
    pairs (as fp32); the output rounds by 2^-11 of itself (half the smallest
    subnormal step, 2^-25, where that is larger).
  * results below fp32's smallest normal number are multiples of 2^-149, so
    each of at most d + T roundings on the way is off by up to 2^-150 whatever
    its size: (d + T) * 2^-149.
States are fp32 for every type and take the fp32 tolerance.
"""
import pytest
import torch

from oracle import linattn as oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def assert_near(got, ref, size, d, T, dtype, what, floor=0.0):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    chunks = -(-T // d)
    tol = (32 * 2.0 ** -24 + (d + 64 + 2 * chunks) * 2.0 ** -23) * size + 2.0 ** -30 * size.amax((-1,), keepdim=True)
    tol = tol + (d + T) * 2.0 ** -149 + floor
    if dtype == BF16:
        score = 2.0 ** -8 if d == 64 and T >= 128 else 2.0 ** -11
        tol = tol + (2.0 ** -11 + score) * size + 2.0 ** -8 * ref.abs()
    elif dtype == F16:
        tol = tol + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    over = ((got - ref).abs() - tol)
    worst = int(over.argmax())
    assert (over <= 0).all(), (f"{what}: off by {float((got - ref).abs().flatten()[worst]):.3e} at flat index {worst}, "
                               f"allowed {float(tol.flatten()[worst]):.3e}")


def make(seed, B, T, H, d, dtype, decay="mixed", packed=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if packed:
        q, k, v = n(B, T, 3, H, d).to(dtype).unbind(2)
    else:
        q, k, v = (n(B, T, H, d).to(dtype) for _ in range(3))
    if decay == "mixed":      # from no memory loss to a loss of most of it per token
        lg = torch.tensor([0.0, -0.01, -0.3, -2.0, -0.001, -7.0, -0.1, -1.0], device=DEV).repeat(-(-H // 8))[:H]
    else:
        lg = torch.full((H,), float(decay), device=DEV)
    return q, k, v, lg.contiguous(), n(B, H, d, d), n(B, T, H, d).to(dtype), n(B, H, d, d)


def check_forward(q, k, v, lg, S0=None, lengths=None, scale=None, **kw):
    B, T, H, d = q.shape
    sc = d ** -0.5 if scale is None else scale
    o, S = binding.srwm_linattn_forward(q, k, v, lg, scale=scale, S_init=S0, lengths=lengths, **kw)
    ro, rS = oracle.forward(q, k, v, lg, sc, S0, lengths)
    clean = [torch.nan_to_num(x.float(), 0.0, 0.0, 0.0) for x in (q, k, v)]
    ao, aS = oracle.sizes(*clean, lg, sc, S0, lengths)
    assert o.dtype == q.dtype and S.dtype == F32
    assert_near(o, ro, ao, d, T, q.dtype, "o")
    assert_near(S, rS, aS, d, T, F32, "S_final")
    return o, S


def check_backward(q, k, v, lg, do, S0=None, lengths=None, dS=None, scale=None, **kw):
    B, T, H, d = q.shape
    sc = d ** -0.5 if scale is None else scale
    got = binding.srwm_linattn_backward(q, k, v, lg, do, scale=scale, S_init=S0, lengths=lengths, dS_final=dS, **kw)
    ref = oracle.grads(q, k, v, lg, sc, do, S0, lengths, dS)
    size = oracle.grad_sizes(*(torch.nan_to_num(x.float(), 0.0, 0.0, 0.0) for x in (q, k, v)), lg, sc,
                             torch.nan_to_num(do.float(), 0.0, 0.0, 0.0), S0, lengths, dS)
    for name, x, r, a, dt in zip(("dq", "dk", "dv", "dS_init"), got, ref, size, (q.dtype,) * 3 + (F32,)):
        assert x.dtype == dt
        assert_near(x, r, a, d, T, dt, name)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 33, 63, 64, 65, 200])
def test_forward_lengths_and_types(T, d, dtype):
    q, k, v, lg, S0, _, _ = make(T + d, 3, T, 5, d, dtype)
    check_forward(q, k, v, lg, S0)
    check_forward(q, k, v, lg)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 17, 64, 65, 130])
def test_backward_lengths_and_types(T, d, dtype):
    q, k, v, lg, S0, do, dS = make(T + d, 3, T, 5, d, dtype)
    check_backward(q, k, v, lg, do, S0, None, dS)
    check_backward(q, k, v, lg, do)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 32, 64])
def test_ragged_batches(d, dtype):
    """Lengths below 0, 0, 1, inside and at the end of a chunk, T and above;
    masked rows hold NaN, infinities and the type's lowest value."""
    T = 150
    lengths = torch.tensor([-4, 0, 1, d - 1, d, d + 1, 2 * d, T - 1, T, T + 9], dtype=torch.int32, device=DEV)
    B = len(lengths)
    q, k, v, lg, S0, do, dS = make(7 + d, B, T, 3, d, dtype)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min], device=DEV).to(dtype)
    rows = (torch.arange(T, device=DEV) >= lengths[:, None].clamp(0, T))
    for i, x in enumerate((q, k, v, do)):
        x[rows] = bad[(torch.arange(3 * d, device=DEV) + i) % 4].view(3, d)
    o, _ = check_forward(q, k, v, lg, S0, lengths)
    assert (o[rows] == 0).all()
    got = check_backward(q, k, v, lg, do, S0, lengths, dS)
    for x in got[:3]:
        assert (x[rows] == 0).all()
    _, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0, lengths=lengths)
    assert torch.equal(S[1], S0[1]) and torch.equal(got[3][1], dS[1])      # the empty sequence passes them on
    _, S = binding.srwm_linattn_forward(q, k, v, lg, lengths=lengths)
    assert (S[:2] == 0).all()


@pytest.mark.parametrize("decay", [0.0, -float("inf"), -1e30, -20.0, -1e-6, 0.5])
@pytest.mark.parametrize("d", [16, 64])
def test_decay_extremes(d, decay):
    """No decay, the current token alone, and values above 0 taken as 0."""
    q, k, v, lg, S0, do, dS = make(3 + d, 2, 100, 3, d, F32, decay)
    check_forward(q, k, v, lg, S0)
    ref = lg.clamp(max=0)
    ref = torch.where(ref < -1000, torch.full_like(ref, -1000.0), ref)     # autograd of exp(-inf) * S is fine, 0 * inf is not
    got = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS)
    want = oracle.grads(q, k, v, ref, d ** -0.5, do, S0, None, dS)
    size = oracle.grad_sizes(q, k, v, ref, d ** -0.5, do, S0, None, dS)
    for name, x, r, a in zip(("dq", "dk", "dv", "dS_init"), got, want, size):
        assert_near(x, r, a, d, 100, F32, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 32, 64])
def test_packed_projection_views(d, dtype):
    """q, k, v as views of one [B,T,3,H,d] array, gradients into views of
    another: bit for bit what contiguous copies give; the rest of the packed
    gradients' array is not touched."""
    B, T, H = 3, 77, 3
    q, k, v, lg, S0, do, dS = make(11 + d, B, T, H, d, dtype, packed=True)
    o, S = check_forward(q, k, v, lg, S0)
    o2, S2 = binding.srwm_linattn_forward(q.contiguous(), k.contiguous(), v.contiguous(), lg, S_init=S0)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    pack = torch.full((B, T, 4, H, d), 7.0, device=DEV, dtype=dtype)
    dq, dk, dv, spare = pack.unbind(2)
    got = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS, dq=dq, dk=dk, dv=dv)
    want = binding.srwm_linattn_backward(q.contiguous(), k.contiguous(), v.contiguous(), lg, do, S_init=S0, dS_final=dS)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (spare == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H,d", [(1, 3000, 1, 64), (2, 2111, 3, 32), (1, 4099, 2, 16), (3, 1500, 8, 64)])
def test_long_sequences_of_few_streams(B, T, H, d, dtype):
    """The long axis split over the GPU and joined, whole and ragged."""
    q, k, v, lg, S0, do, dS = make(T, B, T, H, d, dtype)
    check_forward(q, k, v, lg, S0)
    check_backward(q, k, v, lg, do, S0, None, dS)
    lengths = torch.tensor([T - 700, 1, 900][:B], dtype=torch.int32, device=DEV)
    check_forward(q, k, v, lg, S0, lengths)
    check_backward(q, k, v, lg, do, S0, lengths, dS)


@pytest.mark.parametrize("d", [16, 64])
def test_magnitudes_far_apart(d):
    """Token groups of very different sizes, groups of zeros, large and tiny
    inputs: the scaling to fp16's range loses nothing that fp32 holds."""
    B, T, H = 2, 160, 2
    q, k, v, lg, S0, do, dS = make(23 + d, B, T, H, d, F32)
    e = torch.tensor([0, 4, -5, 9, -12, 2, 0, -3, 6, -8], device=DEV).repeat_interleave(16).float()
    for x, s in ((q, e), (k, e.roll(16)), (v, e.flip(0)), (do, -e)):
        x.mul_((10.0 ** s).view(1, T, 1, 1))
    k[:, 32:64] = 0
    q[:, 96:112] = 0
    check_forward(q, k, v, lg, S0)
    check_backward(q, k, v, lg, do, S0, None, dS)
    z = torch.zeros_like(q)
    check_forward(z, z, z, lg, S0)
    check_forward(q * 1e-18, k * 1e-12, v * 1e-10, lg)


def test_large_16_bit_values():
    """fp16 inputs at the top of the type's range whose states and scores are
    far beyond it; bf16 likewise."""
    q, k, v, lg, _, _, _ = make(5, 2, 70, 2, 32, F16, -0.5)
    check_forward(q * 0.001, k * 1000, v * 8, lg, scale=2.0 ** -10)
    check_forward(*((x.float() * s).to(BF16) for x, s in ((q, 1e-6), (k, 1e15), (v, 1e-4))), lg)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 32, 64])
def test_windows_and_single_tokens_continue_a_prompt(d, dtype):
    """A prompt, a second window from its state, then single tokens."""
    B, T, H = 3, 90, 5
    q, k, v, lg, _, _, _ = make(31 + d, B, T, H, d, dtype)
    ro, rS = oracle.forward(q, k, v, lg, d ** -0.5)
    ao, aS = oracle.sizes(q, k, v, lg, d ** -0.5)
    outs, S = [], None
    for lo, hi in ((0, 40), (40, 81)):
        o, S = binding.srwm_linattn_forward(*(x[:, lo:hi].contiguous() for x in (q, k, v)), lg, S_init=S)
        outs.append(o)
    for t in range(81, T):
        o, S2 = binding.srwm_linattn_step(q[:, t], k[:, t], v[:, t], lg, S, S_out=S)     # in place
        assert S2 is S
        outs.append(o.unsqueeze(1))
    assert_near(torch.cat(outs, 1), ro, ao, d, T, dtype, "o")
    assert_near(S, rS, aS, d, T, F32, "S")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (70, 9)])
def test_step(B, H, d, dtype):
    q, k, v, lg, S0, _, _ = make(B + d, B, 1, H, d, dtype)
    o, S = binding.srwm_linattn_step(q[:, 0], k[:, 0], v[:, 0], lg, S0, scale=0.7)
    ro, rS = oracle.forward(q, k, v, lg, 0.7, S0)
    ao, aS = oracle.sizes(q, k, v, lg, 0.7, S0)
    assert_near(o.unsqueeze(1), ro, ao, d, 1, dtype, "o")
    assert_near(S, rS, aS, d, 1, F32, "S_out")
    packed = torch.stack((q[:, 0], k[:, 0], v[:, 0]), 1)                       # [B, 3, H, d]
    o2, S2 = binding.srwm_linattn_step(*packed.unbind(1), lg, S0, scale=0.7)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    binding.srwm_linattn_step(q[:, 0], k[:, 0], v[:, 0], lg, S0, scale=0.7, S_out=S0)
    assert torch.equal(S0, S)


def test_gradients_against_differences():
    """o is linear in each of q, k, v and S_init alone, so a central difference
    along a direction is exact but for roundings: outputs of sum of squares n
    rounded by 2^-20 of their sizes change L by a small multiple of 2^-20
    |do| |o|, over the step 2h = 2."""
    B, T, H, d = 2, 75, 3, 32
    q, k, v, lg, S0, do, dS = make(41, B, T, H, d, F32)
    grads = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS)

    def loss(*x):
        o, S = binding.srwm_linattn_forward(*x[:3], lg, S_init=x[3])
        return (o.double() * do.double()).sum() + (S.double() * dS.double()).sum(), \
            o.double().norm() * do.double().norm() + S.double().norm() * dS.double().norm()

    base = [q, k, v, S0]
    for i in range(4):
        u = torch.randn_like(base[i])
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + u, base[i] - u
        (lu, su), (ld, _) = loss(*up), loss(*dn)
        want = float((grads[i].double() * u.double()).sum())
        assert abs(float(lu - ld) / 2 - want) <= 2.0 ** -18 * float(su), ("q", "k", "v", "S_init")[i]


def test_zero_tokens():
    q, k, v, lg, S0, do, dS = make(2, 3, 0, 2, 16, BF16)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    assert o.shape == q.shape and torch.equal(S, S0)
    _, S = binding.srwm_linattn_forward(q, k, v, lg)
    assert (S == 0).all()
    *_, d0 = binding.srwm_linattn_backward(q, k, v, lg, do, dS_final=dS)
    assert torch.equal(d0, dS)


def test_not_finite_inputs_stay_in_their_stream():
    q, k, v, lg, S0, do, _ = make(13, 3, 100, 4, 32, F32)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    k[1, 70, 2, 5] = float("nan")
    v[2, 50, 0, 3] = float("inf")
    o2, S2 = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    touched = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    touched[1, 2] = touched[2, 0] = True
    assert torch.equal(S[~touched], S2[~touched])
    assert torch.equal(o.transpose(1, 2)[~touched], o2.transpose(1, 2)[~touched])
    assert not torch.isfinite(S2[1, 2]).all() and not torch.isfinite(S2[2, 0]).all()
    assert torch.equal(o[1, :64, 2], o2[1, :64, 2]) and torch.equal(o[2, :32, 0], o2[2, :32, 0])   # the chunks before
    assert torch.isnan(o2[1, 70:, 2]).any(-1).all()


@pytest.mark.parametrize("B,T", [(5, 90), (1, 2500)])
def test_same_bits_streams_and_graphs(B, T):
    """The same call gives the same bits, on another stream and replayed from a
    graph with new inputs; two graphs with workspaces of their own, replayed on
    two streams at once, do not disturb each other."""
    H, d = 3, 64
    q, k, v, lg, S0, do, dS = make(17, B, T, H, d, BF16)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    grads = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, S2 = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)

    def graph(seed):
        ins = list(make(seed, B, T, H, d, BF16))
        outs = [torch.empty_like(o), torch.empty_like(S)] + [torch.empty_like(x) for x in grads]
        ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in
              (binding.srwm_linattn_workspace_bytes(B, T, H, d), binding.srwm_linattn_backward_workspace_bytes(B, T, H, d))]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q1, k1, v1, lg1, S1, do1, dS1 = ins
            binding.srwm_linattn_forward(q1, k1, v1, lg1, S_init=S1, o=outs[0], S_final=outs[1], workspace=ws[0])
            binding.srwm_linattn_backward(q1, k1, v1, lg1, do1, S_init=S1, dS_final=dS1, dq=outs[2], dk=outs[3],
                                          dv=outs[4], dS_init=outs[5], workspace=ws[1])
        return g, ins, outs, ws

    g1, in1, out1, w1 = graph(18)
    g2, in2, out2, w2 = graph(19)
    for x, y in zip(in1, (q, k, v, lg, S0, do, dS)):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            g2.replay()
    for _ in range(3):
        g1.replay()
    torch.cuda.synchronize()
    for x, y in zip(out1, (o, S) + tuple(grads)):
        assert torch.equal(x, y)
    q2, k2, v2, lg2, S2, do2, dS2 = in2
    want = binding.srwm_linattn_forward(q2, k2, v2, lg2, S_init=S2) + \
        binding.srwm_linattn_backward(q2, k2, v2, lg2, do2, S_init=S2, dS_final=dS2)
    for x, y in zip(out2, want):
        assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """More than 2^31 elements per tensor: the last sequence against a call of its own."""
    B, T, H, d = 33, 1 << 17, 8, 64
    assert B * T * H * d > 1 << 31
    q = torch.randn(B, T, H, d, device=DEV, dtype=BF16)
    lg = make(1, 1, 1, H, d, BF16)[3]
    o, S = binding.srwm_linattn_forward(q, q, q, lg)
    one = q[-1:].contiguous()
    o1, S1 = binding.srwm_linattn_forward(one, one, one, lg)
    size = S1.abs().amax((-1, -2), keepdim=True)
    # the two split the axis differently: fp32 sums of T positive squares, in other orders
    assert ((S[-1:] - S1).abs() <= 2.0 ** -12 * size).all()
    err = (o[-1:].double() - o1.double()).abs()
    assert (err <= 2.0 ** -7 * o1.double().abs().amax((-1,), keepdim=True)).all()
    del o, S
    dq, dk, dv, d0 = binding.srwm_linattn_backward(q, q, q, lg, q)
    e = binding.srwm_linattn_backward(one, one, one, lg, one)
    for a, b in zip((dq, dk, dv), e):
        assert ((a[-1:].double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs().amax((-1,), keepdim=True)).all()


def test_binding_refuses():
    q, k, v, lg, S0, do, dS = make(1, 2, 8, 3, 16, F32)
    f = binding.srwm_linattn_forward
    for bad in (lambda: f(q, k, v.to(BF16), lg), lambda: f(q.double(), k.double(), v.double(), lg),
                lambda: f(q, k[:, :4], v, lg), lambda: f(q, k, v, lg[:2]), lambda: f(q, k, v, lg, S_init=S0.to(BF16)),
                lambda: f(q, k, v, lg, lengths=torch.tensor([1, 2], device=DEV)),
                lambda: f(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, lg),
                lambda: f(q.cpu(), k.cpu(), v.cpu(), lg),
                lambda: binding.srwm_linattn_backward(q, k, v, lg, do, dq=torch.empty_like(q))):
        with pytest.raises(ValueError):
            bad()
    q48 = torch.randn(2, 8, 3, 48, device=DEV)
    for bad, status in ((lambda: f(q48, q48, q48, lg), 3),
                        (lambda: f(q, k, v, lg, o=q), 5),
                        (lambda: f(q, k, v, lg, S_init=S0, S_final=S0), 5),
                        (lambda: f(q, k, v, lg, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), 2)):
        with pytest.raises(binding.SrwmError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T", [127, 128, 129, 255, 256, 257, 390])
def test_lengths_around_wide_chunks(T, dtype):
    """d = 64 around multiples of 128 tokens, views of packed arrays."""
    q, k, v, lg, S0, do, dS = make(T, 2, T, 3, 64, dtype, packed=True)
    check_forward(q, k, v, lg, S0)
    check_backward(q, k, v, lg, do, S0, None, dS)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_streams_than_the_gpu_holds(dtype):
    """Several streams for each CTA, their lengths from nothing to T, masked
    rows NaN."""
    T, lens = 300, [0, 300, 1, 128, 0, -3, 127, 129, 256, 299, 300, 17, 0, 257, 255, 64]
    lengths = torch.tensor(lens * 3, dtype=torch.int32, device=DEV)
    B = len(lengths)
    q, k, v, lg, S0, do, dS = make(3, B, T, 9, 64, dtype)
    rows = torch.arange(T, device=DEV) >= lengths[:, None]
    for x in (q, k, v, do):
        x[rows] = float("nan")
    o, _ = check_forward(q, k, v, lg, S0, lengths)
    assert (o[rows] == 0).all()
    for x in check_backward(q, k, v, lg, do, S0, lengths, dS)[:3]:
        assert (x[rows] == 0).all()
    check_forward(q, k, v, lg, None, lengths)
    for x in (q, k, v, do):
        x[rows] = 0
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)      # all T tokens, zeros among them
    sc = 64 ** -0.5
    (ro, rS), (ao, aS) = oracle.forward(q, k, v, lg, sc, S0), oracle.sizes(q, k, v, lg, sc, S0)
    top = [float(x.abs().max()) for x in (q, k, v, do)]
    assert_near(o, ro, ao, 64, T, dtype, "o", 2.0 ** -31 * sc * 64 * top[0] * top[1] * top[2])
    assert_near(S, rS, aS, 64, T, F32, "S_final", 2.0 ** -31 * top[1] * top[2])
    got = binding.srwm_linattn_backward(q, k, v, lg, do)
    ref, size = oracle.grads(q, k, v, lg, sc, do), oracle.grad_sizes(q, k, v, lg, sc, do)
    for name, x, r, a, i in zip(("dq", "dk", "dv"), got, ref, size, range(3)):
        floor = 2.0 ** -31 * sc * 64 * top[0] * top[1] * top[2] * top[3] / top[i]
        assert_near(x, r, a, 64, T, dtype, name, floor)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
def test_padding_stays_zero_beside_values_that_are_not_finite(d, dtype):
    T = 300
    lengths = torch.tensor([290, 130, 5], dtype=torch.int32, device=DEV)
    q, k, v, lg, S0, do, dS = make(29 + d, 3, T, 2, d, dtype)
    for x, t in ((k, 3), (v, 4), (do, 2)):
        x[:, t, 0, 5] = float("inf")
        x[:, t, 1, 5] = float("nan")
    rows = torch.arange(T, device=DEV) >= lengths[:, None]
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0, lengths=lengths)
    assert (o[rows] == 0).all() and not torch.isfinite(S).flatten(2).all(-1).any()
    for x in binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, lengths=lengths, dS_final=dS)[:3]:
        assert (x[rows] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [100, 300])
def test_not_finite_inputs_stay_in_their_stream_at_width_64(T, dtype):
    q, k, v, lg, S0, _, _ = make(14, 60, T, 4, 64, dtype)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    k[1, T - 10, 2, 5] = float("nan")
    v[2, 50, 0, 3] = float("inf")
    o2, S2 = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    touched = torch.zeros(60, 4, dtype=torch.bool, device=DEV)
    touched[1, 2] = touched[2, 0] = True
    assert torch.equal(S[~touched], S2[~touched])
    assert torch.equal(o.transpose(1, 2)[~touched], o2.transpose(1, 2)[~touched])
    assert not torch.isfinite(S2[1, 2]).all() and not torch.isfinite(S2[2, 0]).all()
    before = (T - 10) // 128 * 128 if T >= 128 else (T - 10) // 64 * 64
    assert torch.equal(o[1, :before, 2], o2[1, :before, 2])
    assert torch.isnan(o2[1, T - 10:, 2]).any(-1).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 64])
def test_a_decay_that_is_nan_is_not_hidden(d, dtype):
    q, k, v, lg, S0, _, _ = make(6, 2, 200, 3, d, dtype)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    o1, S1 = binding.srwm_linattn_step(q[:, 0], k[:, 0], v[:, 0], lg, S0)
    lg[1] = float("nan")
    o2, S2 = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0)
    o3, S3 = binding.srwm_linattn_step(q[:, 0], k[:, 0], v[:, 0], lg, S0)
    for x in (S2, S3, o2.transpose(1, 2), o3):
        assert torch.isnan(x[:, 1]).all()
    for x, y in ((S, S2), (S1, S3), (o.transpose(1, 2), o2.transpose(1, 2)), (o1, o3)):
        assert torch.equal(x[:, ::2], y[:, ::2])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams_at_once(dtype):
    """Calls that run beside one another on two CUDA streams give what each
    gives alone, and no wait runs out."""
    sets = [make(s, 60, 400, 4, 64, dtype) for s in (50, 51)]
    alone = [binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS) for q, k, v, lg, S0, do, dS in sets]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in sets]
    both = [[], []]
    for _ in range(4):
        for i, (q, k, v, lg, S0, do, dS) in enumerate(sets):
            with torch.cuda.stream(side[i]):
                both[i] = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, dS_final=dS)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert binding.srwm_last_device_status() == 0


def test_first_call_inside_a_capture():
    """A process whose first calls are captured into a graph."""
    code = """
import torch
from self_referential_weight_gb300 import binding
q = torch.randn(2, 200, 3, 64, device="cuda")
lg = torch.full((3,), -0.1, device="cuda")
x = [t for dt in (torch.float32, torch.bfloat16) for t in (q.to(dt),)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = [binding.srwm_linattn_forward(t, t, t, lg)[0] for t in x]
g.replay()
torch.cuda.synchronize()
want = [binding.srwm_linattn_forward(t, t, t, lg)[0] for t in x]
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""
    import pathlib
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], cwd=pathlib.Path(__file__).parent.parent, capture_output=True, text=True,
                       timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 32, 64])
def test_repeats_give_the_same_bits(d, dtype):
    """Ragged batches of more streams than the GPU holds, where the kernels'
    warps meet in changing orders."""
    T, lens = 300, [0, 300, 1, 128, 0, 257, 127, 129, 256, 299, 300, 17, 0, 257, 255, 64]
    lengths = torch.tensor(lens * 5, dtype=torch.int32, device=DEV)
    q, k, v, lg, S0, do, dS = make(71, len(lengths), T, 9, d, dtype)

    def run():
        return binding.srwm_linattn_forward(q, k, v, lg, S_init=S0, lengths=lengths) + \
            binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, lengths=lengths, dS_final=dS)

    first = run()
    for _ in range(25):
        assert all(torch.equal(x, y) for x, y in zip(first, run()))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T,B,H", [(3, 2, 3), (8, 1, 1), (9, 401, 5), (17, 331, 7), (19, 601, 3), (27, 301, 7), (40, 303, 5)])
def test_short_sequences(T, B, H, d, dtype):
    """Few and many streams of a few tokens, whole and ragged, views of packed arrays."""
    q, k, v, lg, S0, do, dS = make(T + d, B, T, H, d, dtype, packed=True)
    check_forward(q, k, v, lg, S0)
    check_backward(q, k, v, lg, do, S0, None, dS)
    lengths = (torch.arange(B, device=DEV) * 7 % (T + 3) - 1).int()
    rows = torch.arange(T, device=DEV) >= lengths[:, None]
    for x in (q, k, v, do):
        x[rows] = float("nan")
    o, _ = check_forward(q, k, v, lg, None, lengths, scale=-0.3)
    assert (o[rows] == 0).all()
    for x in check_backward(q, k, v, lg, do, None, lengths, scale=-0.3)[:3]:
        assert (x[rows] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,d", [(128, 16), (255, 32), (449, 64), (1201, 64)])
def test_a_few_streams_of_some_hundred_tokens(T, d, dtype):
    """The shortest axes that are split, whole and with lengths that end inside, at and before a segment."""
    q, k, v, lg, S0, do, dS = make(T + d, 4, T, 1, d, dtype)
    check_forward(q, k, v, lg, S0)
    check_backward(q, k, v, lg, do, S0, None, dS)
    lengths = torch.tensor([T // 2, 0, T - 1, 2 * d], dtype=torch.int32, device=DEV)
    check_forward(q, k, v, lg, S0, lengths)
    check_backward(q, k, v, lg, do, S0, lengths, dS)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("decay", [0.0, -0.3])
@pytest.mark.parametrize("by", [10, 15])
@pytest.mark.parametrize("at", [16, 112, 176])
def test_later_tokens_do_not_cost_earlier_ones_their_bits(at, by, decay, dtype):
    """Sixteen tokens far above their neighbours, which do not see them: in
    order tokens at .. at + 15 for the sixteen before, in reverse at - 16 ..
    at - 1 for the sixteen behind.  No state, so that those rows stay small;
    each row's tolerance is that of the tokens it sees."""
    T, d = 200, 64
    q, k, v, lg, _, do, _ = make(at + by, 2, T, 3, d, dtype, decay)
    if dtype == F16:
        by //= 3      # values and outputs stay below 65504
    big = torch.ones(T, 1, 1, device=DEV)
    big[at:at + 16] = 2.0 ** by
    check_forward(q, (k.float() * big).to(dtype), (v.float() * big).to(dtype), lg)
    dq = binding.srwm_linattn_backward(q, (k.float() * big).to(dtype), (v.float() * big).to(dtype), lg, do)[0]
    args = (q, (k.float() * big).to(dtype), (v.float() * big).to(dtype), lg, d ** -0.5, do)
    assert_near(dq, oracle.grads(*args)[0], oracle.grad_sizes(*args)[0], d, T, dtype, "dq")
    big = torch.ones(T, 1, 1, device=DEV)
    big[at - 16:at] = 2.0 ** by
    args = ((q.float() * big).to(dtype), k, v, lg, d ** -0.5, (do.float() * big).to(dtype))
    got = binding.srwm_linattn_backward(args[0], k, v, lg, args[5])
    for name, x, r, a in list(zip(("dq", "dk", "dv"), got, oracle.grads(*args), oracle.grad_sizes(*args)))[1:]:
        assert_near(x, r, a, d, T, dtype, name)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T", [8, 26, 100, 300, 1201])
def test_an_empty_sequence_passes_its_state_on_whatever_the_decay(T, d, dtype):
    """No token, no decay: also of a head whose decay is NaN, beside sequences that have tokens."""
    q, k, v, lg, S0, do, dS = make(T + d, 3, T, 3, d, dtype)
    lg[1] = float("nan")
    lengths = torch.tensor([T, 0, (T + 1) // 2], dtype=torch.int32, device=DEV)
    o, S = binding.srwm_linattn_forward(q, k, v, lg, S_init=S0, lengths=lengths)
    got = binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, lengths=lengths, dS_final=dS)
    assert torch.equal(S[1], S0[1]) and torch.equal(got[3][1], dS[1])
    assert all((x[1] == 0).all() for x in (o,) + tuple(got[:3]))
    assert torch.isnan(S[::2, 1]).all() and torch.isnan(got[3][::2, 1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 8, 26, 100, 200])
def test_gradients_under_a_decay_that_is_nan(T, d, dtype):
    """All of that head's gradients are NaN, whichever kernel a length takes;
    the other heads' are as they were."""
    q, k, v, lg, S0, do, dS = make(T + d, 3, T, 3, d, dtype)
    lengths = torch.tensor([T, 1, (T + 1) // 2], dtype=torch.int32, device=DEV)
    run = lambda: binding.srwm_linattn_backward(q, k, v, lg, do, S_init=S0, lengths=lengths, dS_final=dS)  # noqa: E731
    was = run()
    lg[1] = float("nan")
    got = run()
    for b, n in enumerate(lengths.tolist()):
        for x in got[:3]:
            assert torch.isnan(x[b, :n, 1]).all() and (x[b, n:, 1] == 0).all()
        assert torch.isnan(got[3][b, 1]).all()
    for x, y in zip(got, was):
        heads = (lambda t: t[:, ::2]) if x is got[3] else (lambda t: t[:, :, ::2])
        assert torch.equal(heads(x), heads(y))


@pytest.mark.parametrize("T", [128, 200, 390])
def test_scores_of_wide_chunks_keep_their_bits(T):
    """bf16, d = 64, T >= 128: the score and the state enter their products as
    pairs of bf16, off by half a step of a half step, 2^-16 each; sums and
    weighted rows as in fp32 (see above); the output rounds by 2^-8 of itself."""
    d, q, k, v, lg, S0, do, dS = 64, *make(T, 3, T, 5, 64, BF16)
    tol = 2 * 2.0 ** -16 + (d + 64 + 2 * -(-T // d)) * 2.0 ** -23 + 32 * 2.0 ** -24

    def near(x, ref, size):
        room = (1 + 2.0 ** -7) * tol * size + 2.0 ** -8 * ref.abs() + (d + T) * 2.0 ** -133
        assert ((x.double() - ref).abs() <= room).all(), float(((x.double() - ref).abs() / room).max())

    for S, D in ((S0, dS), (None, None)):
        args = (q, k, v, lg, d ** -0.5)
        near(binding.srwm_linattn_forward(*args[:4], S_init=S)[0], oracle.forward(*args, S)[0],
             oracle.sizes(*(x.float() for x in args[:3]), *args[3:], S)[0])
        got = binding.srwm_linattn_backward(*args[:4], do, S_init=S, dS_final=D)
        for x, r, a in list(zip(got, oracle.grads(*args, do, S, None, D), oracle.grad_sizes(*args, do, S, None, D)))[:3]:
            near(x, r, a)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_values_in_wide_chunks(dtype):
    """d = 64, T >= 128: scores and states far from 1, in fp32's range."""
    q, k, v, lg, S0, do, dS = make(5, 2, 200, 2, 64, dtype, -0.5)
    for a, b, c in ((1e-6, 1e15, 1e-4), (1e12, 1e-3, 1e8), (1e-12, 1e-9, 1e5)):
        check_forward(*((x.float() * s).to(dtype) for x, s in ((q, a), (k, b), (v, c))), lg)
        check_backward(*((x.float() * s).to(dtype) for x, s in ((q, a), (k, b), (v, c))), lg, (do.float() / a).to(dtype))

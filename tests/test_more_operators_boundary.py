"""Host-only checks of the short convolution, selective scan and RMS norm entry
points (no GPU needed): bad arguments are refused before CUDA is touched; and
their oracles' pins: gradients against differences, closed forms."""
import ctypes

import pytest
import torch

from oracle import conv as conv_oracle
from oracle import rmsnorm as norm_oracle
from oracle import ssm as ssm_oracle
from self_referential_weight_gb300 import binding
from self_referential_weight_gb300 import build as lib_build

A = 0x100000  # fake, 16-byte aligned "device" addresses: never dereferenced
M = 0x1000000
BIG = 1 << 40
ARGUMENTS = (1, 2, 3, 4, 5)   # the statuses of refused arguments


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(lib_build.build())
    P, I, LL, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    L.srwm_conv_forward.argtypes = [P, LL, P, P, P, P, I, I, I, I, I, I, P, P, P]
    L.srwm_conv_step.argtypes = [P, LL, P, P, P, I, I, I, I, I, P, P, P]
    L.srwm_conv_backward.argtypes = [P, LL, P, P, P, P, I, I, I, I, I, I, P, P, P, LL, P, P, P, P, SZ, P]
    L.srwm_conv_backward_workspace_bytes.argtypes, L.srwm_conv_backward_workspace_bytes.restype = [I] * 4, SZ
    L.srwm_ssm_forward.argtypes = [P, LL, P, LL, P, P, P, LL, P, P, LL, P, I, P, P, I, I, I, I, I, I, P, P, P, SZ, P]
    L.srwm_ssm_step.argtypes = [P, LL, P, LL, P, P, P, LL, P, P, LL, P, I, P, I, I, I, I, I, P, P, P]
    L.srwm_ssm_backward.argtypes = ([P, LL, P, LL, P, P, P, LL, P, P, LL, P, I, P, P, I, I, I, I, I, I] +
                                    [P, P, P, P, P, P, P, LL, P, P, LL, P, P, P, SZ, P])
    for n in ("srwm_ssm_workspace_bytes", "srwm_ssm_backward_workspace_bytes"):
        getattr(L, n).argtypes, getattr(L, n).restype = [I] * 5, SZ
    L.srwm_rmsnorm_forward.argtypes = [P, P, P, I, LL, I, F, I, I, P, P, P, P, P]
    L.srwm_rmsnorm_backward.argtypes = [P, P, P, P, P, I, LL, I, P, P, P, SZ, P]
    L.srwm_rmsnorm_backward_workspace_bytes.argtypes, L.srwm_rmsnorm_backward_workspace_bytes.restype = [LL, I], SZ
    return L


def caller(f, base):
    return lambda **kw: f(*dict(base, **kw).values(), None)


def test_conv_refuses(lib):
    f = caller(lib.srwm_conv_forward, dict(x=A, ld=16, w=A + M, b=A + 2 * M, s=None, n=None, dt=0, B=2, T=5, D=16, W=4, act=1,
                                           y=A + 3 * M, so=A + 4 * M))
    s = caller(lib.srwm_conv_step, dict(x=A, ld=16, w=A + M, b=A + 2 * M, s=A + 5 * M, dt=0, B=2, D=16, W=4, act=1, y=A + 3 * M,
                                        so=A + 4 * M))
    g = caller(lib.srwm_conv_backward, dict(x=A, ld=16, w=A + M, b=A + 2 * M, s=None, n=None, dt=0, B=2, T=5, D=16, W=4, act=1,
                                            dy=A + 3 * M, ds=None, dx=A + 4 * M, ldg=16, dw=A + 5 * M, db=A + 6 * M, d0=None,
                                            ws=A + 7 * M, wb=BIG))
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1
    assert s(x=None) == 1 and s(s=None) == 1 and s(so=None) == 1
    assert g(dy=None) == 1 and g(dx=None) == 1 and g(ws=None) == 1
    for call in (f, s, g):
        assert call(B=0) == 2 and call(D=0) == 2 and call(B=1 << 29, D=1 << 20) == 2
        assert call(D=12) == 3 and call(W=1) == 3 and call(W=5) == 3 and call(act=2) == 3 and call(dt=3) == 3
        assert call(ld=8) == 2 and call(ld=18) == 2 and call(x=A + 4) == 4 and call(w=A + M + 8) == 4
    assert f(D=1 << 25, ld=1 << 25) == 2 and f(T=-1) == 2 and f(n=A + 5 * M + 2) == 4 and f(B=1 << 10, T=1 << 29, D=1 << 10, ld=1 << 10) == 2
    assert f(y=A) == 5 and f(so=A + 3 * M + 64) == 5 and f(y=A + 16, ld=64) == 5 and f(s=A + 4 * M) == 5
    assert s(so=A + 5 * M + 16) == 5 and s(y=A) == 5 and s(so=A + 5 * M) not in ARGUMENTS   # exactly in place
    assert g(ldg=8) == 2 and g(wb=16) == 2 and g(dx=A) == 5 and g(db=A + 5 * M) == 5 and g(ws=A + 4 * M) == 5
    # a slice beside x's in one packed array interleaves without overlap; half over it does not
    assert g(ld=32, dx=A + 64, ldg=32) not in ARGUMENTS and g(ld=32, dx=A + 32, ldg=32) == 5
    assert lib.srwm_conv_backward_workspace_bytes(2, 5, 16, 4) > 0 and lib.srwm_conv_backward_workspace_bytes(2, 5, 16, 5) == 0


def test_ssm_refuses(lib):
    inputs = dict(u=A, ldu=16, dt=A + M, ldt=16, A=A + 2 * M, B=A + 3 * M, C=A + 4 * M, ldb=16, skip=A + 5 * M, z=A + 6 * M, ldz=16,
                  bias=A + 7 * M, sp=1)
    sizes = dict(ty=0, nb=2, T=5, D=16, N=16, G=1)
    one = {k: v for k, v in sizes.items() if k != "T"}
    f = caller(lib.srwm_ssm_forward, dict(inputs, h0=None, n=None, **sizes, y=A + 8 * M, h=A + 9 * M, ws=A + 10 * M, wb=BIG))
    s = caller(lib.srwm_ssm_step, dict(inputs, h0=A + 11 * M, **one, y=A + 8 * M, h=A + 9 * M))
    g = caller(lib.srwm_ssm_backward, dict(inputs, h0=None, n=None, **sizes, dy=A + 8 * M, dh=None, du=A + 9 * M, ddt=A + 10 * M,
                                           dA=A + 11 * M, dB=A + 12 * M, dC=A + 13 * M, ldg=16, dsk=None, dz=A + 14 * M, ldgz=16,
                                           dbi=None, d0=None, ws=A + 15 * M, wb=BIG))
    for call in (f, s, g):
        for p in ("u", "dt", "A", "B", "C"):
            assert call(**{p: None}) == 1, p
            assert call(**{p: A + 20 * M + 8}) == 4, p
        assert call(nb=0) == 2 and call(D=0) == 2 and call(N=0) == 2 and call(G=0) == 2 and call(G=3) == 2
        assert call(nb=1 << 20, D=1 << 12, ldu=1 << 12, ldt=1 << 12, ldz=1 << 12) == 2
        assert call(N=8, ldb=16) == 3 and call(N=48, ldb=48) == 3 and call(N=128, ldb=128) == 3 and call(ty=3) == 3
        assert call(D=12) == 3 and call(G=4, ldb=64) == 3 and call(sp=2) == 3
        assert call(ldu=8) == 2 and call(ldt=18) == 2 and call(ldz=8) == 2 and call(ldb=8) == 2 and call(N=32) == 2
    assert f(y=None) == 1 and f(ws=None) == 1 and f(T=-1) == 2 and f(wb=16) == 2 and f(n=A + 20 * M + 2) == 4
    assert f(y=A) == 5 and f(y=A + 6 * M) == 5 and f(h=A + 8 * M + 64) == 5 and f(ws=A + 3 * M) == 5 and f(h0=A + 9 * M) == 5
    assert s(h0=None) == 1 and s(h=None) == 1 and s(y=A + M) == 5 and s(h=A + 11 * M + 16) == 5
    assert s(h=A + 11 * M) not in ARGUMENTS
    for p in ("dy", "du", "ddt", "dA", "dB", "dC", "dz", "ws"):
        assert g(**{p: None}) == 1, p
    assert g(z=None, dz=None) not in ARGUMENTS and g(ldg=8) == 2 and g(ldgz=8) == 2 and g(wb=16) == 2
    assert g(du=A) == 5 and g(ddt=A + 9 * M) == 5 and g(dB=A + 13 * M) == 5 and g(dz=A + 8 * M) == 5 and g(dA=A + 15 * M) == 5
    pack = dict(dB=A + 12 * M, dC=A + 12 * M + 64, ldg=32)
    assert g(**pack) not in ARGUMENTS and g(**dict(pack, dC=A + 12 * M + 32)) == 5
    assert lib.srwm_ssm_workspace_bytes(2, 5, 16, 16, 1) > 0 and lib.srwm_ssm_workspace_bytes(2, 5, 16, 16, 4) == 0
    assert lib.srwm_ssm_backward_workspace_bytes(2, 5, 16, 8, 1) == 0 and lib.srwm_ssm_backward_workspace_bytes(2, 5, 16, 64, 2) > 0


def test_rmsnorm_refuses(lib):
    f = caller(lib.srwm_rmsnorm_forward, dict(x=A, r=A + M, g=A + 2 * M, dt=1, N=4, C=256, eps=1e-5, out=1, block=128, y=A + 3 * M,
                                              s=A + 4 * M, t=A + 5 * M, rs=A + 6 * M))
    g = caller(lib.srwm_rmsnorm_backward, dict(t=A, g=A + M, rs=A + 2 * M, dy=A + 3 * M, dt_=None, ty=1, N=4, C=256, dx=A + 4 * M,
                                               dg=A + 5 * M, ws=A + 6 * M, wb=BIG))
    assert f(x=None) == 1 and f(y=None) == 1 and f(s=None) == 1 and f(s=None, out=0, block=0) not in ARGUMENTS
    assert f(N=-1) == 2 and f(C=0) == 2 and f(N=1 << 31) == 2 and f(C=200) == 2
    assert f(C=12) == 3 and f(C=16384) == 3 and f(dt=3) == 3 and f(eps=0.0) == 3 and f(eps=float("nan")) == 3
    assert f(out=2) == 3 and f(block=64) == 3 and f(out=0) == 3 and f(r=A + M + 8) == 4
    assert f(y=A) == 5 and f(t=A) == 5 and f(t=A + M + 16) == 5 and f(rs=A + 4 * M) == 5 and f(s=A + 2 * M) == 5
    assert f(t=A + M) not in ARGUMENTS        # the residual stream in place
    for p in ("t", "rs", "dy", "dx", "ws"):
        assert g(**{p: None}) == 1, p
    assert g(N=-1) == 2 and g(wb=16) == 2 and g(C=12) == 3 and g(ty=7) == 3 and g(dy=A + 3 * M + 4) == 4
    assert g(dx=A) == 5 and g(dx=A + 3 * M) == 5 and g(dg=A + M) == 5 and g(ws=A + 4 * M) == 5
    assert lib.srwm_rmsnorm_backward_workspace_bytes(4, 256) > 0 and lib.srwm_rmsnorm_backward_workspace_bytes(4, 20) == 0


@pytest.mark.parametrize("B,T,D,N,G", [
    (65536, 26, 256, 16, 1), (1 << 20, 8, 1024, 16, 1), (65536, 16, 1024, 64, 1), (4096, 26, 1024, 64, 1), (512, 8192, 2048, 64, 1),
    (1 << 20, 0, 1024, 16, 1), (1 << 20, 1, 64, 32, 2), (70000, 257, 256, 16, 4), (64, 1024, 1024, 16, 1), (3, 100000, 512, 32, 1)])
def test_ssm_gradients_workspace_is_bounded(lib, B, T, D, N, G):
    """What the header says each sequence takes, for as many as fill the GPU (912 ranges of 1024 / N channels) or as 2 GB
    hold; and what the segments of at most one such wave take beside it."""
    ranges = G * -(-(D // G) // (1024 // N))
    each = -(-T // 8) * D * N * 4 + T * ranges * 8 * N + max(1, -(-T // 256)) * D * (N + 2) * 4
    wave = min(B, -(-912 // ranges))
    segments = 912 * (1024 // N) * 4 * ((2 * N + 1) + (N + 2) * (T // 512 + 2))
    need = lib.srwm_ssm_backward_workspace_bytes(B, T, D, N, G)
    assert 0 < need <= max(2e9, wave * each) + segments + 4096


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(2, 3, 16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.srwm_conv_forward(x, torch.zeros(16, 4))
    with pytest.raises(ValueError, match="CUDA"):
        binding.srwm_ssm_forward(x, x, torch.zeros(16, 16), torch.zeros(2, 3, 1, 16), torch.zeros(2, 3, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        binding.srwm_rmsnorm_forward(x[0], None)
    with pytest.raises(ValueError, match="activation"):
        binding.srwm_conv_step(x[0], torch.zeros(16, 4), None, torch.zeros(3, 3, 16), activation="tanh")
    with pytest.raises(ValueError, match="out"):
        binding.srwm_rmsnorm_forward(x[0], None, out="fp8")


# ------------------------------------------------------------------ the oracles
def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def _differences(loss, base, grads, h=1e-5):
    n = _rand(77)
    for i, g in enumerate(grads):
        u = n(*base[i].shape)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * u, base[i] - h * u
        want, high, low = float((g * u).sum()), loss(*up), loss(*dn)
        # the losses' own roundings, a few 2^-53 of them, are divided by 2 h: at a loss of 2e7 that is 2e-4
        tol = 1e-6 * (1 + abs(want)) + (abs(high) + abs(low)) * 2.0 ** -51 / (2 * h)
        assert abs((high - low) / (2 * h) - want) < tol, i


@pytest.mark.parametrize("W", [2, 4])
def test_conv_oracle_against_torch_and_differences(W):
    n = _rand(W)
    x, w, b, s, dy, ds = n(3, 7, 5), n(5, W), n(5), n(3, W - 1, 5), n(3, 7, 5), n(3, W - 1, 5)
    lengths = torch.tensor([7, 1, 0])
    y, last = conv_oracle.forward(x, w, b, "silu", s)
    full = torch.cat([s, x], 1)
    want = torch.nn.functional.silu(torch.nn.functional.conv1d(full.transpose(1, 2), w[:, None], b, groups=5)).transpose(1, 2)
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12) and torch.equal(last, full[:, 7:])
    y, last = conv_oracle.forward(x, w, b, "silu", s, lengths)
    assert torch.allclose(y[1, :1], want[1, :1]) and (y[1, 1:] == 0).all() and torch.equal(last[2], s[2])
    assert torch.equal(last[1], full[1, 1:W])
    grads = conv_oracle.grads(x, w, b, "silu", dy, s, lengths, ds)

    def loss(x, w, b, s):
        y, last = conv_oracle.forward(x, w, b, "silu", s, lengths)
        return float((y * dy).sum() + (last * ds).sum())

    _differences(loss, [x, w, b, s], grads)


def test_rmsnorm_oracle_against_torch_and_differences():
    n = _rand(1)
    x, r, g, dy, dt = n(4, 6), n(4, 6), n(6), n(4, 6), n(4, 6)
    y, h, rstd = norm_oracle.forward(x, g, r, 1e-5)
    assert torch.allclose(y, torch.nn.functional.rms_norm(x + r, (6,), g, 1e-5), rtol=1e-12) and torch.equal(h, x + r)
    assert torch.allclose(y, h * rstd[:, None] * g, rtol=1e-12)
    grads = norm_oracle.grads(h, g, 1e-5, dy, dt)
    _differences(lambda h, g: float((norm_oracle.forward(h, g, None, 1e-5)[0] * dy).sum() + (h * dt).sum()), [h, g], grads)


def test_e4m3_values_are_those_of_the_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    table = norm_oracle.e4m3_values()
    assert torch.equal(torch.isnan(codes), torch.isnan(table))
    assert torch.equal(torch.nan_to_num(codes), torch.nan_to_num(table)) and float(table[126]) == 448


def _scan(seed, B=2, T=6, D=6, N=3, G=2):
    n = _rand(seed)
    return dict(u=n(B, T, D), dt=n(B, T, D), A=-torch.exp(n(D, N)), Bt=n(B, T, G, N), Ct=n(B, T, G, N), skip=n(D), z=n(B, T, D),
                dt_bias=n(D), h_init=n(B, D, N)), n(B, T, D), n(B, D, N)


def test_ssm_oracle_against_the_sum_over_pairs():
    """y_t = sum over s <= t of C_t . (exp(A (S_t - S_s)) x_s B_s), S the steps' running sum, and the state that came in."""
    a, _, _ = _scan(1)
    y, h = ssm_oracle.forward(**a)
    s = torch.nn.functional.softplus(a["dt"] + a["dt_bias"])
    S = s.cumsum(1)
    D, G = 6, 2
    B, C = (a[k].repeat_interleave(D // G, 2) for k in ("Bt", "Ct"))
    gap = torch.exp(a["A"] * (S[:, :, None] - S[:, None, :])[..., None]) * (torch.arange(6)[:, None] >= torch.arange(6))[None, :, :, None, None]
    hs = torch.einsum("btsdn,bsd,bsdn->btdn", gap, s * a["u"], B) + torch.exp(a["A"] * S[..., None]) * a["h_init"][:, None]
    want = ((C * hs).sum(-1) + a["skip"] * a["u"]) * torch.nn.functional.silu(a["z"])
    assert torch.allclose(y, want, rtol=1e-10, atol=1e-12) and torch.allclose(h, hs[:, -1], rtol=1e-10, atol=1e-12)
    lengths = torch.tensor([4, 0])
    y, h = ssm_oracle.forward(**a, lengths=lengths)
    assert torch.allclose(y[0, :4], want[0, :4], rtol=1e-10, atol=1e-12) and (y[0, 4:] == 0).all() and (y[1] == 0).all()
    assert torch.allclose(h[0], hs[0, 3], rtol=1e-10, atol=1e-12) and torch.equal(h[1], a["h_init"][1])


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, torch.tensor([6, 3]), torch.tensor([0, 5])])
def test_ssm_oracle_gradients_against_differences(lengths, softplus):
    a, dy, dh = _scan(2)
    grads = ssm_oracle.grads(dy, a, softplus, lengths, dh)
    assert tuple(grads) == ssm_oracle.NAMES

    def loss(*v):
        y, h = ssm_oracle.forward(**dict(zip(ssm_oracle.NAMES, v)), softplus=softplus, lengths=lengths)
        return float((y * dy).sum() + (h * dh).sum())

    _differences(loss, [a[k] for k in ssm_oracle.NAMES], [grads[k] for k in ssm_oracle.NAMES])


def test_ssm_error_bounds_hold_for_a_plain_computation_in_32_bits():
    """The same recurrence in float32: inside the bounds, and not a hundred times inside them everywhere."""
    a, dy, dh = _scan(3, B=2, T=40, D=8, N=4, G=1)
    a = {k: v.float() for k, v in a.items()}
    leaves = {k: v.clone().requires_grad_(True) for k, v in a.items()}
    s = torch.nn.functional.softplus(leaves["dt"] + leaves["dt_bias"])
    h, out = leaves["h_init"], []
    for t in range(40):
        B, C = (leaves[k][:, t].expand(2, 8, 4) for k in ("Bt", "Ct"))
        h = torch.exp(s[:, t, :, None] * leaves["A"]) * h + (s[:, t] * leaves["u"][:, t])[..., None] * B
        out.append((C * h).sum(-1) + leaves["skip"] * leaves["u"][:, t])
    y = torch.stack(out, 1) * torch.nn.functional.silu(leaves["z"])
    grads = dict(zip(leaves, torch.autograd.grad((y * dy.float()).sum() + (h * dh.float()).sum(), list(leaves.values()))))
    ry, rh = ssm_oracle.forward(**a)
    ref = ssm_oracle.grads(dy.float(), a, True, None, dh.float())
    ey, eh, err = ssm_oracle.errors(dy.float(), a, True, None, dh.float())
    for name, got, want, e in [("y", y, ry, ey), ("h", h, rh, eh)] + [(k, grads[k], ref[k], err[k]) for k in grads]:
        share = ((got.detach().double() - want).abs() / (e * 2.0 ** -24)).max()
        assert 0.002 < float(share) < 1, (name, float(share))

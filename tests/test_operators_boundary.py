"""Host-only checks of the linear attention and group norm entry points (no GPU
needed): bad arguments are refused before CUDA is touched; and their oracles'
pins: gradients against differences, closed forms."""
import ctypes

import pytest
import torch

from oracle import groupnorm as gn_oracle
from oracle import linattn as la_oracle
from self_referential_weight_gb300 import binding
from self_referential_weight_gb300 import build as lib_build

A = 0x100000  # fake, 16-byte aligned "device" addresses: never dereferenced
M = 0x1000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(lib_build.build())
    P, I, LL, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    L.srwm_linattn_forward.argtypes = [P, P, P, LL, P, P, P, I, I, I, I, I, F, P, P, P, SZ, P]
    L.srwm_linattn_step.argtypes = [P, P, P, LL, P, P, I, I, I, I, F, P, P, P]
    L.srwm_linattn_backward.argtypes = [P, P, P, LL, P, P, P, I, I, I, I, I, F, P, P, P, P, P, LL, P, P, SZ, P]
    for n in ("srwm_linattn_workspace_bytes", "srwm_linattn_backward_workspace_bytes"):
        getattr(L, n).argtypes, getattr(L, n).restype = [I] * 4, SZ
    L.srwm_groupnorm_forward.argtypes = [P, P, P, I, LL, LL, I, I, F, I, P, P, P, P, SZ, P]
    L.srwm_groupnorm_backward.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, P, P, P, P, SZ, P]
    for n in ("srwm_groupnorm_workspace_bytes", "srwm_groupnorm_backward_workspace_bytes"):
        getattr(L, n).argtypes, getattr(L, n).restype = [LL, LL, I, I], SZ
    return L


def test_linattn_forward_refuses(lib):
    base = dict(q=A, k=A + M, v=A + 2 * M, ld=32, lg=A + 3 * M, S0=None, n=None, dt=0, B=2, T=3, H=2, d=16, sc=1.0,
                o=A + 4 * M, S=A + 5 * M, ws=A + 6 * M, wb=BIG)

    def call(**kw):
        return lib.srwm_linattn_forward(*dict(base, **kw).values(), None)

    for p in ("q", "k", "v", "lg", "o", "ws"):
        assert call(**{p: None}) == 1, p
    assert call(B=0) == 2 and call(T=-1) == 2 and call(H=0) == 2 and call(d=0) == 2
    assert call(B=1 << 20, H=1 << 12) == 2 and call(B=1 << 15, H=1 << 15, T=1 << 30, ld=1 << 20) == 2
    assert call(d=48, ld=96) == 3 and call(d=128, ld=256) == 3 and call(dt=3) == 3 and call(dt=-1) == 3
    assert call(ld=31) == 2 and call(ld=34) == 2 and call(ld=33, dt=1) == 2 and call(ld=36, dt=1) == 2
    assert call(wb=16) == 2
    assert call(k=A + M + 4) == 4 and call(S=A + 5 * M + 8) == 4 and call(n=A + 7 * M + 2) == 4
    assert call(o=A) == 5 and call(S=A + 4 * M + 64) == 5 and call(ws=A + M) == 5 and call(S0=A + 5 * M) == 5
    assert call(o=A + 16, ld=96) == 5                   # contiguous o over q's strided rows
    assert lib.srwm_linattn_workspace_bytes(2, 3, 2, 16) > 0 and lib.srwm_linattn_workspace_bytes(2, 3, 2, 48) == 0
    assert lib.srwm_linattn_workspace_bytes(0, 3, 2, 16) == 0


def test_linattn_step_refuses(lib):
    base = dict(q=A, k=A + M, v=A + 2 * M, ld=32, lg=A + 3 * M, S=A + 4 * M, dt=1, B=2, H=2, d=16, sc=1.0,
                o=A + 5 * M, So=A + 6 * M)

    def call(**kw):
        return lib.srwm_linattn_step(*dict(base, **kw).values(), None)

    for p in ("q", "k", "v", "lg", "S", "o", "So"):
        assert call(**{p: None}) == 1, p
    assert call(B=0) == 2 and call(d=48, ld=96) == 3 and call(dt=7) == 3 and call(ld=16) == 2
    assert call(v=A + 2 * M + 8) == 4
    assert call(So=A + 4 * M + 16) == 5 and call(o=A + 4 * M) == 5 and call(So=A) == 5
    assert call(So=A + 4 * M) not in (1, 2, 3, 4, 5)    # exactly in place passes the argument checks


def test_linattn_backward_refuses(lib):
    base = dict(q=A, k=A + M, v=A + 2 * M, ld=32, lg=A + 3 * M, S0=None, n=None, dt=0, B=2, T=3, H=2, d=16, sc=1.0,
                do=A + 4 * M, dS=None, dq=A + 5 * M, dk=A + 6 * M, dv=A + 7 * M, ldg=32, d0=None, ws=A + 8 * M, wb=BIG)

    def call(**kw):
        return lib.srwm_linattn_backward(*dict(base, **kw).values(), None)

    for p in ("q", "k", "v", "lg", "do", "dq", "dk", "dv", "ws"):
        assert call(**{p: None}) == 1, p
    assert call(T=-1) == 2 and call(ldg=16) == 2 and call(wb=16) == 2 and call(d=24, ld=48, ldg=48) == 3
    assert call(dq=A + 5 * M + 4) == 4
    assert call(dq=A) == 5 and call(dk=A + 5 * M) == 5 and call(dv=A + 4 * M) == 5 and call(d0=A + 8 * M) == 5
    # slices of one packed array interleave without overlap; a slice half over another does not
    pack = dict(dq=A + 5 * M, dk=A + 5 * M + 128, dv=A + 5 * M + 256, ldg=96)
    assert call(**pack) not in (1, 2, 3, 4, 5)
    assert call(**dict(pack, dk=A + 5 * M + 64)) == 5 and call(**dict(pack, dv=A + 5 * M + 320)) == 5


def test_groupnorm_refuses(lib):
    f = dict(x=A, g=A + M, b=A + 2 * M, dt=0, N=4, L=3, C=16, G=4, eps=1e-5, act=1, y=A + 3 * M, m=A + 4 * M, r=A + 5 * M,
             ws=A + 6 * M, wb=BIG)
    g = dict(x=A, g=A + M, b=A + 2 * M, m=A + 3 * M, r=A + 4 * M, dy=A + 5 * M, dt=0, N=4, L=3, C=16, G=4, act=1,
             dx=A + 6 * M, dg=A + 7 * M, db=A + 8 * M, ws=A + 9 * M, wb=BIG)

    def fwd(**kw):
        return lib.srwm_groupnorm_forward(*dict(f, **kw).values(), None)

    def bwd(**kw):
        return lib.srwm_groupnorm_backward(*dict(g, **kw).values(), None)

    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(ws=None) == 1
    for p in ("x", "m", "r", "dy", "dx", "ws"):
        assert bwd(**{p: None}) == 1, p
    for call in (fwd, bwd):
        assert call(N=-1) == 2 and call(L=0) == 2 and call(G=3) == 2 and call(G=0) == 2 and call(wb=8) == 2
        assert call(N=1 << 32) == 2 and call(N=1 << 30, L=1 << 30) == 2
        assert call(C=12) == 3 and call(C=16384) == 3 and call(dt=5) == 3 and call(act=3) == 3 and call(act=-1) == 3
        assert call(x=A + 2) == 4
    assert fwd(eps=0.0) == 3 and fwd(eps=float("nan")) == 3
    assert fwd(y=A) == 5 and fwd(m=A + 5 * M) == 5 and fwd(ws=A) == 5 and fwd(r=A + M) == 5
    assert bwd(dx=A) == 5 and bwd(dx=A + 5 * M) == 5 and bwd(dg=A + 8 * M) == 5 and bwd(ws=A + 3 * M) == 5
    assert lib.srwm_groupnorm_workspace_bytes(4, 3, 16, 4) > 0 and lib.srwm_groupnorm_workspace_bytes(4, 3, 16, 3) == 0


# ------------------------------------------------------------------ the oracles
def _case(seed=0, B=2, T=6, H=2, d=3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return [n(B, T, H, d) for _ in range(3)], torch.tensor([-0.3, -1.2], dtype=torch.float64), n(B, H, d, d), \
        n(B, T, H, d), n(B, H, d, d)


def test_linattn_oracle_equals_the_masked_matrix_form():
    (q, k, v), lg, S0, _, _ = _case()
    o, S = la_oracle.forward(q, k, v, lg, 0.5)
    t = torch.arange(6)
    gap = t[:, None] - t[None, :]
    D = torch.where(gap >= 0, torch.exp(lg.view(-1, 1, 1) * gap.clamp(min=0)), 0.0)
    want = torch.einsum("bthd,bshd,hts,bshe->bthe", q, k, D, v) * 0.5
    assert torch.allclose(o, want, rtol=1e-12, atol=1e-12)
    n = torch.tensor([4, 0])
    o, S = la_oracle.forward(q, k, v, lg, 0.5, S0, n)
    o4, S4 = la_oracle.forward(q[:, :4], k[:, :4], v[:, :4], lg, 0.5, S0)
    assert torch.equal(o[0, :4], o4[0]) and torch.equal(S[0], S4[0]) and torch.equal(S[1], S0[1])
    assert (o[0, 4:] == 0).all() and (o[1] == 0).all()


@pytest.mark.parametrize("lengths", [None, torch.tensor([6, 3]), torch.tensor([0, 5])])
def test_linattn_oracle_gradients_against_differences_and_the_stated_formulas(lengths):
    (q, k, v), lg, S0, do, dS = _case(1)
    grads = la_oracle.grads(q, k, v, lg, 0.5, do, S0, lengths, dS)

    def loss(q, k, v, S0):
        o, S = la_oracle.forward(q, k, v, lg, 0.5, S0, lengths)
        return float((o * do).sum() + (S * dS).sum())

    base, h = [q, k, v, S0], 1e-5
    for i, g in enumerate(grads):
        u = torch.randn_like(base[i])
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * u, base[i] - h * u
        assert abs((loss(*up) - loss(*dn)) / (2 * h) - float((g * u).sum())) < 1e-7 * (1 + abs(float((g * u).sum())))
    if lengths is None:      # D_t = scale q_t do_t^T + g D_{t+1}
        D, g = dS.clone(), torch.exp(lg).view(1, -1, 1, 1)
        for t in range(5, -1, -1):
            D = D + 0.5 * q[:, t].unsqueeze(-1) * do[:, t].unsqueeze(-2)
            assert torch.allclose(grads[1][:, t], (D @ v[:, t].unsqueeze(-1)).squeeze(-1), rtol=1e-10, atol=1e-12)
            assert torch.allclose(grads[2][:, t], (k[:, t].unsqueeze(-2) @ D).squeeze(-2), rtol=1e-10, atol=1e-12)
            D = g * D
        assert torch.allclose(grads[3], D, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("act", ["none", "silu", "relu"])
def test_groupnorm_oracle_against_torch_and_differences(act):
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, gamma, beta, dy = n(3, 5, 8), n(8), n(8), n(3, 5, 8)
    y, mean, rstd = gn_oracle.forward(x, gamma, beta, 2, 1e-5, act)
    z = torch.nn.functional.group_norm(x.transpose(1, 2), 2, gamma, beta, 1e-5).transpose(1, 2)
    want = {"none": z, "silu": torch.nn.functional.silu(z), "relu": torch.relu(z)}[act]
    assert torch.allclose(y, want, rtol=1e-10, atol=1e-12) and mean.shape == rstd.shape == (3, 2)
    grads = gn_oracle.grads(x, gamma, beta, 2, 1e-5, act, dy)
    base, h = [x, gamma, beta], 1e-6
    for i, gr in enumerate(grads):
        u = n(*base[i].shape)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * u, base[i] - h * u
        f = lambda a: float((gn_oracle.forward(a[0], a[1], a[2], 2, 1e-5, act)[0] * dy).sum())  # noqa: E731
        assert abs((f(up) - f(dn)) / (2 * h) - float((gr * u).sum())) < 1e-6 * (1 + abs(float((gr * u).sum())))


def test_groupnorm_wants_an_eps():
    """None is no eps (it was taken as 1)."""
    x = torch.zeros(2, 3, 16)
    for eps in (None, "small"):
        with pytest.raises(TypeError):
            binding.srwm_groupnorm_forward(x, None, None, 2, eps=eps)
    with pytest.raises(ValueError, match="CUDA"):
        binding.srwm_groupnorm_forward(x, None, None, 2)

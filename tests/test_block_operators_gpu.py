"""The convolution, the scan and the norm together, as a block uses them: norm with the residual, an input
projection, convolution, the step's and B's and C's projection, scan with its gate, an output projection.  A prompt
and then single tokens on the GPU, against the same block in float64 from the operators' definitions; and its
gradients, chained operator by operator, against autograd through the definitions.

The prompt's 12 tokens and the single ones pass two blocks in fp32, with values of the order of 1 and products of up
to 96 terms: each of some 10 operations loses less than (96 + 64) 2^-24 of its magnitude, 1e-5, and the block's
derivatives stay below about 10: 1e-3 of the largest magnitude bounds both passes, and is far below what a wrong
state, row or gradient would give."""
import pytest
import torch

from oracle import conv as conv_oracle
from oracle import rmsnorm as norm_oracle
from oracle import ssm as ssm_oracle
from self_referential_weight_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
C, D, N, R, W = 64, 96, 16, 8, 4


def params(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(gamma=1 + 0.1 * n(C), w_in=n(2 * D, C) / 8, taps=n(D, W) / 2, bias=0.1 * n(D), w_x=n(R + 2 * N, D) / 10,
                w_dt=n(D, R) / 4, dt_bias=n(D) - 2, A=-torch.exp(n(D, N)), skip=n(D), w_out=n(C, D) / 10)


def gpu_prompt(p, x, stream):
    B, T, _ = x.shape
    y, _, total, rstd = binding.srwm_rmsnorm_forward(x.view(-1, C), p["gamma"], residual=stream.view(-1, C))
    xz = (y @ p["w_in"].T).view(B, T, 2 * D)
    u, conv_state = binding.srwm_conv_forward(xz[..., :D], p["taps"], p["bias"])
    xp = u @ p["w_x"].T
    dt = (xp[..., :R] @ p["w_dt"].T).contiguous()
    Bt, Ct = xp[..., R:R + N].unflatten(-1, (1, N)), xp[..., R + N:].unflatten(-1, (1, N))
    o, h = binding.srwm_ssm_forward(u, dt, p["A"], Bt, Ct, skip=p["skip"], z=xz[..., D:], dt_bias=p["dt_bias"])
    kept = dict(y=y, total=total, rstd=rstd, xz=xz, u=u, xp=xp, dt=dt, Bt=Bt, Ct=Ct, o=o)
    return o @ p["w_out"].T, total.view(B, T, C), (conv_state, h), kept


def gpu_token(p, x, stream, state):
    conv_state, h = state
    y, _, total, _ = binding.srwm_rmsnorm_forward(x, p["gamma"], residual=stream)
    xz = y @ p["w_in"].T
    u, _ = binding.srwm_conv_step(xz[:, :D], p["taps"], p["bias"], conv_state, state_out=conv_state)
    xp = u @ p["w_x"].T
    o, _ = binding.srwm_ssm_step(u, xp[:, :R] @ p["w_dt"].T, p["A"], xp[:, R:R + N].unflatten(-1, (1, N)),
                                 xp[:, R + N:].unflatten(-1, (1, N)), h, skip=p["skip"], z_t=xz[:, D:], dt_bias=p["dt_bias"], h_out=h)
    return o @ p["w_out"].T, total


def defined(p, x, stream):
    B, T, _ = x.shape
    y, total, _ = norm_oracle.forward(x.reshape(-1, C), p["gamma"], stream.reshape(-1, C), 1e-5)
    xz = (y @ p["w_in"].T).view(B, T, 2 * D)
    u, _ = conv_oracle.forward(xz[..., :D], p["taps"], p["bias"], "silu")
    xp = u @ p["w_x"].T
    o, h = ssm_oracle.forward(u, xp[..., :R] @ p["w_dt"].T, p["A"], xp[..., R:R + N].unflatten(-1, (1, N)),
                              xp[..., R + N:].unflatten(-1, (1, N)), p["skip"], xz[..., D:], p["dt_bias"])
    return o @ p["w_out"].T, total.view(B, T, C)


def close(got, want, what):
    assert float((got.double() - want).abs().max()) <= 1e-3 * float(want.abs().max()), what


def test_a_prompt_and_the_tokens_after_it():
    g = torch.Generator(device=DEV).manual_seed(1)
    blocks = [params(s) for s in (2, 3)]
    x = torch.randn(3, 17, C, generator=g, device=DEV)
    want, stream = x.double(), torch.zeros(3, 17, C, device=DEV, dtype=torch.float64)
    for p in blocks:
        want, stream = defined({k: v.double() for k, v in p.items()}, want, stream)
    out, stream_g, states = x[:, :12].contiguous(), torch.zeros(3, 12, C, device=DEV), []
    for p in blocks:
        out, stream_g, state, _ = gpu_prompt(p, out.contiguous(), stream_g)
        states.append(state)
    close(out, want[:, :12], "prompt")
    close(stream_g, stream[:, :12], "residual stream")
    for t in range(12, 17):
        o, s = x[:, t].contiguous(), torch.zeros(3, C, device=DEV)
        for p, state in zip(blocks, states):
            o, s = gpu_token(p, o, s, state)
        close(o, want[:, t], f"token {t}")


def test_gradients_through_the_block():
    g = torch.Generator(device=DEV).manual_seed(5)
    p = params(6)
    x, stream = (torch.randn(2, 12, C, generator=g, device=DEV) for _ in range(2))
    dout, dstream = (torch.randn(2, 12, C, generator=g, device=DEV) for _ in range(2))
    leaves = {k: v.double().requires_grad_(True) for k, v in {**p, "x": x, "stream": stream}.items()}
    o, t = defined({k: leaves[k] for k in p}, leaves["x"], leaves["stream"])
    ref = dict(zip(leaves, torch.autograd.grad((o * dout.double()).sum() + (t * dstream.double()).sum(), list(leaves.values()))))

    _, total, _, k = gpu_prompt(p, x, stream)
    got = {"w_out": torch.einsum("btc,btd->cd", dout, k["o"])}
    dxz, dxp = torch.empty_like(k["xz"]), torch.empty_like(k["xp"])
    du, ddt, got["A"], dB, dC, got["skip"], _, got["dt_bias"], _ = binding.srwm_ssm_backward(
        k["u"], k["dt"], p["A"], k["Bt"], k["Ct"], dout @ p["w_out"], skip=p["skip"], z=k["xz"][..., D:], dt_bias=p["dt_bias"],
        dB=dxp[..., R:R + N].unflatten(-1, (1, N)), dC=dxp[..., R + N:].unflatten(-1, (1, N)), dz=dxz[..., D:])
    got["w_dt"] = torch.einsum("btd,btr->dr", ddt, k["xp"][..., :R])
    dxp[..., :R] = ddt @ p["w_dt"]
    got["w_x"] = torch.einsum("btr,btd->rd", dxp, k["u"])
    _, got["taps"], got["bias"], _ = binding.srwm_conv_backward(k["xz"][..., :D], p["taps"], p["bias"], du + dxp @ p["w_x"],
                                                                dx=dxz[..., :D])
    got["w_in"] = torch.einsum("bti,btc->ic", dxz, k["y"].view(2, 12, C))
    dx, got["gamma"] = binding.srwm_rmsnorm_backward(k["total"], p["gamma"], k["rstd"], (dxz @ p["w_in"]).view(-1, C),
                                                     dtotal=dstream.view(-1, C))
    got["x"] = got["stream"] = dx.view(2, 12, C)
    assert set(got) == set(ref)
    for name in ref:
        close(got[name], ref[name], name)


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured into a graph: no operator needs one outside it."""
    code = """
import torch
from self_referential_weight_gb300 import binding as b
torch.manual_seed(0)
n = lambda *s: torch.randn(*s, device="cuda")
x, w, wb, gamma = n(2, 300, 64), n(64, 4), n(64), n(64)
A, B, C, dtb, z = -torch.exp(n(64, 16)), n(2, 300, 1, 16), n(2, 300, 1, 16), n(64) - 2, n(2, 300, 64)
def run():
    y, _, t, r = b.srwm_rmsnorm_forward(x.view(-1, 64), gamma, residual=z.view(-1, 64))
    y8, s, _, _ = b.srwm_rmsnorm_forward(x.view(-1, 64), gamma, out="e4m3")
    u, cs = b.srwm_conv_forward(y.view(2, 300, 64), w, wb)
    o, h = b.srwm_ssm_forward(u, x, A, B, C, z=z, dt_bias=dtb)
    g = b.srwm_ssm_backward(u, x, A, B, C, o, z=z, dt_bias=dtb)
    d = b.srwm_conv_backward(y.view(2, 300, 64), w, wb, g[0])
    e = b.srwm_rmsnorm_backward(t, gamma, r, d[0].view(-1, 64))
    ut, _ = b.srwm_conv_step(x[:, 0], w, wb, cs)
    ot, ht = b.srwm_ssm_step(ut, x[:, 0], A, B[:, 0], C[:, 0], h, z_t=z[:, 0], dt_bias=dtb)
    return [v for v in (y, y8.view(torch.uint8), s, u, cs, o, h, *g, *d, *e, ut, ot, ht) if v is not None]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, run()))
"""
    import pathlib
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], cwd=pathlib.Path(__file__).parent.parent, capture_output=True, text=True,
                       timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_graphs_share_a_workspace():
    """Graphs that are replayed one after the other may hold the same workspace; what they leave in it does not matter."""
    g = torch.Generator(device=DEV).manual_seed(9)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    sets = []
    for T in (40, 700):
        a = [n(2, T, 64), n(2, T, 64), -torch.exp(n(64, 16)), n(2, T, 1, 16), n(2, T, 1, 16)]
        sets.append((a, n(2, T, 64), binding.srwm_ssm_forward(*a), binding.srwm_ssm_backward(*a, a[0])))
    need = max(max(binding.srwm_ssm_backward_workspace_bytes(2, T, 64, 16, 1), binding.srwm_ssm_workspace_bytes(2, T, 64, 16, 1)) for T in (40, 700))
    ws = torch.full((need,), 255, device=DEV, dtype=torch.uint8)      # NaN where it is read before it is written
    graphs, outs = [], []
    for a, _, _, _ in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append((*binding.srwm_ssm_forward(*a, workspace=ws), *binding.srwm_ssm_backward(*a, a[0], workspace=ws)))
    for i in (0, 1, 0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        for x, r in zip(outs[i], (*sets[i][2], *sets[i][3])):
            assert (x is None) == (r is None) and (x is None or torch.equal(x, r))


def test_offsets_past_32_bits():
    """More than 2^31 elements in a tensor: the last sequence (or rows) against calls of their own."""
    B, T, width = 300, 1000, 7200
    assert B * T * width > 1 << 31
    x = torch.randn(B, T, width, device=DEV, dtype=torch.bfloat16)
    one = x[-1:].contiguous()
    w, b, A = torch.randn(width, 4, device=DEV), torch.randn(width, device=DEV), -torch.exp(torch.randn(width, 16, device=DEV))
    y, s = binding.srwm_conv_forward(x, w, b)
    y1, s1 = binding.srwm_conv_forward(one, w, b)
    assert torch.equal(y[-1:], y1) and torch.equal(s[-1:], s1)
    d, d1 = binding.srwm_conv_backward(x, w, b, y)[0], binding.srwm_conv_backward(one, w, b, y1)[0]
    assert torch.equal(d[-1:], d1)
    del y, d
    rows = x.view(B * T, width)
    y, _, t, r = binding.srwm_rmsnorm_forward(rows, b, residual=rows)
    y1, _, t1, r1 = binding.srwm_rmsnorm_forward(rows[-700:].contiguous(), b, residual=rows[-700:].contiguous())
    assert torch.equal(y[-700:], y1) and torch.equal(t[-700:], t1) and torch.equal(r[-700:], r1)
    e = binding.srwm_rmsnorm_backward(t, b, r, rows)[0]
    assert torch.equal(e[-700:], binding.srwm_rmsnorm_backward(t1, b, r1, rows[-700:].contiguous())[0])
    del y, t, e
    bc = torch.randn(B, T, 2, 16, device=DEV, dtype=torch.bfloat16).unsqueeze(3).unbind(2)
    ones = [v[-1:] for v in bc]
    y, h = binding.srwm_ssm_forward(x, x, A, *bc)
    y1, h1 = binding.srwm_ssm_forward(one, one, A, *ones)

    def close(p, q):          # one sequence alone is cut along its axis: other roundings, then bf16's
        assert float((p.double() - q.double()).norm()) <= 2.0 ** -8 * float(q.double().norm())

    close(y[-1:], y1)
    close(h[-1:], h1)
    got, want = binding.srwm_ssm_backward(x, x, A, *bc, y), binding.srwm_ssm_backward(one, one, A, *ones, y1)
    for i in (0, 1, 3, 4):
        close(got[i][-1:], want[i])

"""Bounded waits: a TMA load that never arrives ends the kernel with a status,
not a hang, and leaves the context usable.

The fault is made on the host: srwm_debug_skip_x_chunk(1) makes the kernels
skip issuing the load of input chunk 1, so the wait for it runs out after the
(shortened) wait limit.  Nothing faults or traps on the GPU.
"""
import numpy as np
import pytest
import torch

import oracle
from self_referential_weight_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def short_waits():
    binding.srwm_set_wait_limit_ns(50_000_000)  # 50 ms
    yield
    binding.srwm_debug_skip_x_chunk(-1)
    binding.srwm_set_wait_limit_ns(1_000_000_000)


@pytest.mark.parametrize("d,B,smx", [(16, 2, False), (32, 2, False), (64, 2, False), (64, 110, False),
                                     (64, 110, True)])
def test_missing_chunk_times_out_then_recovers(short_waits, d, B, smx):
    """B = 110 (330 streams at H = 3, more than two per SM on a GB300) runs the
    two-warp d = 64 kernel, whose CTAs agree on a timeout at chunk boundaries,
    with and without the input softmax."""
    wl = inputs.Workload("t", B, 100, 3, d, 4, smx, 40 + d, "normal")
    x, W0 = inputs.make_inputs(wl)
    xd, W0d = torch.from_numpy(x).to(DEV), torch.from_numpy(W0).to(DEV)
    assert binding.srwm_last_device_status() == 0

    binding.srwm_debug_skip_x_chunk(1)
    binding.srwm_forward(xd, W0d, 4, smx)
    assert binding.srwm_last_device_status() == binding.SRWM_ERR_TIMEOUT
    assert binding.srwm_last_device_status() == 0  # reading clears it

    binding.srwm_debug_skip_x_chunk(-1)
    y, Wf = binding.srwm_forward(xd, W0d, 4, smx)
    assert binding.srwm_last_device_status() == 0
    yo, Wo = oracle.forward(x, W0, 4, smx)
    assert np.abs(y.cpu().numpy() - yo).max() / np.abs(yo).max() <= 1e-4
    assert np.abs(Wf.cpu().numpy() - Wo).max() / np.abs(Wo).max() <= 1e-4


@pytest.mark.parametrize("d,H,slots_per_sm", [(32, 4, 12), (16, 16, 16)])
def test_missing_chunk_wrap_schedule(short_waits, d, H, slots_per_sm):
    """The d = 32 and d = 16 kernels on the wrap-around schedule (more streams
    than warp slots): a missing chunk ends every slot with the timeout status,
    also the slots whose next piece's chunks were already issued, and the next
    call is correct."""
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    B = (slots_per_sm * n_sm) // H + 7
    wl = inputs.Workload("t", B, 100, H, d, 1, True, 77 + d, "normal")
    x, W0 = inputs.make_inputs(wl)
    xd, W0d = torch.from_numpy(x).to(DEV), torch.from_numpy(W0).to(DEV)
    assert binding.srwm_last_device_status() == 0

    binding.srwm_debug_skip_x_chunk(1)
    binding.srwm_forward_balanced(xd, W0d, 1, True)
    assert binding.srwm_last_device_status() == binding.SRWM_ERR_TIMEOUT
    assert binding.srwm_last_device_status() == 0

    binding.srwm_debug_skip_x_chunk(-1)
    y, Wf = binding.srwm_forward_balanced(xd, W0d, 1, True)
    assert binding.srwm_last_device_status() == 0
    rng = np.random.default_rng(3)
    for b in sorted(set(int(v) for v in rng.integers(0, B, 6)) | {0, B - 1}):
        yo, Wo = oracle.forward(x[b:b + 1], W0, 1, True)
        assert np.abs(y[b].cpu().numpy() - yo[0]).max() / np.abs(yo).max() <= 1e-4
        assert np.abs(Wf[b].cpu().numpy() - Wo[0]).max() / np.abs(Wo).max() <= 1e-4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [2, 90])
def test_missing_chunk_of_linear_attention(short_waits, B, dtype):
    """The kernels on 128-token chunks, a stream or several per SM (the first
    stream that has a second chunk ends its CTA), forward and backward: the
    timeout status, then calls that are right again."""
    T, H, d = 300, 5, 64
    g = torch.Generator(device=DEV).manual_seed(B)
    q, k, v, do = (torch.randn(B, T, H, d, generator=g, device=DEV).to(dtype) for _ in range(4))
    lg = torch.full((H,), -0.05, device=DEV)
    assert binding.srwm_last_device_status() == 0
    o, S = binding.srwm_linattn_forward(q, k, v, lg)
    grads = binding.srwm_linattn_backward(q, k, v, lg, do)
    assert binding.srwm_last_device_status() == 0
    for call in (lambda: binding.srwm_linattn_forward(q, k, v, lg), lambda: binding.srwm_linattn_backward(q, k, v, lg, do)):
        binding.srwm_debug_skip_x_chunk(1)
        call()
        assert binding.srwm_last_device_status() == binding.SRWM_ERR_TIMEOUT
        assert binding.srwm_last_device_status() == 0
        binding.srwm_debug_skip_x_chunk(-1)
        o2, S2 = binding.srwm_linattn_forward(q, k, v, lg)
        again = binding.srwm_linattn_backward(q, k, v, lg, do)
        assert binding.srwm_last_device_status() == 0
        assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(x, y) for x, y in zip(grads, again))
    short = torch.full((B,), 128, dtype=torch.int32, device=DEV)      # no sequence has a second chunk
    want = binding.srwm_linattn_forward(q, k, v, lg, lengths=short)
    binding.srwm_debug_skip_x_chunk(1)
    got = binding.srwm_linattn_forward(q, k, v, lg, lengths=short)
    assert binding.srwm_last_device_status() == 0 and all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_attention_under_the_shortest_limit(short_waits, dtype):
    """Waits that run out anywhere, at or beside the end of what they wait for:
    each call ends, says so or is right, and the next ones are right."""
    B, T, H, d = 60, 400, 5, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    q, k, v, do = (torch.randn(B, T, H, d, generator=g, device=DEV).to(dtype) for _ in range(4))
    lg = torch.full((H,), -0.05, device=DEV)
    lengths = (torch.arange(B, device=DEV) * 37 % (T + 1)).int()

    def run():
        return (binding.srwm_linattn_forward(q, k, v, lg, lengths=lengths) +
                binding.srwm_linattn_backward(q, k, v, lg, do, lengths=lengths))

    want = run()
    assert binding.srwm_last_device_status() == 0
    for limit in (1000, 1500, 2500, 5000, 20000):
        binding.srwm_set_wait_limit_ns(limit)
        got = run()
        status = binding.srwm_last_device_status()
        assert status in (0, binding.SRWM_ERR_TIMEOUT)
        assert status or all(torch.equal(x, y) for x, y in zip(want, got))
    binding.srwm_set_wait_limit_ns(50_000_000)
    got = run()
    assert binding.srwm_last_device_status() == 0 and all(torch.equal(x, y) for x, y in zip(want, got))

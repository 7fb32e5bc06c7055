"""The windowed attention's bounded waits, without a fault: with gla_set_stall_step the tensor-core
issuer of every CTA waits on a barrier that completes only after its loop, gives up after the
limit (2 ms here) and raises the CTA's abort flag; every role leaves its loop, copies and products
drain, tensor memory is freed.  The host reads GLA_ERR_TIMEOUT and the next calls are right."""
import time

import pytest

pytestmark = pytest.mark.gpu

GLA_ERR_TIMEOUT = 5


@pytest.mark.parametrize("call", ["fwd", "bwd"])
@pytest.mark.parametrize("step,sink", [(0, 0), (1, 40), (3, 0)])
def test_waits_give_up_and_the_next_call_is_the_same(call, step, sink):
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dO = r(2, 900, 2, 96) * 0.1, r(2, 900, 1, 96), r(2, 900, 1, 192), r(2, 900, 2, 192)
    lens = torch.tensor([900, 700], dtype=torch.int32, device="cuda")

    def run(which):
        if which == "fwd":
            return gla.window_attn_fwd(q, k, v, 600, sink, lens)
        return gla.window_attn_bwd(q, k, v, o, lse, dO, 600, sink, lens)
    o, lse = run("fwd")
    want = run(call)
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    try:
        gla.set_wait_timeout_ns(2_000_000)
        gla.set_stall_step(step)
        t0 = time.perf_counter()
        run(call)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
        assert gla.get_device_error() == GLA_ERR_TIMEOUT
        assert dt < 5.0
    finally:
        gla.set_stall_step(-1)
        gla.set_wait_timeout_ns(0)
    got = run(call)
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))

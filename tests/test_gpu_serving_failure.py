"""The bounded waits of the attention over pages, without a fault: with gla_set_stall_step the tensor-core
issuer of every CTA (over 8-bit pages of few rows: the warp that sends the loads off) waits on a barrier
that completes only after its loop, gives up after the limit (2 ms here), and the others after it; loads
and products drain, tensor memory is freed.  The host reads GLA_ERR_TIMEOUT and the next calls are
right."""
import time

import pytest

pytestmark = pytest.mark.gpu

GLA_ERR_TIMEOUT = 5
WINDOW, SINK = 700, 4


@pytest.mark.parametrize("call", ["chunk16", "chunk8", "few8", "step8"])
@pytest.mark.parametrize("step", [0, 1, 3])
def test_waits_give_up_and_the_next_call_is_the_same(call, step):
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    codes = lambda *s: torch.randint(-127, 128, s, generator=gen, device="cuda").to(torch.int8)  # noqa: E731
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # (enough rows that some are not cut into fewer tiles or rounds than the steps)
    new = {"chunk16": [3000, 900, 1], "chunk8": [3000, 900, 1], "few8": [4, 3] * 120, "step8": [1] * 240}[call]
    n = len(new)
    start = [sum(new[:b]) for b in range(n + 1)]
    N, slots = start[-1], WINDOW + SINK
    q, k, v = r(N, 8, 96) * 0.1, r(N, 2, 96), r(N, 2, 192)
    if call == "chunk16":
        pools, e = (r(n, 1, slots, 2, 96), r(n, 1, slots, 2, 192)), None
    else:
        pools = codes(n, 1, slots, 2, 96), codes(n, 1, slots, 2, 192)
        e = torch.full((n, 1, 2, slots, 2), -6, dtype=torch.int8, device="cuda")
    page, pos = ints(*range(n)), ints(*([5000, 699, 650] * n)[:n])

    def run():
        if call != "step8":
            return [gla.window_attn_chunk(*pools, page, pos, ints(*start), q, k, v, WINDOW, SINK, pool_e=e)]
        pk, pv, pe = (x.clone() for x in (*pools, e))
        return [gla.window_attn8_decode_step(pk, pv, page, pe, pos, q, k, v, WINDOW, SINK), pk, pv, pe]
    want = run()
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    try:
        gla.set_wait_timeout_ns(2_000_000)
        gla.set_stall_step(step)
        t0 = time.perf_counter()
        run()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
        assert gla.get_device_error() == GLA_ERR_TIMEOUT
        assert dt < 5.0
    finally:
        gla.set_stall_step(-1)
        gla.set_wait_timeout_ns(0)
    got = run()
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))

"""The bounded waits of the gated scan and the layer norm, without a fault: with gla_set_stall_step
one CTA of every cluster (every CTA that awaits tiles, without clusters) waits for what never comes, gives up after
the limit (2 ms here) and leaves without its pair; the others' waits run out as well.  The norm's
rings stop fetching.  No CTA leaves while something may still be written into its memory.  The host reads GLA_ERR_TIMEOUT and the next calls are right."""
import time

import pytest

pytestmark = pytest.mark.gpu

GLA_ERR_TIMEOUT = 5


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch


def _stalled(gla, torch, step, run):
    """`run` stalls at `step`; before and after it gives the same bits."""
    want = run()
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    for _ in range(2):
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


SCANS = [  # B, T, D, type, steps: with 152 SMs
    (1, 2000, 64, "bfloat16", (0, 1, 3)),     # a cluster of 8, TMA tiles, four rounds
    (1, 2000, 68, "float32", (2,)),
    (3, 700, 66, "float32", (0, 1)),          # 8, rows of pairs
    (3, 700, 65, "float16", (0, 1)),          # 8, odd rows
    (60, 130, 64, "float16", (0, 1)),         # a cluster of 2
    (60, 300, 256, "bfloat16", (0, 2, 4)),    # none, TMA
]


@pytest.mark.parametrize("call", ["fwd", "bwd"])
@pytest.mark.parametrize("B,T,D,dt,step", [(*s[:4], k) for s in SCANS for k in s[4]])
def test_scan_gives_up_and_the_next_call_is_the_same(env, call, B, T, D, dt, step):
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, g = (r(B, T, D).to(getattr(torch, dt)) for _ in range(2))
    dy, init = r(B, T, D), r(B, D)
    y, _ = gla.gated_scan_fwd(x, g, init)
    if call == "fwd":
        _stalled(gla, torch, step, lambda: gla.gated_scan_fwd(x, g, init))
    else:
        _stalled(gla, torch, step, lambda: gla.gated_scan_bwd(x, g, y, dy, init, init))


@pytest.mark.parametrize("call", ["fwd", "bwd"])
@pytest.mark.parametrize("n,D,dt,step", [(5000, 2048, "bfloat16", 0), (5000, 2048, "bfloat16", 1),
                                         (20000, 512, "float16", 3), (9000, 1020, "float32", 4)])
def test_norm_rings_give_up_and_the_next_call_is_the_same(env, call, n, D, dt, step):
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, dy = (torch.randn(n, D, generator=gen, device="cuda").to(getattr(torch, dt))
             for _ in range(2))
    w = torch.randn(D, generator=gen, device="cuda")
    _, m, r = gla.layer_norm_fwd(x, w)
    if call == "fwd":
        _stalled(gla, torch, step, lambda: gla.layer_norm_fwd(x, w))
    else:
        _stalled(gla, torch, step, lambda: gla.layer_norm_bwd(dy, x, w, m, r))


def test_window_waits_last_as_long_as_an_item(env):
    """With a window of all of T an item streams 1,024 tiles forward and 4,096 in the gradient (0.9 and
    2.7 ms); a limit of 0.2 ms, two hundred tiles, does not end it."""
    gla, torch = env
    T = 131072
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dO = r(1, T, 2, 96) * 0.1, r(1, T, 1, 96), r(1, T, 1, 192), r(1, T, 2, 192)
    o, lse = gla.window_attn_fwd(q, k, v, T)
    want = gla.window_attn_bwd(q, k, v, o, lse, dO, T)
    assert gla.get_device_error() == 0
    try:
        gla.set_wait_timeout_ns(200_000)
        o2, lse2 = gla.window_attn_fwd(q, k, v, T)
        assert gla.get_device_error() == 0
        got = gla.window_attn_bwd(q, k, v, o, lse, dO, T)
        assert gla.get_device_error() == 0
    finally:
        gla.set_wait_timeout_ns(0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_window_waits_last_through_sequences_without_tokens(env):
    """Between the batch's first and last sequences the output rows of some 400 items a CTA are zeros
    (0.4 ms of stores), while the next item's sums wait for them; a limit of 0.2 ms does not end it."""
    gla, torch = env
    B, T = 2000, 2048
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[:20] = lens[-20:] = T
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dO = r(B, T, 2, 96) * 0.1, r(B, T, 1, 96), r(B, T, 1, 192), r(B, T, 2, 192)
    o, lse = gla.window_attn_fwd(q, k, v, 256, 3, lens)
    want = gla.window_attn_bwd(q, k, v, o, lse, dO, 256, 3, lens)
    assert gla.get_device_error() == 0
    try:
        gla.set_wait_timeout_ns(200_000)
        o2, lse2 = gla.window_attn_fwd(q, k, v, 256, 3, lens)
        got = gla.window_attn_bwd(q, k, v, o, lse, dO, 256, 3, lens)
        assert gla.get_device_error() == 0
    finally:
        gla.set_wait_timeout_ns(0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))

"""Packed sequences that overlap, where `start` decreases: each of them is within the call's rows, but together
they have more tiles, and more rows, than the plan and the workspace have room for.  The call is reported, writes
nothing behind its workspace, its output or its pages, and the next one is right."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

RANGE = 6
GUARD = 1 << 26  # bytes behind a workspace: more than the tiles of all sequences would need


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch


# sequences, tokens, H, KV, window: keys cut into parts and not; over 8 bits the few rows' kernel, the one that
# turns codes into operands in shared memory, and the one over the pages written out
CASES = [(16, 64, 256, 4, 1, 4096), (16, 64, 256, 4, 1, 100), (16, 300, 256, 4, 2, 700),
         (8, 64, 256, 4, 1, 4096), (8, 64, 256, 16, 1, 4096), (8, 64, 512, 8, 1, 60), (8, 3, 600, 4, 2, 1000),
         (8, 700, 600, 8, 2, 200), (16, 2000, 1500, 4, 2, 40)]


@pytest.mark.parametrize("bits,n,N,H,KV,window", CASES)
def test_overlapping_sequences_stay_within_their_buffers(env, bits, n, N, H, KV, window):
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(n + N)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    sink, P = 2, 3
    slots = window + sink
    if bits == 16:
        pool = [r(P, 1, slots, KV, 96), r(P, 1, slots, KV, 192), None]
    else:
        pool = [torch.randint(-127, 128, (P, 1, slots, KV, d), generator=gen, device="cuda").to(torch.int8)
                for d in (96, 192)]
        pool.append(torch.full((P, 1, KV, slots, 2), -6, dtype=torch.int8, device="cuda"))
    before = [None if x is None else x.clone() for x in pool]
    q, k, v = r(N, H, 96) * 0.1, r(N, KV, 96), r(N, KV, 192)
    page, pos = ints([1] * n), ints([5 * slots] * n)
    size = gla.window_attn_chunk_workspace_size(n, N, H, KV, window, sink, bits=bits)
    room = torch.full((size + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    rows = torch.full((N + 64, H, 192), 7.0, device="cuda").bfloat16()
    args = (*pool[:2], page, pos)

    def call(start):
        return gla.window_attn_chunk(*args, ints(start), q, k, v, window, sink, pool_e=pool[2], out=rows[:N],
                                     workspace=room[:size]).clone()
    even = np.linspace(0, N, n + 1).astype(int).tolist()
    want = call(even)
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    for start in ([N * (b % 2) for b in range(n + 1)],                       # all of the rows, again and again
                  [0] * (n // 2) + [N, 0] * ((n + 1 - n // 2) // 2) + [N] * ((n + 1 - n // 2) % 2),
                  [(N * (7 * b % 5)) // 4 for b in range(n + 1)]):
        assert len(start) == n + 1 and any(a > b for a, b in zip(start, start[1:]))
        call(start)
        torch.cuda.synchronize()
        assert gla.get_device_error() == RANGE
        assert bool((room[size:] == 0x5A).all()) and bool((rows[N:] == 7).all())
        assert all(x is None or torch.equal(x, y) for x, y in zip(pool, before))
    assert torch.equal(call(even), want) and gla.get_device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_overlapping_sequences_append_to_their_own_pages(env, bits):
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(bits)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randn(40, 2, d, generator=gen, device="cuda").bfloat16() for d in (96, 192))
    kind = torch.bfloat16 if bits == 16 else torch.int8
    pool = [torch.zeros(6, 1, 9, 2, d, dtype=kind, device="cuda") for d in (96, 192)]
    e = None if bits == 16 else torch.zeros(6, 1, 2, 9, 2, dtype=torch.int8, device="cuda")
    gla.window_cache_append(*pool, ints(0, 1, 3, 4), ints(0, 3, 70, 2), ints(0, 40, 0, 40, 20), k, v, 8, 1, pool_e=e)
    torch.cuda.synchronize()
    assert gla.get_device_error() == RANGE
    for x in (*pool, e):
        assert x is None or not x[[2, 5]].any()

"""The workspace of chunks whose keys are cut into parts: it grows with the rows that are there, not with the tiles of
128 that might be, and parts that gain next to nothing are not made.  Results in parts against the definition, as in
test_gpu_serving.py."""
import random

import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import serving_ops as ref

pytestmark = pytest.mark.gpu
U, F = 2.0 ** -8, 1024 * 2.0 ** -24
ROW = 776  # bytes of a (token, query head) and part: 192 sums, reference and sum


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch


def test_sizes(env):
    gla, _ = env
    size = lambda *a: gla.window_attn_chunk_workspace_size(*a, bits=16)  # noqa: E731
    # single tokens, many and few of them; a large batch of long chunks
    assert size(1000, 1000, 16, 4, 65536, 0) <= 2 * 1000 * 16 * ROW
    assert 0 < size(100, 100, 16, 1, 65536, 0) <= 6 * 100 * 16 * ROW
    assert size(256, 20000, 32, 4, 131072, 0) <= 2 * 20000 * 32 * ROW
    assert size(1, 1, 16, 4, 5000, 4) > 0
    rng = random.Random(1)
    for _ in range(300):
        n, H, KV = rng.randint(1, 300), rng.choice([4, 12, 16, 128]), rng.choice([1, 2, 4])
        N = n + int(rng.choice([0, 1, 50]) * rng.random() * n)
        need = size(n, N, H, KV, int(2 ** rng.uniform(4, 20)), rng.choice([0, 4]))
        assert need <= 64 * N * H * ROW + 16 * (N + n + 32) * KV, (n, N, H, KV)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,H,KV,window,sink", [
    ([5] * 8, 16, 1, 3000, 2), ([1, 9, 0, 30, 2, 1, 1], 12, 2, 2900, 4), ([40], 40, 1, 3000, 0), ([47, 3], 6, 2, 2100, 1)])
def test_parts_of_uneven_sequences(env, new, H, KV, window, sink, bits):
    gla, torch = env
    rng = np.random.default_rng(len(new) + H + bits)
    n, N, slots = len(new), sum(new), window + sink
    start = np.concatenate([[0], np.cumsum(new)]) + 1
    pos, page = [int(x) for x in rng.integers(0, 3 * slots, n)], rng.permutation(n + 1)[:n]
    if bits == 16:
        k, v = (as_dtype_values(rng.standard_normal((n + 1, 1, slots, KV, d)).astype(np.float32), "bf16")
                for d in (96, 192))
        pool, values = (to_dev(k, torch.bfloat16), to_dev(v, torch.bfloat16), None), (k, v)
    else:
        k, v = (rng.integers(-127, 128, (n + 1, 1, slots, KV, d)).astype(np.int8) for d in (96, 192))
        e = rng.integers(-8, -5, (n + 1, 1, KV, slots, 2)).astype(np.int8)
        two = 2.0 ** e.astype(np.float64).transpose(0, 1, 3, 2, 4)
        pool, values = tuple(torch.from_numpy(x).cuda() for x in (k, v, e)), (k * two[..., :1], v * two[..., 1:])
    q = as_dtype_values(rng.standard_normal((N + 2, H, 96)).astype(np.float32) * np.float32(0.25), "bf16")
    k, v = (as_dtype_values(rng.standard_normal((N + 2, KV, d)).astype(np.float32), "bf16") for d in (96, 192))
    dev = [to_dev(x, torch.bfloat16) for x in (q, k, v)]
    ints = lambda x: torch.tensor([int(y) for y in x], dtype=torch.int32, device="cuda")  # noqa: E731
    size = gla.window_attn_chunk_workspace_size(n, N + 2, H, KV, window, sink, bits=bits)
    assert size > 0
    outs = []
    for fill in (0x00, 0xFF):
        room = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
        o = torch.full((N + 2, H, 192), 7.0, device="cuda").bfloat16()
        gla.window_attn_chunk(*pool[:2], ints(page), ints(pos), ints(start), *dev, window, sink, pool_e=pool[2], out=o,
                              workspace=room[:size])
        assert bool((room[size:] == fill).all()) and bool((o[[0, -1]] == 7).all())
        outs.append(o)
    assert torch.equal(*outs) and gla.get_device_error() == 0
    want, pv, _ = ref.chunk(*values, page, pos, start, q, k, v, window, sink)
    live = slice(1, N + 1)
    off = np.abs(outs[0].float().cpu().numpy().astype(np.float64) - want)[live]
    assert np.all(off <= ((U + F) * pv + U * np.abs(want) + 2.0 ** -25)[live])

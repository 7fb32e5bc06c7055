"""Serving with the windowed attention at the ends of its ranges: pools past 2^31 elements, more sequences
than a CTA lists, many query heads, one long sequence among short ones, no tokens at all, a page that two
sequences share, workspaces full of anything.  Against the definition as in test_gpu_serving.py, or for the
same bits as a call that test compares."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import serving_ops as ref

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
F = 1024 * 2.0 ** -24
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch, {"bf16": torch.bfloat16, "fp16": torch.float16}


def _ints(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(torch, rng, P, slots, KV, dt, t, bits):
    """(keys, values, exponents or None) on the device and the values in 64 bits."""
    if bits == 16:
        k, v = (as_dtype_values(rng.standard_normal((P, 1, slots, KV, d)).astype(np.float32), dt) for d in (96, 192))
        return (to_dev(k, t), to_dev(v, t), None), (k, v)
    k, v = (rng.integers(-127, 128, (P, 1, slots, KV, d)).astype(np.int8) for d in (96, 192))
    e = rng.integers(-8, -5, (P, 1, KV, slots, 2)).astype(np.int8)
    two = 2.0 ** e.astype(np.float64).transpose(0, 1, 3, 2, 4)
    return tuple(torch.from_numpy(x).cuda() for x in (k, v, e)), (k * two[..., :1], v * two[..., 1:])


def _new(torch, rng, N, H, KV, dt, t):
    q = as_dtype_values(rng.standard_normal((N, H, 96)).astype(np.float32) * np.float32(0.25), dt)
    k, v = (as_dtype_values(rng.standard_normal((N, KV, d)).astype(np.float32), dt) for d in (96, 192))
    return (q, k, v), tuple(to_dev(x, t) for x in (q, k, v))


def _close(o, want, pv, av, dt):
    room = (U[dt] + F) * pv + TINY[dt] * av + U[dt] * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(o.float().cpu().numpy().astype(np.float64) - want) <= room)


# Wholly short batches and ones with a long sequence inside; rows that end in a group, that fill several,
# tokens that lie across units; heads of one key head up to the most.
MIXED = [  # new tokens, positions, H, KV, window, sink, type
    ([1] * 20 + [130] + [2] * 20, [40 * b for b in range(41)], 4, 1, 150, 3, "bf16"),
    ([3, 0, 1, 60, 0, 2] + [1] * 30, [7 * b for b in range(36)], 6, 2, 90, 70, "fp16"),   # sinks past new tokens
    ([11], [900], 3, 1, 400, 5, "bf16"),            # 33 rows: one in a unit of its own
    ([2, 3], [500, 20], 10, 1, 257, 0, "fp16"),     # units that end inside a token's heads
    ([1, 1, 1], [0, 70, 5000], 128, 1, 133, 2, "bf16"),
    ([5], [3000], 128, 1, 1000, 1, "fp16"),
    ([4] * 9, [64 * b for b in range(9)], 8, 1, 511, 1, "bf16"),  # pages that end at a round, before and behind
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,pos,H,KV,window,sink,dt", MIXED)
def test_mixed_batches_match_the_definition(env, new, pos, H, KV, window, sink, dt, bits):
    gla, torch, types = env
    rng = np.random.default_rng(len(new) + H + bits)
    P, start = len(new) + 1, np.concatenate([[0], np.cumsum(new)])
    page = rng.permutation(P)[:len(new)]
    pool, values = _pool(torch, rng, P, window + sink, KV, dt, types[dt], bits)
    (q, k, v), dev = _new(torch, rng, int(start[-1]), H, KV, dt, types[dt])
    args = (*pool[:2], _ints(torch, page.tolist()), _ints(torch, pos), _ints(torch, start.tolist()), *dev,
            window, sink)
    o = gla.window_attn_chunk(*args, pool_e=pool[2])
    _close(o, *ref.chunk(*values, page, pos, start, q, k, v, window, sink), dt)
    # a workspace of just the size that is asked for, full of NaN, twice
    size = gla.window_attn_chunk_workspace_size(len(new), len(q), H, KV, window, sink)
    ws = torch.full((max(size, 4) // 4,), float("nan"), device="cuda")
    for _ in range(2):
        assert torch.equal(gla.window_attn_chunk(*args, pool_e=pool[2], workspace=ws), o)
    assert gla.get_device_error() == 0


@pytest.mark.parametrize("H,KV,dt", [(128, 1, "bf16"), (24, 1, "fp16"), (9, 3, "bf16")])
def test_steps_of_many_heads_are_chunks_of_one(env, H, KV, dt):
    """A step and a chunk of one token each are the same attention; only the step's codes are new."""
    gla, torch, types = env
    rng = np.random.default_rng(H)
    n, window, sink = 5, 321, 2
    pool, values = _pool(torch, rng, n, window + sink, KV, dt, types[dt], 8)
    (q, k, v), dev = _new(torch, rng, n, H, KV, dt, types[dt])
    pos = [0, 1, 64, 322, 9000]
    want = ref.chunk(*values, np.arange(n), pos, np.arange(n + 1), q, k, v, window, sink)
    page = _ints(torch, list(range(n)))
    size = gla.window_attn8_decode_workspace_size(n, H, KV, window, sink)
    ws = torch.full((max(size, 4) // 4,), float("nan"), device="cuda")
    o = gla.window_attn8_decode_step(*pool[:2], page, pool[2], _ints(torch, pos), *dev, window, sink, workspace=ws)
    _close(o, *want, dt)
    assert gla.get_device_error() == 0


@pytest.mark.parametrize("bits,H", [(16, 4), (8, 4), (8, 40)])
def test_thousands_of_sequences(env, bits, H):
    """More items than all the CTAs' lists hold at once, every third sequence empty: each part of the batch has
    the bits of a call on it alone."""
    gla, torch, types = env
    rng = np.random.default_rng(H + bits)
    n, window, sink = 9000, 16, 1
    new = [b % 3 for b in range(n)]
    start = np.concatenate([[0], np.cumsum(new)])
    pos = [(7 * b) % 100 for b in range(n)]
    page = [b % 50 for b in range(n)]
    pool, values = _pool(torch, rng, 50, window + sink, 1, "bf16", types["bf16"], bits)
    (q, k, v), dev = _new(torch, rng, int(start[-1]), H, 1, "bf16", types["bf16"])
    o = gla.window_attn_chunk(*pool[:2], _ints(torch, page), _ints(torch, pos), _ints(torch, start.tolist()), *dev,
                              window, sink, pool_e=pool[2])
    for lo in (0, 4321, 8990):
        hi = lo + 10
        rows = slice(int(start[lo]), int(start[hi]))
        _close(o[rows], *ref.chunk(*values, page[lo:hi], pos[lo:hi], start[lo:hi + 1] - start[lo],
                                   q[rows], k[rows], v[rows], window, sink), "bf16")
    assert gla.get_device_error() == 0


def test_no_tokens(env):
    gla, torch, types = env
    pk, pv = (torch.zeros(2, 1, 9, 1, d, dtype=torch.int8, device="cuda") for d in (96, 192))
    e = torch.zeros(2, 1, 1, 9, 2, dtype=torch.int8, device="cuda")
    z = lambda n, h, d: torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for n in (0, 2):
        page, pos, start = _ints(torch, [0, 1][:n]), _ints(torch, [3, 4][:n]), _ints(torch, [0] * (n + 1))
        assert gla.window_attn_chunk(pk, pv, page, pos, start, z(0, 2, 96), z(0, 1, 96), z(0, 1, 192), 8, 1,
                                     pool_e=e).shape == (0, 2, 192)
        gla.window_cache_append(pk, pv, page, pos, start, z(0, 1, 96), z(0, 1, 192), 8, 1, pool_e=e)
    none = _ints(torch, [])
    assert gla.window_attn8_decode_step(pk, pv, none, e, none, z(0, 2, 96), z(0, 1, 96), z(0, 1, 192), 8,
                                        1).shape == (0, 2, 192)
    assert [x.shape[0] for x in gla.window_cache8_read(pk, pv, none, e, 8, 1)] == [0, 0]
    # two sequences of which none has a token in the rows that are there
    o = torch.full((3, 2, 192), 7.0, device="cuda").bfloat16()
    gla.window_attn_chunk(pk, pv, _ints(torch, [0, 1]), _ints(torch, [3, 4]), _ints(torch, [1, 1, 1]), z(3, 2, 96),
                          z(3, 1, 96), z(3, 1, 192), 8, 1, pool_e=e, out=o)
    assert bool((o == 7).all()) and gla.get_device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_one_page_for_two_sequences(env, bits):
    """Drafts that go on from one prompt: reads of the page only, so both may have it."""
    gla, torch, types = env
    rng = np.random.default_rng(3)
    pool, _ = _pool(torch, rng, 2, 200, 2, "bf16", types["bf16"], bits)
    _, (q, k, v) = _new(torch, rng, 6, 4, 2, "bf16", types["bf16"])
    twice = [torch.cat([x, x]) for x in (q, k, v)]
    o = gla.window_attn_chunk(*pool[:2], _ints(torch, [1, 1]), _ints(torch, [777, 777]), _ints(torch, [0, 6, 12]),
                              *twice, 199, 1, pool_e=pool[2])
    assert torch.equal(o[:6], o[6:]) and gla.get_device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_pools_past_32_bits(env, bits):
    """The last page of pools of 2^31 elements and more has the results of a pool of one page."""
    gla, torch, types = env
    gen = torch.Generator(device="cuda").manual_seed(bits)
    window, sink, KV, H, t = 4000, 4, 4, 16, torch.bfloat16
    slots = window + sink
    P = 2 ** 31 // (slots * KV * 192) + 3
    kind = t if bits == 16 else torch.int8
    big = [torch.zeros(P, 1, slots, KV, d, dtype=kind, device="cuda") for d in (96, 192)]
    one = [torch.randn(1, 1, slots, KV, d, generator=gen, device="cuda").to(t) if bits == 16 else
           torch.randint(-127, 128, (1, 1, slots, KV, d), generator=gen, device="cuda").to(torch.int8)
           for d in (96, 192)]
    if bits == 8:
        big.append(torch.zeros(P, 1, KV, slots, 2, dtype=torch.int8, device="cuda"))
        one.append(torch.randint(-8, -5, (1, 1, KV, slots, 2), generator=gen, device="cuda").to(torch.int8))
    else:
        big.append(None)
        one.append(None)
    assert big[1].numel() > 2 ** 31
    for x, y in zip(big, one):
        if x is not None:
            x[-1] = y[0]
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)  # noqa: E731
    for n in (2, 300):
        q, k, v = r(n, H, 96) * 0.1, r(n, KV, 96), r(n, KV, 192)
        outs = []
        for pool, page in ((big, P - 1), (one, 0)):
            page, pos, start = _ints(torch, [page]), _ints(torch, [12345]), _ints(torch, [0, n])
            o = [gla.window_attn_chunk(*pool[:2], page, pos, start, q, k, v, window, sink, pool_e=pool[2])]
            gla.window_cache_append(*pool[:2], page, pos, start, k, v, window, sink, pool_e=pool[2])
            if bits == 8:
                o.append(gla.window_attn8_decode_step(*pool[:2], page, pool[2], pos + n, q[:1], k[:1], v[:1],
                                                      window, sink))
                o += gla.window_cache8_read(*pool[:2], page, pool[2], window, sink)
            outs.append(o + [x[-1].clone() for x in pool if x is not None])
        assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert not big[1][:-1].any() and gla.get_device_error() == 0


def test_rotary_past_32_bits(env):
    gla, torch, types = env
    B, T, H, D = 3, 70000, 110, 96  # 2.2 10^9 elements
    turns = gla.rotary_turns(96).cuda()
    x = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[-1, -50:] = torch.randn(50, H, D, generator=gen, device="cuda").bfloat16()
    tail = x[-1:, -50:].contiguous()
    pos = torch.arange(T - 50, T, dtype=torch.int32, device="cuda")[None]
    want, _ = gla.rotary(tail, None, turns, pos)
    got, _ = gla.rotary(x, None, turns, q_out=x)
    assert torch.equal(got[-1:, -50:], want) and not got[:-1, -50:].any()


def test_long_chunks_over_codes_and_a_page_that_is_not_there(env):
    """Long chunks over 8-bit pages go by a copy of the pages in the workspace: pages that are not full, a
    workspace full of NaN, a layer of several, and a sequence whose page is out of range."""
    gla, torch, types = env
    rng = np.random.default_rng(21)
    new, pos, H, KV, window, sink = [400, 1, 300], [90, 700, 0], 4, 2, 300, 3
    pool, values = _pool(torch, rng, 4, window + sink, KV, "fp16", types["fp16"], 8)
    two = [torch.stack([x[:, 0], torch.full_like(x[:, 0], 127)], 1) for x in pool]  # (layer 1: anything)
    two[2][0, 0, :, 90:] = 127  # exponents of slots that no token has reached
    start = np.concatenate([[0], np.cumsum(new)])
    (q, k, v), dev = _new(torch, rng, int(start[-1]), H, KV, "fp16", types["fp16"])
    size = gla.window_attn_chunk_workspace_size(3, len(q), H, KV, window, sink, bits=8)
    assert size >= 3 * (window + sink) * KV * 288 * 2 > 0
    assert gla.window_attn_chunk_workspace_size(3, len(q), H, KV, window, sink, bits=16) < size
    assert gla.window_attn_chunk_workspace_size(3, len(q), H, KV, window, sink) == size

    def call(page):
        o = torch.full((len(q), H, 192), 7.0, device="cuda").half()
        ws = torch.full((size // 4,), float("nan"), device="cuda")
        gla.window_attn_chunk(two[0], two[1], _ints(torch, page), _ints(torch, pos), _ints(torch, start.tolist()),
                              *dev, window, sink, pool_e=two[2], out=o, workspace=ws)
        return o
    o = call([0, 3, 1])
    _close(o, *ref.chunk(*values, [0, 3, 1], pos, start, q, k, v, window, sink), "fp16")
    assert gla.get_device_error() == 0
    for bad in (4, -1):
        b = call([0, 3, bad])
        assert gla.get_device_error() == 6
        assert bool((b[401:] == 7).all()) and torch.equal(b[:401], o[:401])


def test_a_last_round_of_parts_among_packed_tokens(env):
    """Whole units and parts of the others, of which more might have come than did."""
    gla, torch, types = env
    rng = np.random.default_rng(31)
    n, H, KV, window, sink = 116, 16, 4, 600, 4
    pos = [(37 * b) % 1300 for b in range(n)]
    pool, values = _pool(torch, rng, n, window + sink, KV, "bf16", types["bf16"], 8)
    (q, k, v), dev = _new(torch, rng, n, H, KV, "bf16", types["bf16"])
    page = rng.permutation(n)
    o = gla.window_attn_chunk(*pool[:2], _ints(torch, page.tolist()), _ints(torch, pos),
                              _ints(torch, list(range(n + 1))), *dev, window, sink, pool_e=pool[2])
    _close(o, *ref.chunk(*values, page, pos, np.arange(n + 1), q, k, v, window, sink), "bf16")
    assert gla.get_device_error() == 0


@pytest.mark.parametrize("new,dt", [(4, "bf16"), (4, "fp16"), (5, "fp16"), (6, "bf16"), (7, "bf16"), (8, "fp16")])
@pytest.mark.parametrize("n", [20, 80])
def test_drafts_of_many_sequences(env, n, new, dt):
    """Units of 16, 24 and 32 rows, fewer than two to an SM of 152 and more, and with some sequences a token short."""
    gla, torch, types = env
    rng = np.random.default_rng(n + new)
    H, KV, window, sink = 16, 4, 150, 2
    sizes = [new - (b % 5 == 4) for b in range(n)]
    start = np.concatenate([[0], np.cumsum(sizes)])
    pos = [(53 * b) % 400 for b in range(n)]
    pool, values = _pool(torch, rng, n, window + sink, KV, dt, types[dt], 8)
    (q, k, v), dev = _new(torch, rng, int(start[-1]), H, KV, dt, types[dt])
    page = rng.permutation(n)
    o = gla.window_attn_chunk(*pool[:2], _ints(torch, page.tolist()), _ints(torch, pos),
                              _ints(torch, start.tolist()), *dev, window, sink, pool_e=pool[2])
    _close(o, *ref.chunk(*values, page, pos, start, q, k, v, window, sink), dt)
    assert gla.get_device_error() == 0

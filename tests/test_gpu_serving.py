"""GPU parity of serving with the windowed attention: packed tokens into pages of 16 and 8 bits, pages
read back, chunks of tokens and single ones over them.

What goes into pages is exact on both sides (codes and exponents are whole numbers), so it is compared for
equality.  Attention is bounded as in test_gpu_window_attn.py, with u half a step of the 16-bit type: the
weights round once for the product with v, the output once, |do| <= u (sum p |v| + |o|), sums and scores
in fp32 add less than 1024 roundings of 2^-24 of the sums of magnitudes, and below 2^-14 fp16 rounds by
up to 2^-25 whatever the value (TINY, times |v|; with 8-bit pages the products take c 2^e or c, exactly)."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import layer_ops, serving_ops as ref

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
F = 1024 * 2.0 ** -24
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}
RANGE = 6


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch, {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _npy(t):
    return t.float().cpu().numpy().astype(np.float64)


def _ints(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _draw(rng, dt, *s):
    return as_dtype_values(rng.standard_normal(s).astype(np.float32), dt)


class Pool:
    """Pools of 16 or 8 bits on the device, and the values that they stand for."""

    def __init__(self, torch, rng, P, PL, slots, KV, dt, t, bits):
        self.torch, self.bits, self.t = torch, bits, t
        shape = lambda d: (P, PL, slots, KV, d)  # noqa: E731
        if bits == 16:
            self.k, self.v = (to_dev(_draw(rng, dt, *shape(d)), t) for d in (96, 192))
            self.e = None
        else:
            self.k, self.v = (torch.from_numpy(rng.integers(-127, 128, shape(d)).astype(np.int8)).cuda()
                              for d in (96, 192))
            self.e = torch.from_numpy(rng.integers(-8, -5, (P, PL, KV, slots, 2)).astype(np.int8)).cuda()

    def values(self):
        k, v = _npy(self.k), _npy(self.v)
        if self.e is not None:
            two = 2.0 ** _npy(self.e).transpose(0, 1, 3, 2, 4)
            k, v = k * two[..., :1], v * two[..., 1:]
        return k, v

    def spoil(self, page, layer, slot):
        """Bytes of slots that no token has reached."""
        if self.bits == 16:
            self.k[page, layer, slot:] = float("nan")
            self.v[page, layer, slot:] = float("nan")
        else:
            self.e[page, layer, :, slot:] = 127

    def clone(self):
        p = object.__new__(Pool)
        p.torch, p.bits, p.t = self.torch, self.bits, self.t
        p.k, p.v, p.e = self.k.clone(), self.v.clone(), None if self.e is None else self.e.clone()
        return p

    def same(self, other):
        bits = lambda x: x.view(self.torch.int16) if self.bits == 16 else x  # noqa: E731
        return (self.torch.equal(bits(self.k), bits(other.k)) and
                self.torch.equal(bits(self.v), bits(other.v)) and
                (self.e is None or self.torch.equal(self.e, other.e)))


# ------------------------------------------------------------------------------- pages
APPEND = [  # new tokens, positions, counts, KV, window, sink, layers, type, rows in front and behind
    ([1], [0], None, 1, 1, 0, 1, "bf16", 0, 0),
    ([5, 0, 3], [0, 7, 2], None, 2, 4, 2, 2, "fp16", 2, 3),
    ([40, 33], [3, 100], None, 3, 16, 0, 1, "bf16", 0, 1),          # more than the ring holds
    ([40, 33, 9], [0, 2, 5], [40, 1, 0], 1, 7, 20, 2, "fp16", 1, 0),  # sinks past the window; drafts
    ([1] * 70, list(range(70)), None, 4, 33, 1, 1, "bf16", 0, 0),
    ([2], [2 ** 31 - 3], None, 2, 5, 1, 1, "bf16", 0, 0),           # the last positions of 32 bits
    ([300, 1, 257], [0, 1000, 90], [299, 1, 257], 5, 100, 3, 1, "fp16", 5, 5),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,pos,count,KV,window,sink,PL,dt,front,behind", APPEND)
def test_append(env, new, pos, count, KV, window, sink, PL, dt, front, behind, bits):
    gla, torch, types = env
    rng = np.random.default_rng(sum(new) + bits)
    n, P, slots, layer = len(new), len(new) + 2, window + sink, PL - 1
    start = front + np.concatenate([[0], np.cumsum(new)])
    N = int(start[-1]) + behind
    size = np.exp(rng.standard_normal((N, KV, 1)) * 4).astype(np.float32)  # into fp16's subnormals
    k = as_dtype_values(rng.standard_normal((N, KV, 96)).astype(np.float32) * size, dt)
    v = as_dtype_values(rng.standard_normal((N, KV, 192)).astype(np.float32) / size, dt)
    k[start[0], 0], v[start[0], 0, 3:] = 0, 0
    if dt == "fp16":
        v[start[0], -1, :2] = 65504, -512
        k[start[0], -1] *= np.float32(2.0 ** -12)
        k = as_dtype_values(k, dt)
    page = rng.permutation(P)[:n].astype(np.int32)
    pool = Pool(torch, rng, P, PL, slots, KV, dt, types[dt], bits)
    want = pool.clone()
    kd, vd = to_dev(k, types[dt]), to_dev(v, types[dt])
    if bits == 16:
        rows = [(kd, want.k), (vd, want.v)]
    else:
        (ck, ek), (cv, ev) = ref.codes(k, ref.LOWEST[dt]), ref.codes(v, ref.LOWEST[dt])
        dev = lambda x: torch.from_numpy(x.astype(np.int8)).cuda()  # noqa: E731
        rows = [(dev(ck), want.k), (dev(cv), want.v)]
        e = dev(np.stack([ek, ev], -1))
    for b in range(n):
        for i in range(new[b] if count is None else count[b]):
            s = layer_ops.window_slot(pos[b] + i, window, sink)
            for x, p in rows:
                p[page[b], layer, s] = x[start[b] + i]
            if bits == 8:
                want.e[page[b], layer, :, s] = e[start[b] + i]
    args = (_ints(torch, page.tolist()), _ints(torch, pos), _ints(torch, start.tolist()), kd, vd, window,
            sink, None if count is None else _ints(torch, count))
    gla.window_cache_append(pool.k, pool.v, *args, layer=layer, pool_e=pool.e)
    assert pool.same(want) and gla.get_device_error() == 0
    if bits == 8:
        again = torch.from_numpy(np.concatenate([page, page[:1]])).cuda()  # pages may repeat
        gk, gv = gla.window_cache8_read(pool.k, pool.v, again, pool.e, window, sink, layer=layer,
                                        out_dtype=types[dt])
        rk, rv = pool.values()
        at = np.concatenate([page, page[:1]])
        assert np.array_equal(_npy(gk), rk[at, layer]) and np.array_equal(_npy(gv), rv[at, layer])


@pytest.mark.parametrize("bits", [16, 8])
def test_append_leaves_what_is_out_of_range(env, bits):
    gla, torch, types = env
    rng = np.random.default_rng(5)
    kd, vd = (to_dev(_draw(rng, "bf16", 12, 2, d), types["bf16"]) for d in (96, 192))

    def call(page, pos, start, count=None):
        pool = Pool(torch, np.random.default_rng(6), 3, 1, 5, 2, "bf16", types["bf16"], bits)
        before = pool.clone()
        gla.window_cache_append(pool.k, pool.v, _ints(torch, page), _ints(torch, pos), _ints(torch, start),
                                kd, vd, 4, 1, None if count is None else _ints(torch, count), pool_e=pool.e)
        return [torch.equal(pool.k[p], before.k[p]) and torch.equal(pool.v[p], before.v[p])
                for p in range(3)]
    assert call([1, 0], [0, 3], [0, 4, 8]) == [False, False, True] and gla.get_device_error() == 0
    assert call([3, 0], [0, 3], [0, 4, 8]) == [False, True, True] and gla.get_device_error() == RANGE
    assert call([-1, 0], [0, 3], [0, 4, 8]) == [False, True, True] and gla.get_device_error() == RANGE
    assert call([1, 0], [0, -1], [0, 4, 8]) == [True, False, True] and gla.get_device_error() == RANGE
    assert call([1, 0], [0, 2 ** 31 - 4], [0, 4, 8]) == [True, False, True]
    assert gla.get_device_error() == RANGE
    assert call([1, 0], [0, 3], [0, 4, 13]) == [True, False, True] and gla.get_device_error() == RANGE
    assert call([1, 0], [0, 3], [-1, 4, 8])[0] is False and gla.get_device_error() == RANGE
    # counts past the ends are read as the nearer end
    assert call([1, 0], [0, 3], [0, 4, 8], [-2, 5]) == [False, True, True]
    assert gla.get_device_error() == RANGE
    # a sequence without rows that is out of range is reported too
    assert call([1, 7], [0, 3], [0, 4, 4]) == [True, False, True] and gla.get_device_error() == RANGE


def test_codes_of_what_is_not_finite(env):
    gla, torch, types = env
    for dt in ("fp16", "bf16"):
        rng = np.random.default_rng(9)
        k, v = _draw(rng, dt, 6, 1, 96), _draw(rng, dt, 6, 1, 192)
        k[1, 0, 7], k[2, 0, 30:33], k[3], v[1, 0, 191] = np.inf, np.nan, np.nan, -np.inf
        v[4, 0, ::2], v[5, 0, 0], v[5, 0, 1] = np.nan, np.nan, np.inf
        pool = Pool(torch, rng, 1, 1, 6, 1, dt, types[dt], 8)
        kd, vd = to_dev(k, types[dt]), to_dev(v, types[dt])
        gla.window_cache_append(pool.k, pool.v, _ints(torch, [0]), _ints(torch, [0]), _ints(torch, [0, 6]),
                                kd, vd, 6, 0, pool_e=pool.e)
        for x, c, j in ((k, pool.k, 0), (v, pool.v, 1)):
            want, e = ref.codes(x, ref.LOWEST[dt])
            assert np.array_equal(_npy(c)[0, 0], want) and np.array_equal(_npy(pool.e)[0, 0, :, :, j].T, e)


def test_read_leaves_pages_out_of_range(env):
    gla, torch, types = env
    pool = Pool(torch, np.random.default_rng(7), 3, 2, 6, 2, "fp16", types["fp16"], 8)
    k, v = gla.window_cache8_read(pool.k, pool.v, _ints(torch, [2, 3, -1, 0]), pool.e, 5, 1, layer=1,
                                  out_dtype=torch.float16)
    rk, rv = pool.values()
    assert gla.get_device_error() == RANGE
    assert np.array_equal(_npy(k[0]), rk[2, 1]) and np.array_equal(_npy(v[3]), rv[0, 1])


# ------------------------------------------------------------------------------- chunk
CHUNK = [  # new tokens, positions, H, KV, window, sink, layers, type, output type, rows in front, behind
    ([1], [0], 1, 1, 1, 0, 1, "bf16", "bf16", 0, 0),
    ([1], [7], 2, 1, 1, 0, 1, "fp16", "fp32", 0, 0),                # sees itself alone
    ([3, 0, 5], [0, 4, 2], 3, 1, 4, 2, 2, "fp16", "fp16", 2, 3),
    ([64, 65], [0, 10], 2, 2, 1000, 0, 1, "bf16", "fp32", 0, 0),    # a ring that is not full
    ([130, 1], [128, 129], 4, 2, 128, 0, 1, "fp16", "fp32", 1, 1),
    ([70, 40], [500, 33], 2, 1, 33, 4, 1, "bf16", "bf16", 0, 2),    # sinks far from the window
    ([90], [60], 4, 1, 40, 200, 2, "fp16", "fp16", 0, 0),           # sinks among the new tokens
    ([300], [5], 2, 2, 20, 160, 1, "bf16", "bf16", 3, 0),
    ([17], [100], 5, 1, 100, 3, 1, "bf16", "fp32", 0, 0),           # heads that 128 does not divide
    ([9, 9], [1000, 2], 64, 1, 150, 1, 1, "fp16", "fp16", 0, 0),    # many heads on one key head
    ([1] * 40, [11 * b for b in range(40)], 8, 2, 200, 4, 1, "bf16", "bf16", 0, 0),
    ([5, 4, 3] * 7, [3000 + b for b in range(21)], 16, 4, 260, 4, 3, "fp16", "fp16", 0, 5),
    ([37], [40000], 4, 2, 5000, 16, 1, "bf16", "bf16", 0, 0),       # few rows over a long page
    ([2], [2 ** 31 - 3], 2, 1, 70, 2, 1, "bf16", "bf16", 0, 0),     # the last positions of 32 bits
    ([700, 3], [129, 1], 3, 1, 129, 1, 1, "fp16", "fp16", 0, 0),
]


def _chunk_inputs(env, new, pos, H, KV, window, sink, PL, dt, front, behind, bits):
    gla, torch, types = env
    rng = np.random.default_rng(sum(new) + window + bits)
    n, P, slots, layer = len(new), len(new) + 2, window + sink, PL - 1
    start = front + np.concatenate([[0], np.cumsum(new)])
    N = int(start[-1]) + behind
    q = _draw(rng, dt, N, H, 96) * np.float32(0.25)
    k, v = _draw(rng, dt, N, KV, 96), _draw(rng, dt, N, KV, 192)
    page = rng.permutation(P)[:n].astype(np.int32)
    pool = Pool(torch, rng, P, PL, slots, KV, dt, types[dt], bits)
    values = pool.values()
    for b in range(n):
        if pos[b] < slots:
            pool.spoil(int(page[b]), layer, pos[b])
    qd, kd, vd = (to_dev(x, types[dt]) for x in (q, k, v))
    for x in (qd, kd, vd):  # rows of no sequence
        x[:front], x[int(start[-1]):] = float("nan"), float("nan")
    return q, k, v, page, pool, values, start, N, (qd, kd, vd), layer


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new,pos,H,KV,window,sink,PL,dt,out,front,behind", CHUNK)
def test_chunk_matches_the_definition(env, new, pos, H, KV, window, sink, PL, dt, out, front, behind, bits):
    gla, torch, types = env
    q, k, v, page, pool, values, start, N, dev, layer = _chunk_inputs(
        env, new, pos, H, KV, window, sink, PL, dt, front, behind, bits)
    before = pool.clone()
    o = torch.full((N, H, 192), 7.0, device="cuda").to(types[out])
    args = (pool.k, pool.v, _ints(torch, page.tolist()), _ints(torch, pos), _ints(torch, start.tolist()),
            *dev, window, sink)
    kw = dict(layer=layer, pool_e=pool.e)
    gla.window_attn_chunk(*args, out=o, **kw)
    again = gla.window_attn_chunk(*args, out_dtype=types[out], **kw)
    live = slice(front, int(start[-1]))
    assert torch.equal(o[live], again[live]) and gla.get_device_error() == 0 and pool.same(before)
    assert bool((o[:front] == 7).all()) and bool((o[int(start[-1]):] == 7).all())
    want, pv, av = ref.chunk(*values, page, pos, start, q, k, v, window, sink, layer)
    uo = 2.0 ** -24 if out == "fp32" else U[out]
    room = (U[dt] + F) * pv + TINY[dt] * av + uo * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(_npy(o)[live] - want[live]) <= room[live])


@pytest.mark.parametrize("bits", [16, 8])
def test_chunk_leaves_what_is_out_of_range(env, bits):
    gla, torch, types = env
    new, pos = [5, 3, 70], [9, 50, 2]
    q, k, v, page, pool, _, start, N, dev, layer = _chunk_inputs(env, new, pos, 4, 2, 40, 3, 1, "bf16", 0, 0,
                                                                bits)

    def call(page=page.tolist(), pos=pos, start=start.tolist()):
        o = torch.full((N, 4, 192), 7.0, device="cuda").bfloat16()
        gla.window_attn_chunk(pool.k, pool.v, _ints(torch, page), _ints(torch, pos), _ints(torch, start),
                              *dev, 40, 3, pool_e=pool.e, out=o)
        return o
    want = call()
    assert gla.get_device_error() == 0
    p = page.tolist()
    for bad in (dict(page=[p[0], 99, p[2]]), dict(page=[p[0], -1, p[2]]), dict(pos=[9, -50, 2]),
                dict(pos=[9, 2 ** 31 - 3, 2])):
        o = call(**bad)
        assert gla.get_device_error() == RANGE
        assert bool((o[5:8] == 7).all()) and torch.equal(o[:5], want[:5]) and torch.equal(o[8:], want[8:])
    o = call(start=[0, 5, 8, N + 1])
    assert gla.get_device_error() == RANGE and bool((o[8:] == 7).all()) and torch.equal(o[:8], want[:8])


def test_chunks_of_many_sequences_are_independent(env):
    """A batch of long, short and empty chunks: each sequence has the bits of a call on it alone, with
    the same cut of its keys (none: the batch and the single calls both fill the device or are short)."""
    gla, torch, types = env
    rng = np.random.default_rng(11)
    new = [700] + [0] * 5 + [1, 1, 130, 0, 64] + [1] * 30 + [0, 300, 0]
    pos = [int(x) for x in rng.integers(0, 900, len(new))]
    q, k, v, page, pool, values, start, N, dev, layer = _chunk_inputs(
        env, new, pos, 4, 2, 250, 5, 1, "bf16", 0, 0, 16)
    o = gla.window_attn_chunk(pool.k, pool.v, _ints(torch, page.tolist()), _ints(torch, pos),
                              _ints(torch, start.tolist()), *dev, 250, 5)
    for b, m in enumerate(new):
        if m == 0:
            continue
        rows = slice(int(start[b]), int(start[b + 1]))
        one = gla.window_attn_chunk(pool.k, pool.v, _ints(torch, [int(page[b])]), _ints(torch, [pos[b]]),
                                    _ints(torch, [0, m]), *(x[rows].contiguous() for x in dev), 250, 5)
        # parts of the keys are joined in fp32 where the one call cuts them and the other does not: then a
        # few weights round against another maximum, each by u at most on both sides
        assert (one - o[rows]).abs().max().item() <= 2 * (2 * U["bf16"] + F) * 6
    assert gla.get_device_error() == 0


# -------------------------------------------------------------------------- one token
DECODE = [  # active, pages, layers, H, KV, window, sink, type, output type
    (1, 1, 1, 1, 1, 1, 0, "bf16", "bf16"),
    (3, 7, 2, 4, 2, 5, 2, "fp16", "fp32"),
    (2, 3, 1, 40, 2, 101, 0, "bf16", "bf16"),     # 20 query heads on a key head; an odd number of slots
    (5, 5, 1, 16, 1, 200, 64, "bf16", "fp32"),
    (2, 2, 3, 6, 2, 3001, 4, "fp16", "fp16"),     # slots cut into many parts
    (320, 330, 1, 2, 2, 70, 3, "bf16", "bf16"),   # whole ones, and a last round of parts
    (100, 101, 1, 40, 2, 190, 11, "fp16", "fp32"),
    (152, 152, 1, 2, 2, 70, 3, "fp16", "fp16"),   # a full round of whole ones
]


@pytest.mark.parametrize("N,P,PL,H,KV,window,sink,dt,out", DECODE)
def test_decode8_matches_the_definition(env, N, P, PL, H, KV, window, sink, dt, out):
    gla, torch, types = env
    rng = np.random.default_rng(N + window)
    slots, layer = window + sink, PL - 1
    pool = Pool(torch, rng, P, PL, slots, KV, dt, types[dt], 8)
    q = _draw(rng, dt, N, H, 96) * np.float32(0.25)
    k, v = _draw(rng, dt, N, KV, 96), _draw(rng, dt, N, KV, 192)
    page = rng.permutation(P)[:N].astype(np.int32)
    pos = rng.integers(0, 3 * slots, N).astype(np.int32)
    pos[0] = 0  # an empty page
    if N > 1:
        pos[1] = 2 ** 31 - 2
    values = pool.values()
    for n in range(N):
        if pos[n] < slots:
            pool.spoil(int(page[n]), layer, int(pos[n]))
    start = list(range(N + 1))
    pd, sd = torch.from_numpy(page).cuda(), _ints(torch, start)
    posd = torch.from_numpy(pos).cuda()
    qd, kd, vd = (to_dev(x, types[dt]) for x in (q, k, v))
    want_pool = pool.clone()
    gla.window_cache_append(want_pool.k, want_pool.v, pd, posd, sd, kd, vd, window, sink, layer=layer,
                            pool_e=want_pool.e)
    args = (pool.k, pool.v, pd, pool.e, posd, qd, kd, vd, window, sink)
    o = gla.window_attn8_decode_step(*args, layer=layer, out_dtype=types[out])
    assert pool.same(want_pool) and gla.get_device_error() == 0
    o2 = gla.window_attn8_decode_step(*args, layer=layer, out_dtype=types[out])
    assert torch.equal(o, o2) and pool.same(want_pool)
    want, pv, av = ref.chunk(*values, page, pos.tolist(), start, q, k, v, window, sink, layer)
    uo = 2.0 ** -24 if out == "fp32" else U[out]
    room = (U[dt] + F) * pv + TINY[dt] * av + uo * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(_npy(o) - want) <= room)


def test_decode8_leaves_what_is_out_of_range(env):
    gla, torch, types = env
    for window in (40, 900):  # one part of the slots, several
        pool = Pool(torch, np.random.default_rng(3), 3, 1, window + 1, 1, "fp16", types["fp16"], 8)
        before = pool.clone()
        r = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
        out = torch.full((4, 2, 192), 7.0, device="cuda").half()
        gla.window_attn8_decode_step(pool.k, pool.v, _ints(torch, [3, 1, -1, 0]), pool.e,
                                     _ints(torch, [9, 5, 9, -1]), r(4, 2, 96), r(4, 1, 96), r(4, 1, 192),
                                     window, 1, out=out)
        assert gla.get_device_error() == RANGE
        assert bool((out[[0, 2, 3]] == 7).all()) and not bool((out[1] == 7).any())
        for a, b in ((pool.k, before.k), (pool.v, before.v), (pool.e, before.e)):
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and not torch.equal(a[1], b[1])


# ------------------------------------------------------------------------ all together
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("window,sink", [(40, 3), (300, 0), (7, 30)])
def test_serving_in_chunks_is_one_pass(env, window, sink, bits):
    """Three sequences, rotary positions, prompts in chunks of unequal lengths, then single tokens: with
    pages of 16 bits the rows of one pass over whole sequences.  With 8 bits each key is off by half a
    step, 2^-7 of its row's largest, and the scores by that of sum |q|: bounded through the oracle on the
    pages' own values, token by token."""
    gla, torch, types = env
    B, T, H, KV, split = 3, 90, 4, 2, [[50, 0, 30], [13, 61, 1], [0, 0, 32]]
    rng = np.random.default_rng(window + bits)
    q = to_dev(_draw(rng, "bf16", B, T, H, 96) * np.float32(0.25), types["bf16"])
    k, v = (to_dev(_draw(rng, "bf16", B, T, KV, d), types["bf16"]) for d in (96, 192))
    turns = gla.rotary_turns(96).cuda()
    qr, kr = gla.rotary(q, k, turns)
    whole, _ = gla.window_attn_fwd(qr, kr, v, window, sink, out_dtype=torch.float32)
    pool = Pool(torch, rng, 4, 2, window + sink, KV, "bf16", types["bf16"], bits)
    pool0 = pool.clone()
    page, pos = [2, 0, 3], [0, 0, 0]
    pd = _ints(torch, page)
    steps = [[c[i] for c in split] for i in range(3)]
    while any(p + sum(s[b] for s in steps) < T for b, p in enumerate(pos)):
        left = [T - p - sum(s[b] for s in steps) for b, p in enumerate(pos)]
        steps.append([min(1, x) for x in left])
    for new in steps:
        rows = [(b, pos[b] + i) for b in range(B) for i in range(new[b])]
        bi, ti = (torch.tensor(x, device="cuda") for x in zip(*rows))
        start = [0, *np.cumsum(new).tolist()]
        a, c = gla.rotary(q[bi, ti], k[bi, ti], turns, ti.int())
        val = v[bi, ti].contiguous()
        assert torch.equal(a, qr[bi, ti]) and torch.equal(c, kr[bi, ti])
        args = (pd, _ints(torch, pos), _ints(torch, start))
        values = pool.values()
        single = all(x == 1 for x in new)
        if single and bits == 8:
            o = gla.window_attn8_decode_step(pool.k, pool.v, pd, pool.e, args[1], a, c, val, window, sink,
                                             layer=1, out_dtype=torch.float32)
        else:
            o = gla.window_attn_chunk(pool.k, pool.v, *args, a, c, val, window, sink, layer=1,
                                      pool_e=pool.e, out_dtype=torch.float32)
            gla.window_cache_append(pool.k, pool.v, *args, c, val, window, sink, layer=1, pool_e=pool.e)
        want, pv, _ = ref.chunk(*values, page, pos, start, _npy(a), _npy(c), _npy(val), window, sink, 1)
        assert np.all(np.abs(_npy(o) - want) <= (U["bf16"] + F) * pv + 2.0 ** -24 * np.abs(want) + 2.0 ** -25)
        if bits == 16:
            # both round the weights, each by at most u, and |v| < 5.5
            assert (o - whole[bi, ti]).abs().max().item() <= 2 * (U["bf16"] + F) * 5.5
        pos = [p + m for p, m in zip(pos, new)]
    assert pos == [T] * B and gla.get_device_error() == 0
    assert torch.equal(pool.k[1], pool0.k[1]) and torch.equal(pool.k[:, 0], pool0.k[:, 0])


def test_streams_and_graphs_give_the_same_bits(env):
    gla, torch, types = env
    rng = np.random.default_rng(8)
    pool = Pool(torch, rng, 2, 1, 1204, 2, "bf16", types["bf16"], 8)
    pool16 = Pool(torch, rng, 2, 1, 1204, 2, "bf16", types["bf16"], 16)
    q, k, v = (to_dev(_draw(rng, "bf16", 30, h, d), types["bf16"]) for h, d in ((4, 96), (2, 96), (2, 192)))
    page, pos, start = _ints(torch, [1, 0]), _ints(torch, [1300, 30]), _ints(torch, [0, 10, 30])

    def step(qq, kk, stream=None):
        kw = dict(stream=stream)
        outs = [gla.window_attn_chunk(p.k, p.v, page, pos, start, qq, kk, v, 1200, 4, pool_e=p.e, **kw)
                for p in (pool, pool16)]
        c, c16 = (p.clone() for p in (pool, pool16)) if stream is None else (pool.clone(), pool16.clone())
        for p in (c, c16):
            gla.window_cache_append(p.k, p.v, page, pos, start, kk, v, 1200, 4, pool_e=p.e, **kw)
        outs += [c.k, c.v, c.e, c16.k, c16.v]
        outs.append(gla.window_attn8_decode_step(c.k, c.v, page, c.e, pos + 10, qq[:2].contiguous(),
                                                 kk[:2].contiguous(), v[:2].contiguous(), 1200, 4, **kw))
        return outs + list(gla.window_cache8_read(c.k, c.v, page, c.e, 1200, 4, **kw))
    want = step(q, k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(q, k)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    bq = torch.zeros_like(q)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(bq, k))
        graphs.append(g)
    bq.copy_(q)
    for g, out in zip(graphs, outs):
        g.replay()
        again = step(q, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, out, again))
    assert gla.get_device_error() == 0

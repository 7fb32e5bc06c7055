"""Attention over 8-bit pages whose rows are of unlike sizes: exponents up to the largest that an append writes,
values that grow and shrink along a page, queries and keys far from 1.

Bounds as in test_gpu_serving.py: u of the call's type for the weights and the output, F for sums and scores, and
2^-25 |v| for a weight below fp16's 2^-14.  Over few rows a slot's weight also takes its value's 2^e, relative to a
2^r that is at least 2^-60 and otherwise at most the page's largest 2^e: what falls below fp16's normal range rounds by
up to 2^-25 2^r, times a code of at most 2^7, in units of a sum of weights of at least 1 (the weight of the score
that the others are relative to)."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import serving_ops as ref

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
F = 1024 * 2.0 ** -24
# new tokens of two sequences at H = 4, KV = 2: rows of the few rows' kernel, of the one that turns codes into operands
# in shared memory, and of the one over the pages written out
ROUTES = {"few": 3, "codes": 60, "copy": 200}
LOWEST = {"bf16": -126, "fp16": -24}


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


class Case:
    """n sequences of `new` tokens each on full pages, H = 4, KV = 2."""

    def __init__(self, env, dt, new, window=290, sink=6, n=2, seed=0):
        self.gla, self.torch, types = env
        self.dt, self.t, self.n, self.window, self.sink = dt, types[dt], n, window, sink
        self.rng = rng = np.random.default_rng(100 * new + seed)
        slots, self.N = window + sink, n * new
        self.start, self.pos, self.page = list(range(0, self.N + 1, new)), [3 * slots + 11 * b for b in range(n)], None
        self.page = rng.permutation(n + 1)[:n].tolist()
        self.ck, self.cv = (rng.integers(-127, 128, (n + 1, 1, slots, 2, d)) for d in (96, 192))
        self.e = rng.integers(-8, -5, (n + 1, 1, 2, slots, 2))
        self.q = as_dtype_values(rng.standard_normal((self.N, 4, 96)).astype(np.float32) * np.float32(0.25), dt)
        self.k, self.v = (as_dtype_values(rng.standard_normal((self.N, 2, d)).astype(np.float32), dt)
                          for d in (96, 192))

    def pools(self):
        return [self.torch.from_numpy(x.astype(np.int8)).cuda() for x in (self.ck, self.cv, self.e)]

    def new(self):
        return [to_dev(x.astype(np.float32), self.t) for x in (self.q, self.k, self.v)]

    def want(self):
        two = 2.0 ** self.e.astype(np.float64).transpose(0, 1, 3, 2, 4)
        return ref.chunk(self.ck * two[..., :1], self.cv * two[..., 1:], self.page, self.pos, self.start, self.q,
                         self.k, self.v, self.window, self.sink)

    def chunk(self):
        pk, pv, pe = self.pools()
        return self.gla.window_attn_chunk(pk, pv, *(_ints(self.torch, x) for x in (self.page, self.pos, self.start)),
                                          *self.new(), self.window, self.sink, pool_e=pe)

    def step(self):
        assert self.N == self.n
        pk, pv, pe = self.pools()
        return self.gla.window_attn8_decode_step(pk, pv, _ints(self.torch, self.page), pe, _ints(self.torch, self.pos),
                                                 *self.new(), self.window, self.sink)

    def check(self, o, few):
        want, pv, av = self.want()
        room = (U[self.dt] + F) * pv + U[self.dt] * np.abs(want)
        if few or self.dt == "fp16":
            room = room + 2.0 ** -25 * av
        if few:
            r = max(int(self.e[self.page, 0, :, :, 1].max()), -60)
            room = room + (self.window + self.sink) * 2.0 ** (r + 7 - 25)
        got = o.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        # (fp16 outputs below its normal values round by half of 2^-24)
        off = np.abs(got - want) - room - (2.0 ** -25 if self.dt == "fp16" else 0.0)
        assert np.all(off <= 0), (off.max(), np.abs(want).max())
        assert self.gla.get_device_error() == 0


@pytest.mark.parametrize("route", list(ROUTES))
@pytest.mark.parametrize("e", [103, 104, 105, 112, 121])
def test_large_values_of_bf16(env, route, e):
    """A few rows of values of up to 2^112 or 2^121 among ordinary ones.  (Scores within about 1 of each other, and codes
    of at most 7 with 2^121: the sums of weighted values stay below fp32's 2^128.)"""
    c = Case(env, "bf16", ROUTES[route], seed=e)
    c.q *= np.float32(2.0 ** -5)
    big = c.rng.permutation(296)[:1 if e == 121 else 8]
    c.e[:, 0, :, big, 1] = e
    if e == 121:
        c.cv[:, 0, big] = c.cv[:, 0, big] // 18
    c.check(c.chunk(), route == "few")


@pytest.mark.parametrize("route,up", [("few", 80), ("few", 100), ("few", 112), ("codes", 96), ("codes", 105), ("codes", 112),
                                      ("copy", 112)])
def test_large_keys_of_bf16(env, route, up):
    """Keys of about 2^up and queries as much smaller: the scores of ordinary ones."""
    c = Case(env, "bf16", ROUTES[route], seed=up)
    c.e[..., 0] += up + 7
    c.k = c.k * 2.0 ** (up + 7)
    c.q = as_dtype_values(c.q * np.float32(2.0 ** -(up + 7)), "bf16")  # (the smallest are subnormal)
    c.check(c.chunk(), route == "few")


@pytest.mark.parametrize("dt,held", [("bf16", 127 * 2.0 ** 121), ("fp16", 127 * 2.0 ** 9)])
@pytest.mark.parametrize("route", list(ROUTES))
def test_an_infinity_is_held_as_the_largest_code(env, route, dt, held):
    """A value that was infinite counts with its weight; weights are all the same here (no query)."""
    c = Case(env, dt, ROUTES[route])
    c.q[:] = 0
    pk, pv, pe = c.pools()
    inf = c.torch.zeros(1, 2, 192, dtype=c.t, device="cuda")
    inf[0, 0, 5], inf[0, 0, 7] = float("inf"), float("-inf")
    at = 2 * 296 + 100  # a token that all of these see; its slot
    c.gla.window_cache_append(pk, pv, _ints(c.torch, [c.page[0]]), _ints(c.torch, [at]), _ints(c.torch, [0, 1]),
                              c.torch.zeros(1, 2, 96, dtype=c.t, device="cuda"), inf, c.window, c.sink, pool_e=pe)
    o = c.gla.window_attn_chunk(pk, pv, *(_ints(c.torch, x) for x in (c.page, c.pos, c.start)), *c.new(), c.window,
                                c.sink, pool_e=pe)
    slot = ref.window_slot(at, c.window, c.sink)
    c.ck[c.page[0], 0, slot], c.cv[c.page[0], 0, slot] = 0, 0
    c.e[c.page[0], 0, :, slot] = LOWEST[dt]
    c.cv[c.page[0], 0, slot, 0, 5], c.cv[c.page[0], 0, slot, 0, 7] = 127, -127
    c.e[c.page[0], 0, 0, slot, 1] = 121 if dt == "bf16" else 9
    assert 127 * 2.0 ** c.e[c.page[0], 0, 0, slot, 1] == held
    for x, y in zip((pk, pv, pe), c.pools()):
        assert c.torch.equal(x, y)
    c.check(o, route == "few")


def _sizes(rng, how, slots, lo, hi):
    ramp = np.linspace(lo, hi, slots).round().astype(int)
    if how == "one":
        e = np.full(slots, lo)
        e[rng.integers(slots)] = hi
        return e
    return {"up": ramp, "down": ramp[::-1], "any": rng.integers(lo, hi + 1, slots)}[how]


@pytest.mark.parametrize("how", ["up", "down", "any", "one"])
@pytest.mark.parametrize("dt,lo,hi", [("bf16", -30, 10), ("bf16", -68, -57), ("bf16", -126, 60), ("fp16", -24, 8)])
@pytest.mark.parametrize("new,n,window", [(1, 2, 290), (3, 2, 290), (16, 2, 700), (9, 40, 130), (1, 300, 1100)])
def test_values_that_grow_and_shrink(env, new, n, window, dt, lo, hi, how):
    """Over few rows: the reference of the weights moves up along the page, in parts of it too."""
    c = Case(env, dt, new, window=window, n=n, seed=n)
    for p in range(n + 1):
        for kv in range(2):
            c.e[p, 0, kv, :, 1] = _sizes(c.rng, how, window + c.sink, lo, hi)
    c.v = as_dtype_values(c.v * np.float32(2.0 ** max(lo + 7, -90)), dt)  # as small as the smallest there
    c.check(c.chunk(), True)
    if new == 1:
        c.check(c.step(), True)


@pytest.mark.parametrize("route", list(ROUTES))
@pytest.mark.parametrize("up", [-60, -20, 30, 90])
def test_queries_far_from_one(env, route, up):
    """Queries times 2^up, another power for each head, and keys as much smaller.  (Queries of a head are taken into
    fp16's range by a power of two.)"""
    c = Case(env, "bf16", ROUTES[route], seed=abs(up))
    by = up + np.array([0, 0, 5, 5])  # of the heads; KV heads 0 and 1
    c.q = c.q * 2.0 ** by[:, None]
    c.e[..., 0] -= by[::2][:, None]
    c.k = c.k * 2.0 ** -by[::2][:, None]
    c.check(c.chunk(), route == "few")

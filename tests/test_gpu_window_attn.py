"""GPU parity of the windowed attention (forward, gradient, cache fill, decode step) against the
fp64 definition.

Bounds, with u half a step of the 16-bit type and p the softmax weights: the kernels round p once
(relative u) for the product with v, and the output once, so |do| <= u (sum p |v| + |o|).  dv has
the same form.  The gradient's delta takes the rounded o, off by sum |dO| |do|, and dz = p (dp -
delta) rounds once, so dq is off by u (sum |dz| |k| + |dq|) + sum p ddelta |k|, dk alike.  Sums
and scores in fp32 add less than 1024 roundings of 2^-24 of the sums of magnitudes.  Below 2^-14
fp16 has steps of 2^-24, so there a rounding is off by up to 2^-25 whatever the value: each p and
dz (for o: each exp(z - m), divided by a sum of at least 1) adds TINY times what it multiplies."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import layer_ops as ref

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
    return gla, torch, {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(seed, B, T, H, KV, dt):
    rng = np.random.default_rng(seed)
    draw = lambda s, *n: as_dtype_values((s * rng.standard_normal(n)).astype(np.float32), dt)  # noqa: E731
    return (draw(2 * 96 ** -0.5, B, T, H, 96), draw(1, B, T, KV, 96), draw(1, B, T, KV, 192),
            draw(1, B, T, H, 192))


def _npy(t):
    return t.float().cpu().numpy().astype(np.float64)


def _weights(q, k, b, h, G, window, sink, n):
    """Dense softmax weights [n, n] of one head."""
    t = np.arange(n)
    ok = (t[None] <= t[:, None]) & ((t[:, None] - t[None] < window) | (t[None] < sink))
    z = q[b, :n, h].astype(np.float64) @ k[b, :n, h // G].astype(np.float64).T
    z = np.where(ok, z, -np.inf)
    p = np.exp(z - z.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


CASES = [  # B, T, H, KV, window, sink, type, output type, lengths
    (1, 1, 1, 1, 1, 0, "bf16", "bf16", None),
    (2, 5, 3, 1, 2, 1, "fp16", "fp16", [5, 0]),
    (1, 64, 2, 2, 1, 0, "bf16", "fp32", None),          # every query sees itself alone
    (1, 65, 2, 1, 64, 0, "bf16", "bf16", None),
    (2, 130, 4, 2, 500, 0, "fp16", "fp32", [130, 1]),   # a window past T: plain causal attention
    (1, 300, 2, 1, 33, 4, "bf16", "bf16", None),        # sinks in a tile far from the window
    (2, 257, 4, 1, 40, 70, "fp16", "fp16", [257, 129]), # more sinks than one tile, than the window
    (1, 200, 2, 2, 7, 1000, "bf16", "bf16", None),      # every token a sink
    (3, 150, 6, 2, 64, 16, "bf16", "fp32", [64, 128, 150]),
    (1, 700, 1, 1, 129, 1, "fp16", "fp16", None),
    (1, 700, 2, 1, 20, 600, "bf16", "bf16", [650]),     # more tiles of sinks than are cut up
    (2, 900, 2, 2, 1, 140, "fp16", "fp32", [900, 333]), # far queries in many parts
]


@pytest.mark.parametrize("B,T,H,KV,window,sink,dt,out,lens", CASES)
def test_matches_the_definition(env, B, T, H, KV, window, sink, dt, out, lens):
    gla, torch, types = env
    q, k, v, dO = _inputs(T + window, B, T, H, KV, dt)
    qd, kd, vd, gd = (to_dev(x, types[dt]) for x in (q, k, v, dO))
    ld = None
    if lens is not None:
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):  # nothing there may be read
            for x in (qd, kd, vd, gd):
                x[b, n:] = float("nan")
    o, lse = gla.window_attn_fwd(qd, kd, vd, window, sink, ld, out_dtype=types[out])
    ob, lb = o.clone(), lse.clone()
    for b, n in enumerate(lens or []):
        ob[b, n:] = float("nan")
        lb[b, :, n:] = float("nan")
    got = gla.window_attn_bwd(qd, kd, vd, ob, lb, gd, window, sink, ld)
    again = gla.window_attn_bwd(qd, kd, vd, ob, lb, gd, window, sink, ld)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # o as a view of a [B,H,T,192] tensor gives the same bits
    view = ob.transpose(1, 2).contiguous().transpose(1, 2)
    again = gla.window_attn_bwd(qd, kd, vd, view, lb, gd, window, sink, ld)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert o.dtype == got[0].dtype == types[out] and gla.get_device_error() == 0
    o_r, lse_r = ref.window_attn_fwd(q, k, v, window, sink, lens)
    g_r = ref.window_attn_bwd(q, k, v, dO, window, sink, lens)
    u, uo, G = U[dt], 2.0 ** -24 if out == "fp32" else U[out], H // KV
    do = uo * np.abs(o_r)
    slack = [uo * np.abs(x) for x in g_r]
    for b in range(B):
        n = T if lens is None else lens[b]
        for h in range(H):
            if n == 0:
                continue
            p = _weights(q, k, b, h, G, window, sink, n)
            K, V, D = (np.abs(x.astype(np.float64)) for x in (k[b, :n, h // G], v[b, :n, h // G],
                                                            dO[b, :n, h]))
            do[b, :n, h] += (u + F) * (p @ V) + TINY[dt] * ((p > 0) @ V)
            dd = (D * do[b, :n, h]).sum(1)[:, None] + F * (D * (p @ V)).sum(1)[:, None]
            dp = dO[b, :n, h].astype(np.float64) @ v[b, :n, h // G].astype(np.float64).T
            dz = np.abs(p * (dp - (p * dp).sum(1)[:, None]))
            ez = (u + F) * dz + p * dd + F * p * (D @ V.T) + TINY[dt] * (p > 0)
            slack[0][b, :n, h] += ez @ K
            slack[1][b, :n, h // G] += ez.T @ np.abs(q[b, :n, h].astype(np.float64))
            slack[2][b, :n, h // G] += (u + F) * (p.T @ D) + TINY[dt] * ((p > 0).T @ D)
    assert np.all(np.abs(_npy(o) - o_r) <= do + 2.0 ** -25)
    live = np.isfinite(lse_r)
    lg = _npy(lse)
    assert np.array_equal(live, np.isfinite(lg)) and np.all(lg[~live] == -np.inf)
    A = (np.abs(q).sum(-1).max() * np.abs(k).max())
    assert np.all(np.abs(lg[live] - lse_r[live]) <= 2.0 ** -24 * (96 * A + T + 64))
    for name, x, r, s in zip(("dq", "dk", "dv"), got, g_r, slack):
        worst = np.max(np.abs(_npy(x) - r) - s)
        assert worst <= 2.0 ** -25, (name, worst)


def test_bad_length_is_recorded_and_clamped(env):
    gla, torch, types = env
    q, k, v, _ = (to_dev(x, types["bf16"]) for x in _inputs(1, 2, 70, 2, 1, "bf16"))
    lens = torch.tensor([-1, 71], dtype=torch.int32, device="cuda")
    o, lse = gla.window_attn_fwd(q, k, v, 16, 2, lens)
    assert gla.get_device_error() == 6
    o2, lse2 = gla.window_attn_fwd(q, k, v, 16, 2, lens.clamp(0, 70))
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and gla.get_device_error() == 0


DECODE = [  # active, pages, layers, H, KV, window, sink, type, output type
    (1, 1, 1, 1, 1, 1, 0, "bf16", "bf16"),
    (3, 7, 2, 4, 2, 5, 2, "fp16", "fp32"),
    (2, 3, 1, 40, 2, 100, 0, "bf16", "bf16"),     # 20 query heads on a key head: two groups
    (5, 5, 1, 16, 1, 200, 64, "bf16", "fp32"),
    (2, 2, 3, 6, 2, 3000, 4, "fp16", "fp16"),     # slots cut into many parts
    (320, 330, 1, 2, 2, 70, 3, "bf16", "bf16"),   # whole ones, and a last round of parts
    (100, 101, 1, 40, 2, 190, 10, "bf16", "fp32"),  # the same with two groups
    (152, 152, 1, 2, 2, 70, 3, "fp16", "fp16"),   # a full round of whole ones
]


@pytest.mark.parametrize("N,P,PL,H,KV,window,sink,dt,out", DECODE)
def test_decode_matches_the_definition(env, N, P, PL, H, KV, window, sink, dt, out):
    gla, torch, types = env
    rng = np.random.default_rng(N + window)
    slots, layer, G = window + sink, PL - 1, H // KV
    draw = lambda *s: as_dtype_values(rng.standard_normal(s).astype(np.float32), dt)  # noqa: E731
    pk, pv = draw(P, PL, slots, KV, 96), draw(P, PL, slots, KV, 192)
    q, k, v = draw(N, H, 96) * np.float32(0.25), draw(N, KV, 96), draw(N, KV, 192)
    page = rng.permutation(P)[:N].astype(np.int32)
    pos = rng.integers(0, 3 * slots, N).astype(np.int32)
    pos[0] = 0  # an empty cache
    if N > 1:
        pos[1] = 2 ** 31 - 1  # the last position of 32 bits
    o_r, pk_r, pv_r = ref.window_attn_decode_step(pk, pv, page, pos, q, k, v, window, sink, layer)
    # slots that a sequence has not filled yet are not read
    pkd, pvd = to_dev(pk, types[dt]), to_dev(pv, types[dt])
    for n in range(N):
        pkd[page[n], layer, int(pos[n]) + 1:] = float("nan")
        pvd[page[n], layer, int(pos[n]) + 1:] = float("nan")
    want_k, want_v = pkd.clone(), pvd.clone()
    kd, vd = to_dev(k, types[dt]), to_dev(v, types[dt])
    for n in range(N):
        s = ref.window_slot(int(pos[n]), window, sink)
        want_k[page[n], layer, s], want_v[page[n], layer, s] = kd[n], vd[n]
    args = (pkd, pvd, torch.from_numpy(page).cuda(), torch.from_numpy(pos).cuda(),
            to_dev(q, types[dt]), kd, vd, window, sink)
    o = gla.window_attn_decode_step(*args, layer=layer, out_dtype=types[out])
    o2 = gla.window_attn_decode_step(*args, layer=layer, out_dtype=types[out])
    assert torch.equal(o, o2) and gla.get_device_error() == 0
    bits = lambda x: x.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(pkd), bits(want_k)) and torch.equal(bits(pvd), bits(want_v))
    u, uo = U[dt], 2.0 ** -24 if out == "fp32" else U[out]
    for n in range(N):
        m = min(int(pos[n]) + 1, slots)
        for h in range(H):
            z = pk_r[page[n], layer, :m, h // G] @ q[n, h].astype(np.float64)
            p = np.exp(z - z.max())
            p /= p.sum()
            V = np.abs(pv_r[page[n], layer, :m, h // G])
            slack = (u + F) * (p @ V) + TINY[dt] * V.sum(0) + uo * np.abs(o_r[n, h])
            assert np.all(np.abs(_npy(o[n, h]) - o_r[n, h]) <= slack + 2.0 ** -25)


def test_bad_pages_and_positions_are_left_alone(env):
    gla, torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    for window in (40, 900):  # one part of the slots, several
        pk, pv = r(3, 1, window + 1, 1, 96), r(3, 1, window + 1, 1, 192)
        page = torch.tensor([3, 1, -1, 0], dtype=torch.int32, device="cuda")
        pos = torch.tensor([9, 5, 9, -1], dtype=torch.int32, device="cuda")
        bk, bv = pk.clone(), pv.clone()
        out = torch.full((4, 2, 192), 7.0, device="cuda").half()
        gla.window_attn_decode_step(pk, pv, page, pos, r(4, 2, 96), r(4, 1, 96), r(4, 1, 192),
                                    window, 1, out=out)
        assert gla.get_device_error() == 6
        assert bool((out[[0, 2, 3]] == 7).all()) and not bool((out[1] == 7).any())
        assert torch.equal(pk[[0, 2]], bk[[0, 2]]) and torch.equal(pv[[0, 2]], bv[[0, 2]])
        assert not torch.equal(pk[1], bk[1])
        bk, bv = pk.clone(), pv.clone()
        gla.window_cache_fill(pk, pv, page[:3].contiguous(), r(3, 9, 1, 96), r(3, 9, 1, 192),
                              window, 1)
        assert gla.get_device_error() == 6
        assert torch.equal(pk[[0, 2]], bk[[0, 2]]) and not torch.equal(pk[1], bk[1])


@pytest.mark.parametrize("T,window,sink,lens", [
    (1, 1, 0, None), (50, 64, 4, None), (300, 33, 4, [300, 40, 0]), (129, 128, 1, [129, 5, 64])])
def test_fill_then_decode_goes_on_as_one_pass(env, T, window, sink, lens):
    """Prompts into the caches, then tokens one at a time = one pass over the whole sequences."""
    gla, torch, types = env
    B, H, KV, more = 3, 4, 2, 40
    lens = lens or [T] * B
    q, k, v, _ = _inputs(T, B, T + more, H, KV, "bf16")
    qd, kd, vd = (to_dev(x, types["bf16"]) for x in (q, k, v))
    pk = torch.full((4, 2, window + sink, KV, 96), 3.0, device="cuda").bfloat16()
    pv = torch.full((4, 2, window + sink, KV, 192), 3.0, device="cuda").bfloat16()
    page = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gla.window_cache_fill(pk, pv, page, kd[:, :T].contiguous(), vd[:, :T].contiguous(), window,
                          sink, ld, layer=1)
    wk, wv = ref.window_cache_fill(np.full(pk.shape, 3.0), np.full(pv.shape, 3.0), page.tolist(),
                                   k[:, :T], v[:, :T], window, sink, 1, lens)
    assert np.array_equal(_npy(pk), wk) and np.array_equal(_npy(pv), wv)
    o, _ = gla.window_attn_fwd(qd, kd, vd, window, sink, out_dtype=torch.float32)
    rows = torch.arange(B, device="cuda")
    for step in range(more):
        pos = ld + step
        at = pos.long()
        one = gla.window_attn_decode_step(pk, pv, page, pos, qd[rows, at], kd[rows, at],
                                          vd[rows, at], window, sink, layer=1,
                                          out_dtype=torch.float32)
        # both sides round the weights, each by at most u, and |v| < 5.5
        assert (one - o[rows, at]).abs().max().item() <= 2 * (U["bf16"] + F) * 5.5
    assert bool((pk[1] == 3).all()) and bool((pk[:, 0] == 3).all())


def test_streams_and_graphs_give_the_same_bits(env):
    gla, torch, types = env
    q, k, v, dO = (to_dev(x, types["bf16"]) for x in _inputs(3, 2, 200, 4, 2, "bf16"))
    pk = torch.randn(2, 1, 604, 2, 96, device="cuda").bfloat16()
    pv = torch.randn(2, 1, 604, 2, 192, device="cuda").bfloat16()
    page, pos = torch.tensor([[1, 0], [700, 30]], dtype=torch.int32, device="cuda")

    def step(qq, stream=None):
        o, lse = gla.window_attn_fwd(qq, k, v, 50, 4, stream=stream)
        grads = gla.window_attn_bwd(qq, k, v, o, lse, dO, 50, 4, stream=stream)
        one = gla.window_attn_decode_step(pk, pv, page, pos, qq[:, 0].contiguous(),
                                          k[:, 0].contiguous(), v[:, 0].contiguous(), 600, 4,
                                          stream=stream)
        return [o, lse, *grads, one]
    want = step(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(q, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    bq = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(bq)
    bq.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("sink", [0, 5])
def test_sequences_of_a_ragged_batch_are_independent(env, sink):
    """Many empty and short sequences between long ones, more items than CTAs: every sequence has
    the bits of the call on it alone, padding is zero."""
    gla, torch, _ = env
    B, T, H, KV = 30, 1500, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dO = r(B, T, H, 96) * 0.2, r(B, T, KV, 96), r(B, T, KV, 192), r(B, T, H, 192)
    lens = [1500] + [0] * 9 + [640, 1, 0, 129] + [0] * 7 + [1499] + [64] * 4 + [0, 1000, 0, 0]
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = gla.window_attn_fwd(q, k, v, 200, sink, ld)
    got = gla.window_attn_bwd(q, k, v, o, lse, dO, 200, sink, ld)
    assert gla.get_device_error() == 0
    for b, n in enumerate(lens):
        assert not o[b, n:].any() and all(not g[b, n:].any() for g in got)
        if n == 0:
            continue
        one = [x[b:b + 1] for x in (q, k, v)]
        ob, lb = gla.window_attn_fwd(*one, 200, sink, ld[b:b + 1])
        gb = gla.window_attn_bwd(*one, ob, lb, dO[b:b + 1], 200, sink, ld[b:b + 1])
        assert torch.equal(ob[0], o[b]) and torch.equal(lb[0], lse[b])
        assert all(torch.equal(x[0], y[b]) for x, y in zip(gb, got))

"""GPU parity of the gated scan (forward, gradient, decode step, paged decode step) against the
fp64 definition, and the calls at its edges: lengths of zero and one, padding full of NaN, gates
that keep or reset the state, bad lengths and pages, streams and graphs.

Bound: in fp32 a token's gate is off by at most 32 roundings (the exponent |g| log2(e) carries
|g| <= 20 of them), which the sums sum(u_t prod f) <= 1 pass on once; each step and each join of
partial scans adds at most four roundings of the largest value M in play.  So no value is off by
more than (4 T + 64) 2^-24 M."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu


def _bound(T, M):
    return (4 * T + 64) * 2.0 ** -24 * M


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch


def _inputs(seed, B, T, D, dt):
    rng = np.random.default_rng(seed)
    draw = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    x = as_dtype_values(draw(B, T, D), dt)
    g = as_dtype_values(2 * draw(B, T, D) + 2, dt)
    return x, g, draw(B, T, D), draw(B, D), draw(B, D)


CASES = [  # B, T, D, type, states, lengths
    (1, 1, 1, "fp32", True, None),
    (2, 1, 64, "bf16", False, None),
    (2, 31, 63, "bf16", True, None),           # one lane short of a slab, odd rows
    (3, 33, 65, "fp16", True, [33, 0, 1]),
    (1, 64, 130, "bf16", True, None),
    (2, 257, 96, "fp32", True, [257, 100]),    # clusters of several CTAs, ragged tiles
    (1, 1025, 66, "bf16", False, None),
    (5, 128, 200, "fp16", True, [128, 127, 65, 64, 2]),
    (40, 70, 512, "bf16", True, None),         # one CTA per sequence and slab
    (1, 700, 33, "bf16", True, [650]),         # odd rows, a cluster of 8
    (2, 300, 66, "fp32", True, [300, 129]),    # rows of pairs, a cluster of 4
    (30, 200, 130, "fp16", True, None),
    (60, 130, 66, "bf16", False, None),        # ... and of 2
    (60, 130, 64, "bf16", True, [130] * 30 + [64] * 29 + [0]),  # the same from 16-byte rows
    (30, 129, 65, "fp32", True, None),
    (1, 1400, 72, "fp16", True, [1399]),       # more rounds than the ring holds
]


@pytest.mark.parametrize("B,T,D,dt,states,lens", CASES)
def test_matches_the_definition(env, B, T, D, dt, states, lens):
    gla, torch = env
    x, g, dy, init, dfin = _inputs(T + D, B, T, D, dt)
    if not states:
        init = dfin = None
    td = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dt]
    f32 = torch.float32
    xd, gd, dyd = to_dev(x, td), to_dev(g, td), to_dev(dy, f32)
    idd = None if init is None else to_dev(init, f32)
    fdd = None if dfin is None else to_dev(dfin, f32)
    ld = None
    if lens is not None:
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):  # nothing there may be read
            for p in (xd, gd, dyd):
                p[b, n:] = float("nan")
    y, fin = gla.gated_scan_fwd(xd, gd, idd, ld)
    ybwd = y.clone()
    if lens is not None:
        for b, n in enumerate(lens):
            ybwd[b, n:] = float("nan")
    dx, dg, dinit = gla.gated_scan_bwd(xd, gd, ybwd, dyd, idd, fdd, ld)
    again = gla.gated_scan_bwd(xd, gd, ybwd, dyd, idd, fdd, ld)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, dinit), again))
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    y_r, fin_r = ref.gated_scan_fwd(x, g, init, lens)
    dx_r, dg_r, dinit_r = ref.gated_scan_bwd(x, g, dy, init, dfin, lens)
    M = max(np.abs(x).max(), 0 if init is None else np.abs(init).max())
    # |G| <= what ones for gates of keeping, the largest memory, would give: taken from dx / u
    G = np.abs(dx_r / ref.sigmoid(-g)).max() + 0.0
    G = max(G, 0 if dfin is None else np.abs(dfin).max())
    for name, got, want, m in (("y", y, y_r, M), ("final", fin, fin_r, M), ("dx", dx, dx_r, G),
                               ("d_init", dinit, dinit_r, G), ("dg", dg, dg_r, G * 2 * M)):
        err = np.abs(got.cpu().numpy().astype(np.float64) - want).max()
        assert err <= _bound(T, m), (name, err, _bound(T, m))


def test_gates_of_infinity_keep_and_reset_exactly(env):
    gla, torch = env
    x = torch.randn(2, 100, 40, device="cuda")
    init = torch.randn(2, 40, device="cuda")
    y, fin = gla.gated_scan_fwd(x, torch.full_like(x, float("inf")), init)
    assert torch.equal(y, init[:, None].expand_as(y)) and torch.equal(fin, init)
    y, _ = gla.gated_scan_fwd(x, torch.full_like(x, float("-inf")), init)
    assert torch.equal(y, x)
    dx, dg, di = gla.gated_scan_bwd(x, torch.full_like(x, float("inf")), y, torch.ones_like(x),
                                    init)
    assert not dx.any() and not dg.any() and torch.equal(di, torch.full_like(di, 100.0))


def test_long_sequence_matches_its_pieces(env):
    """The clustered scan over a long sequence = the pieces run one after the other."""
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 5001, 64, generator=gen, device="cuda").bfloat16()
    g = (torch.randn(1, 5001, 64, generator=gen, device="cuda") + 3).bfloat16()
    y, fin = gla.gated_scan_fwd(x, g)
    state, parts = None, []
    for lo in range(0, 5001, 700):
        p, state = gla.gated_scan_fwd(x[:, lo:lo + 700].contiguous(),
                                      g[:, lo:lo + 700].contiguous(), state)
        parts.append(p)
    M = x.float().abs().max().item()
    assert (torch.cat(parts, 1) - y).abs().max().item() <= 2 * _bound(5001, M)
    assert (state - fin).abs().max().item() <= 2 * _bound(5001, M)


def test_bad_length_is_recorded_and_clamped(env):
    gla, torch = env
    x = torch.randn(3, 10, 8, device="cuda")
    lens = torch.tensor([11, -4, 5], dtype=torch.int32, device="cuda")
    y, fin = gla.gated_scan_fwd(x, x, None, lens)
    assert gla.get_device_error() == 6
    want, wfin = gla.gated_scan_fwd(x, x, None, lens.clamp(0, 10))
    assert torch.equal(y, want) and torch.equal(fin, wfin) and gla.get_device_error() == 0


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (7, "fp16"), (100, "fp32"), (2, "bf16")])
def test_decode_is_the_scan_token_by_token(env, D, dt):
    gla, torch = env
    x, g, _, init, _ = _inputs(D, 3, 6, D, dt)
    td = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dt]
    y_r, _ = ref.gated_scan_fwd(x, g, init)
    xd, gd, state = to_dev(x, td), to_dev(g, td), to_dev(init, torch.float32)
    pool = torch.randn(5, 3, D, device="cuda")
    page = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[page.long(), 1] = state
    before = pool.clone()
    for t in range(6):
        y = gla.gated_scan_decode_step(state, xd[:, t].contiguous(), gd[:, t].contiguous())
        yp = gla.gated_scan_decode_step_paged(pool, page, xd[:, t:t + 1].contiguous(),
                                              gd[:, t:t + 1].contiguous(), layer0=1)
        assert torch.equal(y, state) and torch.equal(yp[:, 0], y)
        err = np.abs(y.cpu().numpy() - y_r[:, t]).max()
        assert err <= _bound(t + 1, max(np.abs(x).max(), np.abs(init).max()))
    assert torch.equal(pool[page.long(), 1], state)
    before[page.long(), 1] = state
    assert torch.equal(pool, before)  # other pages and layers as they were
    assert gla.get_device_error() == 0


def test_bad_page_is_left_alone(env):
    gla, torch = env
    pool = torch.randn(4, 1, 8, device="cuda")
    page = torch.tensor([1, 4, -1, 3], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 1, 8, device="cuda")
    before, y = pool.clone(), torch.full((4, 1, 8), 7.0, device="cuda")
    gla.gated_scan_decode_step_paged(pool, page, x, x, out=y)
    assert gla.get_device_error() == 6
    assert torch.equal(pool[[0, 2]], before[[0, 2]]) and bool((y[1:3] == 7).all())
    assert not torch.equal(pool[[1, 3]], before[[1, 3]])


def test_streams_and_graphs_give_the_same_bits(env):
    gla, torch = env
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g, dy = (torch.randn(2, 300, 96, generator=gen, device="cuda") for _ in range(3))
    init = torch.randn(2, 96, generator=gen, device="cuda")
    y, fin = gla.gated_scan_fwd(x, g, init)
    grads = gla.gated_scan_bwd(x, g, y, dy, init, fin)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, fin2 = gla.gated_scan_fwd(x, g, init, stream=side)
    grads2 = gla.gated_scan_bwd(x, g, y2, dy, init, fin2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    bx = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yc, fc = gla.gated_scan_fwd(bx, g, init)
        gc = gla.gated_scan_bwd(bx, g, yc, dy, init, fc)
    bx.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yc, y) and torch.equal(fc, fin)
    assert all(torch.equal(a, b) for a, b in zip(gc, grads))

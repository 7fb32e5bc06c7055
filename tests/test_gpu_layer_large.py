"""The operators around the mixer on tensors of more than 2^31 elements, and in calls that run at
the same time: each result has the bits of the same call on a small tensor, alone."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    yield gla, torch
    torch.cuda.empty_cache()


def _rand(torch, *s, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(s))
    return torch.randn(*s, generator=gen, device="cuda").to(dtype)


def _behind(torch, B, one):
    """[B, ...] whose last entry is `one` [1, ...]; the others are not set."""
    t = torch.empty(B, *one.shape[1:], dtype=one.dtype, device="cuda")
    t[-1:] = one
    return t


@pytest.mark.parametrize("D", [2048, 2046])
def test_gated_scan(env, D):
    gla, torch = env
    T = 4096
    B = 2 ** 31 // (T * D) + 2
    x1, g1 = (_rand(torch, 1, T, D, dtype=torch.bfloat16) for _ in range(2))
    dy1 = _rand(torch, 1, T, D, dtype=torch.float32)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = T - 3
    x, g, dy = _behind(torch, B, x1), _behind(torch, B, g1 + 1), _behind(torch, B, dy1)
    assert x.numel() > 2 ** 31
    y, fin = gla.gated_scan_fwd(x, g, None, lens)
    got = gla.gated_scan_bwd(x, g, y, dy, None, None, lens)
    # the cut into clusters depends on B: other joins of the partial scans, each step and join four
    # roundings of values of at most 6
    y1, fin1 = gla.gated_scan_fwd(x1, g1 + 1, None, lens[-1:].clone())
    tol = (4 * T + 64) * 2.0 ** -24 * 6
    assert (y[-1] - y1[0]).abs().max() <= tol and (fin[-1] - fin1[0]).abs().max() <= tol
    one = gla.gated_scan_bwd(x1, g1 + 1, y1, dy1, None, None, lens[-1:].clone())
    G = 60  # |G| <= sum of |dy| over a gate's memory, kept far below this by gates around 0.7
    for a, b in zip(got, one):
        assert (a[-1] - b[0]).abs().max() <= (4 * T + 64) * 2.0 ** -24 * G * 12
    assert not y[:-1].any() and not got[0][:-1].any()
    assert gla.get_device_error() == 0


@pytest.mark.parametrize("D", [2048, 2047])
def test_layer_norm(env, D):
    gla, torch = env
    n = 2 ** 31 // D + 300
    x = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    x[-200:] = _rand(torch, 200, D, dtype=torch.bfloat16)
    w, b = _rand(torch, D, dtype=torch.float32), _rand(torch, D, dtype=torch.float32)
    y, m, r = gla.layer_norm_fwd(x, w, b)
    dx, dw, db = gla.layer_norm_bwd(x, x, w, m, r)
    last = x[-200:].clone()
    y1, m1, r1 = gla.layer_norm_fwd(last, w, b)
    dx1, dw1, db1 = gla.layer_norm_bwd(last, last, w, m1, r1)
    # other variants for few rows: the statistics to 64 roundings, the outputs to a step of bf16
    assert (m[-200:] - m1).abs().max() <= 64 * 2.0 ** -24 * 6
    assert (r[-200:] - r1).abs().max() <= 64 * 2.0 ** -24 * 6 * r1.max()
    for a, c in ((y[-200:], y1), (dx[-200:], dx1)):
        assert ((a.float() - c.float()).abs() <= 2.0 ** -7 * c.float().abs() + 1e-4).all()
    # zero rows add nothing; 200 terms of at most 36
    assert (dw - dw1).abs().max() <= 3000 * 2.0 ** -24 * 200 * 36
    assert (db - db1).abs().max() <= 3000 * 2.0 ** -24 * 200 * 6
    assert gla.get_device_error() == 0


def test_window_attention(env):
    gla, torch = env
    T, H, KV, W, S = 8192, 16, 16, 100, 4
    B = 2 ** 31 // (T * H * 96) + 2
    one = [_rand(torch, 1, T, h, d, dtype=torch.bfloat16) * s
           for h, d, s in ((H, 96, 0.1), (KV, 96, 1), (KV, 192, 1), (H, 192, 1))]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = 3000
    q, k, v, dO = (_behind(torch, B, t) for t in one)
    assert q.numel() > 2 ** 31
    o, lse = gla.window_attn_fwd(q, k, v, W, S, lens)
    got = gla.window_attn_bwd(q, k, v, o, lse, dO, W, S, lens)
    o1, lse1 = gla.window_attn_fwd(*one[:3], W, S, lens[-1:].clone())
    want = gla.window_attn_bwd(*one[:3], o1, lse1, one[3], W, S, lens[-1:].clone())
    assert torch.equal(o[-1], o1[0]) and torch.equal(lse[-1], lse1[0])
    assert all(torch.equal(a[-1], b[0]) for a, b in zip(got, want))
    assert not o[:-1].any() and not any(a[:-1].any() for a in got)
    assert gla.get_device_error() == 0


def test_pools(env):
    gla, torch = env
    W, S, KV, H = 1020, 4, 4, 16
    P = 2 ** 31 // (1024 * KV * 96) + 3
    pk = torch.empty(P, 1, 1024, KV, 96, dtype=torch.bfloat16, device="cuda")
    pv = torch.empty(P, 1, 1024, KV, 192, dtype=torch.bfloat16, device="cuda")
    assert pk.numel() > 2 ** 31
    k, v = (_rand(torch, 2, 1500, KV, d, dtype=torch.bfloat16) for d in (96, 192))
    q = _rand(torch, 2, H, 96, dtype=torch.bfloat16) * 0.1
    pos = torch.tensor([1500, 1500], dtype=torch.int32, device="cuda")
    out = []
    for a, b, page in ((pk, pv, [P - 1, 0]), (pk[:2].clone(), pv[:2].clone(), [1, 0])):
        page = torch.tensor(page, dtype=torch.int32, device="cuda")
        gla.window_cache_fill(a, b, page, k, v, W, S)
        o = gla.window_attn_decode_step(a, b, page, pos, q, k[:, 7].contiguous(),
                                        v[:, 7].contiguous(), W, S)
        out.append((o, a[page.long()], b[page.long()]))
    assert all(torch.equal(x, y) for x, y in zip(*out))
    D = 2048
    pool = torch.empty(2 ** 31 // D + 9, 1, D, device="cuda")
    pool[-1], pool[0] = 1.5, 2.5
    small = torch.stack([pool[-1], pool[0]])
    x, g = (_rand(torch, 2, 1, D, dtype=torch.bfloat16) for _ in range(2))
    page = torch.tensor([len(pool) - 1, 0], dtype=torch.int32, device="cuda")
    y = gla.gated_scan_decode_step_paged(pool, page, x, g)
    assert torch.equal(y, gla.gated_scan_decode_step(small, x, g))
    assert torch.equal(pool[page.long()], small) and gla.get_device_error() == 0


def test_calls_on_two_streams_at_once(env):
    """Two streams with tensors and workspaces of their own, calls of every operator in flight on
    both, chained launches included."""
    gla, torch = env

    def work(seed):
        r = lambda *s: _rand(torch, seed, *s, dtype=torch.bfloat16)[0]  # noqa: E731
        x, g = r(2, 700, 520), r(2, 700, 520)
        q, k, v, dO = r(2, 700, 4, 96) * 0.2, r(2, 700, 2, 96), r(2, 700, 2, 192), r(2, 700, 4, 192)
        pk, pv = r(3, 1, 300, 2, 96), r(3, 1, 300, 2, 192)
        page = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
        pos = torch.tensor([700, 90], dtype=torch.int32, device="cuda")
        q1, k1, v1 = (t[:, 0].contiguous() for t in (q, k, v))

        def run(stream=None):
            y, fin = gla.gated_scan_fwd(x, g, stream=stream)
            n, m, s = gla.layer_norm_fwd(x, stream=stream)
            o, lse = gla.window_attn_fwd(q, k, v, 150, 5, stream=stream)
            return [y, fin, n, o, lse, *gla.gated_scan_bwd(x, g, y, y, None, fin, stream=stream),
                    *gla.layer_norm_bwd(x, x, None, m, s, stream=stream),
                    *gla.window_attn_bwd(q, k, v, o, lse, dO, 150, 5, stream=stream),
                    gla.window_attn_decode_step(pk, pv, page, pos, q1, k1, v1, 296, 4,
                                                stream=stream)]
        return run
    runs = [work(1), work(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for _ in range(3):  # several steps queued on each before any is waited for
            got = [r(s) for r, s in zip(runs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, h in zip(want, got) for a, b in zip(w, h))
    assert gla.get_device_error() == 0


def test_a_workspace_serves_calls_and_graphs_in_turn(env):
    """One caller's workspace, left dirty by other calls: eager calls and two captured graphs."""
    gla, torch = env
    r = lambda *s: _rand(torch, *s, dtype=torch.bfloat16)  # noqa: E731
    sizes = [(1, 900, 4, 2), (3, 300, 2, 1)]
    need = max(gla.window_attn_bwd_workspace_size(*s, 100, 9) for s in sizes)
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")

    def make(B, T, H, KV):
        q, k, v, dO = r(B, T, H, 96) * 0.2, r(B, T, KV, 96), r(B, T, KV, 192), r(B, T, H, 192)
        o, lse = gla.window_attn_fwd(q, k, v, 100, 9)
        return lambda w: gla.window_attn_bwd(q, k, v, o, lse, dO, 100, 9, workspace=w)
    calls = [make(*s) for s in sizes]
    want = [c(None) for c in calls]
    graphs, outs = [], []
    for c in calls:
        c(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c(ws))
        graphs.append(g)
    for _ in range(2):
        for g, out, w, c in zip(graphs, outs, want, calls):
            g.replay()
            again = c(ws)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) and torch.equal(a, e) for a, b, e in zip(w, out, again))
            ws.fill_(255)

"""The operators around the mixer run together as a layer uses them, on the GPU against the same
layer in 64 bits: layer norm -> conv -> gated scan -> projections -> windowed attention -> layer
norm, ragged lengths; a training step with every gradient, and serving (prompts, then tokens one at
a time over the pools).

Bound: the kernels compute in fp32 and round q, k, v, the softmax weights, dO and dz to bf16, each by
at most u = 2^-8 relative.  To first order a result's error is a linear form in these roundings.
`noisy` moves each of them by exactly +-u with random signs, which gives that form's size for
independent roundings of full size; real ones are smaller (a third of the variance), so four times
that size leaves room for the draw.  fp32 adds at most 2^-24 times the 64 (scan, sums of 384) or
so roundings along each path: 2^-16 of the norm is far above it."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
B, T, H, KV, D, WINDOW, SINK = 2, 150, 2, 1, 384, 40, 3
LENS = [150, 97]


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    gen = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).float().double()  # noqa: E731
    p = {"x": r(B, T, D) * 2 + 1, "w": 1 + 0.2 * r(D), "b": 0.2 * r(D), "cw": 0.5 * r(D, 4),
         "cb": 0.1 * r(D), "wq": r(D, H * 96) * (D * 96) ** -0.5 * 3, "wk": r(D, KV * 96) * D ** -0.5,
         "wv": r(D, KV * 192) * D ** -0.5, "w2": 1 + 0.2 * r(H * 192), "b2": 0.2 * r(H * 192),
         "R": r(B, T, H * 192)}
    p = {k: v.float().double() for k, v in p.items()}
    for b, n in enumerate(LENS):
        p["R"][b, n:] = 0
    return gla, torch, p


def _reference(torch, p, lens, noise=None):
    """(z, gradients of sum(z R)) in 64 bits; noise: a generator, moves every rounded value."""
    def rounded(t):
        if noise is None:
            return t
        f = 1 + U * (2.0 * torch.randint(0, 2, t.shape, generator=noise) - 1)
        h = 1 + U * (2.0 * torch.randint(0, 2, t.shape, generator=noise) - 1)
        t = t + (t * (f - 1)).detach()  # the value moved, its gradient through unchanged
        if t.requires_grad:
            t.register_hook(lambda g: g * h)
        return t

    def norm(t, w, b):
        c = t - t.mean(-1, keepdim=True)
        return c / (c.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * w + b
    leaves = {k: v.clone().requires_grad_() for k, v in p.items() if k != "R"}
    L = leaves
    n = norm(L["x"], L["w"], L["b"])
    xe = torch.cat([torch.zeros(B, 3, D, dtype=n.dtype), n], 1)
    c = torch.nn.functional.silu(sum(L["cw"][:, j] * xe[:, j:j + n.shape[1]] for j in range(4)) +
                                 L["cb"])
    f, h, ys = torch.sigmoid(n), torch.zeros(B, D, dtype=n.dtype), []
    for t in range(n.shape[1]):
        h = f[:, t] * h + (1 - f[:, t]) * c[:, t]
        ys.append(h)
    y = torch.stack(ys, 1)
    Tn = n.shape[1]
    q, k, v = (rounded(y @ L[s]).view(B, Tn, -1, d) for s, d in (("wq", 96), ("wk", 96),
                                                                 ("wv", 192)))
    k, v = k.repeat_interleave(H // KV, 2), v.repeat_interleave(H // KV, 2)
    z = torch.einsum("bthd,bshd->bhts", q, k)
    if noise is not None:  # dz
        hz = 1 + U * (2.0 * torch.randint(0, 2, z.shape, generator=noise) - 1)
        z.register_hook(lambda g: g * hz)
    t = torch.arange(Tn)
    sees = (t[None] <= t[:, None]) & ((t[:, None] - t[None] < WINDOW) | (t[None] < SINK))
    pr = torch.softmax(z.masked_fill(~sees, -torch.inf), -1)
    if noise is not None:
        pr = pr + (pr * U * (2.0 * torch.randint(0, 2, pr.shape, generator=noise) - 1)).detach()
    o = torch.einsum("bhts,bshd->bthd", pr, v).reshape(B, Tn, H * 192)
    if noise is not None:  # dO
        ho = 1 + U * (2.0 * torch.randint(0, 2, o.shape, generator=noise) - 1)
        o.register_hook(lambda g: g * ho)
    out = norm(o, L["w2"], L["b2"])
    keep = (t[None] < torch.tensor(lens)[:, None])[..., None]
    (out * p["R"] * keep).sum().backward()
    return out.detach(), {k: v.grad for k, v in leaves.items()}


def _step(gla, torch, p, lens):
    """The same with the kernels: (z, gradients by name)."""
    d = {k: v.float().cuda() for k, v in p.items()}
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n, m1, r1 = gla.layer_norm_fwd(d["x"], d["w"], d["b"])
    c, _ = gla.conv_fwd(n, d["cw"], d["cb"])
    y, _ = gla.gated_scan_fwd(c, n, None, ld)
    q, k, v = ((y @ d[s]).bfloat16().view(B, T, -1, e) for s, e in (("wq", 96), ("wk", 96),
                                                                   ("wv", 192)))
    o, lse = gla.window_attn_fwd(q, k, v, WINDOW, SINK, ld, out_dtype=torch.float32)
    flat = o.view(B, T, H * 192)
    z, m2, r2 = gla.layer_norm_fwd(flat, d["w2"], d["b2"])
    g = {}
    do, g["w2"], g["b2"] = gla.layer_norm_bwd(d["R"], flat, d["w2"], m2, r2)
    dq, dk, dv = gla.window_attn_bwd(q, k, v, o, lse, do.bfloat16().view(o.shape), WINDOW, SINK, ld)
    dy = torch.zeros_like(y)
    for s, e in (("wq", dq), ("wk", dk), ("wv", dv)):
        e = e.reshape(B * T, -1)
        g[s] = y.view(B * T, D).T @ e
        dy += (e @ d[s].T).view(B, T, D)
    dc, dg, _ = gla.gated_scan_bwd(c, n, y, dy, None, None, ld)
    dn, _, g["cw"], g["cb"] = gla.conv_bwd(n, d["cw"], dc, d["cb"])
    g["x"], g["w"], g["b"] = gla.layer_norm_bwd(dn + dg, d["x"], d["w"], m1, r1)
    return z, g


def test_training_step_matches_64_bits(env):
    gla, torch, p = env
    z, g = _step(gla, torch, p, LENS)
    torch.cuda.synchronize()
    assert gla.get_device_error() == 0
    zr, gr = _reference(torch, p, LENS)
    zn, gn = _reference(torch, p, LENS, torch.Generator().manual_seed(1))
    live = torch.arange(T)[None] < torch.tensor(LENS)[:, None]
    err, room = (z.cpu().double() - zr)[live].norm(), (zn - zr)[live].norm()
    assert err <= 4 * room + 2 ** -16 * zr[live].norm(), (err, room)
    assert set(g) == set(gr)
    for name in g:
        err, room = (g[name].cpu().double() - gr[name]).norm(), (gn[name] - gr[name]).norm()
        assert err <= 4 * room + 2 ** -16 * gr[name].norm(), (name, err, room)
    assert not g["x"][1, LENS[1]:].any()  # padding gets no gradient

    # and against differences of the 64-bit loss, along a random direction of every input: the
    # quotient's own error is of the order of the square of its step
    gen, eps = torch.Generator().manual_seed(2), 1e-5
    way = {k: torch.randn(v.shape, generator=gen, dtype=torch.float64) for k, v in p.items() if k != "R"}
    loss = []
    for s in (eps, -eps):
        moved = {k: v + s * way[k] if k in way else v for k, v in p.items()}
        out, _ = _reference(torch, moved, LENS)
        loss.append((out * p["R"] * live[..., None]).sum())
    slope = (loss[0] - loss[1]) / (2 * eps)
    along = sum((g[k].cpu().double() * way[k]).sum() for k in way)
    room = 4 * sum((gn[k] - gr[k]).norm().item() * way[k].norm().item() for k in way)
    assert abs(along - slope) <= room + 1e-6 * abs(slope), (along, slope, room)


def test_a_captured_step_and_an_eager_one_between_give_the_same_bits(env):
    """The whole step captured, its inputs changed, an eager step between replays."""
    gla, torch, p = env
    want = _step(gla, torch, p, LENS)
    d = {k: v.clone() for k, v in p.items()}
    dev = {k: v.float().cuda() for k, v in d.items()}
    zero = dev["x"].clone()
    ld = torch.tensor(LENS, dtype=torch.int32, device="cuda")

    def run(x):
        n, m, r = gla.layer_norm_fwd(x, dev["w"], dev["b"])
        y, fin = gla.gated_scan_fwd(n, n, None, ld)
        q = y[..., :H * 96].bfloat16().reshape(B, T, H, 96)
        k = y[..., :96].bfloat16().reshape(B, T, 1, 96)
        v = y[..., :192].bfloat16().reshape(B, T, 1, 192)
        o, lse = gla.window_attn_fwd(q, k, v, WINDOW, SINK, ld)
        return [n, y, fin, o, lse, *gla.window_attn_bwd(q, k, v, o, lse, o, WINDOW, SINK, ld),
                *gla.gated_scan_bwd(n, n, y, y, None, fin, ld), *gla.layer_norm_bwd(n, x, dev["w"], m, r)]
    eager = run(dev["x"])
    graphs, outs = [], []
    for _ in range(2):  # two graphs, with workspaces of the capture's pool
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(zero))
        graphs.append(g)
    for rep in range(2):
        for g, out in zip(graphs, outs):
            g.replay()
            again = run(dev["x"])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(eager, out, again))
    z, g = _step(gla, torch, p, LENS)
    assert torch.equal(z, want[0]) and all(torch.equal(g[k], want[1][k]) for k in g)
    assert gla.get_device_error() == 0


def test_serving_goes_on_from_prompts(env):
    """Prompts of different lengths into the pools, then tokens one at a time."""
    gla, torch, p = env
    prompts, more = [90, 2], 30  # one longer than the window, one shorter than the conv's reach
    d = {k: v.float().cuda() for k, v in p.items()}
    page = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    ld = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    scan = torch.zeros(6, 2, D, device="cuda")
    pk = torch.zeros(6, 2, WINDOW + SINK, KV, 96, device="cuda").bfloat16()
    pv = torch.zeros(6, 2, WINDOW + SINK, KV, 192, device="cuda").bfloat16()
    x = d["x"][:, :max(prompts)].contiguous()
    n, _, _ = gla.layer_norm_fwd(x, d["w"], d["b"], want_stats=False)
    c, _ = gla.conv_fwd(n, d["cw"], d["cb"])
    y, fin = gla.gated_scan_fwd(c, n, None, ld)
    scan[page.long(), 1] = fin
    conv = torch.zeros(B, 3, D, device="cuda")
    for b, m in enumerate(prompts):
        m3 = min(m, 3)
        conv[b, 3 - m3:] = n[b, m - m3:m]

    def project(s):
        return ((s @ d[w]).bfloat16().view(*s.shape[:-1], -1, e)
                for w, e in (("wq", 96), ("wk", 96), ("wv", 192)))
    _, k, v = project(y)
    gla.window_cache_fill(pk, pv, page, k, v, WINDOW, SINK, ld, layer=1)
    rows, got = torch.arange(B, device="cuda"), []
    for step in range(more):
        pos = ld + step
        n, _, _ = gla.layer_norm_fwd(d["x"][rows, pos.long()], d["w"], d["b"], want_stats=False)
        c = gla.conv_decode_step(conv, n, d["cw"], d["cb"])
        y = gla.gated_scan_decode_step_paged(scan, page, c[:, None], n[:, None], layer0=1)[:, 0]
        q, k, v = project(y)
        o = gla.window_attn_decode_step(pk, pv, page, pos, q, k, v, WINDOW, SINK, layer=1,
                                        out_dtype=torch.float32)
        z, _, _ = gla.layer_norm_fwd(o.view(B, H * 192), d["w2"], d["b2"], want_stats=False)
        got.append(z.cpu().double())
    assert gla.get_device_error() == 0
    assert not scan[:, 0].any() and not pk[:, 0].any() and not scan[0].any()
    zr, _ = _reference(torch, p, LENS)
    zn, _ = _reference(torch, p, LENS, torch.Generator().manual_seed(3))
    for b, m in enumerate(prompts):
        z = torch.stack([s[b] for s in got])
        err, room = (z - zr[b, m:m + more]).norm(), (zn - zr)[b, m:m + more].norm()
        assert err <= 4 * room + 2 ** -16 * z.norm(), (b, err, room)

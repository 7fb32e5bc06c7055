"""GPU parity of the rotary positions against the definition in 64 bits.

Bound: the phase is a whole number, the same on both sides.  In the kernel what is left of it after the
nearest quarter turn is cut to 2^-34 turns (4e-10 radians) and rounded to fp32 (2^-24 of at most pi / 4);
sincospi is off by at most 2 units in the last place (2^-23) and the scale's product rounds once: below
6 x 2^-24 of the scale in all.  Two products and a sum add 2 x 2^-24 of their sizes, the output u of
itself, or 2^-25 where fp16 is below its normal numbers."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    return gla, torch, {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _definition(x, turns, pos, inter, inverse, scale):
    """(y, sum of magnitudes) in fp64; x [B,T,H,D], turns int64 [n], pos [B,T]."""
    n = len(turns)
    with np.errstate(over="ignore"):
        phase = pos.astype(np.int64).astype(np.uint64)[..., None] * turns.astype(np.uint64)
    w = phase.astype(np.int64).astype(np.float64) * (2 * np.pi / 2.0 ** 64)  # modulo a turn
    c, s = np.cos(w)[:, :, None] * scale, np.sin(w)[:, :, None] * scale * (-1 if inverse else 1)
    x = x.astype(np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = abs(scale) * (np.abs(a) + np.abs(b))
    return y, mag


CASES = [  # B, T, H, KV, D, R, interleaved, inverse, scale, type, output type, positions
    (1, 1, 1, 0, 2, 2, False, False, 1.0, "fp32", "fp32", "none"),
    (2, 3, 2, 1, 96, 96, False, False, 1.0, "bf16", "bf16", "none"),
    (2, 3, 2, 1, 96, 96, True, False, 1.0, "bf16", "bf16", "far"),
    (1, 77, 5, 5, 96, 64, False, True, 1.2, "fp16", "fp32", "none"),
    (1, 77, 5, 5, 96, 64, True, True, 1.2, "fp16", "fp16", "far"),
    (3, 50, 16, 4, 96, 48, True, False, 0.5, "bf16", "fp32", "none"),
    (3, 50, 16, 4, 96, 62, False, False, 1.0, "bf16", "bf16", "negative"),  # 31 pairs: by the element
    (3, 50, 3, 1, 97, 62, True, False, 1.0, "fp16", "fp16", "far"),         # odd channels that pass
    (2, 9, 1, 3, 33, 6, False, False, 1.0, "fp32", "fp32", "far"),
    (1, 4, 2, 2, 200, 8, True, True, -1.0, "fp32", "fp32", "none"),
    (2, 130, 7, 2, 128, 128, False, False, 1.0, "fp32", "fp32", "far"),
    (5, 1, 33, 2, 96, 32, False, False, 1.0, "fp16", "fp16", "far"),
    (1, 40000, 2, 1, 96, 96, True, False, 1.0, "bf16", "bf16", "none"),
]


@pytest.mark.parametrize("B,T,H,KV,D,R,inter,inverse,scale,dt,out,where", CASES)
def test_matches_the_definition(env, B, T, H, KV, D, R, inter, inverse, scale, dt, out, where):
    gla, torch, types = env
    rng = np.random.default_rng(T + H + R)
    draw = lambda *s: as_dtype_values(rng.standard_normal(s).astype(np.float32), dt)  # noqa: E731
    q, k = draw(B, T, H, D), draw(B, T, max(KV, 1), D)
    turns = gla.rotary_turns(R, 10000.0)
    pos = np.broadcast_to(np.arange(T), (B, T)).astype(np.int32)
    if where == "far":
        pos = rng.integers(0, 2 ** 31, (B, T)).astype(np.int32)
        pos[0, 0] = 2 ** 31 - 1
    elif where == "negative":
        pos = (pos - 1000).astype(np.int32)
    pd = None if where == "none" else torch.from_numpy(np.ascontiguousarray(pos)).cuda()
    qd, kd = to_dev(q, types[dt]), to_dev(k, types[dt]) if KV else None
    kw = dict(interleaved=inter, inverse=inverse, scale=scale)
    got = gla.rotary(qd, kd, turns.cuda(), pd, out_dtype=types[out], **kw)
    assert (got[1] is None) == (KV == 0) and got[0].dtype == types[out]
    for x, y in ((q, got[0]), (k, got[1]))[:2 if KV else 1]:
        want, mag = _definition(x, turns.numpy(), pos, inter, inverse, np.float32(scale))
        off = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
        tiny = 2.0 ** -25 if out == "fp16" else 0.0
        assert np.all(off <= 8 * 2.0 ** -24 * mag + U[out] * (1 + 2.0 ** -9) *
                      np.abs(want) * (mag > 0) + tiny * (mag > 0))
    # in place, and from views of wider rows
    if out == dt:
        a, b = qd.clone(), None if kd is None else kd.clone()
        gla.rotary(a, b, turns.cuda(), pd, q_out=a, k_out=b, **kw)
        assert torch.equal(a, got[0]) and (b is None or torch.equal(b, got[1]))
    for front in (0, 3, 16):
        row = torch.full((B, T, front + (H + KV) * D + 5), 9.0, device="cuda").to(types[dt])
        vq = row[..., front:front + H * D].view(B, T, H, D)
        vk = row[..., front + H * D:front + (H + KV) * D].view(B, T, KV, D) if KV else None
        vq.copy_(qd)
        if KV:
            vk.copy_(kd)
        again = gla.rotary(vq, vk, turns.cuda(), pd, out_dtype=types[out], **kw)
        assert torch.equal(again[0], got[0]) and (not KV or torch.equal(again[1], got[1]))
    # heads in front of tokens
    vq = qd.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(gla.rotary(vq, None, turns.cuda(), pd, out_dtype=types[out], **kw)[0], got[0])


def test_packed_tokens_and_nothing(env):
    gla, torch, _ = env
    turns = gla.rotary_turns(64).cuda()
    q, k = torch.randn(2, 7, 4, 96, device="cuda").bfloat16(), torch.randn(2, 7, 1, 96, device="cuda").bfloat16()
    pos = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7) * 1000
    a, b = gla.rotary(q, k, turns, pos)
    c, d = gla.rotary(q.view(14, 4, 96), k.view(14, 1, 96), turns, pos.view(14))
    assert c.shape == (14, 4, 96) and torch.equal(a.view_as(c), c) and torch.equal(b.view_as(d), d)
    e, f = gla.rotary(q[:, :0], k[:, :0], turns)
    assert e.shape == (2, 0, 4, 96) and f.shape == (2, 0, 1, 96)
    assert gla.get_device_error() == 0


def test_values_that_are_not_finite_stay_in_their_pair(env):
    gla, torch, _ = env
    x = torch.ones(1, 3, 2, 96, device="cuda").half()
    x[0, 1, 0, 5], x[0, 1, 0, 90] = float("nan"), float("inf")
    y, _ = gla.rotary(x, None, gla.rotary_turns(64).cuda())
    bad = ~y.isfinite()
    assert bad.sum() == 3 and bool(bad[0, 1, 0, [5, 37, 90]].all())


def test_gradient_against_differences(env):
    """<dy, d rotary(x)> along a random direction, in fp32: the map is linear, so a difference quotient is
    off by roundings only: 2^-24 x 8 of each term's size (above), of 2 x 96 x 60 terms."""
    gla, torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, w, dy = (torch.randn(1, 30, 2, 96, generator=gen, device="cuda") for _ in range(3))
    turns = gla.rotary_turns(80, scaling="parts", factor=4.0).cuda()
    for inter in (False, True):
        kw = dict(interleaved=inter, scale=1.1)
        dx, _ = gla.rotary(dy, None, turns, inverse=True, **kw)
        up, _ = gla.rotary(x + w, None, turns, **kw)
        down, _ = gla.rotary(x - w, None, turns, **kw)
        slope = ((up.double() - down.double()) / 2 * dy.double()).sum()
        size = 1.1 * 2 * (dy.abs() * (x.abs() + w.abs())).double().sum() * 2
        assert abs((dx.double() * w.double()).sum() - slope) <= 16 * 2.0 ** -24 * size


def test_streams_and_graphs(env):
    gla, torch, _ = env
    turns = gla.rotary_turns(96).cuda()
    q, k = torch.randn(3, 40, 16, 96, device="cuda").half(), torch.randn(3, 40, 4, 96, device="cuda").half()
    want = gla.rotary(q, k, turns)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = gla.rotary(q, k, turns, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    bq = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gla.rotary(bq, k, turns)
    bq.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))

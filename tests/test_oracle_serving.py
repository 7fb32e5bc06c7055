"""Pins of the oracle of serving with the windowed attention (oracle/serving_ops.py), and the host-side
table of the rotary positions."""
import numpy as np
import pytest

from oracle import layer_ops, serving_ops as ref


def test_rotary_keeps_lengths_and_depends_on_distances():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 7, 1, 10))
    ang = np.array([1.0, 0.3, 0.01])
    for inter in (False, True):
        a, b = ref.rotary(q, ang, interleaved=inter), ref.rotary(k, ang, interleaved=inter)
        assert np.array_equal(a[..., 6:], q[..., 6:]) and np.array_equal(a[:, 0], q[:, 0])
        assert np.allclose((a ** 2).sum(-1), (q ** 2).sum(-1))
        far = np.arange(7)[None] + 1000
        a2, b2 = ref.rotary(q, ang, far, inter), ref.rotary(k, ang, far, inter)
        assert np.allclose(np.einsum("bthd,bshd->ts", a, b), np.einsum("bthd,bshd->ts", a2, b2))
        assert np.allclose(ref.rotary(a, ang, None, inter, True), q)  # turned back
    # position 1, one pair: the angle itself
    x = np.array([1.0, 0.0]).reshape(1, 1, 1, 2)
    assert np.allclose(ref.rotary(x, [0.5], [[1]], scale=2.0)[0, 0, 0], [2 * np.cos(.5), 2 * np.sin(.5)])


def test_rotary_gradient_is_the_turn_back():
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 1, 3, 2, 8))
    ang, h = np.array([0.7, 0.2]), 1e-6
    for inter in (False, True):
        g = ref.rotary(dy, ang, None, inter, True, 1.3)
        for at in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[at] = h
            d = ((ref.rotary(x + e, ang, None, inter, False, 1.3) -
                  ref.rotary(x - e, ang, None, inter, False, 1.3)) * dy).sum() / (2 * h)
            assert abs(d - g[at]) < 1e-8


def test_codes_are_within_half_a_step():
    rng = np.random.default_rng(3)
    for dt, low, size in (("bf16", -126, 96), ("fp16", -24, 192)):
        x = rng.standard_normal((50, size)) * np.exp(rng.standard_normal((50, 1)) * 3)
        x = x.astype(np.float16).astype(np.float64)
        x[0] = 0
        c, e = ref.codes(x, low)
        assert np.abs(c).max() <= 127 and e.min() >= low
        step = 2.0 ** e[:, None]
        off = np.abs(c * step - x)
        top = np.abs(x) > 127.5 * step
        assert np.all(off[~top] <= (step / 2 + 0 * x)[~top]) and np.all(off[top] < (step + 0 * x)[top])
        assert not c[0].any() and e[0] == low
    # the largest of a row has at least 64 steps; ties to even; the ends of the types
    c, e = ref.codes([[64.0, 0.5, 1.5, -63.5]], -24)
    assert e[0] == 0 and c[0].tolist() == [64, 0, 2, -64]
    c, e = ref.codes([[65504.0, -512.0]], -24)
    assert e[0] == 9 and c[0].tolist() == [127, -1]
    c, e = ref.codes([[2.0 ** -24, 0.0]], -24)
    assert e[0] == -24 and c[0].tolist() == [1, 0]


@pytest.mark.parametrize("window,sink,cuts", [(3, 0, (0, 4, 5)), (4, 2, (1, 6)), (16, 3, (5, 5)),
                                              (1, 1, (0, 9)), (5, 20, (2, 3))])
def test_chunks_are_one_pass(window, sink, cuts):
    """A sequence cut anywhere, chunk by chunk over its page, gives the rows of one pass."""
    rng = np.random.default_rng(4)
    T, H, KV = 12, 4, 2
    q, k, v = (rng.standard_normal((T, n, d)) for n, d in ((H, 3), (KV, 3), (KV, 5)))
    want, _ = layer_ops.window_attn_fwd(q[None], k[None], v[None], window, sink)
    pk, pv = (rng.standard_normal((2, 2, window + sink, KV, d)) for d in (3, 5))
    edges = [0, *cuts, T]
    for a, b in zip(edges, edges[1:]):
        args = ([1], [a], [0, b - a], *(x[a:b] for x in (q, k, v)), window, sink, 1)
        got, _, _ = ref.chunk(pk, pv, *args)
        assert b == a or np.abs(got - want[0, a:b]).max() < 1e-13
        pk, pv = ref.append(pk, pv, [1], [a], [0, b - a], k[a:b], v[a:b], window, sink, 1)
    full = layer_ops.window_cache_fill(pk * 0, pv * 0, [1], k[None], v[None], window, sink, 1)
    held = min(T, window + sink)
    assert np.array_equal(full[0][1, 1, :held], pk[1, 1, :held])


def _turns(R, *a, **kw):
    gla = pytest.importorskip("gated_linear_attention_chunked_gb300")
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    return gla.rotary_turns(R, *a, **kw).numpy().astype(np.float64) / 2.0 ** 64 * 2 * np.pi


def test_table_of_turns():
    """The table against the formulas in radians; each entry is off by 2^-53 of itself and 2^-64."""
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    near = lambda a, b: np.all(np.abs(a - b) <= 1e-15 * b + 2.0 ** -61)  # noqa: E731
    assert near(_turns(64), f)
    assert near(_turns(64, 500.0), 500.0 ** (-np.arange(0, 64, 2) / 64))
    assert near(_turns(64, scaling="linear", factor=4.0), f / 4)
    g = _turns(64, scaling="base", factor=8.0)
    assert near(g[:1], f[:1]) and near(g[-1:], f[-1:] / 8) and np.all(np.diff(g) < 0)
    g = _turns(64, scaling="parts", factor=8.0, context=2048, low=2.0, high=16.0)
    n = 2048 * f / (2 * np.pi)
    assert near(g[n >= 16], f[n >= 16]) and near(g[n <= 2], f[n <= 2] / 8)
    mid = (n > 2) & (n < 16)
    keep = (n[mid] - 2) / 14
    assert mid.any() and np.allclose(g[mid], f[mid] * keep + f[mid] / 8 * (1 - keep), rtol=1e-14)
    assert near(_turns(2, scaling="base", factor=8.0), np.ones(1))


def test_table_refuses():
    gla = pytest.importorskip("gated_linear_attention_chunked_gb300")
    for bad in (dict(R=3), dict(R=0), dict(R=8, scaling="dynamic")):
        with pytest.raises(ValueError):
            gla.rotary_turns(**bad)
    for bad in (dict(base=1.0), dict(base=float("inf")), dict(scaling="linear", factor=0.5),
                dict(scaling="base", factor=float("nan")), dict(scaling="parts", low=3.0, high=3.0),
                dict(scaling="parts", context=0), dict(scaling="parts", low=-1.0)):
        with pytest.raises(gla.GlaError) as e:
            gla.rotary_turns(8, **{"factor": 2.0, **bad})
        assert e.value.code == 1


def test_codes_of_what_is_not_finite():
    c, e = ref.codes([[np.inf, 1000.0, np.nan, -np.inf]], -24)
    assert e[0] == 9 and c[0].tolist() == [127, 2, 0, -127]
    c, e = ref.codes([[np.nan, 2.0]], -126)
    assert e[0] == -5 and c[0].tolist() == [0, 64]

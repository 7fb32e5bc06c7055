"""Pins of the fp64 definitions of the operators around the mixer: closed forms, central finite
differences of every gradient, and decode = prefill token by token.  CPU only."""
import numpy as np
import pytest

from oracle import layer_ops as ref


def _differences(f, x, h=1e-6):
    """Central differences of the scalar f() in the entries of the array x (changed in place)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


# Second differences leave h^2 f''' / 6 ~ 1e-12 and rounding eps f / h ~ 1e-9 on sums of order 10.
FD = 1e-7


def test_gated_scan_closed_forms():
    rng = np.random.default_rng(1)
    x, init = rng.standard_normal((2, 9, 3)), rng.standard_normal((2, 3))
    y, fin = ref.gated_scan_fwd(x, np.full(x.shape, np.inf), init)   # keeps its state
    assert np.array_equal(y, np.repeat(init[:, None], 9, 1)) and np.array_equal(fin, init)
    y, fin = ref.gated_scan_fwd(x, np.full(x.shape, -np.inf), init)  # resets it
    assert np.array_equal(y, x)
    y, _ = ref.gated_scan_fwd(np.ones_like(x), np.zeros(x.shape))    # f = 1/2: 1 - 2^-t
    assert np.allclose(y[0, :, 0], 1 - 0.5 ** np.arange(1, 10), rtol=0, atol=1e-15)
    # a sequence cut in two carries its state; a shorter length is the shorter sequence
    g = rng.standard_normal(x.shape)
    y, fin = ref.gated_scan_fwd(x, g, init)
    ya, mid = ref.gated_scan_fwd(x[:, :4], g[:, :4], init)
    yb, end = ref.gated_scan_fwd(x[:, 4:], g[:, 4:], mid)
    assert np.array_equal(y, np.concatenate([ya, yb], 1)) and np.array_equal(end, fin)
    yl, fl = ref.gated_scan_fwd(x, g, init, [4, 0])
    assert np.array_equal(yl[0, :4], ya[0]) and not yl[0, 4:].any() and not yl[1].any()
    assert np.array_equal(fl[0], mid[0]) and np.array_equal(fl[1], init[1])


@pytest.mark.parametrize("lens", [None, [5, 2, 0]])
def test_gated_scan_gradient(lens):
    rng = np.random.default_rng(2)
    x, g, dy = (rng.standard_normal((3, 5, 2)) for _ in range(3))
    init, dfin = rng.standard_normal((3, 2)), rng.standard_normal((3, 2))

    def loss():
        y, fin = ref.gated_scan_fwd(x, g, init, lens)
        return (y * dy).sum() + (fin * dfin).sum()
    for got, by in zip(ref.gated_scan_bwd(x, g, dy, init, dfin, lens), (x, g, init)):
        assert np.abs(got - _differences(loss, by)).max() < FD


def test_layer_norm():
    rng = np.random.default_rng(3)
    x, w, b, dy = (rng.standard_normal(s) for s in ((4, 7), 7, 7, (4, 7)))
    y, mean, rstd = ref.layer_norm_fwd(x, eps=0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-14) and np.allclose(y.var(-1), 1, atol=1e-14)
    assert np.allclose(ref.layer_norm_fwd(3 * x + 5, eps=0.0)[0], y, atol=1e-13)
    for got, by in zip(ref.layer_norm_bwd(dy, x, w), (x, w, b)):
        d = _differences(lambda: (ref.layer_norm_fwd(x, w, b)[0] * dy).sum(), by)
        assert np.abs(got - d).max() < FD


def test_window_sees_what_it_says():
    assert ref.visible(0, 1, 0) == [0] and ref.visible(5, 1, 0) == [5]
    assert ref.visible(5, 3, 0) == [3, 4, 5] and ref.visible(5, 3, 2) == [0, 1, 3, 4, 5]
    assert ref.visible(5, 3, 4) == [0, 1, 2, 3, 4, 5]
    # equal keys: the mean of the visible values
    rng = np.random.default_rng(4)
    q, v = rng.standard_normal((1, 6, 2, 3)), rng.standard_normal((1, 6, 1, 4))
    o, lse = ref.window_attn_fwd(q, np.zeros((1, 6, 1, 3)), v, 3, 1)
    assert np.allclose(o[0, 5, 1], v[0, [0, 3, 4, 5], 0].mean(0)) and np.allclose(
        lse[0, :, 5], np.log(4))
    o, lse = ref.window_attn_fwd(q, np.zeros((1, 6, 1, 3)), v, 3, 1, [2])
    assert not o[0, 2:].any() and np.all(lse[0, :, 2:] == -np.inf)


@pytest.mark.parametrize("window,sink,lens", [(3, 0, None), (2, 2, [6, 4]), (9, 1, [1, 0])])
def test_window_gradient(window, sink, lens):
    rng = np.random.default_rng(5)
    q, k, v, dO = (rng.standard_normal(s) for s in ((2, 6, 4, 3), (2, 6, 2, 3), (2, 6, 2, 5),
                                                    (2, 6, 4, 5)))

    def loss():
        return (ref.window_attn_fwd(q, k, v, window, sink, lens)[0] * dO).sum()
    for got, by in zip(ref.window_attn_bwd(q, k, v, dO, window, sink, lens), (q, k, v)):
        assert np.abs(got - _differences(loss, by)).max() < FD


@pytest.mark.parametrize("window,sink,prompt", [(3, 0, 0), (4, 2, 5), (16, 3, 4), (1, 1, 9)])
def test_window_decode_is_prefill_token_by_token(window, sink, prompt):
    """A prompt put into the cache, then tokens one at a time, give the rows of one pass."""
    rng = np.random.default_rng(6)
    B, T, H, KV = 2, 11, 4, 2
    q, k, v = (rng.standard_normal((B, T, n, d)) for n, d in ((H, 3), (KV, 3), (KV, 5)))
    o, _ = ref.window_attn_fwd(q, k, v, window, sink)
    page = [2, 0]
    pk, pv = (rng.standard_normal((3, 2, window + sink, KV, d)) for d in (3, 5))
    other = pk[:, 0].copy(), pk[1].copy()
    pk, pv = ref.window_cache_fill(pk, pv, page, k[:, :prompt], v[:, :prompt], window, sink, 1)
    for t in range(prompt, T):
        got, pk, pv = ref.window_attn_decode_step(pk, pv, page, [t, t], q[:, t], k[:, t], v[:, t],
                                                  window, sink, 1)
        assert np.abs(got - o[:, t]).max() < 1e-13
    assert np.array_equal(pk[:, 0], other[0]) and np.array_equal(pk[1], other[1])

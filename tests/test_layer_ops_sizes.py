"""Sizes, windows and indexes past 32 bits through the binding of the operators around the mixer: the
C ABI's int does not hold them, and they must not be cut off.  CPU only: a library that notes the
arguments of its calls, and tensors without memory."""
import pytest

torch = pytest.importorskip("torch")
import gated_linear_attention_chunked_gb300 as gla  # noqa: E402
from gated_linear_attention_chunked_gb300 import _build, layer_ops  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
MOST = 2 ** 31 - 1


@pytest.fixture()
def calls(monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if not name.endswith("_size"):
                    seen.append((name, args))
                return 0
            return call
    monkeypatch.setattr(layer_ops, "_lib", Lib())
    monkeypatch.setattr(layer_ops, "_begin", lambda t, name, stream: (t.get_device(), None))
    monkeypatch.setattr(layer_ops, "_stream", lambda dev: 0)
    empty = torch.empty
    monkeypatch.setattr(layer_ops, "_empty",
                        lambda *s, dtype, device: empty(*s, dtype=dtype, device="meta"))
    return seen


def _t(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


BIG = 2 ** 32 + 5  # cut off to 5


def _refused(calls, f, *args, **kw):
    with pytest.raises(ValueError, match="32 bits"):
        f(*args, **kw)
    assert not calls


def test_tensors_longer_than_an_int(calls):
    for s in ((1, BIG, 1), (BIG, 1, 1), (1, 1, BIG)):
        x, y = _t(*s), _t(*s, dtype=F32)
        _refused(calls, gla.gated_scan_fwd, x, x)
        _refused(calls, gla.gated_scan_bwd, x, x, y, y)
    x, s = _t(1, BIG), _t(1, BIG, dtype=F32)
    _refused(calls, gla.gated_scan_decode_step, s, x, x)
    _refused(calls, gla.layer_norm_fwd, x)
    _refused(calls, gla.layer_norm_bwd, x, x, None, _t(1, dtype=F32), _t(1, dtype=F32))
    q, k, v = _t(1, BIG, 1, 96), _t(1, BIG, 1, 96), _t(1, BIG, 1, 192)
    _refused(calls, gla.window_attn_fwd, q, k, v, 4)
    o, lse = _t(1, BIG, 1, 192), _t(1, 1, BIG, dtype=F32)
    _refused(calls, gla.window_attn_bwd, q, k, v, o, lse, o, 4)
    with pytest.raises(ValueError, match="32 bits"):
        gla.layer_norm_bwd_workspace_size(1, BIG)
    # long batches of rows are sizes of 64 bits
    gla.layer_norm_fwd(_t(BIG, 1))
    gla.gated_scan_decode_step(_t(BIG, 1, dtype=F32), _t(BIG, 1), _t(BIG, 1))
    assert calls[0][1][-3] == BIG and calls[1][1][-3] == BIG


@pytest.mark.parametrize("layer", [2 ** 32, -2 ** 32, 2 ** 31])
def test_layers(calls, layer):
    pool, page, x = _t(3, 2, 8, dtype=F32), _t(1, dtype=I32), _t(1, 1, 8)
    _refused(calls, gla.gated_scan_decode_step_paged, pool, page, x, x, layer0=layer)
    pk, pv = _t(3, 2, 9, 1, 96), _t(3, 2, 9, 1, 192)
    k, v, q = _t(1, 1, 96), _t(1, 1, 192), _t(1, 2, 96)
    _refused(calls, gla.window_cache_fill, pk, pv, page, k[None], v[None], 8, 1, layer=layer)
    _refused(calls, gla.window_attn_decode_step, pk, pv, page, page, q, k, v, 8, 1, layer=layer)
    # a window and sinks whose sum is the pool's but which are none
    _refused(calls, gla.window_cache_fill, pk, pv, page, k[None], v[None], 2 ** 32 + 9, -2 ** 32)
    _refused(calls, gla.window_attn_decode_step, pk, pv, page, page, q, k, v, 2 ** 32 + 9, -2 ** 32)


@pytest.mark.parametrize("window,want", [(7, 7), (MOST, MOST), (2 ** 32 + 7, MOST),
                                         (2 ** 63 - 1, MOST), (0, 0), (-2 ** 32 + 7, -1)])
def test_windows_and_sinks_past_an_int_mean_all(calls, window, want):
    q, k, v = _t(1, 9, 2, 96), _t(1, 9, 1, 96), _t(1, 9, 1, 192)
    o, lse = _t(1, 9, 2, 192), _t(1, 2, 9, dtype=F32)
    for args in ((window, 0), (3, window)):
        gla.window_attn_fwd(q, k, v, *args)
        gla.window_attn_bwd(q, k, v, o, lse, o, *args)
    at = [a.index(None, 3) + 1 for _, a in calls]  # behind lens
    assert [a[i:i + 2] for i, (_, a) in zip(at, calls)] == [(want, 0)] * 2 + [(3, want)] * 2


def test_workspace_sizes_of_endless_windows():
    _build.build()
    layer_ops._lib = None
    size = gla.window_attn_bwd_workspace_size
    for w in (9, MOST, 2 ** 32 + 1, 2 ** 63 - 1):
        assert size(1, 9, 4, 2, w, 0) == size(1, 9, 4, 2, 9, 0) > 0
        assert size(1, 9, 4, 2, 8, w) == size(1, 9, 4, 2, 8, 9) > 0
    assert size(1, 9, 4, 2, -2 ** 32 + 8, 0) == 0
    for args in ((2 ** 32 + 1, 4, 2, 8), (1, 4, 2, 2 ** 32 + 8)):
        with pytest.raises(ValueError, match="32 bits"):
            gla.window_attn_decode_workspace_size(*args)

"""Serving with the windowed attention refuses bad calls before it touches a device: status codes of the
C ABI (fake addresses that nothing reads) and the binding's checks.  CPU only."""
import ctypes

import pytest

import gated_linear_attention_chunked_gb300 as gla
from gated_linear_attention_chunked_gb300 import _build

A = 0x1000  # a 16-byte aligned fake address
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gla.load()


def test_rotary(lib):
    def rot(q=A, qs=None, qo=A + 0x1000, H=2, k=A, ks=None, ko=A + 0x2000, KV=1, dt=0, ot=0, turns=A,
            pos=None, scale=1.0, B=2, T=3, D=96, R=96):
        st = lambda s: None if s is None else (ctypes.c_longlong * 3)(*s)  # noqa: E731
        return lib.gla_rotary(q, st(qs), qo, H, k, st(ks), ko, KV, dt, ot, turns, pos, scale, 0, 0, B, T,
                              D, R, None)
    assert rot(B=0) == 0 and rot(T=0) == 0 and rot(B=-1) == INVALID
    assert rot(H=0) == INVALID and rot(KV=-1) == INVALID and rot(D=0) == INVALID
    assert rot(R=95) == INVALID and rot(R=0) == INVALID and rot(R=98) == INVALID
    assert rot(scale=float("nan")) == INVALID and rot(scale=float("inf")) == INVALID
    assert rot(dt=3) == UNSUPPORTED and rot(dt=1, ot=0) == UNSUPPORTED and rot(dt=0, ot=2) == UNSUPPORTED
    assert rot(D=4098, R=2) == UNSUPPORTED and rot(H=32768) == UNSUPPORTED
    assert rot(B=1 << 30, T=1 << 20) == UNSUPPORTED
    assert rot(q=None) == INVALID and rot(qo=None) == INVALID and rot(k=None) == INVALID
    assert rot(ko=None) == INVALID and rot(turns=None) == INVALID
    assert rot(q=A + 1) == ALIGN and rot(k=A + 1) == ALIGN and rot(dt=1, ot=1, q=A + 2) == ALIGN
    assert rot(qo=A + 8) == ALIGN and rot(ko=A + 2) == ALIGN and rot(pos=A + 2) == ALIGN
    assert rot(turns=A + 4) == ALIGN
    # in place: not with strides, not into another type
    assert rot(qo=A, qs=(576, 192, 96)) == INVALID and rot(ko=A, ks=(288, 96, 96)) == INVALID
    assert rot(qo=A, ot=1) == INVALID and rot(ko=A, ot=1) == INVALID
    assert rot(qs=(-1, 192, 96)) == INVALID and rot(ks=(288, 96, -96)) == INVALID


def test_append_and_read(lib):
    def app(k=A, v=A, dt=0, pos=A, start=A, count=None, pk=A, pv=A, pe=None, page=A, n=2, N=9, P=3, PL=2,
            layer=0, window=8, sink=1, KV=2, dk=96, dv=192):
        return lib.gla_window_cache_append(k, v, dt, pos, start, count, pk, pv, pe, page, n, N, P, PL,
                                           layer, window, sink, KV, dk, dv, None)
    assert app(n=0) == 0 and app(N=0) == 0 and app(n=-1) == INVALID and app(N=-1) == INVALID
    assert app(layer=2) == INVALID and app(layer=-1) == INVALID and app(P=0) == INVALID
    assert app(PL=0) == INVALID and app(window=0) == INVALID and app(sink=-1) == INVALID
    assert app(KV=0) == INVALID
    assert app(dt=1) == UNSUPPORTED and app(dk=64) == UNSUPPORTED and app(dv=96) == UNSUPPORTED
    assert app(N=(1 << 30) + 1) == UNSUPPORTED and app(n=1 << 30) == UNSUPPORTED
    assert app(window=(1 << 30) + 1) == UNSUPPORTED and app(P=1 << 30, window=1 << 12) == UNSUPPORTED
    for name in ("k", "v", "pos", "start", "pk", "pv", "page"):
        assert app(**{name: None}) == INVALID
        assert app(**{name: A + 2}) == ALIGN
    assert app(pe=A + 2) == ALIGN and app(count=A + 2) == ALIGN

    def read(pk=A, pv=A, pe=A, page=A, n=2, P=3, PL=2, layer=0, window=8, sink=1, k=A, v=A, dt=0, KV=2,
             dk=96):
        return lib.gla_window_cache8_read(pk, pv, pe, page, n, P, PL, layer, window, sink, k, v, dt, KV,
                                          dk, 192, None)
    assert read(n=0) == 0 and read(n=-1) == INVALID and read(layer=2) == INVALID
    assert read(dt=1) == UNSUPPORTED and read(dk=64) == UNSUPPORTED
    assert read(n=1 << 30, window=1 << 8) == UNSUPPORTED
    for name in ("pk", "pv", "pe", "page", "k", "v"):
        assert read(**{name: None}) == INVALID
        assert read(**{name: A + 2}) == ALIGN


def test_chunk(lib):
    def chunk(pk=A, pv=A, pe=None, page=A, pos=A, start=A, n=2, N=9, P=3, PL=2, layer=0, window=8, sink=1,
              q=A, k=A, v=A, dt=0, o=A, ot=0, ws=A, wb=1 << 40, H=4, KV=2, dk=96, dv=192):
        return lib.gla_window_attn_chunk(pk, pv, pe, page, pos, start, n, N, P, PL, layer, window, sink,
                                         q, k, v, dt, o, ot, ws, wb, H, KV, dk, dv, None)
    assert chunk(n=0) == 0 and chunk(N=0) == 0 and chunk(n=-1) == INVALID and chunk(N=-1) == INVALID
    assert chunk(KV=3) == INVALID and chunk(H=0) == INVALID and chunk(window=0) == INVALID
    assert chunk(sink=-1) == INVALID and chunk(layer=2) == INVALID and chunk(P=0) == INVALID
    assert chunk(dt=1) == UNSUPPORTED and chunk(ot=2) == UNSUPPORTED and chunk(dk=64) == UNSUPPORTED
    assert chunk(dv=96) == UNSUPPORTED and chunk(H=1024, KV=2) == UNSUPPORTED
    assert chunk(N=(1 << 30) + 1) == UNSUPPORTED and chunk(n=1 << 26) == UNSUPPORTED
    assert chunk(window=1 << 30, sink=1) == UNSUPPORTED
    for name in ("pk", "pv", "page", "pos", "start", "q", "k", "v", "o"):
        assert chunk(**{name: None}) == INVALID
        assert chunk(**{name: A + 2}) == ALIGN
    assert chunk(pe=A + 8) == ALIGN
    assert lib.gla_window_attn_chunk_workspace_size(2, 9, 4, 3, 8, 1) == 0
    assert lib.gla_window_attn_chunk_workspace_size(0, 9, 4, 2, 8, 1) == 0
    assert lib.gla_window_attn_chunk_workspace_size(3, 40, 16, 4, 5000, 1) >= 0  # without a device too


def test_decode8(lib):
    def dec(pk=A, pv=A, pe=A, page=A, pos=A, n=2, P=3, PL=2, layer=0, window=8, sink=1, q=A, k=A, v=A,
            dt=0, o=A, ot=0, ws=None, wb=0, H=4, KV=2, dk=96):
        return lib.gla_window_attn8_decode_step(pk, pv, pe, page, pos, n, P, PL, layer, window, sink, q, k,
                                                v, dt, o, ot, ws, wb, H, KV, dk, 192, None)
    assert dec(n=0) == 0 and dec(n=-1) == INVALID and dec(KV=3) == INVALID
    assert dec(layer=2) == INVALID and dec(PL=0) == INVALID and dec(window=-1) == INVALID
    assert dec(dk=64) == UNSUPPORTED and dec(dt=1) == UNSUPPORTED and dec(ot=2) == UNSUPPORTED
    assert dec(n=1 << 29, H=16) == UNSUPPORTED and dec(window=1 << 30, sink=1) == UNSUPPORTED
    for name in ("pk", "pv", "pe", "page", "pos", "q", "k", "v", "o"):
        assert dec(**{name: None}) == INVALID
        assert dec(**{name: A + 2}) == ALIGN
    assert lib.gla_window_attn8_decode_workspace_size(2, 4, 3, 8, 1) == 0
    assert lib.gla_window_attn8_decode_workspace_size(3, 16, 4, 1000, 4) >= 0  # without a device too


def test_the_binding_refuses_host_tensors_and_misfits():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(2, 3, 4), torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(2, 1, 4, 3, 4)
    for call in (lambda: gla.rotary(x, x, torch.zeros(2, dtype=torch.int64)),
                 lambda: gla.window_cache_append(pool, pool, i, i, i, x, x, 4),
                 lambda: gla.window_cache8_read(pool, pool, i, pool, 4),
                 lambda: gla.window_attn_chunk(pool, pool, i, i, i, x, x, x, 4),
                 lambda: gla.window_attn8_decode_step(pool, pool, i, pool, i, x, x, x, 4)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(AttributeError):
        gla.rotary_sideways


# ------------------------------------------------------- sizes and indexes past 32 bits
BIG = 2 ** 32 + 5  # cut off to 5


@pytest.fixture()
def calls(monkeypatch):
    """A library that notes the arguments of its calls, and tensors without memory."""
    torch = pytest.importorskip("torch")
    from gated_linear_attention_chunked_gb300 import layer_ops, serving_ops
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if not name.endswith("_size"):
                    seen.append((name, args))
                return 0
            return call
    monkeypatch.setattr(layer_ops, "_lib", Lib())
    monkeypatch.setattr(serving_ops, "_begin", lambda t, name, stream: (t.get_device(), None))
    monkeypatch.setattr(layer_ops, "_stream", lambda dev: 0)
    empty = torch.empty
    monkeypatch.setattr(layer_ops, "_empty", lambda *s, dtype, device: empty(*s, dtype=dtype, device="meta"))
    return seen


def test_sizes_past_32_bits_are_not_cut_off(calls):
    import torch

    def t(*s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="meta")

    def i(n):
        return t(n, dtype=torch.int32)

    def pools(P=2, PL=1, slots=5, KV=1, dtype=torch.bfloat16):
        return t(P, PL, slots, KV, 96, dtype=dtype), t(P, PL, slots, KV, 192, dtype=dtype)

    def refused(f, *a, **kw):
        with pytest.raises(ValueError, match="32 bits"):
            f(*a, **kw)
        assert not calls
    turns = t(2, dtype=torch.int64)
    for s in ((BIG, 1, 1, 4), (1, BIG, 1, 4), (1, 1, BIG, 4), (1, 1, 1, BIG)):
        refused(gla.rotary, t(*s), None, turns)
    e = t(2, 1, 1, 5, 2, dtype=torch.int8)
    codes = pools(dtype=torch.int8)
    for N, n, layer, window, sink in ((BIG, 1, 0, 4, 1), (3, BIG, 0, 4, 1), (3, 1, BIG, 4, 1),
                                      (3, 1, 0, BIG, 1), (3, 1, 0, 4, BIG)):
        q, k, v = t(N, 1, 96), t(N, 1, 96), t(N, 1, 192)
        refused(gla.window_cache_append, *pools(), i(n), i(n), i(n + 1), k, v, window, sink, layer=layer)
        refused(gla.window_attn_chunk, *pools(), i(n), i(n), i(n + 1), q, k, v, window, sink, layer=layer)
        if n == 1:
            refused(gla.window_attn8_decode_step, *codes, i(N), e, i(N), q, k, v, window, sink, layer=layer)
        if N == 3:
            refused(gla.window_cache8_read, *codes, i(n), e, window, sink, layer=layer)
    for f, args in ((gla.window_attn_chunk_workspace_size, (1, 9, 4, 2, 8, 0)),
                    (gla.window_attn8_decode_workspace_size, (1, 4, 2, 8, 0))):
        for at in range(len(args)):
            refused(f, *args[:at], BIG, *args[at + 1:])
    # and what fits is called as it is
    k, v = t(3, 1, 96), t(3, 1, 192)
    gla.window_cache_append(*codes, i(1), i(1), i(2), k, v, 4, 1, pool_e=e)
    assert calls and calls[0][0] == "gla_window_cache_append" and calls[0][1][10:20] == (1, 3, 2, 1, 0, 4, 1,
                                                                                         1, 96, 192)


def test_misfits(calls):
    import torch

    def t(*s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="meta")
    i, I8 = t(1, dtype=torch.int32), torch.int8
    k, v, q = t(3, 1, 96), t(3, 1, 192), t(3, 2, 96)
    start = t(2, dtype=torch.int32)
    pk, pv = t(2, 1, 5, 1, 96), t(2, 1, 5, 1, 192)
    ck, cv, e = t(2, 1, 5, 1, 96, dtype=I8), t(2, 1, 5, 1, 192, dtype=I8), t(2, 1, 1, 5, 2, dtype=I8)
    app = lambda *p, **kw: gla.window_cache_append(*p, i, i, start, k, v, 4, 1, **kw)  # noqa: E731
    with pytest.raises(TypeError, match="pool_k must be torch.bfloat16"):
        app(ck, cv)
    with pytest.raises(TypeError, match="pool_k must be torch.int8"):
        app(pk, pv, pool_e=e)
    with pytest.raises(ValueError, match="pool_v must be"):
        app(pk, t(2, 1, 4, 1, 192))
    with pytest.raises(ValueError, match="pool_e must be"):
        app(ck, cv, pool_e=t(2, 1, 5, 1, 2, dtype=I8))
    with pytest.raises(ValueError, match="start must be"):
        gla.window_cache_append(pk, pv, i, i, i, k, v, 4, 1)
    with pytest.raises(ValueError, match="count must be"):
        app(pk, pv, count=start)
    with pytest.raises(TypeError, match="v must be"):
        gla.window_attn_chunk(pk, pv, i, i, start, q, k, v.half(), 4, 1)
    with pytest.raises(ValueError, match="pool_e is missing"):
        gla.window_attn8_decode_step(ck, cv, i, None, i, t(1, 2, 96), t(1, 1, 96), t(1, 1, 192), 4, 1)
    with pytest.raises(ValueError, match="pool_e is missing"):
        gla.window_cache8_read(ck, cv, i, None, 4, 1)
    x, turns = t(2, 3, 4, 8), t(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="k must be"):
        gla.rotary(x, x.half(), turns)
    with pytest.raises(ValueError, match="pos must be"):
        gla.rotary(x, x, turns, t(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="turns must be"):
        gla.rotary(x, x, t(4, dtype=torch.float32))
    with pytest.raises(ValueError, match="last axis contiguous"):
        gla.rotary(x.transpose(2, 3), None, turns[:2])
    assert not calls

"""The operators around the mixer refuse bad calls before they touch a device: status codes of
the C ABI (fake addresses that nothing reads) and the binding's checks.  CPU only."""
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


def test_gated_scan(lib):
    def fwd(x=A, g=A, dt=0, init=None, lens=None, y=A, fin=None, B=2, T=5, D=7):
        return lib.gla_gated_scan_fwd(x, g, dt, init, lens, y, fin, B, T, D, None)
    assert fwd(B=0) == INVALID and fwd(T=0) == INVALID and fwd(D=-1) == INVALID
    assert fwd(dt=3) == UNSUPPORTED
    assert fwd(B=1 << 30, D=64) == UNSUPPORTED and fwd(B=1 << 14, T=1 << 22, D=64) == UNSUPPORTED
    assert fwd(T=(1 << 31) - 2) == UNSUPPORTED
    assert fwd(x=None) == INVALID and fwd(g=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(x=A + 2) == ALIGN and fwd(init=A + 4) == ALIGN and fwd(lens=A + 2) == ALIGN
    assert fwd(fin=A + 8) == ALIGN

    def bwd(y=A, dy=A, dx=A, dg=A, dfin=None, dinit=None, T=5, dt=0):
        return lib.gla_gated_scan_bwd(A, A, dt, y, dy, None, dfin, None, dx, dg, dinit, 2, T, 7,
                                      None)
    assert bwd(T=0) == INVALID and bwd(dt=9) == UNSUPPORTED
    assert bwd(y=None) == INVALID and bwd(dy=None) == INVALID and bwd(dg=None) == INVALID
    assert bwd(dfin=A + 4) == ALIGN and bwd(dinit=A + 12) == ALIGN


def test_gated_scan_decode(lib):
    def dec(s=A, x=A, dt=1, y=A, N=3, D=5):
        return lib.gla_gated_scan_decode_step(s, x, A, dt, y, N, D, None)
    assert dec(N=0) == 0 and dec(N=-1) == INVALID and dec(D=0) == INVALID
    assert dec(dt=7) == UNSUPPORTED and dec(N=1 << 38, D=64) == UNSUPPORTED
    assert dec(s=None) == INVALID and dec(y=None) == INVALID and dec(x=A + 4) == ALIGN

    def paged(pool=A, page=A, n=2, P=4, PL=3, l0=0, L=2, D=5, dt=0):
        return lib.gla_gated_scan_decode_step_paged(pool, page, n, P, PL, l0, A, A, dt, A, L, D,
                                                    None)
    assert paged(n=0) == 0 and paged(n=-1) == INVALID and paged(P=0) == INVALID
    assert paged(l0=2) == INVALID and paged(l0=-1) == INVALID and paged(L=0) == INVALID
    assert paged(l0=2, L=(1 << 31) - 1) == INVALID  # layer0 + L past 32 bits
    assert paged(page=None) == INVALID and paged(page=A + 2) == ALIGN and paged(pool=A + 8) == ALIGN
    assert paged(dt=4) == UNSUPPORTED


def test_layer_norm(lib):
    def fwd(x=A, xt=0, w=None, b=None, eps=1e-5, y=A, yt=0, m=None, r=None, n=3, D=9):
        return lib.gla_layer_norm_fwd(x, xt, w, b, eps, y, yt, m, r, n, D, None)
    assert fwd(n=0) == 0 and fwd(n=-1) == INVALID and fwd(D=0) == INVALID
    assert fwd(D=16385) == UNSUPPORTED and fwd(xt=5) == UNSUPPORTED
    assert fwd(xt=0, yt=2) == UNSUPPORTED and fwd(xt=1, yt=0) == UNSUPPORTED
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(w=A + 4) == ALIGN and fwd(m=A + 4) == ALIGN

    def bwd(dy=A, dt=0, x=A, xt=0, m=A, r=A, dx=A, dw=A, db=A, ws=None, wb=0, n=3, D=9):
        return lib.gla_layer_norm_bwd(dy, dt, x, xt, None, m, r, dx, dw, db, ws, wb, n, D, None)
    assert bwd(n=-2) == INVALID and bwd(D=16385) == UNSUPPORTED and bwd(dt=2) == UNSUPPORTED
    assert bwd(m=None) == INVALID and bwd(dx=None) == INVALID
    assert bwd() == WORKSPACE and bwd(ws=0x10010, wb=1 << 30) == ALIGN
    assert bwd(dw=A + 4) == ALIGN
    assert lib.gla_layer_norm_bwd_workspace_size(0, 9) == 0


def test_window_attn(lib):
    def fwd(q=A, dt=0, lens=None, window=8, sink=0, o=A, ot=0, lse=None, B=1, T=9, H=4, KV=2,
            dk=96, dv=192):
        return lib.gla_window_attn_fwd(q, A, A, dt, lens, window, sink, o, ot, lse, B, T, H, KV,
                                       dk, dv, None)
    assert fwd(B=0) == INVALID and fwd(T=0) == INVALID and fwd(H=0) == INVALID
    assert fwd(KV=3) == INVALID and fwd(KV=0) == INVALID and fwd(KV=-2) == INVALID
    assert fwd(window=0) == INVALID and fwd(sink=-1) == INVALID
    assert fwd(dk=64) == UNSUPPORTED and fwd(dv=96) == UNSUPPORTED
    assert fwd(dt=1) == UNSUPPORTED and fwd(dt=0, ot=2) == UNSUPPORTED and fwd(dt=5, ot=5) == UNSUPPORTED
    assert fwd(T=(1 << 30) + 1) == UNSUPPORTED and fwd(B=1 << 20, T=1 << 12) == UNSUPPORTED
    assert fwd(B=1 << 28, T=1, H=16) == UNSUPPORTED
    assert fwd(q=None) == INVALID and fwd(o=None) == INVALID
    assert fwd(q=A + 8) == ALIGN and fwd(lens=A + 2) == ALIGN and fwd(lse=A + 2) == ALIGN

    def bwd(lse=A, dO=A, dq=A, dk=A, dv=A, ws=A, wb=1 << 30, H=4, KV=2, dt=0, ot=0, st=None):
        strides = None if st is None else (ctypes.c_longlong * 3)(*st)
        return lib.gla_window_attn_bwd(A, A, A, dt, None, 8, 0, A, strides, ot, lse, dO, dq, dk, dv, ws, wb,
                                       1, 9, H, KV, 96, 192, None)
    assert bwd(KV=3) == INVALID and bwd(dt=1) == UNSUPPORTED and bwd(ot=2) == UNSUPPORTED
    assert bwd(lse=None) == INVALID and bwd(dO=None) == INVALID and bwd(dv=None) == INVALID
    assert bwd(st=(-192, 192, 192)) == INVALID and bwd(st=(192, 192, 194)) == ALIGN
    need = lib.gla_window_attn_bwd_workspace_size(1, 9, 4, 2, 8, 0)
    assert need > 0 and bwd(ws=None) == WORKSPACE and bwd(wb=need - 1) == WORKSPACE
    assert bwd(ws=A + 16, wb=need) == ALIGN and bwd(dk=A + 8) == ALIGN
    assert lib.gla_window_attn_bwd_workspace_size(1, 9, 4, 3, 8, 0) == 0


def test_window_cache(lib):
    def fill(pk=A, page=A, dt=0, P=3, PL=2, layer=0, window=8, sink=1, B=2, T=9, KV=2, lens=None):
        return lib.gla_window_cache_fill(A, A, dt, lens, pk, A, page, P, PL, layer, window, sink,
                                         B, T, KV, 96, 192, None)
    assert fill(layer=2) == INVALID and fill(layer=-1) == INVALID and fill(P=0) == INVALID
    assert fill(T=0) == INVALID and fill(window=0) == INVALID and fill(dt=1) == UNSUPPORTED
    assert fill(window=(1 << 30) + 1) == UNSUPPORTED and fill(P=1 << 30, window=1 << 12) == UNSUPPORTED
    assert fill(pk=None) == INVALID and fill(page=None) == INVALID
    assert fill(pk=A + 8) == ALIGN and fill(page=A + 2) == ALIGN and fill(lens=A + 1) == ALIGN

    def dec(pk=A, dt=0, page=A, pos=A, n=2, P=3, PL=2, layer=0, window=8, sink=1, o=A, ot=0,
            ws=None, wb=0, H=4, KV=2, dk=96):
        return lib.gla_window_attn_decode_step(pk, A, dt, page, pos, n, P, PL, layer, window, sink,
                                               A, A, A, o, ot, ws, wb, H, KV, dk, 192, None)
    assert dec(n=0) == 0 and dec(n=-1) == INVALID and dec(KV=3) == INVALID
    assert dec(layer=2) == INVALID and dec(PL=0) == INVALID and dec(window=-1) == INVALID
    assert dec(dk=64) == UNSUPPORTED and dec(dt=1) == UNSUPPORTED and dec(ot=2) == UNSUPPORTED
    assert dec(n=1 << 29, H=16) == UNSUPPORTED
    assert dec(window=1 << 30, sink=1) == UNSUPPORTED
    assert dec(pos=None) == INVALID and dec(o=None) == INVALID
    assert dec(pos=A + 2) == ALIGN and dec(pk=A + 8) == ALIGN
    assert lib.gla_window_attn_decode_workspace_size(2, 4, 3, 8, 1) == 0
    assert lib.gla_window_attn_decode_workspace_size(3, 16, 4, 1000, 4) >= 0  # without a device too


def test_the_binding_refuses_host_tensors_and_misfits():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 4)
    for call in (lambda: gla.gated_scan_fwd(x, x), lambda: gla.layer_norm_fwd(x),
                 lambda: gla.gated_scan_decode_step(x, x, x),
                 lambda: gla.gated_scan_decode_step_paged(x, x, x, x),
                 lambda: gla.window_attn_fwd(x[None], x[None], x[None], 4),
                 lambda: gla.window_attn_decode_step(x, x, x, x, x, x, x, 4),
                 lambda: gla.window_cache_fill(x, x, x, x[None], x[None], 4)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(AttributeError):
        gla.layer_norm_sideways

"""Binding of the operators around the mixer: gated scan, layer norm, windowed attention.

The functions are part of the package's namespace (``gla.gated_scan_fwd`` ...).  As there, this is
argument marshalling only.  All tensors of a call lie on one CUDA device, which need not be the
current one; outputs and workspaces are allocated there, on the stream of the call.
"""
from __future__ import annotations

import ctypes

import torch

CODES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
F32, I32 = torch.float32, torch.int32

_empty = torch.empty
_getdev = torch._C._cuda_getDevice
# the handle of a device's current stream; torch.cuda.current_stream(dev).cuda_stream costs 6 us a
# call, a third of a small call's time
_stream = torch._C._cuda_getCurrentRawStream
_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load
        _lib = load()
    return _lib


def _fail(call: str, rc: int):
    from . import GlaError
    raise GlaError(call, rc)


def _code(t, name) -> int:
    code = CODES.get(t)
    if code is None:
        raise TypeError(f"unsupported {name} dtype {t}")
    return code


def _ptr(t, name, dev, dtype, shape):
    """Pointer of a contiguous tensor of the call's device, type and shape (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _view(t, name, dev, shape):
    """Pointer and strides (None: contiguous) of a tensor whose last axis is contiguous."""
    if t.is_contiguous():
        return _ptr(t, name, dev, t.dtype, shape), None
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.shape != shape or t.stride(-1) != 1:
        raise ValueError(f"{name} must be {list(shape)} with its last axis contiguous")
    strides = [s if n > 1 else 0 for s, n in zip(t.stride()[:-1], shape)]
    return t.data_ptr(), (ctypes.c_longlong * len(strides))(*strides)


def _begin(t, name, stream):
    """(device index, context to leave or None) of a call on tensor t's device and `stream` (None:
    that device's current one): what the call allocates and launches goes there."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if stream is None and dev == _getdev():
        return dev, None
    if stream is not None and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, {name} on {t.device}")
    ctx = torch.cuda.device(t.device) if stream is None else torch.cuda.stream(stream)
    ctx.__enter__()
    return dev, ctx


def _end(ctx):
    if ctx is not None:
        ctx.__exit__(None, None, None)


# The C ABI's sizes and indexes are 32-bit, and ctypes cuts off what is above without a word.
_MOST = 2 ** 31 - 1


def _fit(*values):
    """Refuses sizes and indexes that the C ABI's int does not hold.  (Called where a bit above the
    lowest 31 is set in any of them, which costs a call that has none a tenth of a microsecond.)"""
    if any(not -_MOST <= v <= _MOST for v in values):
        raise ValueError(f"sizes and indexes must fit 32 bits, got {values}")


def _reach(window, sink):
    """Window and sinks of a call on whole sequences, where any value past T means all of T."""
    return max(min(window, _MOST), -1), max(min(sink, _MOST), -1)


def _scratch(nbytes, dev, workspace):
    """(pointer, bytes, tensor) of the caller's workspace or a new one."""
    if workspace is None:
        workspace = _empty(nbytes, dtype=torch.uint8, device=dev)
        return workspace.data_ptr(), nbytes, workspace
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{dev}")
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError("workspace too small")
    return workspace.data_ptr(), have, workspace


# ------------------------------------------------------------------------- gated scan
def gated_scan_fwd(x, g, init_state=None, lens=None, *, want_final_state=True, out=None,
                   stream=None):
    """Gated scan h_t = f_t h_{t-1} + (1 - f_t) x_t, f = sigmoid(g) (gla_gated_scan_fwd).
    x, g [B,T,D] (bf16/fp16/fp32), init_state [B,D] fp32, lens [B] int32: tokens of each sequence,
    the rest is padding.  Returns (y fp32 [B,T,D], final_state fp32 [B,D] or None)."""
    B, T, D = x.shape
    if (B | T | D) >> 31:
        _fit(B, T, D)
    t = x.dtype
    dev, ctx = _begin(x, "x", stream)
    try:
        y = _empty((B, T, D), dtype=F32, device=dev) if out is None else out
        fin = _empty((B, D), dtype=F32, device=dev) if want_final_state else None
        rc = _library().gla_gated_scan_fwd(
            _ptr(x, "x", dev, t, x.shape), _ptr(g, "g", dev, t, x.shape), _code(t, "input"),
            _ptr(init_state, "init_state", dev, F32, (B, D)), _ptr(lens, "lens", dev, I32, (B,)),
            _ptr(y, "out", dev, F32, x.shape), None if fin is None else fin.data_ptr(), B, T, D,
            _stream(dev))
        if rc:
            _fail("gla_gated_scan_fwd", rc)
    finally:
        _end(ctx)
    return y, fin


def gated_scan_bwd(x, g, y, dy, init_state=None, d_final_state=None, lens=None, *,
                   want_d_init_state=True, stream=None):
    """Gradient of gated_scan_fwd (gla_gated_scan_bwd); y: the forward's output, dy [B,T,D] fp32.
    Returns (dx, dg, d_init_state or None), fp32."""
    B, T, D = x.shape
    if (B | T | D) >> 31:
        _fit(B, T, D)
    t = x.dtype
    dev, ctx = _begin(x, "x", stream)
    try:
        dx = _empty((B, T, D), dtype=F32, device=dev)
        dg = _empty((B, T, D), dtype=F32, device=dev)
        dinit = _empty((B, D), dtype=F32, device=dev) if want_d_init_state else None
        rc = _library().gla_gated_scan_bwd(
            _ptr(x, "x", dev, t, x.shape), _ptr(g, "g", dev, t, x.shape), _code(t, "input"),
            _ptr(y, "y", dev, F32, x.shape), _ptr(dy, "dy", dev, F32, x.shape),
            _ptr(init_state, "init_state", dev, F32, (B, D)),
            _ptr(d_final_state, "d_final_state", dev, F32, (B, D)),
            _ptr(lens, "lens", dev, I32, (B,)), dx.data_ptr(), dg.data_ptr(),
            None if dinit is None else dinit.data_ptr(), B, T, D, _stream(dev))
        if rc:
            _fail("gla_gated_scan_bwd", rc)
    finally:
        _end(ctx)
    return dx, dg, dinit


def gated_scan_decode_step(state, x, g, *, out=None, stream=None):
    """One token of the gated scan (gla_gated_scan_decode_step): state [..., D] fp32 is updated in
    place, x, g the same shape (bf16/fp16/fp32).  Returns y fp32 (the new state)."""
    D = x.shape[-1]
    if D >> 31:
        _fit(D)
    t = x.dtype
    dev, ctx = _begin(x, "x", stream)
    try:
        y = _empty(x.shape, dtype=F32, device=dev) if out is None else out
        rc = _library().gla_gated_scan_decode_step(
            _ptr(state, "state", dev, F32, x.shape), _ptr(x, "x", dev, t, x.shape),
            _ptr(g, "g", dev, t, x.shape), _code(t, "input"), _ptr(y, "out", dev, F32, x.shape),
            x.numel() // max(D, 1), D, _stream(dev))
        if rc:
            _fail("gla_gated_scan_decode_step", rc)
    finally:
        _end(ctx)
    return y


def gated_scan_decode_step_paged(pool, page, x, g, *, layer0=0, out=None, stream=None):
    """The same over a state pool (gla_gated_scan_decode_step_paged): pool [P,pool_layers,D] fp32 is
    updated in place for pages page[n] (int32 [n_active], distinct) and layers layer0..layer0+L-1;
    x, g [n_active,L,D].  Returns y fp32 [n_active,L,D]."""
    n, L, D = x.shape
    P, PL, _ = pool.shape
    if (n | P | PL | layer0 | L | D) >> 31:
        _fit(n, P, PL, layer0, L, D)
    t = x.dtype
    dev, ctx = _begin(x, "x", stream)
    try:
        y = _empty(x.shape, dtype=F32, device=dev) if out is None else out
        rc = _library().gla_gated_scan_decode_step_paged(
            _ptr(pool, "pool", dev, F32, (P, PL, D)), _ptr(page, "page", dev, I32, (n,)), n, P, PL,
            layer0, _ptr(x, "x", dev, t, x.shape), _ptr(g, "g", dev, t, x.shape),
            _code(t, "input"), _ptr(y, "out", dev, F32, x.shape), L, D, _stream(dev))
        if rc:
            _fail("gla_gated_scan_decode_step_paged", rc)
    finally:
        _end(ctx)
    return y


# ------------------------------------------------------------------------- layer norm
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, *, out_dtype=None, want_stats=True,
                   out=None, stream=None):
    """Layer norm over the last axis (gla_layer_norm_fwd): x [..., D] (bf16/fp16/fp32), weight,
    bias [D] fp32.  out_dtype: x's type (default) or fp32.  Returns (y, mean, rstd), the last two
    fp32 [...] or None."""
    D = x.shape[-1]
    if D >> 31:
        _fit(D)
    t = x.dtype
    dev, ctx = _begin(x, "x", stream)
    try:
        if out is None:
            out = _empty(x.shape, dtype=out_dtype or t, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        mean = _empty(x.shape[:-1], dtype=F32, device=dev) if want_stats else None
        rstd = _empty(x.shape[:-1], dtype=F32, device=dev) if want_stats else None
        rc = _library().gla_layer_norm_fwd(
            _ptr(x, "x", dev, t, x.shape), _code(t, "input"),
            _ptr(weight, "weight", dev, F32, (D,)), _ptr(bias, "bias", dev, F32, (D,)), eps,
            _ptr(out, "out", dev, out.dtype, x.shape), _code(out.dtype, "output"),
            None if mean is None else mean.data_ptr(), None if rstd is None else rstd.data_ptr(),
            x.numel() // max(D, 1), D, _stream(dev))
        if rc:
            _fail("gla_layer_norm_fwd", rc)
    finally:
        _end(ctx)
    return out, mean, rstd


def layer_norm_bwd_workspace_size(n_tokens, D) -> int:
    if D >> 31:
        _fit(D)
    return _library().gla_layer_norm_bwd_workspace_size(n_tokens, D)


def layer_norm_bwd(dy, x, weight, mean, rstd, *, workspace=None, stream=None):
    """Gradient of layer_norm_fwd (gla_layer_norm_bwd): dy [..., D] of x's type or fp32, which is
    also dx's type; mean, rstd as the forward returned them.  Returns (dx, d_weight, d_bias), the
    last two fp32 [D]."""
    D = x.shape[-1]
    if D >> 31:
        _fit(D)
    t = x.dtype
    n = x.numel() // max(D, 1)
    dev, ctx = _begin(x, "x", stream)
    try:
        dx = _empty(x.shape, dtype=dy.dtype, device=dev)
        dw = _empty((D,), dtype=F32, device=dev)
        db = _empty((D,), dtype=F32, device=dev)
        lib = _library()
        wp, wb, hold = _scratch(lib.gla_layer_norm_bwd_workspace_size(n, D), dev, workspace)
        rc = lib.gla_layer_norm_bwd(
            _ptr(dy, "dy", dev, dy.dtype, x.shape), _code(dy.dtype, "dy"),
            _ptr(x, "x", dev, t, x.shape), _code(t, "input"),
            _ptr(weight, "weight", dev, F32, (D,)),
            _ptr(mean, "mean", dev, F32, x.shape[:-1]), _ptr(rstd, "rstd", dev, F32, x.shape[:-1]),
            dx.data_ptr(), dw.data_ptr(), db.data_ptr(), wp, wb, n, D, _stream(dev))
        if rc:
            _fail("gla_layer_norm_bwd", rc)
    finally:
        _end(ctx)
    return dx, dw, db


# ------------------------------------------------------------------ windowed attention
def window_attn_fwd(q, k, v, window, sink=0, lens=None, *, out_dtype=None, want_lse=True,
                    out=None, stream=None):
    """Causal attention over the last `window` tokens and the first `sink` (gla_window_attn_fwd).
    q [B,T,H,96], k [B,T,KV,96], v [B,T,KV,192] (bf16/fp16, q pre-scaled; KV divides H), lens [B]
    int32: tokens of each sequence, the rest is padding.  out_dtype: q's type (default) or fp32.
    Returns (o [B,T,H,192], lse fp32 [B,H,T] or None)."""
    B, T, H, dk = q.shape
    KV, dv = v.shape[2], v.shape[3]
    if (B | T | H | KV | dk | dv) >> 31:
        _fit(B, T, H, KV, dk, dv)
    window, sink = _reach(window, sink)
    t = q.dtype
    dev, ctx = _begin(q, "q", stream)
    try:
        if out is None:
            out = _empty((B, T, H, dv), dtype=out_dtype or t, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        lse = _empty((B, H, T), dtype=F32, device=dev) if want_lse else None
        rc = _library().gla_window_attn_fwd(
            _ptr(q, "q", dev, t, q.shape), _ptr(k, "k", dev, t, (B, T, KV, dk)),
            _ptr(v, "v", dev, t, (B, T, KV, dv)), _code(t, "input"),
            _ptr(lens, "lens", dev, I32, (B,)), window, sink,
            _ptr(out, "out", dev, out.dtype, (B, T, H, dv)), _code(out.dtype, "output"),
            None if lse is None else lse.data_ptr(), B, T, H, KV, dk, dv, _stream(dev))
        if rc:
            _fail("gla_window_attn_fwd", rc)
    finally:
        _end(ctx)
    return out, lse


def window_attn_bwd_workspace_size(B, T, H, KV, window, sink=0) -> int:
    if (B | T | H | KV) >> 31:
        _fit(B, T, H, KV)
    window, sink = _reach(window, sink)
    return _library().gla_window_attn_bwd_workspace_size(B, T, H, KV, window, sink)


def window_attn_bwd(q, k, v, o, lse, dO, window, sink=0, lens=None, *, workspace=None,
                    stream=None):
    """Gradient of window_attn_fwd (gla_window_attn_bwd): o, lse as the forward returned them (o may
    be a view of another layout whose channels are adjacent), dO of q's type.  Returns (dq, dk,
    dv), of o's type."""
    B, T, H, dk_ = q.shape
    KV, dv_ = v.shape[2], v.shape[3]
    if (B | T | H | KV | dk_ | dv_) >> 31:
        _fit(B, T, H, KV, dk_, dv_)
    window, sink = _reach(window, sink)
    t = q.dtype
    dev, ctx = _begin(q, "q", stream)
    try:
        dq = _empty(q.shape, dtype=o.dtype, device=dev)
        dk = _empty(k.shape, dtype=o.dtype, device=dev)
        dv = _empty(v.shape, dtype=o.dtype, device=dev)
        lib = _library()
        wp, wb, hold = _scratch(lib.gla_window_attn_bwd_workspace_size(B, T, H, KV, window, sink),
                                dev, workspace)
        rc = lib.gla_window_attn_bwd(
            _ptr(q, "q", dev, t, q.shape), _ptr(k, "k", dev, t, (B, T, KV, dk_)),
            _ptr(v, "v", dev, t, (B, T, KV, dv_)), _code(t, "input"),
            _ptr(lens, "lens", dev, I32, (B,)), window, sink,
            *_view(o, "o", dev, (B, T, H, dv_)), _code(o.dtype, "output"),
            _ptr(lse, "lse", dev, F32, (B, H, T)), _ptr(dO, "dO", dev, t, (B, T, H, dv_)),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), wp, wb, B, T, H, KV, dk_, dv_,
            _stream(dev))
        if rc:
            _fail("gla_window_attn_bwd", rc)
    finally:
        _end(ctx)
    return dq, dk, dv


def window_cache_fill(pool_k, pool_v, page, k, v, window, sink=0, lens=None, *, layer=0,
                      stream=None):
    """The keys and values of prompts into their pages (gla_window_cache_fill).  pool_k, pool_v
    [P,pool_layers,sink+window,KV,96|192] (bf16/fp16) are updated in place in layer `layer` of
    pages page[b] (int32 [B], distinct); k [B,T,KV,96], v [B,T,KV,192], lens [B] int32."""
    B, T, KV, dk = k.shape
    dv = v.shape[-1]
    P, PL = pool_k.shape[:2]
    if (B | T | KV | dk | dv | P | PL | layer | window | sink) >> 31:
        _fit(B, T, KV, dk, dv, P, PL, layer, window, sink)
    t = k.dtype
    slots = window + sink
    dev, ctx = _begin(k, "k", stream)
    try:
        rc = _library().gla_window_cache_fill(
            _ptr(k, "k", dev, t, k.shape), _ptr(v, "v", dev, t, (B, T, KV, dv)),
            _code(t, "input"), _ptr(lens, "lens", dev, I32, (B,)),
            _ptr(pool_k, "pool_k", dev, t, (P, PL, slots, KV, dk)),
            _ptr(pool_v, "pool_v", dev, t, (P, PL, slots, KV, dv)),
            _ptr(page, "page", dev, I32, (B,)), P, PL, layer, window, sink, B, T, KV, dk, dv,
            _stream(dev))
        if rc:
            _fail("gla_window_cache_fill", rc)
    finally:
        _end(ctx)


def window_attn_decode_workspace_size(n_active, H, KV, window, sink=0) -> int:
    if (n_active | H | KV | window | sink) >> 31:
        _fit(n_active, H, KV, window, sink)
    return _library().gla_window_attn_decode_workspace_size(n_active, H, KV, window, sink)


def window_attn_decode_step(pool_k, pool_v, page, pos, q, k, v, window, sink=0, *, layer=0,
                            out_dtype=None, out=None, workspace=None, stream=None):
    """One token of the windowed attention over its caches (gla_window_attn_decode_step).  pool_k,
    pool_v as in window_cache_fill get the token's key and value in place; page, pos int32
    [n_active]: its page and its position from 0; q [n_active,H,96], k [n_active,KV,96], v
    [n_active,KV,192].  out_dtype: q's type (default) or fp32.  Returns o [n_active,H,192]."""
    n, H, dk = q.shape
    KV, dv = v.shape[1], v.shape[2]
    P, PL = pool_k.shape[:2]
    if (n | H | KV | dk | dv | P | PL | layer | window | sink) >> 31:
        _fit(n, H, KV, dk, dv, P, PL, layer, window, sink)
    t = q.dtype
    slots = window + sink
    dev, ctx = _begin(q, "q", stream)
    try:
        if out is None:
            out = _empty((n, H, dv), dtype=out_dtype or t, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        lib = _library()
        wp, wb, hold = _scratch(lib.gla_window_attn_decode_workspace_size(n, H, KV, window, sink),
                                dev, workspace)
        rc = lib.gla_window_attn_decode_step(
            _ptr(pool_k, "pool_k", dev, t, (P, PL, slots, KV, dk)),
            _ptr(pool_v, "pool_v", dev, t, (P, PL, slots, KV, dv)), _code(t, "input"),
            _ptr(page, "page", dev, I32, (n,)), _ptr(pos, "pos", dev, I32, (n,)), n, P, PL, layer,
            window, sink, _ptr(q, "q", dev, t, q.shape), _ptr(k, "k", dev, t, (n, KV, dk)),
            _ptr(v, "v", dev, t, (n, KV, dv)), _ptr(out, "out", dev, out.dtype, (n, H, dv)),
            _code(out.dtype, "output"), wp, wb, H, KV, dk, dv, _stream(dev))
        if rc:
            _fail("gla_window_attn_decode_step", rc)
    finally:
        _end(ctx)
    return out

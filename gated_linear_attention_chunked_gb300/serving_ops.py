"""Binding of serving with the windowed attention: rotary positions, packed tokens into pages of 16
and 8 bits, chunks of tokens and single ones over them.

The functions are part of the package's namespace (``gla.rotary`` ...).  As in layer_ops.py this is
argument marshalling only, with the same rules for devices, streams and workspaces.
"""
from __future__ import annotations

import ctypes

import torch

from . import layer_ops as _ops
from .layer_ops import I32, _begin, _code, _end, _fail, _fit, _ptr

I8, I64 = torch.int8, torch.int64
_Three = ctypes.c_longlong * 3
SCALING = {"plain": 0, "linear": 1, "base": 2, "parts": 3}


def _view3(t, name, dev, shape):
    """_view of a [B,T,heads,D] tensor, whose three strides are put down without a list (half a microsecond)."""
    if t.is_contiguous() or t.get_device() != dev or t.shape != shape or t.stride(-1) != 1:
        return _ops._view(t, name, dev, shape)
    a, b, c, _ = t.stride()
    return t.data_ptr(), _Three(a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, c if shape[2] > 1 else 0)


def _scratch(size, dev, workspace):
    """_ops._scratch, but for nothing where nothing is needed: an empty tensor costs as much as any."""
    return (None, 0, None) if size == 0 and workspace is None else _ops._scratch(size, dev, workspace)


# ------------------------------------------------------------------------------ rotary
def rotary_turns(R, base=10000.0, scaling="plain", factor=1.0, *, context=4096, low=1.0, high=32.0):
    """The table of `rotary` for R channels (gla_rotary_turns): a HOST int64 tensor [R / 2], turns per
    position in units of 2^-64.  scaling: "plain", or for contexts `factor` times as long as those trained
    on "linear", "base" or "parts" (by how often a pair turns within `context` tokens: at least `high`
    times it stays, at most `low` times it is divided by factor)."""
    if scaling not in SCALING:
        raise ValueError(f"scaling must be one of {sorted(SCALING)}, got {scaling!r}")
    if R >> 31:
        _fit(R)
    if R < 2 or R % 2:
        raise ValueError(f"R must be even and at least 2, got {R}")
    out = torch.empty(R // 2, dtype=I64)
    rc = _ops._library().gla_rotary_turns(R, base, SCALING[scaling], factor, context, low, high,
                                          out.data_ptr())
    if rc:
        _fail("gla_rotary_turns", rc)
    return out


def rotary(q, k, turns, pos=None, *, interleaved=False, inverse=False, scale=1.0, out_dtype=None,
           q_out=None, k_out=None, stream=None):
    """Rotary positions (gla_rotary): q [B,T,H,D] and k [B,T,KV,D] (or None; bf16/fp16/fp32) have the pairs
    of their first R = 2 len(turns) channels turned by the angles of positions pos (int32 [B,T]; None:
    token t of each sequence at t).  turns: int64 [R / 2] on the device, from rotary_turns.  Packed
    tokens are q [N,H,D], k [N,KV,D], pos [N].  inverse: the gradient, (dq, dk) from those of the results.
    q and k may be views whose channels are adjacent; q_out may be q itself, where that is contiguous
    and keeps its type, and k_out k.  out_dtype: q's type (default) or fp32.  Returns (q', k')."""
    packed = q.dim() == 3
    if packed:
        q, k = q[None], None if k is None else k[None]
        pos = None if pos is None else pos[None]
        q_out = None if q_out is None else q_out[None]
        k_out = None if k_out is None else k_out[None]
    B, T, H, D = q.shape
    KV = 0 if k is None else k.shape[-2]
    R = 2 * turns.shape[0]
    if (B | T | H | D | KV | R) >> 31:
        _fit(B, T, H, D, KV, R)
    t = q.dtype
    dev, ctx = _begin(q, "q", stream)
    try:
        out = (out_dtype or t) if q_out is None else q_out.dtype
        if out_dtype is not None and out != out_dtype:
            raise TypeError(f"q_out must be {out_dtype}, got {out}")
        if q_out is None:
            q_out = _ops._empty((B, T, H, D), dtype=out, device=dev)
            qo = q_out.data_ptr()
        else:
            qo = _ptr(q_out, "q_out", dev, out, (B, T, H, D))
        if k is None:
            kp, ks, ko = None, None, None
        else:
            if k.dtype != t:
                raise TypeError(f"k must be {t}, got {k.dtype}")
            kp, ks = _view3(k, "k", dev, (B, T, KV, D))
            if k_out is None:
                k_out = _ops._empty((B, T, KV, D), dtype=out, device=dev)
                ko = k_out.data_ptr()
            else:
                ko = _ptr(k_out, "k_out", dev, out, (B, T, KV, D))
        rc = _ops._library().gla_rotary(
            *_view3(q, "q", dev, q.shape), qo, H, kp, ks, ko, KV,
            _code(t, "input"), _code(out, "output"), _ptr(turns, "turns", dev, I64, (R // 2,)),
            _ptr(pos, "pos", dev, I32, (B, T)), scale, 1 if interleaved else 0, 1 if inverse else 0,
            B, T, D, R, _ops._stream(dev))
        if rc:
            _fail("gla_rotary", rc)
    finally:
        _end(ctx)
    if packed:
        return q_out[0], None if k is None else k_out[0]
    return q_out, k_out if k is not None else None


# ------------------------------------------------------------------------------- pages
def _pools(pool_k, pool_v, pool_e, dev, t, P, PL, slots, KV, dk, dv):
    """Pointers of the pools: 16-bit ones of type t, or codes and exponents."""
    row = t if pool_e is None else I8
    return (_ptr(pool_k, "pool_k", dev, row, (P, PL, slots, KV, dk)),
            _ptr(pool_v, "pool_v", dev, row, (P, PL, slots, KV, dv)),
            _ptr(pool_e, "pool_e", dev, I8, (P, PL, KV, slots, 2)))


def window_cache_append(pool_k, pool_v, page, pos, start, k, v, window, sink=0, count=None, *,
                        layer=0, pool_e=None, stream=None):
    """Packed tokens' keys and values into their sequences' pages (gla_window_cache_append).  k [N,KV,96],
    v [N,KV,192] (bf16/fp16); sequence b has rows start[b] .. start[b+1] - 1 (int32 [n+1]), the first at
    position pos[b], and of them the first count[b] (None: all) go into layer `layer` of page page[b].
    Pools as in window_cache_fill, or of 8 bits: int8 pool_k, pool_v and their exponents pool_e int8
    [P,pool_layers,KV,sink+window,2].  Updated in place."""
    N, KV, dk = k.shape
    dv, n = v.shape[-1], page.shape[0]
    P, PL = pool_k.shape[:2]
    if (N | KV | dk | dv | n | P | PL | layer | window | sink) >> 31:
        _fit(N, KV, dk, dv, n, P, PL, layer, window, sink)
    t = k.dtype
    dev, ctx = _begin(k, "k", stream)
    try:
        kp, vp, ep = _pools(pool_k, pool_v, pool_e, dev, t, P, PL, window + sink, KV, dk, dv)
        rc = _ops._library().gla_window_cache_append(
            _ptr(k, "k", dev, t, k.shape), _ptr(v, "v", dev, t, (N, KV, dv)), _code(t, "input"),
            _ptr(pos, "pos", dev, I32, (n,)), _ptr(start, "start", dev, I32, (n + 1,)),
            _ptr(count, "count", dev, I32, (n,)), kp, vp, ep, _ptr(page, "page", dev, I32, (n,)), n, N,
            P, PL, layer, window, sink, KV, dk, dv, _ops._stream(dev))
        if rc:
            _fail("gla_window_cache_append", rc)
    finally:
        _end(ctx)


def window_cache8_read(pool_k, pool_v, page, pool_e, window, sink=0, *, layer=0,
                       out_dtype=torch.bfloat16, stream=None):
    """Layer `layer` of 8-bit pages page[n] (int32 [n], they may repeat) as 16-bit rows by slot
    (gla_window_cache8_read).  Returns (k [n,sink+window,KV,96], v [n,sink+window,KV,192])."""
    P, PL, slots, KV, dk = pool_k.shape
    dv, n = pool_v.shape[-1], page.shape[0]
    if (P | PL | KV | dk | dv | n | layer | window | sink) >> 31:
        _fit(P, PL, KV, dk, dv, n, layer, window, sink)
    slots = window + sink
    dev, ctx = _begin(pool_k, "pool_k", stream)
    try:
        if pool_e is None:
            raise ValueError("pool_e is missing: only pages of 8 bits are read back")
        kp, vp, ep = _pools(pool_k, pool_v, pool_e, dev, None, P, PL, slots, KV, dk, dv)
        k = _ops._empty((n, slots, KV, dk), dtype=out_dtype, device=dev)
        v = _ops._empty((n, slots, KV, dv), dtype=out_dtype, device=dev)
        rc = _ops._library().gla_window_cache8_read(
            kp, vp, ep, _ptr(page, "page", dev, I32, (n,)), n, P, PL, layer, window, sink,
            k.data_ptr(), v.data_ptr(), _code(out_dtype, "output"), KV, dk, dv, _ops._stream(dev))
        if rc:
            _fail("gla_window_cache8_read", rc)
    finally:
        _end(ctx)
    return k, v


# --------------------------------------------------------------------------- attention
def window_attn_chunk_workspace_size(n, n_tokens, H, KV, window, sink=0, bits=None) -> int:
    """Bytes of `workspace` of window_attn_chunk over pages of `bits` 16 or 8 (None: enough for either)."""
    if (n | n_tokens | H | KV | window | sink) >> 31:
        _fit(n, n_tokens, H, KV, window, sink)
    if bits not in (None, 8, 16):
        raise ValueError(f"bits must be 8 or 16, got {bits}")
    size = getattr(_ops._library(), f"gla_window_attn_chunk{bits or ''}_workspace_size")
    return size(n, n_tokens, H, KV, window, sink)


def window_attn_chunk(pool_k, pool_v, page, pos, start, q, k, v, window, sink=0, *, layer=0,
                      pool_e=None, out_dtype=None, out=None, workspace=None, stream=None):
    """The windowed attention of packed new tokens over their sequences' pages and each other
    (gla_window_attn_chunk): q [N,H,96], k [N,KV,96], v [N,KV,192] (bf16/fp16); pools, page, pos and start
    as in window_cache_append, which puts the tokens into the pages afterwards (this call only reads
    them).  out_dtype: q's type (default) or fp32.  Returns o [N,H,192]."""
    N, H, dk = q.shape
    KV, dv, n = v.shape[1], v.shape[2], page.shape[0]
    P, PL = pool_k.shape[:2]
    if (N | H | KV | dk | dv | n | P | PL | layer | window | sink) >> 31:
        _fit(N, H, KV, dk, dv, n, P, PL, layer, window, sink)
    t = q.dtype
    dev, ctx = _begin(q, "q", stream)
    try:
        if out is None:
            out = _ops._empty((N, H, dv), dtype=out_dtype or t, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        kp, vp, ep = _pools(pool_k, pool_v, pool_e, dev, t, P, PL, window + sink, KV, dk, dv)
        lib = _ops._library()
        size = (lib.gla_window_attn_chunk16_workspace_size if pool_e is None else
                lib.gla_window_attn_chunk8_workspace_size)
        wp, wb, hold = _scratch(size(n, N, H, KV, window, sink), dev, workspace)
        rc = lib.gla_window_attn_chunk(
            kp, vp, ep, _ptr(page, "page", dev, I32, (n,)), _ptr(pos, "pos", dev, I32, (n,)),
            _ptr(start, "start", dev, I32, (n + 1,)), n, N, P, PL, layer, window, sink,
            _ptr(q, "q", dev, t, q.shape), _ptr(k, "k", dev, t, (N, KV, dk)),
            _ptr(v, "v", dev, t, (N, KV, dv)), _code(t, "input"),
            _ptr(out, "out", dev, out.dtype, (N, H, dv)), _code(out.dtype, "output"), wp, wb, H, KV,
            dk, dv, _ops._stream(dev))
        if rc:
            _fail("gla_window_attn_chunk", rc)
    finally:
        _end(ctx)
    return out


def window_attn8_decode_workspace_size(n_active, H, KV, window, sink=0) -> int:
    if (n_active | H | KV | window | sink) >> 31:
        _fit(n_active, H, KV, window, sink)
    return _ops._library().gla_window_attn8_decode_workspace_size(n_active, H, KV, window, sink)


def window_attn8_decode_step(pool_k, pool_v, page, pool_e, pos, q, k, v, window, sink=0, *, layer=0,
                             out_dtype=None, out=None, workspace=None, stream=None):
    """window_attn_decode_step over 8-bit pages (gla_window_attn8_decode_step): int8 pool_k, pool_v and
    exponents pool_e as in window_cache_append, which get the token's key and value in place; page, pos,
    q, k, v, out_dtype as there.  Returns o [n_active,H,192]."""
    n, H, dk = q.shape
    KV, dv = v.shape[1], v.shape[2]
    P, PL = pool_k.shape[:2]
    if (n | H | KV | dk | dv | P | PL | layer | window | sink) >> 31:
        _fit(n, H, KV, dk, dv, P, PL, layer, window, sink)
    t = q.dtype
    dev, ctx = _begin(q, "q", stream)
    try:
        if pool_e is None:
            raise ValueError("pool_e is missing: 16-bit pages go to window_attn_decode_step")
        if out is None:
            out = _ops._empty((n, H, dv), dtype=out_dtype or t, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
        kp, vp, ep = _pools(pool_k, pool_v, pool_e, dev, t, P, PL, window + sink, KV, dk, dv)
        lib = _ops._library()
        wp, wb, hold = _scratch(
            lib.gla_window_attn8_decode_workspace_size(n, H, KV, window, sink), dev, workspace)
        rc = lib.gla_window_attn8_decode_step(
            kp, vp, ep, _ptr(page, "page", dev, I32, (n,)), _ptr(pos, "pos", dev, I32, (n,)), n, P, PL,
            layer, window, sink, _ptr(q, "q", dev, t, q.shape), _ptr(k, "k", dev, t, (n, KV, dk)),
            _ptr(v, "v", dev, t, (n, KV, dv)), _code(t, "input"),
            _ptr(out, "out", dev, out.dtype, (n, H, dv)), _code(out.dtype, "output"), wp, wb, H, KV, dk,
            dv, _ops._stream(dev))
        if rc:
            _fail("gla_window_attn8_decode_step", rc)
    finally:
        _end(ctx)
    return out

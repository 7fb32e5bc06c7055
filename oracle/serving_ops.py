"""fp64 numpy definitions of serving with the windowed attention -- TEST INFRASTRUCTURE ONLY.

Written from the formulas, sharing nothing with the CUDA code: rotary positions, rows of 8 bits,
packed tokens into pages, chunks of tokens over pages and single tokens over 8-bit pages.  Pinned by
closed forms, differences and the agreement with one pass over whole sequences
(tests/test_oracle_serving.py).
"""
from __future__ import annotations

import numpy as np

from .layer_ops import visible, window_slot


# ------------------------------------------------------------------------------ rotary
def rotary(x, angles, pos=None, interleaved=False, inverse=False, scale=1.0):
    """x [B,T,H,D] with the pairs of its first 2 len(angles) channels turned by pos * angles
    (radians per position; pos [B,T], None: 0 .. T-1)."""
    x, angles = np.asarray(x, np.float64), np.asarray(angles, np.float64)
    B, T = x.shape[:2]
    pos = np.broadcast_to(np.arange(T), (B, T)) if pos is None else np.asarray(pos)
    n = len(angles)
    y = x.copy()
    for b in range(B):
        for t in range(T):
            for i in range(n):
                a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
                w = int(pos[b, t]) * angles[i] * (-1 if inverse else 1)
                z = scale * np.exp(1j * w) * (x[b, t, :, a] + 1j * x[b, t, :, c])
                y[b, t, :, a], y[b, t, :, c] = z.real, z.imag
    return y


# ------------------------------------------------------------------------- 8-bit rows
def codes(x, lowest):
    """(c, e): a row x is held as whole numbers c, |c| <= 127, times 2^e.  Infinities count as the
    type's largest value, NaN as 0."""
    x = np.asarray(x, np.float64)
    x = np.nan_to_num(x, nan=0.0, posinf=HIGHEST[lowest], neginf=-HIGHEST[lowest])
    top = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.where(top > 0, np.floor(np.log2(top)) - 6, lowest), lowest)
    c = np.clip(np.rint(x * 2.0 ** -e[..., None]), -127, 127)
    return c.astype(np.int64), e.astype(np.int64)


LOWEST = {"bf16": -126, "fp16": -24}
HIGHEST = {-126: (2 - 2.0 ** -7) * 2.0 ** 127, -24: 65504.0}


# ------------------------------------------------------------------------------- pages
def append(pool_k, pool_v, page, pos, start, k, v, window, sink=0, layer=0, count=None):
    """Pools [P,PL,slots,KV,d] after the packed tokens went in, one by one."""
    pool_k, pool_v = pool_k.copy(), pool_v.copy()
    for b, p in enumerate(page):
        n = start[b + 1] - start[b] if count is None else count[b]
        for i in range(n):
            slot = window_slot(pos[b] + i, window, sink)
            pool_k[p, layer, slot], pool_v[p, layer, slot] = k[start[b] + i], v[start[b] + i]
    return pool_k, pool_v


def chunk(pool_k, pool_v, page, pos, start, q, k, v, window, sink=0, layer=0):
    """(o, slack): attention of packed tokens over pages and each other; rows of no sequence are NaN.
    slack: sum of p |v| and of |v| over what a row sees, for bounds on roundings."""
    pool_k, pool_v, q, k, v = (np.asarray(a, np.float64) for a in (pool_k, pool_v, q, k, v))
    N, H, _ = q.shape
    G = H // k.shape[1]
    o, pv, av = (np.full((N, H, v.shape[-1]), np.nan) for _ in range(3))
    for b, p in enumerate(page):
        for i in range(start[b + 1] - start[b]):
            row, t = start[b] + i, pos[b] + i
            seen = [s for s in visible_tokens(t, window, sink)]
            old = [window_slot(s, window, sink) for s in seen if s < pos[b]]
            new = [start[b] + s - pos[b] for s in seen if s >= pos[b]]
            for h in range(H):
                ks = np.concatenate([pool_k[p, layer, old, h // G], k[new, h // G]])
                vs = np.concatenate([pool_v[p, layer, old, h // G], v[new, h // G]])
                z = ks @ q[row, h]
                w = np.exp(z - z.max())
                w /= w.sum()
                o[row, h], pv[row, h], av[row, h] = w @ vs, w @ np.abs(vs), np.abs(vs).sum(0)
    return o, pv, av


def visible_tokens(t, window, sink):
    """As visible(), without walking through the tokens that are not seen."""
    near = range(max(0, t - window + 1), t + 1)
    return [s for s in range(min(sink, t + 1)) if s < near.start] + list(near)


assert all(visible_tokens(t, w, s) == list(visible(t, w, s)) for t in range(6) for w in (1, 3, 9)
           for s in (0, 1, 4, 9))

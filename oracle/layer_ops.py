"""fp64 numpy definitions of the operators around the mixer -- TEST INFRASTRUCTURE ONLY.

Written from the formulas, token by token and head by head, sharing nothing with the CUDA code:
the gated scan, layer norm and windowed attention, each with its hand-derived gradient and the
form for single tokens.  Pinned by central finite differences, closed forms and the agreement of
prefill and decode (tests/test_oracle_layer_ops.py).
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, dtype=np.float64) for x in xs]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


# ------------------------------------------------------------------------- gated scan
def gated_scan_fwd(x, g, init=None, lens=None):
    """(y, final): h_t = f h_{t-1} + (1 - f) x_t with f = sigmoid(g_t); 0 past a sequence's end."""
    x, g, init = _f64(x, g, init)
    B, T, D = x.shape
    y, final = np.zeros((B, T, D)), np.zeros((B, D))
    for b in range(B):
        h = np.zeros(D) if init is None else init[b].copy()
        for t in range(T if lens is None else int(lens[b])):
            h = sigmoid(g[b, t]) * h + sigmoid(-g[b, t]) * x[b, t]
            y[b, t] = h
        final[b] = h
    return y, final


def gated_scan_bwd(x, g, dy, init=None, d_final=None, lens=None):
    """(dx, dg, d_init) of sum(y dy) + sum(final d_final)."""
    x, g, dy, init, d_final = _f64(x, g, dy, init, d_final)
    B, T, D = x.shape
    y, _ = gated_scan_fwd(x, g, init, lens)
    dx, dg, dinit = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, D))
    for b in range(B):
        c = np.zeros(D) if d_final is None else d_final[b].copy()
        for t in range((T if lens is None else int(lens[b])) - 1, -1, -1):
            before = y[b, t - 1] if t else (np.zeros(D) if init is None else init[b])
            f, u = sigmoid(g[b, t]), sigmoid(-g[b, t])
            G = dy[b, t] + c
            dx[b, t] = u * G
            dg[b, t] = f * u * (before - x[b, t]) * G
            c = f * G
        dinit[b] = c
    return dx, dg, dinit


# ------------------------------------------------------------------------- layer norm
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x, weight, bias = _f64(x, weight, bias)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    y = y if weight is None else y * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_bwd(dy, x, weight=None, eps=1e-5):
    """(dx, d_weight, d_bias) of sum(y dy); x [n, D]."""
    dy, x, weight = _f64(dy, x, weight)
    n, mean, rstd = layer_norm_fwd(x, eps=eps)
    d = dy if weight is None else dy * weight
    dx = rstd[..., None] * (d - d.mean(-1, keepdims=True) - n * (d * n).mean(-1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


# ------------------------------------------------------------------ windowed attention
def visible(t, window, sink):
    """Keys that query t sees: itself and the window - 1 tokens before it, and the first `sink`."""
    return [s for s in range(t + 1) if t - s < window or s < sink]


def window_attn_fwd(q, k, v, window, sink=0, lens=None):
    """(o, lse): q [B,T,H,dk], k, v [B,T,KV,d]; zeros and -inf past a sequence's end."""
    q, k, v = _f64(q, k, v)
    B, T, H, _ = q.shape
    G = H // k.shape[2]
    o, lse = np.zeros((B, T, H, v.shape[-1])), np.full((B, H, T), -np.inf)
    for b in range(B):
        for t in range(T if lens is None else int(lens[b])):
            s = visible(t, window, sink)
            for h in range(H):
                z = k[b, s, h // G] @ q[b, t, h]
                top = z.max()
                p = np.exp(z - top)
                lse[b, h, t] = top + np.log(p.sum())
                o[b, t, h] = (p / p.sum()) @ v[b, s, h // G]
    return o, lse


def window_attn_bwd(q, k, v, dO, window, sink=0, lens=None):
    """(dq, dk, dv) of sum(o dO)."""
    q, k, v, dO = _f64(q, k, v, dO)
    B, T, H, _ = q.shape
    G = H // k.shape[2]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        for t in range(T if lens is None else int(lens[b])):
            s = visible(t, window, sink)
            for h in range(H):
                ks, vs, go = k[b, s, h // G], v[b, s, h // G], dO[b, t, h]
                z = ks @ q[b, t, h]
                p = np.exp(z - z.max())
                p /= p.sum()
                dp = vs @ go
                dz = p * (dp - p @ dp)
                dq[b, t, h] = dz @ ks
                np.add.at(dk, (b, s, h // G), np.outer(dz, q[b, t, h]))
                np.add.at(dv, (b, s, h // G), np.outer(p, go))
    return dq, dk, dv


def window_slot(t, window, sink):
    """Slot of token t in a sequence's cache: the sinks in front, then a ring of `window`."""
    return t if t < sink else sink + (t - sink) % window


def window_attn_decode_step(pool_k, pool_v, page, pos, q, k, v, window, sink=0, layer=0):
    """(o, pool_k, pool_v) after token pos[n] of each active sequence; pools [P,PL,slots,KV,d]."""
    pool_k, pool_v, q, k, v = [a.copy() for a in _f64(pool_k, pool_v, q, k, v)]
    N, H, _ = q.shape
    G = H // k.shape[1]
    o = np.zeros((N, H, v.shape[-1]))
    for n in range(N):
        p, t = int(page[n]), int(pos[n])
        pool_k[p, layer, window_slot(t, window, sink)] = k[n]
        pool_v[p, layer, window_slot(t, window, sink)] = v[n]
        held = min(t + 1, window + sink)
        for h in range(H):
            z = pool_k[p, layer, :held, h // G] @ q[n, h]
            w = np.exp(z - z.max())
            o[n, h] = (w / w.sum()) @ pool_v[p, layer, :held, h // G]
    return o, pool_k, pool_v


def window_cache_fill(pool_k, pool_v, page, k, v, window, sink=0, layer=0, lens=None):
    """The pools after a prompt's keys and values went in, token by token."""
    pool_k, pool_v, k, v = [a.copy() for a in _f64(pool_k, pool_v, k, v)]
    for b in range(k.shape[0]):
        for t in range(k.shape[1] if lens is None else int(lens[b])):
            slot = window_slot(t, window, sink)
            pool_k[int(page[b]), layer, slot] = k[b, t]
            pool_v[int(page[b]), layer, slot] = v[b, t]
    return pool_k, pool_v

"""Workloads of the layer's further operators: the gated scan, layer norm and windowed attention.

`listed()` gives fixed cases, `draw(rng)` further ones of the same ranges; `prepare` makes a
case's inputs, `run` takes one pass through the operator.  With `own` false `run` computes the
operator from elementary torch operations in 32 bits, with `own` true it calls the library.
`exact` is the same result from the definition in 64 bits.

  scan_fwd / scan_bwd    h_t = f_t h_{t-1} + (1 - f_t) x_t, f_t = sigmoid(g_t), per channel
  scan_decode            one token of it for the active sequences of a state pool
  norm_fwd / norm_bwd    layer norm over the channels of each token, with weight and bias
  window_fwd / _bwd      causal softmax attention over the last `window` tokens and the first
                         `sink` ones, 96 key and 192 value channels per head
  window_decode          one token of it over a pool of fixed-size caches
"""
import math

import torch

own = False

DK, DV = 96, 192
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one layer's training batch: 8 sequences of 2,048 tokens
        dict(name="scan_fwd_train", op="scan_fwd", B=8, T=2048, D=2048, dtype="bf16", state=False,
             ragged=False),
        # a long prompt of odd length, two padded sequences continuing from a state
        dict(name="scan_fwd_long", op="scan_fwd", B=2, T=50021, D=1536, dtype="bf16", state=True,
             ragged=True),
        # the training batch's gradient, an odd length
        dict(name="scan_bwd_train", op="scan_bwd", B=8, T=2047, D=2048, dtype="bf16", state=True,
             ragged=False),
        # a serving step: 1,280 active sequences, one layer of a two-layer pool
        dict(name="scan_decode_pool", op="scan_decode", N=1280, P=1300, D=2048, dtype="bf16"),
        # the norm ahead of a layer, 32 sequences of 2,048 tokens
        dict(name="norm_fwd_train", op="norm_fwd", N=65536, D=2048, dtype="bf16", out="bf16"),
        # the same for a few decoded tokens: a call of launch latency
        dict(name="norm_fwd_tokens", op="norm_fwd", N=16, D=2048, dtype="bf16", out="bf16"),
        # its gradient, from the fp32 gradient the causal conv hands back
        dict(name="norm_bwd_train", op="norm_bwd", N=65536, D=1536, dtype="bf16", out="fp32"),
        # rows that no vector load divides
        dict(name="norm_bwd_odd", op="norm_bwd", N=4099, D=1001, dtype="fp16", out="fp16"),
        # a local-attention layer at the training shape, every head its own keys
        dict(name="window_fwd_train", op="window_fwd", B=8, T=2048, H=16, KV=16, window=512,
             sink=4, dtype="bf16", ragged=False),
        # prefill of one long prompt of odd length, four heads on each key head
        dict(name="window_fwd_long", op="window_fwd", B=1, T=8191, H=16, KV=4, window=1024,
             sink=16, dtype="fp16", ragged=False),
        # the training gradient with shared key heads and a padded batch
        dict(name="window_bwd_train", op="window_bwd", B=8, T=2048, H=16, KV=4, window=512,
             sink=4, dtype="bf16", ragged=True),
        # serving: 256 sequences of mixed ages over caches of 1,024 + 4 slots
        dict(name="window_decode_pool", op="window_decode", N=256, P=260, H=16, KV=4, window=1024,
             sink=4, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_decode", "norm_fwd", "norm_bwd", "window_fwd",
                     "window_bwd", "window_decode"])
    half = rng.choice(["bf16", "fp16"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("scan_fwd", "scan_bwd"):
        D = _log(rng, 32, 4096)
        if rng.random() < 0.8:
            D = (D + 7) // 8 * 8
        B = _log(rng, 1, 32)
        most = 8 * 2048 * 2048 // (B * D)
        return dict(op=op, B=B, T=_log(rng, 1, max(2, min(50021, most))), D=D, dtype=kind,
                    state=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "scan_decode":
        N = _log(rng, 1, 1280)
        return dict(op=op, N=N, P=N + rng.randrange(1, 9), D=_log(rng, 64, 4096), dtype=kind)
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            D = (D + 7) // 8 * 8
        return dict(op=op, N=_log(rng, 1, 65536 * 1536 // max(D, 1536)), D=D, dtype=kind,
                    out=rng.choice([kind, "fp32"]))
    KV = rng.choice([1, 2, 4, 8, 16])
    H = KV * rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * KV <= 16])
    window, sink = _log(rng, 16, 2048), rng.choice([0, 1, 4, 16, 64])
    if op == "window_decode":
        N = _log(rng, 1, max(1, 256 * 1028 * 4 // ((window + sink) * KV)) if KV > 2 else 256)
        return dict(op=op, N=min(N, 512), P=min(N, 512) + 3, H=H, KV=KV, window=window, sink=sink,
                    dtype=half)
    T = _log(rng, 64, 4096)
    budget = (130 if op == "window_fwd" else 56) * 10 ** 6  # pairs of a query and a key
    T = min(T, budget // (H * min(T, window)))
    return dict(op=op, B=rng.randint(1, max(1, min(8, budget // (H * T * min(T, window))))), T=T,
                H=H, KV=KV, window=window, sink=sink, dtype=half, ragged=rng.random() < 0.4)


# ------------------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.float32, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(scale).add_(shift).to(dtype)


def _lengths(gen, B, T):
    """Lengths of a padded batch: the first sequence is full, the others end anywhere."""
    n = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = T
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * seed + 17)
    op, t = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D = case["B"], case["T"], case["D"]
        s["x"] = _normal(gen, (B, T, D), t)
        # forget gates of a trained layer lean towards remembering: sigmoid(2) = 0.88
        s["g"] = _normal(gen, (B, T, D), t, 1.5, 2.0)
        s["init"] = _normal(gen, (B, D)) if case["state"] else None
        s["lens"] = _lengths(gen, B, T) if case["ragged"] else None
        if op == "scan_bwd":
            s["dy"] = _normal(gen, (B, T, D))
            s["d_final"] = _normal(gen, (B, D)) if case["state"] else None
            # the forward's output, which a training step has kept
            f, u = _gates(s["g"])
            s["y"] = _scan(f, u * s["x"].float(), s["init"], s["lens"])[0]
    elif op == "scan_decode":
        N, P, D = case["N"], case["P"], case["D"]
        s["pool"] = _normal(gen, (P, 2, D))
        s["page"] = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32)
        s["x"] = _normal(gen, (N, 1, D), t)
        s["g"] = _normal(gen, (N, 1, D), t, 1.5, 2.0)
    elif op in ("norm_fwd", "norm_bwd"):
        N, D = case["N"], case["D"]
        # a residual stream: tokens of unlike size, off zero
        size = torch.exp(_normal(gen, (N, 1), scale=0.5))
        s["x"] = (_normal(gen, (N, D)) * size + 0.3 * _normal(gen, (1, D))).to(t)
        s["weight"] = _normal(gen, (D,), scale=0.2, shift=1.0)
        s["bias"] = _normal(gen, (D,), scale=0.1)
        if op == "norm_bwd":
            s["dy"] = _normal(gen, (N, D), DTYPES[case["out"]])
            x = s["x"].float()  # what the forward saves: each token's mean and 1 / deviation
            s["mean"] = x.mean(1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(1) + 1e-5).rsqrt()
    elif op in ("window_fwd", "window_bwd"):
        B, T, H, KV = case["B"], case["T"], case["H"], case["KV"]
        s["q"] = _normal(gen, (B, T, H, DK), t, DK ** -0.5)
        s["k"] = _normal(gen, (B, T, KV, DK), t)
        s["v"] = _normal(gen, (B, T, KV, DV), t)
        s["lens"] = _lengths(gen, B, T) if case["ragged"] else None
        if op == "window_bwd":
            s["dO"] = _normal(gen, (B, T, H, DV), t)
            o, lse = _window(s["q"], s["k"], s["v"], case["window"], case["sink"], s["lens"])
            s["o"], s["lse"] = o.to(t), lse  # what the forward saves
    elif op == "window_decode":
        N, P, H, KV = case["N"], case["P"], case["H"], case["KV"]
        slots = case["window"] + case["sink"]
        s["pool_k"] = _normal(gen, (P, 1, slots, KV, DK), t)
        s["pool_v"] = _normal(gen, (P, 1, slots, KV, DV), t)
        s["page"] = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32)
        # most sequences are past their window, some still fill it
        s["pos"] = torch.randint(0, 4 * slots, (N,), generator=gen, device="cuda",
                                 dtype=torch.int32)
        s["q"] = _normal(gen, (N, H, DK), t, DK ** -0.5)
        s["k"] = _normal(gen, (N, KV, DK), t)
        s["v"] = _normal(gen, (N, KV, DV), t)
    return s


# ------------------------------------------------------------------- the plain forms
def _gates(g):
    """sigmoid(g) and 1 - sigmoid(g), each to its own relative precision."""
    g = g.float()
    return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))


def _live(lens, B, T):
    return torch.arange(T, device="cuda")[None, :] < lens[:, None]


def _prefix(a, b):
    """Inclusive scan along dim 1 of h_t = a_t h_{t-1} + b_t, h_{-1} = 0, by doubling strides.
    Overwrites a and b."""
    T, n = a.shape[1], 1
    while n < T:
        b[:, n:] += a[:, n:] * b[:, :-n].clone()
        a[:, n:] *= a[:, :-n].clone()
        n *= 2
    return a, b


def _scan(f, b, init, lens):
    B, T, D = f.shape
    if lens is not None:
        live = _live(lens, B, T)[:, :, None]
        f = torch.where(live, f, torch.ones_like(f))
        b = torch.where(live, b, torch.zeros_like(b))
    b = b.clone()
    if init is not None:
        b[:, 0] += f[:, 0] * init
    h = _prefix(f.clone(), b)[1]
    final = h[:, -1].clone()
    return (h if lens is None else h * live), final


def _scan_bwd(s):
    x, y, dy, lens = s["x"].float(), s["y"], s["dy"], s["lens"]
    f, u = _gates(s["g"])
    B, T, D = f.shape
    if lens is not None:
        live = _live(lens, B, T)[:, :, None]
        f = torch.where(live, f, torch.ones_like(f))
        dy = dy * live
    before = torch.zeros_like(y)
    before[:, 1:] = y[:, :-1]
    if s["init"] is not None:
        before[:, 0] = s["init"]
    # G_t = dy_t + f_{t+1} G_{t+1}: the same scan from the last token
    a = torch.zeros_like(f)
    a[:, 1:] = f.flip(1)[:, :-1]
    b = dy.flip(1).clone()
    if s["d_final"] is not None:
        b[:, 0] += s["d_final"]
    G = _prefix(a, b)[1].flip(1)
    dx, dg = u * G, f * u * (before - x) * G
    if lens is not None:
        dx, dg = dx * live, dg * live
    return dx, dg, f[:, 0] * G[:, 0]


def _scan_decode(s):
    f, u = _gates(s["g"])
    at = s["page"].long()
    h = f[:, 0] * s["pool"][at, 1] + u[:, 0] * s["x"][:, 0].float()
    s["pool"][at, 1] = h
    return h[:, None], s["pool"]


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / (c.square().mean(1) + 1e-5).sqrt()
    y = c * rstd[:, None] * s["weight"] + s["bias"]
    return y.to(DTYPES[s["out"]]), mean, rstd


def _norm_bwd(s):
    dy, n = s["dy"].float(), (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    d = dy * s["weight"]
    dx = s["rstd"][:, None] * (d - d.mean(1, keepdim=True) - n * (d * n).mean(1, keepdim=True))
    return dx.to(DTYPES[s["out"]]), (dy * n).sum(0), dy.sum(0)


def _visible(T, window, sink, lens):
    """[B or 1, 1, T, T]: whether query t sees key s."""
    t = torch.arange(T, device="cuda")
    ok = (t[None, :] <= t[:, None]) & ((t[:, None] - t[None, :] < window) | (t[None, :] < sink))
    ok = ok[None]
    if lens is not None:
        live = t[None, :] < lens[:, None]
        ok = ok & live[:, :, None] & live[:, None, :]
    return ok[:, None]


def _heads(x, G):
    """[B, T, KV, d] -> [B, KV * G, T, d] in 32 bits."""
    return x.float().transpose(1, 2).repeat_interleave(G, 1)


def _window(q, k, v, window, sink, lens):
    B, T, H, _ = q.shape
    G = H // k.shape[2]
    ok = _visible(T, window, sink, lens)
    z = q.float().transpose(1, 2) @ _heads(k, G).transpose(2, 3)
    z = z.masked_fill(~ok, -math.inf)
    top = z.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(3, keepdim=True)
    o = (p @ _heads(v, G)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.transpose(1, 2), (top + torch.log(total))[..., 0]


def _window_bwd(s):
    q, k, v, t = s["q"], s["k"], s["v"], s["q"].dtype
    B, T, H, _ = q.shape
    KV = k.shape[2]
    G = H // KV
    qf, kf, vf = q.float().transpose(1, 2), _heads(k, G), _heads(v, G)
    dO = s["dO"].float().transpose(1, 2)
    ok = _visible(T, s["window"], s["sink"], s["lens"])
    lse = s["lse"][..., None]
    p = torch.exp((qf @ kf.transpose(2, 3)).masked_fill(~ok, -math.inf) -
                  torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    delta = (dO * s["o"].float().transpose(1, 2)).sum(3, keepdim=True)
    dz = p * (dO @ vf.transpose(2, 3) - delta)
    dq = dz @ kf
    dk = (dz.transpose(2, 3) @ qf).view(B, KV, G, T, DK).sum(2)
    dv = (p.transpose(2, 3) @ dO).view(B, KV, G, T, DV).sum(2)
    return tuple(d.transpose(1, 2).to(t) for d in (dq, dk, dv))


def _window_decode(s):
    N, H, KV, sink, window = s["N"], s["H"], s["KV"], s["sink"], s["window"]
    page, pos = s["page"].long(), s["pos"].long()
    slot = torch.where(pos < sink, pos, sink + (pos - sink) % window)
    s["pool_k"][page, 0, slot] = s["k"]
    s["pool_v"][page, 0, slot] = s["v"]
    kc, vc = s["pool_k"][page, 0].float(), s["pool_v"][page, 0].float()
    held = torch.arange(kc.shape[1], device="cuda")[None, :] <= pos[:, None]
    q = s["q"].float().view(N, KV, H // KV, DK)
    z = q @ kc.permute(0, 2, 3, 1)
    z = z.masked_fill(~held[:, None, None, :], -math.inf)
    p = torch.exp(z - z.amax(3, keepdim=True))
    o = (p @ vc.transpose(1, 2)) / p.sum(3, keepdim=True)
    return o.reshape(N, H, DV).to(s["q"].dtype), s["pool_k"], s["pool_v"]


# ------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        return _run_own(op, s)
    if op == "scan_fwd":
        f, u = _gates(s["g"])
        return _scan(f, u * s["x"].float(), s["init"], s["lens"])
    if op == "window_fwd":
        o, lse = _window(s["q"], s["k"], s["v"], s["window"], s["sink"], s["lens"])
        return o.to(s["q"].dtype), lse
    return {"scan_bwd": _scan_bwd, "scan_decode": _scan_decode, "norm_fwd": _norm_fwd,
            "norm_bwd": _norm_bwd, "window_bwd": _window_bwd,
            "window_decode": _window_decode}[op](s)


def _run_own(op, s):
    import gated_linear_attention_chunked_gb300 as gla
    if op == "scan_fwd":
        return gla.gated_scan_fwd(s["x"], s["g"], s["init"], s["lens"])
    if op == "scan_bwd":
        return gla.gated_scan_bwd(s["x"], s["g"], s["y"], s["dy"], s["init"], s["d_final"],
                                  s["lens"])
    if op == "scan_decode":
        return gla.gated_scan_decode_step_paged(s["pool"], s["page"], s["x"], s["g"],
                                                layer0=1), s["pool"]
    if op == "norm_fwd":
        return gla.layer_norm_fwd(s["x"], s["weight"], s["bias"], 1e-5,
                                  out_dtype=DTYPES[s["out"]])
    if op == "norm_bwd":
        return gla.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    if op == "window_fwd":
        return gla.window_attn_fwd(s["q"], s["k"], s["v"], s["window"], s["sink"], s["lens"])
    if op == "window_bwd":
        return gla.window_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"],
                                   s["window"], s["sink"], s["lens"])
    o = gla.window_attn_decode_step(s["pool_k"], s["pool_v"], s["page"], s["pos"], s["q"],
                                    s["k"], s["v"], s["window"], s["sink"])
    return o, s["pool_k"], s["pool_v"]


# ---------------------------------------------------------------- what a pass must do
def _pairs(T, window, sink):
    """Visible (query, key) pairs of a sequence of T tokens."""
    n = min(T, window)
    near = n * (n + 1) // 2 + (T - n) * window
    far = sum(min(sink, t - window + 1) for t in range(window, min(T, window + sink)))
    return near + far + max(0, T - window - sink) * sink


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op in ("scan_fwd", "scan_bwd"):
        n, edge = case["B"] * case["T"] * case["D"], case["B"] * case["D"] * 4
        if op == "scan_fwd":
            return {"bytes": n * (2 * size + 4) + edge * (2 if case["state"] else 1),
                    "flops": 12 * n}
        return {"bytes": n * (2 * size + 16) + edge * (3 if case["state"] else 1),
                "flops": 18 * n}
    if op == "scan_decode":
        n = case["N"] * case["D"]
        return {"bytes": n * (2 * size + 12) + 4 * case["N"], "flops": 12 * n}
    if op in ("norm_fwd", "norm_bwd"):
        n, out = case["N"] * case["D"], 4 if case["out"] == "fp32" else 2
        if op == "norm_fwd":
            return {"bytes": n * (size + out) + 8 * case["N"] + 8 * case["D"], "flops": 8 * n}
        return {"bytes": n * (size + 2 * out) + 8 * case["N"] + 12 * case["D"], "flops": 14 * n}
    H, KV = case["H"], case["KV"]
    if op == "window_decode":
        # a quarter of the sequences still fill their cache, half full on average
        slots = case["window"] + case["sink"]
        held = case["N"] * slots * (0.75 + 0.25 / 2)
        return {"bytes": held * KV * (DK + DV) * 2 + case["N"] * (H + KV) * (DK + DV) * 2,
                "flops": held * H * 2 * (DK + DV)}
    B, T = case["B"], case["T"]
    # a padded batch: the first sequence full, the others half full on average
    full = 1 + (B - 1) * 0.5 if case["ragged"] else B
    pairs = full * _pairs(T, case["window"], case["sink"]) * H
    tokens = B * T
    if op == "window_fwd":
        return {"bytes": tokens * ((H + KV) * (DK + DV) * 2 + 4 * H),
                "flops": pairs * 2 * (DK + DV)}
    return {"bytes": tokens * ((2 * H + 2 * KV) * (DK + DV) * 2 + 2 * H * DV + 4 * H),
            "flops": pairs * 2 * (3 * DK + 2 * DV)}


# ------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        return _exact_scan(s, op == "scan_bwd")
    if op == "scan_decode":
        h = s["pool"].double()
        for n, p in enumerate(s["page"].tolist()):
            f = torch.sigmoid(s["g"][n, 0].double())
            h[p, 1] = f * h[p, 1] + torch.sigmoid(-s["g"][n, 0].double()) * s["x"][n, 0].double()
        return h[s["page"].long(), 1][:, None], h
    if op in ("norm_fwd", "norm_bwd"):
        x = s["x"].double().requires_grad_()
        w = s["weight"].double().requires_grad_()
        b = s["bias"].double().requires_grad_()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        y = torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w)
        if op == "norm_fwd":
            return y.detach(), mean.detach(), rstd.detach()
        return torch.autograd.grad(y, (x, w, b), s["dy"].double())
    if op == "window_decode":
        return _exact_decode(s)
    return _exact_window(s, op == "window_bwd")


def _exact_scan(s, gradient):
    """Token by token; between two of the batch's lengths the same sequences go on."""
    x, g = s["x"].double(), s["g"].double()
    B, T, D = x.shape
    lens = s["lens"].tolist() if s["lens"] is not None else [T] * B
    f, u = torch.sigmoid(g), torch.sigmoid(-g)
    first = torch.zeros_like(x[:, 0]) if s["init"] is None else s["init"].double()
    edges = sorted({0, *lens})
    spans = [(lo, hi, [b for b in range(B) if lens[b] >= hi]) for lo, hi in zip(edges, edges[1:])]
    y, final = torch.zeros_like(x), first.clone()
    for lo, hi, rows in spans:
        h, fs, add = final[rows], f[rows, lo:hi], (u * x)[rows, lo:hi]
        part = torch.empty_like(fs)
        for t in range(hi - lo):
            h = torch.addcmul(add[:, t], fs[:, t], h, out=part[:, t])
        y[rows, lo:hi] = part
        final[rows] = h
    if not gradient:
        return y, final
    before = torch.cat([first[:, None], y[:, :-1]], 1)
    G, c = torch.zeros_like(x), torch.zeros_like(first)
    if s["d_final"] is not None:
        c += s["d_final"]
    for lo, hi, rows in reversed(spans):
        h, fs, dy = c[rows], f[rows, lo:hi], s["dy"][rows, lo:hi].double()
        part = torch.empty_like(fs)
        for t in range(hi - lo - 1, -1, -1):
            h = fs[:, t] * torch.add(dy[:, t], h, out=part[:, t])
        G[rows, lo:hi] = part
        c[rows] = h
    return u * G, f * u * (before - x) * G, c


def _exact_window(s, gradient):
    """Sequence by sequence and head by head, up to the sequence's length; the gradient by
    automatic differentiation of that."""
    B, T, H, _ = s["q"].shape
    G = H // s["k"].shape[2]
    lens = s["lens"].tolist() if s["lens"] is not None else [T] * B
    if sum(n * n for n in lens) * H > 1.2e9:
        return None
    q, k, v = (s[n].double() for n in "qkv")
    o = torch.zeros(B, T, H, DV, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    for b, n in enumerate(lens):
        age = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None, :]
        hidden = (age < 0) | ((age >= s["window"]) & (torch.arange(n, device="cuda") >= s["sink"]))
        bar = torch.zeros(n, n, dtype=torch.float64, device="cuda").masked_fill_(hidden, -math.inf)
        for h in range(H):
            parts = [x.detach().clone().requires_grad_(gradient)
                     for x in (q[b, :n, h], k[b, :n, h // G], v[b, :n, h // G])]
            z = torch.addmm(bar, parts[0], parts[1].T)
            total = torch.logsumexp(z, 1)
            out = (z - total[:, None]).exp() @ parts[2]
            o[b, :n, h], lse[b, h, :n] = out.detach(), total.detach()
            if gradient:
                d = torch.autograd.grad(out, parts, s["dO"][b, :n, h].double())
                grads[0][b, :n, h] += d[0]
                grads[1][b, :n, h // G] += d[1]
                grads[2][b, :n, h // G] += d[2]
    return tuple(grads) if gradient else (o, lse)


def _exact_decode(s):
    sink, window, G = s["sink"], s["window"], s["H"] // s["KV"]
    pk, pv = s["pool_k"].clone(), s["pool_v"].clone()
    o = torch.zeros(s["N"], s["H"], DV, dtype=torch.float64, device="cuda")
    for n, (p, t) in enumerate(zip(s["page"].tolist(), s["pos"].tolist())):
        at = t if t < sink else sink + (t - sink) % window
        pk[p, 0, at], pv[p, 0, at] = s["k"][n], s["v"][n]
        m = min(t + 1, sink + window)
        for h in range(s["KV"]):
            q = s["q"][n, h * G:(h + 1) * G].double()
            w = torch.softmax(q @ pk[p, 0, :m, h].double().T, 1)
            o[n, h * G:(h + 1) * G] = w @ pv[p, 0, :m, h].double()
    return o, pk, pv

"""Workloads of serving with the windowed attention: rotary positions, chunks of new tokens over the
cached pages, and pages of 8 bits.

`listed()` gives fixed cases, `draw(rng)` further ones of the same ranges; `prepare` makes a
case's inputs, `run` takes one pass through the operator.  With `own` false `run` computes the
operator from elementary torch operations in 32 bits (angles in 64), with `own` true it calls the
library.  `exact` is the same result from the definition in 64 bits.

  rotary         pairs of channels turned by an angle that grows with the token's position, and
                 (inverse) the gradient of that
  chunk          new tokens of several sequences, packed one behind the other, attend to their
                 sequence's page and to each other: causal, the last `window` tokens and the first
                 `sink` ones; pages of 16 bits or (bits 8) of 8
  cache8         keys and values of prompts rounded to 8 bits as they go into their pages, and the
                 pages read back
  decode8        one token of the attention over a pool of 8-bit pages, which gets its key and value

A page holds the first `sink` tokens in slots 0 .. sink-1 and the last `window` others in a ring
behind them.  In 8 bits a row x (a key or value of one head) is held as whole numbers c of at most
127 and an exponent e: x is about c 2^e, e = floor(log2(max |x|)) - 6, at least -24 for fp16 and -126
for bf16 (so that c 2^e is a value of that type), c = x 2^-e rounded to even.
"""
import math

import torch

own = False

DK, DV = 96, 192
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LOWEST = {"bf16": -126, "fp16": -24}


def listed():
    return [
        # training: queries and keys of 8 sequences of 2,048 tokens, four heads on each key head
        dict(name="rotary_train", op="rotary", B=8, T=2048, H=16, KV=4, R=96, interleaved=True,
             inverse=False, dtype="bf16", out="bf16", stream=False, far=0, method="plain"),
        # its gradient, odd length, two thirds of the head, positions scaled for a context 8 times as long
        dict(name="rotary_gradient", op="rotary", B=4, T=4095, H=16, KV=16, R=64, interleaved=False,
             inverse=True, dtype="fp32", out="fp32", stream=False, far=0, method="parts"),
        # 48 decoded tokens far into their sequences, read from the projection that made them: a
        # call of launch latency
        dict(name="rotary_tokens", op="rotary", B=48, T=1, H=16, KV=4, R=96, interleaved=False,
             inverse=False, dtype="bf16", out="bf16", stream=True, far=1 << 20, method="linear"),
        # chunked prefill: the next 2,048 tokens of four long prompts
        dict(name="chunk_prefill", op="chunk", bits=16, n=4, new=2048, mix="equal", H=16, KV=4,
             window=1024, sink=4, dtype="bf16"),
        # a serving batch: one prompt's chunk of odd length beside 60 decoded tokens
        dict(name="chunk_mixed", op="chunk", bits=16, n=61, new=1501, mix="one", H=16, KV=2,
             window=512, sink=1, dtype="fp16"),
        # a question of 37 tokens about one long document
        dict(name="chunk_document", op="chunk", bits=16, n=1, new=37, mix="equal", H=16, KV=4,
             window=65536, sink=16, dtype="bf16"),
        # chunked prefill over 8-bit pages, odd sizes
        dict(name="chunk8_prefill", op="chunk", bits=8, n=3, new=1999, mix="equal", H=16, KV=4,
             window=1000, sink=3, dtype="fp16"),
        # 96 sequences of 3 to 5 drafted tokens each, checked in one call
        dict(name="chunk8_drafts", op="chunk", bits=8, n=96, new=5, mix="some", H=16, KV=4,
             window=2048, sink=4, dtype="bf16"),
        # prompts of mixed lengths into 8-bit pages, and the pages read back
        dict(name="cache8_prompts", op="cache8", n=64, T=2048, KV=4, window=1024, sink=4,
             dtype="bf16"),
        # a few short ones, odd sizes
        dict(name="cache8_few", op="cache8", n=3, T=301, KV=2, window=77, sink=1, dtype="fp16"),
        # serving: 256 sequences of mixed ages over 8-bit pages of 1,024 + 4 slots
        dict(name="decode8_pool", op="decode8", n=256, H=16, KV=4, window=1024, sink=4,
             dtype="bf16"),
        # three sequences with long pages, eight heads on each key head
        dict(name="decode8_few", op="decode8", n=3, H=16, KV=2, window=16384, sink=4, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "chunk", "chunk", "cache8", "decode8"])
    half = rng.choice(["bf16", "fp16"])
    KV = rng.choice([1, 2, 4, 8])
    H = KV * rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * KV <= 16])
    if op == "rotary":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        B = _log(rng, 1, 256)
        T = _log(rng, 1, max(1, min(8192, 8 * 2048 * 20 // (B * (H + KV)))))
        return dict(op=op, B=B, T=T, H=H, KV=KV, R=rng.choice([32, 48, 62, 64, 96]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4, dtype=dtype,
                    out=rng.choice([dtype, "fp32"]), stream=rng.random() < 0.4,
                    far=rng.choice([0, 0, 1 << 20]), method=rng.choice(["plain", "linear", "parts"]))
    if op == "cache8":
        window, sink = _log(rng, 16, 4096), rng.choice([0, 1, 4, 16])
        n = _log(rng, 1, max(1, min(64, 56 * 1028 * 4 // ((window + sink) * KV))))
        T = _log(rng, 1, max(1, min(4096, 64 * 2048 * 4 // (n * KV))))
        return dict(op=op, n=n, T=T, KV=KV, window=window, sink=sink, dtype=half)
    if op == "decode8":
        window, sink = _log(rng, 16, 16384), rng.choice([0, 1, 4, 16])
        n = _log(rng, 1, max(1, min(512, 256 * 1028 * 4 // ((window + sink) * KV))))
        return dict(op=op, n=n, H=H, KV=KV, window=window, sink=sink, dtype=half)
    window, sink = _log(rng, 16, 32768), rng.choice([0, 1, 4, 16, 64])
    S = window + sink
    # of all sequences
    tokens = min(8192 * 1028 * 4 // (S * KV), 8192 * 1028 * 16 // (S * H), 8192 * 20 // (H + KV))
    n = _log(rng, 1, max(1, min(128, tokens, 1028 * 4 * 112 // (S * KV))))
    mix = rng.choice(["equal", "one", "some"])
    most = tokens - n + 1 if mix == "one" else tokens // n
    return dict(op=op, bits=rng.choice([8, 16]), n=n, new=_log(rng, 1, max(1, min(3000, most))), mix=mix,
                H=H, KV=KV, window=window, sink=sink, dtype=half)


# ------------------------------------------------------------------------------- inputs
def _new(case):
    """New tokens of each sequence."""
    n, new = case["n"], case["new"]
    if case["mix"] == "one":
        return [new] + [1] * (n - 1)
    return [new if case["mix"] == "equal" else max(1, new - b % 3) for b in range(n)]


def _ages(case):
    """Tokens that each sequence has in its page: mixed, the first of them past its ring."""
    slots = case["window"] + case["sink"]
    return [int(4 * slots * ((0.73 + 0.618034 * b) % 1)) for b in range(case["n"])]


def _prompts(case):
    return [max(1, int(case["T"] * ((0.999999 + 0.618034 * b) % 1) + 0.5)) for b in range(case["n"])]


def _frequencies(case):
    """Radians per position of each pair of channels, float64 [R / 2]."""
    R, base, factor, context = case["R"], 10000.0, 8.0, 4096
    f = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    if case["method"] == "linear":
        return f / factor
    if case["method"] == "parts":
        # pairs that turn often within the trained context stay, slow ones are stretched
        turns = context * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep)
    return f


def _normal(gen, shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(gen, case, s, bits):
    """Pages with a layer in front of the one in use, and pages that nobody uses."""
    n, KV, slots = case["n"], case["KV"], case["window"] + case["sink"]
    P, t = n + 2, DTYPES[case["dtype"]]
    s["page"] = torch.randperm(P, generator=gen, device="cuda")[:n].to(torch.int32)
    if bits == 16:
        s["pool_k"] = _normal(gen, (P, 2, slots, KV, DK), t)
        s["pool_v"] = _normal(gen, (P, 2, slots, KV, DV), t)
        s["pool_e"] = None
        return
    for name, d in (("pool_k", DK), ("pool_v", DV)):
        c = torch.randn((P, 2, slots, KV, d), generator=gen, device="cuda")
        s[name] = c.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    # rows of normal values have exponents of -6 to -5
    s["pool_e"] = torch.randint(-6, -4, (P, 2, KV, slots, 2), generator=gen, device="cuda",
                                dtype=torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * seed + 29)
    op, t = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op == "rotary":
        B, T, H, KV = case["B"], case["T"], case["H"], case["KV"]
        if case["stream"]:  # views of the fused projection's rows: queries, keys, values
            row = _normal(gen, (B, T, (H + KV) * DK + KV * DV), t)
            s["q"] = row[..., :H * DK].view(B, T, H, DK)
            s["k"] = row[..., H * DK:(H + KV) * DK].view(B, T, KV, DK)
        else:
            s["q"] = _normal(gen, (B, T, H, DK), t)
            s["k"] = _normal(gen, (B, T, KV, DK), t)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda")
        s["pos"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
        s["f"] = _frequencies(case)
        # parts of a turn per position, in units of 2^-64
        s["turns"] = (s["f"] / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64).cuda()
        s["f"] = s["f"].cuda()
        s["scale"] = 0.1 * math.log(8.0) + 1 if case["method"] == "parts" else 1.0
    elif op == "cache8":
        n, T, KV = case["n"], case["T"], case["KV"]
        _pool(gen, case, s, 8)
        # tokens of unlike size
        size = torch.exp(_normal(gen, (n * T, KV, 1), scale=0.7))
        s["k"] = (_normal(gen, (n * T, KV, DK)) * size).to(t)
        s["v"] = (_normal(gen, (n * T, KV, DV)) * size).to(t)
        s["start"] = _ints([b * T for b in range(n + 1)])
        s["count"] = _ints(_prompts(case))
        s["pos"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    else:
        n, H, KV = case["n"], case["H"], case["KV"]
        _pool(gen, case, s, case.get("bits", 8))
        s["pos"] = _ints(_ages(case))
        N = n
        if op == "chunk":
            start = [0]
            for m in _new(case):
                start.append(start[-1] + m)
            s["start"], N = _ints(start), start[-1]
        s["q"] = _normal(gen, (N, H, DK), t, DK ** -0.5)
        s["k"] = _normal(gen, (N, KV, DK), t)
        s["v"] = _normal(gen, (N, KV, DV), t)
    return s


# ------------------------------------------------------------------- the plain forms
def _rotary(s, x):
    angle = s["pos"].double()[..., None] * s["f"]
    c, w = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    c, w = c[:, :, None], (-w if s["inverse"] else w)[:, :, None]
    R, x = s["R"], x.float()
    y = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * w, a * w + b * c
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * c - b * w, a * w + b * c
    return y.to(DTYPES[s["out"]])


def _slot(t, window, sink):
    return torch.where(t < sink, t, sink + (t - sink) % window)


def _codes(x, lowest):
    """Whole numbers and exponents of rows of 16 bits."""
    x = x.float()
    top = x.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 7, torch.full_like(top, lowest)).clamp(lowest)
    c = torch.round(torch.ldexp(x, -e[..., None])).clamp(-127, 127)
    return c.to(torch.int8), e.to(torch.int8)


def _pages(s, layer):
    """Keys and values of the sequences' pages in 32 bits: [n, slots, KV, d]."""
    at = s["page"].long()
    k, v = s["pool_k"][at, layer].float(), s["pool_v"][at, layer].float()
    if s["pool_e"] is not None:
        e = s["pool_e"][at, layer].float().transpose(1, 2)
        k, v = k * torch.exp2(e[..., :1]), v * torch.exp2(e[..., 1:])
    return k, v


def _chunk(s):
    n, H, KV, window, sink = s["n"], s["H"], s["KV"], s["window"], s["sink"]
    slots, N = window + sink, s["q"].shape[0]
    k, v = _pages(s, 1)
    k = torch.cat([k.reshape(n * slots, KV, DK), s["k"].float()])
    v = torch.cat([v.reshape(n * slots, KV, DV), s["v"].float()])
    row = torch.arange(N, device="cuda")
    start, pos = s["start"].long(), s["pos"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    p = (pos[seq] + row - start[seq])[:, None]
    # the tokens that each one may see, by position: sinks, then the window
    near = p - window + 1 + torch.arange(window, device="cuda")
    t = torch.cat([torch.arange(sink, device="cuda").expand(N, sink), near], 1)
    sees = torch.cat([t[:, :sink] <= p, near >= sink], 1)
    before = t < pos[seq][:, None]
    at = torch.where(before, seq[:, None] * slots + _slot(t, window, sink),
                     n * slots + (start[seq] - pos[seq])[:, None] + t)
    at = torch.where(sees, at, torch.full_like(at, n * slots))
    q = s["q"].float().view(N, KV, H // KV, DK)
    z = q @ k[at].permute(0, 2, 3, 1)
    z = z.masked_fill(~sees[:, None, None, :], -math.inf)
    w = torch.exp(z - z.amax(3, keepdim=True))
    o = (w @ v[at].transpose(1, 2)) / w.sum(3, keepdim=True)
    return o.reshape(N, H, DV).to(s["q"].dtype)


def _cache8(s):
    n, T, KV, window, sink = s["n"], s["T"], s["KV"], s["window"], s["sink"]
    slots, low = window + sink, LOWEST[s["dtype"]]
    ck, ek = _codes(s["k"].view(n, T, KV, DK), low)
    cv, ev = _codes(s["v"].view(n, T, KV, DV), low)
    # the last token that belongs in each slot
    slot = torch.arange(slots, device="cuda")[None]
    count = s["count"].long()[:, None]
    t = torch.where(slot < sink, slot, slot + (count - 1 - slot).clamp(min=0) // window * window)
    put = slot < count
    t = torch.where(put, t, torch.zeros_like(t))
    b = torch.arange(n, device="cuda")[:, None]
    at, put = s["page"].long(), put[..., None, None]
    s["pool_k"][at, 1] = torch.where(put, ck[b, t], s["pool_k"][at, 1])
    s["pool_v"][at, 1] = torch.where(put, cv[b, t], s["pool_v"][at, 1])
    e = torch.stack([ek[b, t], ev[b, t]], -1).transpose(1, 2)
    s["pool_e"][at, 1] = torch.where(put.transpose(1, 2), e, s["pool_e"][at, 1])
    k, v = _pages(s, 1)
    t = DTYPES[s["dtype"]]
    return k.to(t), v.to(t)


def _decode8(s):
    n, H, KV, window, sink = s["n"], s["H"], s["KV"], s["window"], s["sink"]
    page, pos, low = s["page"].long(), s["pos"].long(), LOWEST[s["dtype"]]
    slot = _slot(pos, window, sink)
    ck, ek = _codes(s["k"], low)
    cv, ev = _codes(s["v"], low)
    s["pool_k"][page, 1, slot] = ck
    s["pool_v"][page, 1, slot] = cv
    s["pool_e"][page, 1, :, slot] = torch.stack([ek, ev], -1)
    k, v = _pages(s, 1)
    b = torch.arange(n, device="cuda")
    k[b, slot], v[b, slot] = s["k"].float(), s["v"].float()  # the new token itself is not rounded
    held = torch.arange(window + sink, device="cuda")[None, :] <= pos[:, None]
    z = s["q"].float().view(n, KV, H // KV, DK) @ k.permute(0, 2, 3, 1)
    z = z.masked_fill(~held[:, None, None, :], -math.inf)
    w = torch.exp(z - z.amax(3, keepdim=True))
    o = (w @ v.transpose(1, 2)) / w.sum(3, keepdim=True)
    return o.reshape(n, H, DV).to(s["q"].dtype)


# ------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        return _run_own(op, s)
    if op == "rotary":
        return _rotary(s, s["q"]), _rotary(s, s["k"])
    if op == "chunk":
        return _chunk(s)
    if op == "cache8":
        return (*_cache8(s), s["pool_k"], s["pool_v"], s["pool_e"])
    # the pools' codes and exponents are whole numbers, and equal ones stand for equal values
    return _decode8(s), s["pool_k"], s["pool_v"], s["pool_e"]


def _run_own(op, s):
    import gated_linear_attention_chunked_gb300 as gla
    if op == "rotary":
        return gla.rotary(s["q"], s["k"], s["turns"], s["pos"], interleaved=s["interleaved"],
                          inverse=s["inverse"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
    pools, e = (s["pool_k"], s["pool_v"], s["page"]), s["pool_e"]
    if op == "chunk":
        return gla.window_attn_chunk(*pools, s["pos"], s["start"], s["q"], s["k"], s["v"],
                                     s["window"], s["sink"], layer=1, pool_e=e)
    if op == "cache8":
        gla.window_cache_append(*pools, s["pos"], s["start"], s["k"], s["v"], s["window"],
                                s["sink"], s["count"], layer=1, pool_e=e)
        k, v = gla.window_cache8_read(*pools, e, s["window"], s["sink"], layer=1,
                                      out_dtype=DTYPES[s["dtype"]])
        return k, v, s["pool_k"], s["pool_v"], e
    o = gla.window_attn8_decode_step(*pools, e, s["pos"], s["q"], s["k"], s["v"], s["window"],
                                     s["sink"], layer=1)
    return o, s["pool_k"], s["pool_v"], e


# ---------------------------------------------------------------- what a pass must do
def _visible(p, window, sink):
    """Tokens that the one at position p sees, itself among them."""
    return min(p + 1, window) + max(0, min(sink, p + 1 - window))


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "rotary":
        rows = case["B"] * case["T"] * (case["H"] + case["KV"])
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": rows * DK * (size + out) + 4 * case["B"] * case["T"],
                "flops": rows * 3 * case["R"]}
    KV, window, sink = case["KV"], case["window"], case["sink"]
    if op == "cache8":
        slots = window + sink
        kept = sum(min(m, slots) for m in _prompts(case)) * KV
        # the rows that stay are read and written, every page is read back and its values written
        return {"bytes": kept * (288 * 2 + 290) + case["n"] * slots * KV * (290 + 288 * 2),
                "flops": kept * 288 * 3}
    row = 576 if case.get("bits", 8) == 16 else 290
    H = case["H"]
    if op == "decode8":
        seen = [_visible(p, window, sink) for p in _ages(case)]
        return {"bytes": (sum(seen) - case["n"]) * KV * row +
                case["n"] * ((H + KV) * 288 * 2 + KV * 290 + 8), "flops": sum(seen) * H * 2 * 288}
    pairs = cached = 0
    for p, m in zip(_ages(case), _new(case)):
        cached += _visible(p, window, sink) - 1
        pairs += sum(_visible(p + i, window, sink) for i in range(m))
    tokens = sum(_new(case))
    return {"bytes": cached * KV * row + tokens * (H + KV) * 288 * 2, "flops": pairs * H * 2 * 288}


# ------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotary(s, s["q"]), _exact_rotary(s, s["k"])
    if op == "cache8":
        _exact_put(s, s["start"].tolist(), s["count"].tolist())
        k, v = zip(*(_exact_page(s, b) for b in range(s["n"])))
        return torch.stack(k), torch.stack(v), s["pool_k"], s["pool_v"], s["pool_e"]
    if op == "decode8":
        o = _exact_attention(s, list(range(s["n"] + 1)))
        _exact_put(s, list(range(s["n"] + 1)), [1] * s["n"])
        return o, s["pool_k"], s["pool_v"], s["pool_e"]
    if work(case)["flops"] > 2e11:
        return None
    return _exact_attention(s, s["start"].tolist())


def _exact_rotary(s, x):
    """Pairs as complex numbers, times exp(i angle)."""
    R = s["R"]
    turn = torch.polar(torch.full_like(s["f"], s["scale"]).expand(*s["pos"].shape, R // 2),
                       s["pos"].double()[..., None] * s["f"])
    turn = (turn.conj() if s["inverse"] else turn)[:, :, None]
    x = x.double()
    if s["interleaved"]:
        y = torch.view_as_real(turn * torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2))
                                                            .contiguous())).flatten(-2)
    else:
        z = turn * torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous())
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., R:]], -1)


def _exact_page(s, b):
    """Keys and values of a sequence's page by slot."""
    p = int(s["page"][b])
    k, v = s["pool_k"][p, 1].double(), s["pool_v"][p, 1].double()
    if s["pool_e"] is not None:
        two = torch.pow(2.0, s["pool_e"][p, 1].double()).permute(1, 0, 2)
        k, v = k * two[..., 0:1], v * two[..., 1:2]
    return k, v


def _exact_put(s, start, count):
    """Tokens into their slots, sequence by sequence: of several for one slot the last."""
    window, sink, low = s["window"], s["sink"], LOWEST[s["dtype"]]
    for b, p in enumerate(s["page"].tolist()):
        first = int(s["pos"][b])
        where = {}
        for i in range(count[b]):
            t = first + i
            where[t if t < sink else sink + (t - sink) % window] = start[b] + i
        slots = torch.tensor(list(where.keys()), device="cuda")
        rows = torch.tensor(list(where.values()), device="cuda")
        for j, name in enumerate(("k", "v")):
            x = s[name][rows].double()
            top = x.abs().amax(2)
            e = torch.where(top > 0, torch.floor(torch.log2(top)) - 6, low).clamp(min=low)
            c = (x * torch.pow(2.0, -e)[..., None]).round().clamp(-127, 127)
            s["pool_" + name][p, 1, slots] = c.to(torch.int8)
            s["pool_e"][p, 1, :, :, j].index_copy_(1, slots, e.T.to(torch.int8))


def _exact_attention(s, start):
    """Sequence by sequence: the page's tokens in the order of their positions, then the new ones."""
    window, sink, H, KV = s["window"], s["sink"], s["H"], s["KV"]
    G, out = H // KV, []
    for b, first in enumerate(s["pos"].tolist()):
        lo, hi = start[b], start[b + 1]
        k, v = _exact_page(s, b)
        old = list(range(min(first, sink))) + list(range(max(sink, first - window), first))
        t = torch.tensor(old, dtype=torch.long, device="cuda")
        at = torch.where(t < sink, t, sink + (t - sink).remainder(window))
        keys = torch.cat([k[at], s["k"][lo:hi].double()])
        values = torch.cat([v[at], s["v"][lo:hi].double()])
        new = torch.arange(first, first + hi - lo, device="cuda")
        t = torch.cat([t, new])
        age = new[:, None] - t[None, :]
        bar = torch.zeros(age.shape, dtype=torch.float64, device="cuda")
        bar.masked_fill_((age < 0) | ((age >= window) & (t >= sink)), -math.inf)
        o = torch.empty(hi - lo, H, DV, dtype=torch.float64, device="cuda")
        for h in range(H):
            z = torch.addmm(bar, s["q"][lo:hi, h].double(), keys[:, h // G].T)
            o[:, h] = torch.softmax(z, 1) @ values[:, h // G]
        out.append(o)
    return torch.cat(out)

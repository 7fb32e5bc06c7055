"""GPU parity of the layer norm (forward, gradient) against the fp64 definition.

Bounds, with X = max |x| and r = rstd: a sum over the channels adds at most 16 values in a thread
and joins 10 levels of threads and warps, so mean and squares are off by 26 roundings each, and a
normalised value by 64 roundings of X r; the output rounds once more, to its type.  A gradient dx
is r times three such terms; a weight gradient adds ceil(n / 152) tokens in a thread and up to
152 * 16 / 8 + 8 partial sums, each a rounding of the sum of magnitudes."""
import numpy as np
import pytest

from _util import as_dtype_values, to_dev
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}  # half a step, relative


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    types = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    return gla, torch, types


CASES = [  # tokens, channels, type, output type, weights
    (1, 1, "fp32", "fp32", True), (3, 2, "bf16", "bf16", True), (5, 8, "bf16", "fp32", True),
    (7, 31, "fp16", "fp16", True), (400, 96, "bf16", "bf16", True), (33, 100, "fp32", "fp32", False),
    (311, 1001, "fp16", "fp16", True), (700, 1536, "bf16", "fp32", True),
    (65, 2048, "bf16", "bf16", False), (19, 2052, "fp32", "fp32", True),
    (9, 4097, "bf16", "fp32", True), (13, 8192, "fp16", "fp16", True),
    (6, 8200, "bf16", "bf16", True), (5, 9001, "fp32", "fp32", True),
    (4, 16384, "fp32", "fp32", True), (3, 16384, "bf16", "fp32", True),
    (3, 16383, "fp16", "fp16", True),
    # rows enough for a warp each, of each number of accesses
    (1300, 500, "fp32", "fp32", True), (2500, 512, "bf16", "bf16", True),
    (1250, 1000, "fp16", "fp32", False), (1250, 1400, "fp32", "fp32", True),
    (1250, 1528, "bf16", "fp32", True), (5000, 2048, "bf16", "bf16", True),
    (1218, 2044, "fp32", "fp32", False), (4000, 8, "fp16", "fp16", True),
    (700, 4096, "bf16", "bf16", True), (700, 4096, "fp32", "fp32", True),
]


@pytest.mark.parametrize("n,D,dt,out,weights", CASES)
def test_matches_the_definition(env, n, D, dt, out, weights):
    gla, torch, types = env
    rng = np.random.default_rng(n + D)
    x = as_dtype_values((rng.standard_normal((n, D)) * 2 + 3).astype(np.float32), dt)
    dy = as_dtype_values(rng.standard_normal((n, D)).astype(np.float32), out)
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if weights else None
    b = rng.standard_normal(D).astype(np.float32) if weights else None
    xd, dyd = to_dev(x, types[dt]), to_dev(dy, types[out])
    wd, bd = (None if a is None else to_dev(a, torch.float32) for a in (w, b))
    y, mean, rstd = gla.layer_norm_fwd(xd, wd, bd, 1e-3, out_dtype=types[out])
    got = gla.layer_norm_bwd(dyd, xd, wd, mean, rstd)
    again = gla.layer_norm_bwd(dyd, xd, wd, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    assert y.dtype == got[0].dtype == types[out]
    y_r, m_r, r_r = ref.layer_norm_fwd(x, w, b, 1e-3)
    dx_r, dw_r, db_r = ref.layer_norm_bwd(dy, x, w, 1e-3)
    X, W = np.abs(x).max(), 1 if w is None else np.abs(w).max()
    npy = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    # a normalised value: 64 roundings of X r, and of r's own relative error (X r)^2 more
    unit = 64 * U * (X * r_r) * (1 + X * r_r)
    assert np.all(np.abs(npy(mean) - m_r) <= 26 * U * X)
    assert np.all(np.abs(npy(rstd) - r_r) <= unit * r_r)
    slack = HALF[out] * np.abs(y_r) + 2.0 ** -25 + (unit * W)[:, None] * (1 + np.abs(y_r))
    assert np.all(np.abs(npy(y) - y_r) <= slack)
    d = np.abs(dy) if w is None else np.abs(dy * w)
    nmax = np.abs(ref.layer_norm_fwd(x, eps=1e-3)[0]).max(1)
    term = r_r * d.max(1) * (1 + nmax) ** 2
    slack = HALF[out] * np.abs(dx_r) + 2.0 ** -25 + ((64 * U + 4 * unit) * term)[:, None]
    assert np.all(np.abs(npy(got[0]) - dx_r) <= slack)
    chain = -(-n // 152) + 152 * 16 // 8 + 8
    each = np.abs(ref.layer_norm_fwd(x, eps=1e-3)[0])
    assert np.all(np.abs(npy(got[1]) - dw_r) <=
                  (chain * U * (np.abs(dy) * each).sum(0) + (unit[:, None] * np.abs(dy)).sum(0)))
    assert np.all(np.abs(npy(got[2]) - db_r) <= chain * U * np.abs(dy).sum(0))


def test_many_rows_and_leading_axes(env):
    """More rows than the persistent grid holds at once, under two leading axes."""
    gla, torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(7, 1501, 64, generator=gen, device="cuda")
    y, mean, rstd = gla.layer_norm_fwd(x)
    assert mean.shape == rstd.shape == x.shape[:-1]
    y_r, _, _ = ref.layer_norm_fwd(x.cpu().numpy())
    assert np.abs(y.cpu().numpy() - y_r).max() <= 64 * U * 6 * 7
    dy = torch.randn(x.shape, generator=gen, device="cuda")
    dx, dw, db = gla.layer_norm_bwd(dy, x, None, mean, rstd)
    r = ref.layer_norm_bwd(dy.cpu().numpy().reshape(-1, 64), x.cpu().numpy().reshape(-1, 64))
    # |x|, |n|, |dy| < 6, 1 / deviation < 2 for 64 normal channels: one term of dx is < 2 6 7^2
    assert dx.shape == x.shape
    assert np.abs(dx.cpu().numpy().reshape(-1, 64) - r[0]).max() <= 64 * U * (1 + 4 * 12) * 600
    chain = (7 * 1501 // 152 + 152 * 16 // 8 + 8) * U
    assert np.abs(dw.cpu().numpy() - r[1]).max() <= 4 * chain * 7 * 1501
    assert np.abs(db.cpu().numpy() - r[2]).max() <= 4 * chain * 7 * 1501


def test_constant_rows_and_empty_batches(env):
    gla, torch, _ = env
    x = torch.full((5, 40), 3.25, device="cuda")
    y, mean, rstd = gla.layer_norm_fwd(x)
    assert not y.any() and torch.equal(mean, torch.full_like(mean, 3.25))
    none = torch.empty(0, 40, device="cuda")
    y, mean, rstd = gla.layer_norm_fwd(none)
    assert y.shape == (0, 40)
    dx, dw, db = gla.layer_norm_bwd(none, none, None, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_streams_and_graphs_give_the_same_bits(env):
    gla, torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(333, 520, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(520, generator=gen, device="cuda")
    y, m, r = gla.layer_norm_fwd(x, w, w)
    grads = gla.layer_norm_bwd(dy, x, w, m, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, m2, r2 = gla.layer_norm_fwd(x, w, w, stream=side)
    grads2 = gla.layer_norm_bwd(dy, x, w, m2, r2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    bx = torch.ones_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yc, mc, rc = gla.layer_norm_fwd(bx, w, w)
        gc = gla.layer_norm_bwd(dy, bx, w, mc, rc)
    bx.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yc, y) and all(torch.equal(a, b) for a, b in zip(gc, grads))

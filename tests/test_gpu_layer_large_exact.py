"""The gated scan and the layer norm on tensors of more than 2^31 elements against 64 bits, with bounds
taken from the data element by element.

Scan: a term that has gone through k gates is off by at most 40 (k + 1) roundings U = 2^-24 of itself
(each gate 32, of |g| <= 8, and a step's and a join's four).  With A_t the scan of the terms'
magnitudes that is 40 U K_t, K_t = f_t K_{t-1} + A_t.  Outputs add the roundings of their own factors.
Norm: a normalised value is off by 64 roundings; a weight gradient of m rows that are not zero adds
m + 320 numbers at most one after the other (a CTA's rows, 304 CTAs in 32 chains and their join)."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    yield gla, torch
    torch.cuda.empty_cache()


def _scan(torch, f, add):
    h, out = torch.zeros_like(add[0]), torch.empty_like(add)
    for t in range(add.shape[0]):
        h = torch.addcmul(add[t], f[t], h, out=out[t])
    return out


@pytest.mark.parametrize("D", [2048, 2046, 2045])
def test_gated_scan(env, D):
    gla, torch = env
    T = 4096
    B = 2 ** 31 // (T * D) + 2
    gen = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda")
    g, dy = torch.empty_like(x), torch.empty(B, T, D, device="cuda")
    x[-1], g[-1], dy[-1] = r(T, D).bfloat16(), (r(T, D) + 1).bfloat16(), r(T, D)
    n = T - 3
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = n
    y, fin = gla.gated_scan_fwd(x, g, None, lens)
    dx, dg, dinit = gla.gated_scan_bwd(x, g, y, dy, None, None, lens)
    assert gla.get_device_error() == 0
    x1, g1, dy1 = (t[-1, :n].double() for t in (x, g, dy))
    f, u = torch.sigmoid(g1), torch.sigmoid(-g1)
    h = _scan(torch, f, u * x1)
    eh = 40 * U * _scan(torch, f, _scan(torch, f, (u * x1).abs()))
    assert ((y[-1, :n] - h).abs() <= eh).all() and ((fin[-1] - h[-1]).abs() <= eh[-1]).all()
    # G_t = dy_t + f_{t+1} G_{t+1}
    late = torch.zeros_like(f)
    late[1:] = f.flip(0)[:-1]
    G = _scan(torch, late, dy1.flip(0)).flip(0)
    eG = 40 * U * _scan(torch, late, _scan(torch, late, dy1.flip(0).abs())).flip(0)
    before = torch.zeros_like(h)
    before[1:], eb = h[:-1], torch.zeros_like(h)
    eb[1:] = eh[:-1]
    assert ((dx[-1, :n] - u * G).abs() <= u * eG + 34 * U * (u * G).abs()).all()
    want = f * u * (before - x1) * G
    slack = f * u * ((before - x1).abs() * eG + (eb + U * (before - x1).abs()) * (G.abs() + eG))
    assert ((dg[-1, :n] - want).abs() <= slack + 70 * U * want.abs()).all()
    assert ((dinit[-1] - (f * G)[0]).abs() <= f[0] * eG[0] + 34 * U * (f * G)[0].abs()).all()
    assert not y[-1, n:].any() and not dx[-1, n:].any() and not dg[:-1].any()


@pytest.mark.parametrize("D", [2048, 2047])
def test_layer_norm_weights(env, D):
    gla, torch = env
    n, m = 2 ** 31 // D + 300, 200
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    x[-m:] = torch.randn(m, D, generator=gen, device="cuda").bfloat16()
    w = torch.randn(D, generator=gen, device="cuda")
    dy = torch.zeros_like(x)
    dy[-m:] = torch.randn(m, D, generator=gen, device="cuda").bfloat16()
    y, mean, rstd = gla.layer_norm_fwd(x, w)
    dx, dw, db = gla.layer_norm_bwd(dy, x, w, mean, rstd)
    x1, dy1 = x[-m:].double(), dy[-m:].double()
    c = x1 - x1.mean(1, keepdim=True)
    r = (c.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    terms = dy1 * c * r
    # of X r: a value next to its row's mean loses that many digits
    unit = 64 * U * (x1.abs().amax(1, keepdim=True) * r + 1)
    assert ((dw - terms.sum(0)).abs() <= (m + 320) * U * terms.abs().sum(0) +
            (unit * dy1.abs()).sum(0)).all()
    assert ((db - dy1.sum(0)).abs() <= (m + 320) * U * dy1.abs().sum(0)).all()
    d = dy1 * w.double()
    want = r * (d - d.mean(1, keepdim=True) - c * r * (d * c * r).mean(1, keepdim=True))
    slack = 2.0 ** -8 * want.abs() + 4 * unit * r * d.abs().amax(1, keepdim=True) * (
        1 + (c * r).abs().amax(1, keepdim=True)) ** 2
    assert ((dx[-m:].double() - want).abs() <= slack).all() and not dx[:-m].any()
    assert gla.get_device_error() == 0

"""The gated scan with gates near 1 (memory of thousands of tokens), against 64 bits: 1 - f must keep
its digits, or every token errs in the same direction and the errors add up over the memory.

Bounds, with n = min(T, 1 / (1 - f)) the tokens that a state remembers, U = 2^-24 a rounding, M the
largest state (adjoint) and X the largest input: the factor of a thread's 16 tokens (gradient: 8),
a number below 1, is rounded once, by U / 2, its product with the next ones' once more, by U, and the
state once, by U M: at most 2 U M each, of which those within the memory count: n / 8 and n / 4
roundings of M.  Within a thread's tokens each rounds twice, on the way to its pair and to its outputs:
64 of M.  The gate itself is off by 32 roundings (the exponent |g| log2(e) carries |g| <= 20 of them)
and the sum 1 - prod f by 16: the same relative error at every token changes an average over the memory
by at most twice that, 96 of X.  With a product of the f alone the error is up to n / 2 roundings of M."""
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
    return gla, torch


def _inputs(torch, B, T, D):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    x = 1 + torch.randn(B, T, D, generator=gen, device="cuda")
    gates = torch.tensor([10.0, 9.0, 12.0, 8.0, 10.5, 6.0, 11.0, 7.0], device="cuda")
    return x, gates[torch.arange(D, device="cuda") % 8].expand(B, T, D).contiguous()


def _scan64(torch, f, add):
    """h_t = f_t h_{t-1} + add_t over dim 1, 64 bits."""
    h, out = torch.zeros_like(add[:, 0]), torch.empty_like(add)
    for t in range(add.shape[1]):
        h = torch.addcmul(add[:, t], f[:, t], h, out=out[:, t])
    return out


CASES = [
    (1, 50021, 8),    # a cluster of 8, tiles by TMA
    (1, 50021, 6),    # ..., rows of pairs
    (1, 30001, 5),    # ..., odd rows
    (240, 25003, 4),  # no clusters, TMA
    (240, 25003, 3),  # no clusters, odd rows
]


@pytest.mark.parametrize("B,T,D", CASES)
def test_gates_near_one(env, B, T, D):
    gla, torch = env
    x, g = _inputs(torch, B, T, D)
    y, fin = gla.gated_scan_fwd(x, g)
    f, u = torch.sigmoid(g.double()), torch.sigmoid(-g.double())
    n = (1 / u[0, 0]).clamp(max=T)
    want = _scan64(torch, f, u * x.double())
    M, X = want.abs().amax((0, 1)), x.abs().max().double()
    bound = U * ((n / 8 + 64) * M + 96 * X)
    err = (y - want).abs().amax((0, 1))
    assert (err <= bound).all(), (err, bound)
    assert ((fin - want[:, -1]).abs().amax(0) <= bound).all()
    # the gradient: G runs from the last token; x serves as dy
    dx, dg, dinit = gla.gated_scan_bwd(x, g, y, x)
    G = _scan64(torch, f, x.double().flip(1)).flip(1)
    M = G.abs().amax((0, 1))
    bound = U * ((n / 4 + 64) * M + 96 * X * n)  # (G sums over the memory where y averages)
    err = ((dinit - (f * G)[:, 0]).abs()).amax(0)
    assert (err <= bound).all(), (err, bound)
    err = (dx - u * G).abs().amax((0, 1))
    assert (err <= u[0, 0] * (bound + 32 * U * M)).all(), (err, u[0, 0] * bound)


def test_decode_of_a_long_answer(env):
    """Step by step a state is rounded at every token, which no order of operations avoids: of each
    sign alike as x varies, so n / 2 independent errors of at most U M / 2 (M < 2: a step of 2^-23)
    add up to a deviation of sqrt(n / 2) U M / sqrt(3), of which eight are allowed."""
    gla, torch = env
    T, D = 30000, 64
    x, g = _inputs(torch, 1, T, D)
    state = torch.zeros(1, D, device="cuda")
    pool = torch.zeros(2, 1, D, device="cuda")
    page = torch.ones(1, dtype=torch.int32, device="cuda")
    xs, gs = x[0].unsqueeze(1).contiguous(), g[0].unsqueeze(1).contiguous()
    for t in range(T):
        gla.gated_scan_decode_step(state, xs[t], gs[t])
        gla.gated_scan_decode_step_paged(pool, page, xs[t:t + 1], gs[t:t + 1])
    f, u = torch.sigmoid(g.double()), torch.sigmoid(-g.double())
    want = _scan64(torch, f, u * x.double())
    n, M, X = (1 / u[0, 0]).clamp(max=T), want.abs().amax((0, 1)), x.abs().max().double()
    bound = 8 * (n / 2).sqrt() * U * M / 3 ** 0.5 + 96 * U * X
    err = (state - want[:, -1]).abs()[0]
    assert (err <= bound).all(), (err, bound)
    assert torch.equal(pool[1], state) and not pool[0].any()

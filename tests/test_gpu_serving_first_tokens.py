"""The first token of a sequence sees itself alone: its weight is 1, and the output its own value, over 8-bit pages to
the bit.  (Over 16 bits the score, below 2^8 in base 2, and the maximum, a rounded product, differ by a rounding: the
sum of weights is off by less than 2^-16.)"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["step8", "chunk8", "chunk16"])
@pytest.mark.parametrize("n,H,KV,window,sink", [(1, 1, 1, 1, 0), (7, 8, 1, 300, 4), (40, 16, 4, 1024, 0),
                                                (500, 6, 2, 40, 2), (5, 40, 2, 129, 1)])
def test_first_tokens(call, n, H, KV, window, sink):
    import torch
    assert torch.cuda.is_available(), "GPU test without a CUDA device"
    import gated_linear_attention_chunked_gb300 as gla
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    gla.load()
    gen = torch.Generator(device="cuda").manual_seed(n + H)
    slots = window + sink
    for dt in (torch.bfloat16, torch.float16):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
        if call == "chunk16":
            pk, pv, pe = r(n, 1, slots, KV, 96), r(n, 1, slots, KV, 192), None
        else:
            pk, pv = (torch.randint(-127, 128, (n, 1, slots, KV, d), generator=gen, device="cuda").to(torch.int8)
                      for d in (96, 192))
            pe = torch.zeros(n, 1, KV, slots, 2, dtype=torch.int8, device="cuda")
        q, k, v = r(n, H, 96) * 3, r(n, KV, 96), r(n, KV, 192)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        page, pos = ints(list(range(n))), ints([0] * n)
        for out in (dt, torch.float32):
            if call == "step8":
                o = gla.window_attn8_decode_step(pk, pv, page, pe, pos, q, k, v, window, sink, out_dtype=out)
            else:
                o = gla.window_attn_chunk(pk, pv, page, pos, ints(list(range(n + 1))), q, k, v, window, sink,
                                          pool_e=pe, out_dtype=out)
            own = v.repeat_interleave(H // KV, 1)
            if call != "chunk16":
                assert torch.equal(o, own.to(out))
            else:
                room = own.double().abs() * (2.0 ** -16 + torch.finfo(out).eps / 2) + torch.finfo(out).tiny
                assert bool(((o.double() - own.double()).abs() <= room).all())
    assert gla.get_device_error() == 0

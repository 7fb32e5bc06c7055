"""How far the table of the rotary positions is from the formula in 60 digits.  It is made in double: the exponent
-2 i / R rounds (2^-53 of itself, so ln(base) 2 i / R times that of the power), the power (a unit in the last place,
2^-52, at most), a division by 2 pi and the rounding of that constant (2^-53 each), for longer contexts a division
more: 4 + ln(base) 2 i / R units of 2^-53 of an entry, or 5, and half a unit of the table.  A position multiplies that;
the product itself is exact modulo a turn."""
from decimal import Decimal, getcontext

import pytest

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("R,base", [(96, 10000), (64, 500000), (128, 10000), (2, 10000), (62, 1000003)])
@pytest.mark.parametrize("scaling,factor", [("plain", 1), ("linear", 8)])
def test_entries_are_within_roundings_of_double(R, base, scaling, factor):
    gla = pytest.importorskip("gated_linear_attention_chunked_gb300")
    from gated_linear_attention_chunked_gb300 import _build
    _build.build()
    getcontext().prec = 60
    table = gla.rotary_turns(R, float(base), scaling, float(factor)).tolist()
    for i, got in enumerate(table):
        units = (4 if scaling == "plain" else 5) + Decimal(base).ln() * 2 * i / R
        exact = (-(Decimal(2 * i) / R) * Decimal(base).ln()).exp() / (2 * PI) / factor * Decimal(2) ** 64
        assert abs(Decimal(got) - exact) <= exact * units * Decimal(2) ** -53 + Decimal("0.5"), (i, got, exact)

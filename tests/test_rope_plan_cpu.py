"""How exact the table of rope_plan is, against 60 decimal digits: what its docstring states.

base^(-2i / rot): the exponent's rounding (2^-53 of it) counts ln(base) times at most, the power, 2 pi and the quotient
by 2 pi once each (2^-53), the power once more for a library's last bit; scaling by 2^64 is exact, the integer half a
unit."""

import math
from decimal import Decimal, localcontext

import pytest

from qlora_fine_tuning_nf4_b200 import ops

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("rot", [2, 64, 80, 96, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6])
def test_table_against_sixty_digits(rot, base):
    turns = [t % 2 ** 64 for t in ops.rope_plan(rot, base, device="cpu").turns.tolist()]
    far = {20: Decimal(0), 31: Decimal(0)}
    with localcontext() as c:
        c.prec = 60
        for i, t in enumerate(turns):
            exact = Decimal(base) ** (Decimal(-2 * i) / Decimal(rot)) / (2 * PI) * 2 ** 64
            off = abs(t - exact)
            assert off <= Decimal(math.log(base) + 4) / 2 ** 53 * exact + Decimal("0.5")
            for p in far:
                far[p] = max(far[p], off * 2 ** p / 2 ** 64)
    assert far[20] <= Decimal(2) ** -34 and far[31] <= Decimal(2) ** -24

"""The rotation's table against the frequencies in 60 decimal digits.

Bound of an entry for f <= 1, in units of u = 2^-53: pow is off by at most one
unit in the last place (2 u f) and by the rounding of its exponent (|ln f| u f),
2 pi and the division by it add u f each, and a division by the factor u f; so f
(5 + |ln f|) / 2 pi <= 0.8 u.  With "base" the larger base adds f (3 + |ln f|),
with "parts" the blend f (11 + |ln f|): 2.4 u at most.  Larger f scale it."""

from decimal import Decimal, getcontext

import pytest

from token_level_head_phi_gb300 import binding as mb
from token_level_head_phi_gb300 import build as mbuild

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(scope="module", autouse=True)
def lib():
    mbuild.build()
    return mb.load()


def turns(rot, base, scaling, factor, length):
    base, factor, length = Decimal(base), Decimal(factor), Decimal(length)
    if scaling == "base" and rot > 2:
        base *= factor ** (Decimal(rot) / (rot - 2))
    step = base ** (Decimal(-2) / rot)
    for i in range(rot // 2):
        f = step ** i
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            keep = min(max((length * f / TWO_PI - 1) / 31, Decimal(0)), Decimal(1))
            f *= keep + (1 - keep) / factor
        yield f, f / TWO_PI


@pytest.mark.parametrize("rot,base,scaling,factor,length", [
    (2, 10000.0, "none", 1.0, 0.0), (64, 10000.0, "none", 1.0, 0.0), (128, 10000.0, "none", 1.0, 0.0),
    (256, 1e6, "none", 1.0, 0.0), (62, 500000.0, "none", 1.0, 0.0), (16, 0.25, "none", 1.0, 0.0),
    (64, 10000.0, "linear", 3.7, 0.0), (256, 1e6, "linear", 4.0, 0.0), (32, 10000.0, "base", 8.0, 0.0),
    (254, 10000.0, "base", 1.7, 0.0), (2, 10000.0, "base", 8.0, 0.0), (128, 500000.0, "parts", 16.0, 8192.0),
    (64, 10000.0, "parts", 40.0, 4096.0), (96, 10000.0, "parts", 1.3, 2000.0)])
def test_table_and_far_phases(rot, base, scaling, factor, length):
    getcontext().prec = 60
    plan = mb.mhla_rotary_plan(rot, base, scaling, factor, length)
    unit = Decimal(2) ** (-53 if scaling in ("none", "linear") else -51)
    for i, (f, turn) in enumerate(turns(rot, base, scaling, factor, length)):
        bound = unit * max(Decimal(1), f)
        off = abs(Decimal(plan.table.turns[i]) / 2 ** 64 - turn) % 1
        assert min(off, 1 - off) < bound, i
        for position in (1, 12345, (1 << 20) + 1, (1 << 40) - 3):
            phase = Decimal(position * plan.table.turns[i] % 2 ** 64) / 2 ** 64
            off = abs(phase - position * turn) % 1
            assert min(off, 1 - off) < position * bound, (i, position)

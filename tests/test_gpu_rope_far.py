"""The rotary table at far positions and high frequencies, against angles of 60
digits: the header's bound without a slack for the reference."""
from __future__ import annotations

import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def frequency(i, rot, base, scaling, factor, original, low, high):
    base, factor = Decimal(base), Decimal(factor)
    if scaling == "base" and rot > 2:
        base *= factor ** (Decimal(rot) / (rot - 2))
    f = base ** (Decimal(-2 * i) / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        w = (original * f / (2 * PI) - Decimal(low)) / (Decimal(high) - Decimal(low))
    elif scaling == "ramp":
        pair = lambda t: rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
        a, z = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        w = 1 - Decimal(i - a) / max(Decimal(z - a), Decimal("0.001"))
    else:
        return f
    w = min(Decimal(1), max(Decimal(0), w))
    return w * f + (1 - w) * f / factor


def exact(first, positions, rot, base=10000.0, scaling="none", factor=1.0, original_len=1, low=1.0, high=4.0):
    """An angle without its whole turns is exact to 2^-53 of it as a double."""
    out = np.zeros((positions, rot))
    for i in range(rot // 2):
        f = frequency(i, rot, base, scaling, factor, original_len, low, high)
        for p in range(positions):
            a = float((first + p) * f % (2 * PI))
            out[p, i], out[p, rot // 2 + i] = math.cos(a), math.sin(a)
    return out


CASES = [dict(base=500000.0), dict(), dict(scaling="linear", factor=1e-5), dict(scaling="linear", factor=1e-6),
         dict(scaling="linear", factor=16.0), dict(scaling="base", factor=8.0), dict(scaling="base", factor=0.25),
         dict(scaling="bands", factor=16.0, original_len=8192, base=500000.0),
         dict(scaling="ramp", factor=4.0, original_len=4096, high=32.0)]


@pytest.mark.parametrize("how", range(len(CASES)))
@pytest.mark.parametrize("first", [0, 131072 - 8, 2 ** 31 - 8])
@pytest.mark.parametrize("rot", [128, 34])
def test_table_within_its_bound(lib, how, first, rot):
    got = lib.pa_rope_table(8, rot, first_position=first, **CASES[how]).cpu().double().numpy()
    off = np.abs(got - exact(first, 8, rot, **CASES[how])).max()
    assert off <= 2.0 ** -22 + 2.0 ** -52, f"{off * 2 ** 22:.2f} times the bound"

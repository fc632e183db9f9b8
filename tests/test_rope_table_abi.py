"""Host checks of the rotary table (no GPU needed): what a scaling does not read
cannot refuse a call."""
from __future__ import annotations

import pytest

import paged_kv_cache_14_gb300 as pa

NAN = float("nan")


def table(positions=0, rot=128, base=1e4, kind=0, factor=1.0, orig=0, low=1.0, high=4.0, amplitude=1.0, out=0x1000):
    """A call that passes every check launches nothing: it asks for no positions."""
    return pa.load().pa_rope_table(out, 0, positions, rot, base, kind, factor, orig, low, high, amplitude, None)


@pytest.mark.parametrize("factor", [0.0, -1.0, NAN, float("inf")])
def test_plain_table_reads_no_factor(factor):
    assert table(kind=0, factor=factor) == 0
    assert table(kind=0, factor=factor, low=NAN, high=NAN, orig=-1) == 0
    for kind in (1, 2, 3, 4):  # the others do
        assert table(kind=kind, factor=factor, orig=1) == -1


@pytest.mark.parametrize("amplitude", [1e300, -1e300, 3.5e38, float("inf"), NAN])
def test_amplitude_is_finite_in_fp32(amplitude):
    """The entries are fp32: an amplitude beyond its range would be infinite."""
    assert table(amplitude=amplitude) == -1


def test_largest_amplitudes():
    top = float((2 - 2 ** -23) * 2.0 ** 127)
    for amplitude in (top, -top, 1e-300, 0.0):
        assert table(amplitude=amplitude) == 0


def test_extreme_scalings():
    """What leaves the doubles' range on the way without leaving it at the end."""
    assert table(kind=1, factor=1.7e308) == 0 and table(kind=2, factor=1.7e308) == 0
    assert table(kind=3, factor=1e308, orig=8192) == 0 and table(kind=4, factor=1e308, orig=8192, high=32.0) == 0
    assert table(kind=3, factor=4.0, orig=2 ** 31 - 1, low=1e-300, high=1.7e308) == 0
    assert table(kind=3, factor=4.0, orig=1, low=1e-310, high=2e-310) == 0  # a band of no width in normal numbers
    assert table(kind=3, factor=1e-310, orig=2 ** 31 - 1, low=1e-310, high=2e-310) == 0  # (every pair above it)
    assert table(kind=4, factor=4.0, orig=1, low=1e-300, high=1.7e308) == 0
    assert table(base=1.7e308) == 0 and table(base=1.0 + 2 ** -52) == 0
    assert table(rot=4, base=1.7e308, kind=2, factor=1e300) == 0

"""V scales of 8-bit blocks far from 1, with a tolerance that shrinks and grows
with the values: a bf16 output has no smallest step that would matter here."""
from __future__ import annotations

import numpy as np
import pytest

from sparse_helpers import sparse_batch

EXPONENTS = [-120, -60, 0, 60, 100]


def scaled_batch(kv, exponent):
    """V scales times 2^exponent, K scales times half of it, which the queries make up for."""
    b = sparse_batch(12, "bf16", [300, 90], 12, 8, 2, 128, 16, kv)
    b.scales[..., 1] *= np.float32(2.0) ** exponent
    b.scales[..., 0] *= np.float32(2.0) ** (exponent // 2)
    b.q = (b.q.float() * 2.0 ** -(exponent // 2)).bfloat16()
    return b


def times_tolerance(b, got):
    """The output is rounded once (2^-8), a weight to fp16 (2^-11, or 2^-25 where
    it is small, of a row sum of at least 1); a score is off by (d + 8) steps of
    2^-23 of the sum |q k|, and its exponential by 8 steps, in numerator and
    denominator; the sums and the division by 8 steps. Outputs below bf16's normal
    numbers have steps of 2^-133."""
    out, weighted, largest = b.oracle()
    step, d = 2.0 ** -23, b.q.shape[-1]
    es = largest[..., None] * (d + 8) * step + 8 * step
    top = np.abs(b.stored()[1]).max()
    n = int(b.lens.max())
    tol = (2.0 ** -8 + 8 * step) * np.abs(out) + (2.0 ** -11 + 2 * es) * weighted + n * 2.0 ** -25 * top + 2.0 ** -134
    return np.abs(got - out) / tol


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("exponent", EXPONENTS)
def test_tolerance_tells_wrong_outputs(kv, exponent):
    """Zeros, the negated outputs and those of half the scale are outside."""
    b = scaled_batch(kv, exponent)
    out = b.oracle()[0]
    assert times_tolerance(b, out).max() == 0
    for wrong in (0 * out, -out, out / 2):
        assert times_tolerance(b, wrong).max() > 8


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("exponent", EXPONENTS)
def test_scales_far_from_one(lib, kv, exponent):
    b = scaled_batch(kv, exponent)
    got = b.call(lib).double().cpu().numpy()
    assert lib.pa_get_status() == 0
    over = times_tolerance(b, got).max()
    assert over <= 1.0, f"{over:.2f} times the tolerance"

"""How exact the softmax weights of sparse attention over bf16 caches are in the
second product: scores that carry no error of their own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_helpers import sparse_batch

pytestmark = pytest.mark.gpu


def whole_scores(seed, lens, keep, hq, hkv, d, block):
    """q and k of -1, 0 and 1, scale 1/16: products and sums of q k are exact."""
    b = sparse_batch(seed, "bf16", lens, keep, hq, hkv, d, block, ragged=False, scale=1 / 16)
    rng = np.random.default_rng(seed + 1)
    b.q = torch.from_numpy(rng.integers(-1, 2, b.q.shape)).bfloat16()
    b.k = torch.from_numpy(rng.integers(-1, 2, b.k.shape)).bfloat16()
    return b


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (16, 1, 128), (12, 4, 64), (11, 1, 64)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("lens,keep", [([700], 40), ([3, 60, 200], 12)])
def test_weights_of_two_parts(lib, hq, hkv, d, block, lens, keep):
    """Two bf16 parts: the first is off by less than 2^-7 of a weight, the second
    by 2^-8 of that: 2^-15. A score's product with the scale and its difference
    to the reference are off by 3 half steps (2^-24) of at most twice the largest
    sum |q k|, the exponential by 2 steps of 2^-23, and that of numerator and
    denominator both. A product of 16 tokens may lose a step of 2^-22 of the sums
    that it adds to, n / 16 of them and 16 for the joins. The output is rounded
    once: 2^-8."""
    b = whole_scores(40, lens, keep, hq, hkv, d, block)
    got = b.call(lib).double().cpu().numpy()
    assert lib.pa_get_status() == 0
    out, weighted, largest = b.oracle()
    es = 3 * 2.0 ** -24 * 2 * largest[..., None] + 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -15 + 2 * es + (max(lens) / 16 + 16) * 2.0 ** -22) * weighted
    over = np.abs(got - out) / (tol + 1e-30)
    assert over.max() <= 1.0, f"{over.max():.2f} times the tolerance, {(over > 1).mean():.1%} of the outputs"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_values_keep_their_sign(lib, d, value):
    """A weight above 0 times an infinity is that infinity, whatever the weight:
    all alike (each exactly 1), and of every size down to 2^-40."""
    for alike in (True, False):
        b = whole_scores(41, [160], 10, 8, 1, d, 16)
        b.q[:] = 1.0
        b.k[:] = 0.0
        if not alike:
            b.scale = 0.6931471805599453 / 4
            for i in range(10):
                for t in range(16):
                    b.k[b.table[0, i], 0, t, 0] = -float(i * 16 + t)  # weights 2^-(n / 4)
        for n in range(d):
            b.v[b.table[0, n % 10], 0, n // 8 % 16, n] = value  # a row's own in every dimension
        out = b.call(lib).float().cpu()
        assert (out == value).all(), alike


def whole_scores_f16(seed, lens, keep, hq, hkv, d, block, kv):
    """The same in fp16, over fp16 pools or (K codes of -1, 0 and 1, K scales 1) 8-bit ones."""
    b = sparse_batch(seed, "f16", lens, keep, hq, hkv, d, block, kv, ragged=False, scale=1 / 16)
    rng = np.random.default_rng(seed + 1)
    b.q = torch.from_numpy(rng.integers(-1, 2, b.q.shape)).half()
    k = torch.from_numpy(rng.integers(-1, 2, b.k.shape))
    if kv is None:
        b.k = k.half()
    else:
        one = {"e4m3": 0x38, "e5m2": 0x3C}[kv]
        b.k = torch.where(k == 0, 0, torch.where(k > 0, one, one | 0x80)).to(torch.uint8)
        b.scales[..., 0] = 1.0
        assert np.array_equal(b.stored()[0], k.double().numpy())
    return b


@pytest.mark.parametrize("kv,hq,hkv,d", [(None, 8, 1, 128), (None, 16, 1, 128), (None, 12, 4, 64), (None, 11, 1, 64),
                                         ("e4m3", 8, 1, 128), ("e5m2", 12, 1, 128)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("lens,keep", [([700], 40), ([3, 60, 200], 12)])
def test_weights_of_two_fp16_parts(lib, kv, hq, hkv, d, block, lens, keep):
    """The first part is off by less than 2^-10 of a weight, the second by 2^-11 of
    that: 2^-21; weights below fp16's numbers by 2^-39 (times the largest value, a
    token). Scores, exponentials and sums as above, an 8-bit block's product once
    more by its V scale (half a step of 2^-23); the output's rounding is 2^-11, or
    2^-25 below fp16's normal numbers."""
    b = whole_scores_f16(42, lens, keep, hq, hkv, d, block, kv)
    got = b.call(lib).double().cpu().numpy()
    assert lib.pa_get_status() == 0
    out, weighted, largest = b.oracle()
    es = 3 * 2.0 ** -24 * 2 * largest[..., None] + 2.0 ** -22
    top = float(np.abs(np.asarray(b.stored()[1], np.float64)).max())
    sums = (max(lens) / 16 + 16) * 2.0 ** -22 + 2.0 ** -24
    tol = (2.0 ** -11 * np.abs(out) + 2.0 ** -25 + (2.0 ** -21 + 2 * es + sums) * weighted +
           max(lens) * 2.0 ** -39 * top)
    over = np.abs(got - out) / tol
    assert over.max() <= 1.0, f"{over.max():.2f} times the tolerance, {(over > 1).mean():.1%} of the outputs"


@pytest.mark.parametrize("kv,d", [(None, 64), (None, 128), ("e5m2", 128)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_fp16_values_keep_their_sign(lib, kv, d, value):
    """Weights of exactly 1, and of sizes down to 2^-13 (below 2^-14 a weight is no
    normal fp16 number)."""
    for alike in (True, False):
        b = whole_scores_f16(43, [160], 10, 8, 1, d, 16, kv)
        b.q[:] = 1.0
        b.k[:] = 0
        if not alike:
            b.scale = 0.6931471805599453 / 4
            for i in range(10):
                for t in range(16):
                    n = (i * 16 + t) % 53  # weights 2^-(n / 4), as so many dimensions of -1
                    b.k[b.table[0, i], 0, t, :n] = -1.0 if kv is None else 0xBC
        for n in range(d):
            b.v[b.table[0, n % 10], 0, n // 8 % 16, n] = value if kv is None else 0x7C if value > 0 else 0xFC
        out = b.call(lib).float().cpu()
        assert (out == value).all(), alike


@pytest.mark.parametrize("dtype,kv,least", [("bf16", None, 125), ("f16", None, 24.5), ("f16", "e5m2", 24.5)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_values_under_small_weights(lib, dtype, kv, least, value):
    """One infinity a sequence, under a weight of 2^-least to 1: the output is that
    infinity. (A bf16 has numbers down to 2^-126; fp16 ones end at 2^-24, half of
    which a rounding still takes there.)"""
    n, d = 200, 128
    b = sparse_batch(44, dtype, [32] * n, 2, 4, 1, d, 16, kv, ragged=False, scale=0.6931471805599453 / 8)
    b.q[:], b.k[:] = 0.0, 0
    b.q[..., 0] = 8.0
    where, size = np.arange(n) % 32, np.linspace(0.0, least, n)
    for i in range(n):
        one = b.table[i, where[i] // 16], 0, where[i] % 16
        # The score's exponent of 2: a bf16 of up to 125 is off by 2^-2, a value that counts as it is.
        b.k[one][0] = -float(size[i]) if kv is None else int(torch.tensor(-size[i]).to(torch.float8_e5m2).view(torch.uint8))
        b.v[one][:] = value if kv is None else 0x7C if value > 0 else 0xFC
    if kv:
        b.scales[..., 0] = 1.0
    out = b.call(lib).float().cpu()
    assert (out == value).all(), np.unique(np.nonzero((out != value).any(-1).any(-1).numpy())[0])

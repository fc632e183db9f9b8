"""Pins of the long-context oracle: closed forms, torch's own routines, and
planted mistakes that must fail one of them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import oracle.sparse as osp


def turned(x, angle, interleaved):
    """Rows [T, H, D] turned through torch's complex numbers."""
    x = torch.as_tensor(x, dtype=torch.float64)
    pairs = x.reshape(*x.shape[:-1], -1, 2) if interleaved else torch.stack(x.chunk(2, -1), -1)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones(angle.shape, dtype=torch.float64), angle)[:, None]
    y = torch.view_as_real(z)
    return (y.flatten(-2) if interleaved else torch.cat([y[..., 0], y[..., 1]], -1)).numpy()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((7, 3, 32)).astype(np.float32))
    pos = rng.integers(0, 500, 7)
    freqs = osp.rope_frequencies(32)
    got = osp.rotate(x, osp.rope_table(0, 500, freqs), pos, interleaved)
    angle = torch.from_numpy(pos[:, None] * freqs)
    assert np.abs(got - turned(x, angle, interleaved)).max() < 1e-5
    # Products with the positions' difference alone.
    a, b = (osp.rotate(x[:1], osp.rope_table(0, 500, freqs), [p], interleaved)[0, 0] for p in (40, 45))
    c, d = (osp.rotate(x[:1], osp.rope_table(0, 500, freqs), [p], interleaved)[0, 0] for p in (400, 405))
    assert abs(a @ b - c @ d) < 1e-3
    # A part of a head: the rest stays.
    part = osp.rotate(x, osp.rope_table(0, 500, osp.rope_frequencies(8)), pos, interleaved)
    assert np.array_equal(part[..., 8:], x.numpy()[..., 8:]) and not np.array_equal(part[..., :8], x.numpy()[..., :8])


def test_frequencies():
    plain = osp.rope_frequencies(64)
    assert plain[0] == 1.0 and math.isclose(plain[-1], 10000.0 ** (-62 / 64))
    assert np.allclose(osp.rope_frequencies(64, scaling="linear", factor=4.0), plain / 4)
    base = osp.rope_frequencies(64, scaling="base", factor=8.0)
    assert base[0] == 1.0 and math.isclose(base[-1], plain[-1] / 8.0)  # the slowest pair is stretched by the factor
    for kind, kw in (("bands", dict()), ("ramp", dict())):
        f = osp.rope_frequencies(128, scaling=kind, factor=16.0, original_len=8192, **kw)
        r = osp.rope_frequencies(128) / f
        assert np.isclose(r[0], 1.0) and np.isclose(r[-1], 16.0) and (np.diff(r) >= -1e-12).all()
    turns = 8192 * osp.rope_frequencies(128) / (2 * math.pi)
    f = osp.rope_frequencies(128, scaling="bands", factor=16.0, original_len=8192)
    assert np.allclose(f[turns >= 4.0], osp.rope_frequencies(128)[turns >= 4.0])
    assert np.allclose(f[turns <= 1.0], osp.rope_frequencies(128)[turns <= 1.0] / 16)


def test_summaries():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 64)).astype(np.float32)
    codes, scale = osp.summarize(x)
    assert codes.max() == 127 or codes.min() == -127
    hi, lo = codes[0].astype(np.float64) * scale, codes[1].astype(np.float64) * scale
    step = float(scale)
    assert (hi >= x.max(0) - 1e-5 * step).all() and (hi < x.max(0) + 1.001 * step).all()
    assert (lo <= x.min(0) + 1e-5 * step).all() and (lo > x.min(0) - 1.001 * step).all()
    assert osp.summarize(np.zeros((3, 8)))[1] == 0
    x[3, 3] = np.inf
    assert np.isinf(osp.summarize(x)[1]) and (osp.summarize(x)[0] == 0).all()
    # One row is its own range.
    one, s = osp.summarize(x[:1])
    assert (np.abs(one[0].astype(int) - one[1]) <= 1).all()


def bounds(block_scores, alike=False):
    """Whether scores are upper bounds of every key's product with the 8-bit
    query, and no more than that where a block's keys are alike."""
    rng = np.random.default_rng(2)
    k = rng.standard_normal((40, 16, 64)).astype(np.float32)
    if alike:
        k[:] = k[:, :1]
    q = rng.standard_normal((3, 64)).astype(np.float32)
    codes, scale = zip(*(osp.summarize(x) for x in k))
    codes, scale = np.stack(codes), np.array(scale, np.float32)
    score = block_scores(q, codes, scale)
    sq = np.abs(q).max(1, keepdims=True) / np.float32(127)
    best = np.einsum("btd,hd->bht", k.astype(np.float64), np.rint(q / sq) * sq).max((1, 2))
    # A code is off by at most one step of the block's scale (and rounding).
    most = best + 1.01 * scale * np.abs(q).sum(1).max() if alike else np.inf
    return bool((score >= best - 1e-4).all()) and bool((score <= most).all())


def test_scores_bound_products():
    assert bounds(osp.block_scores) and bounds(osp.block_scores, True)
    assert not bounds(lambda q, c, s: osp.block_scores(q, c[:, [1, 1]], s), True)   # lower ends for upper ones
    assert not bounds(lambda q, c, s: osp.block_scores(q[:1], c, s), True)          # one head of the group
    assert not bounds(lambda q, c, s: osp.block_scores(q, c, s * np.float32(0.5)), True)
    assert not bounds(lambda q, c, s: osp.block_scores(q, c, s * np.float32(2)), True)
    assert not bounds(lambda q, c, s: osp.block_scores(np.abs(q), c, s), True)      # the queries' signs lost


def test_choice():
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((2, 4, 32)).astype(np.float32))
    codes = rng.integers(-127, 128, (30, 2, 2, 32)).astype(np.int8)
    codes = np.sort(codes, 2)[:, :, ::-1].copy()
    scales = rng.random((30, 2)).astype(np.float32)
    table = np.stack([rng.permutation(30) for _ in range(2)]).astype(np.int32)
    lens = np.array([470, 50], np.int32)
    lists, n = osp.select_blocks(q, codes, scales, table, lens, 16, 8, 1, 2)
    assert (n == [[8, 8], [4, 4]]).all() and (lists[1, 0] == [0, 1, 2, 3, -1, -1, -1, -1]).all()
    for h in range(2):
        mine = lists[0, h]
        assert mine[0] == 0 and (mine[-2:] == [28, 29]).all() and (np.diff(mine) > 0).all()
        score = osp.block_scores(q[0, 2 * h:2 * h + 2].numpy(), codes[table[0], h], scales[table[0], h])
        rest = np.setdiff1d(np.arange(1, 28), mine)
        assert score[mine[1:-2]].min() >= score[rest].max()
    same = osp.select_blocks(q, codes * 0, scales, table, lens, 16, 8, 1, 2)[0]
    assert (same[0, 0] == [0, 1, 2, 3, 4, 5, 28, 29]).all()  # ties: the lower blocks


def test_all_blocks_is_decode():
    rng = np.random.default_rng(4)
    k, v = (rng.standard_normal((9, 2, 16, 32)) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((2, 4, 32)))
    table = np.array([[3, 1, 7, 0], [8, 2, 5, 6]], np.int32)
    lens = np.array([50, 17], np.int32)
    lists = np.array([[[0, 1, 2, 3]] * 2, [[0, 1, -1, -1]] * 2], np.int32)
    counts = np.array([[4, 4], [2, 2]], np.int32)
    got = osp.decode_sparse(q, k, v, table, lens, lists, counts, 0.3, 16)[0]
    assert np.abs(got - oracle.decode(q, k, v, table, lens, 0.3, 16)).max() < 1e-12
    counts[0, 1] = 0
    assert (osp.decode_sparse(q, k, v, table, lens, lists, counts, 0.3, 16)[0][0, 2:] == 0).all()

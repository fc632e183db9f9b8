"""Block summaries and the choice of blocks, exactly as the oracle has them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.sparse as osp
from sparse_helpers import SUFFIX, dev, normal, pools, values
from tree_helpers import DT, paged

pytestmark = pytest.mark.gpu


def summaries_of(lib, k, sc, kv, table, first, lens, most, codes, scales):
    extra = () if sc is None else (dev(sc),)
    getattr(lib, "pa_block_summaries" + SUFFIX[kv])(dev(k), *extra, *dev(table, first, lens), most, codes, scales)


@pytest.mark.parametrize("dtype,kv,hkv,d", [("f32", None, 2, 32), ("f32", None, 3, 96), ("f32", None, 1, 256),
                                            ("f16", None, 8, 128), ("f16", None, 1, 64), ("bf16", None, 8, 128),
                                            ("bf16", None, 3, 64), ("bf16", "e4m3", 2, 128), ("bf16", "e4m3", 1, 64),
                                            ("bf16", "e5m2", 8, 128), ("bf16", "e5m2", 2, 64)])
@pytest.mark.parametrize("block", [16, 32])
def test_summaries(lib, dtype, kv, hkv, d, block):
    rng = np.random.default_rng(1)
    lens = np.array([1, 15, 16, 17, 32, 33, 64, 100, 257, 5, 0, 40], np.int32)
    first = np.array([0, 14, 0, 16, 3, 33, 63, 37, 0, 2, 0, 31], np.int32)
    table, P = paged(rng, [int(x) for x in lens], block)
    k, _, sc = pools(rng, P, hkv, block, d, dtype, kv)
    codes0 = rng.integers(-128, 128, (P, hkv, 2, d)).astype(np.int8)
    scales0 = rng.random((P, hkv)).astype(np.float32)
    codes, scales = dev(codes0.copy(), scales0.copy())
    summaries_of(lib, k, sc, kv, table, first, lens, 300, codes, scales)
    assert lib.pa_get_status() == 0
    osp.block_summaries(values(k, sc, 0, kv), table, first, lens, block, codes0, scales0)
    assert np.array_equal(codes.cpu().numpy(), codes0)
    assert np.array_equal(scales.cpu().numpy(), scales0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_summaries_of_odd_values(lib, dtype):
    """Infinities, NaN, zeros and the type's smallest values; what lies behind a
    sequence's end is not looked at."""
    rng = np.random.default_rng(2)
    B, hkv, d, P = 16, 2, 64, 9
    k = normal(rng, P, hkv, B, d).to(DT[dtype])
    k[0, 0, 3, 5] = float("inf")
    k[1, 1, 2, 63] = float("nan")
    k[2] = 0.0
    k[3, 0] = 0.0
    k[3, 0, 1, 7] = torch.finfo(DT[dtype]).smallest_normal
    k[4, :, 4:] = float("nan")  # behind the end
    k[5, 0, 0, 0] = -float("inf")
    k[6, 0] = torch.finfo(DT[dtype]).max
    k[7, 1] = -3.0
    if dtype != "f16":
        k[8, 0] = 0.0
        k[8, 0, 3, 3] = 2.0 ** -133  # its quotient by 127 is below fp32's smallest
    table = np.arange(P, dtype=np.int32)[:, None]
    lens = np.full(P, B, np.int32)
    lens[4] = 4
    codes, scales = torch.zeros(P, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(P, hkv, device="cuda")
    summaries_of(lib, k, None, None, table, np.zeros(P, np.int32), lens, B, codes, scales)
    ref, rs = np.zeros((P, hkv, 2, d), np.int8), np.zeros((P, hkv), np.float32)
    osp.block_summaries(k.float().numpy(), table, np.zeros(P, int), lens, B, ref, rs)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), ref)
    assert np.isinf(rs[0, 0]) and np.isinf(rs[1, 1]) and np.isfinite(rs[4]).all() and (rs[2] == 0).all()


def test_summaries_bound_every_product(lib):
    """A block's score is at least any of its keys' products with the 8-bit query."""
    rng = np.random.default_rng(3)
    B, hkv, d, P = 16, 1, 128, 50
    k = normal(rng, P, hkv, B, d)
    table = np.arange(P, dtype=np.int32)[None]
    codes, scales = torch.zeros(P, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(P, hkv, device="cuda")
    summaries_of(lib, k, None, None, table, np.zeros(1, np.int32), np.array([P * B], np.int32), P * B, codes, scales)
    q = rng.standard_normal(d).astype(np.float32)
    score = osp.block_scores(q[None], codes.cpu().numpy()[:, 0], scales.cpu().numpy()[:, 0])
    sq = np.float32(np.abs(q).max() / np.float32(127))
    best = (k[:, 0].double().numpy() @ (np.rint(q / sq) * float(sq))).max(1)
    assert (score >= best - 1e-4).all()


def test_summaries_errors(lib):
    rng = np.random.default_rng(4)
    P, hkv, B, d = 6, 2, 16, 64
    k = normal(rng, P, hkv, B, d).bfloat16()
    for table, first, length, most, code in (([[0, 9]], 0, 20, 64, -7), ([[0, -1]], 0, 20, 64, -7),
                                             ([[0, 1]], 0, 40, 64, -8), ([[0, 1]], 3, 2, 64, -8),
                                             ([[0, 1]], -1, 2, 64, -8), ([[0, 1]], 0, 20, 19, -8)):
        codes, scales = torch.zeros(P, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(P, hkv, device="cuda")
        summaries_of(lib, k, None, None, np.array(table, np.int32), np.array([first], np.int32),
                     np.array([length], np.int32), most, codes, scales)
        assert lib.pa_get_status() == code, (table, first, length)
        assert lib.pa_get_status() == 0


def chosen(seed, lens, hq, hkv, d, block, dtype, keep, sink, recent, spread=1.0):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    table, P = paged(rng, [int(x) for x in lens], block)
    q = normal(rng, len(lens), hq, d).to(DT[dtype])
    codes = np.empty((P, hkv, 2, d), np.int8)
    lo = rng.integers(-127, 100, (P, hkv, d))
    codes[:, :, 1] = lo
    codes[:, :, 0] = np.minimum(lo + rng.integers(0, 60, lo.shape), 127)
    scales = np.exp(spread * rng.standard_normal((P, hkv))).astype(np.float32)
    return q, codes, scales, table, lens


def check_select(lib, q, codes, scales, table, lens, block, keep, sink, recent, **kw):
    lists, counts = lib.pa_select_blocks(*dev(q, codes, scales, table, lens), int(lens.max(initial=1)) or 1, block, keep,
                                         num_sink=sink, num_recent=recent, **kw)
    ref, n = osp.select_blocks(q, codes, scales, table, lens, block, keep, sink, recent)
    assert np.array_equal(counts.cpu().numpy(), n)
    assert np.array_equal(lists.cpu().numpy(), ref)


LENS = [1, 16, 17, 300, 1000, 5000, 0, 2049, 64, 777]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (9, 1, 96), (12, 4, 32), (128, 1, 128), (3, 3, 256)])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 1), (4, 1, 1), (17, 2, 3), (64, 0, 0), (5, 2, 3), (400, 1, 1)])
def test_select(lib, dtype, hq, hkv, d, keep, sink, recent):
    args = chosen(1, LENS, hq, hkv, d, 16, dtype, keep, sink, recent)
    check_select(lib, *args, 16, keep, sink, recent)
    assert lib.pa_get_status() == 0


@pytest.mark.parametrize("spread", [0.0, 30.0])
@pytest.mark.parametrize("block", [16, 32])
def test_select_long(lib, spread, block):
    """Rows split over a cluster; scales over fp32's whole range, and all equal."""
    args = chosen(2, [70001, 33, 40000], 16, 2, 64, block, "bf16", 300, 1, 4, spread)
    check_select(lib, *args, block, 300, 1, 4)


def test_select_ties(lib):
    """Equal scores go to the lower block, wherever the row is split."""
    n, hkv, d, nb = 2, 2, 64, 3000
    q = torch.ones(n, hkv, d)
    table = np.arange(nb, dtype=np.int32)[None].repeat(n, 0)
    lens = np.full(n, nb * 16, np.int32)
    codes = np.ones((nb, hkv, 2, d), np.int8)
    scales = np.ones((nb, hkv), np.float32)
    check_select(lib, q, codes, scales, table, lens, 16, 50, 1, 1)
    rng = np.random.default_rng(5)
    scales = rng.integers(1, 4, (nb, hkv)).astype(np.float32)
    check_select(lib, q, codes, scales, table, lens, 16, 1200, 1, 1)
    check_select(lib, q, codes * 0, scales, table, lens, 16, 700, 3, 0)
    check_select(lib, -q, codes, scales, table, lens, 16, 700, 0, 2)


def test_select_odd_values(lib):
    """Heads that are not finite count as zeros, blocks whose keys are not come
    first; zeros and the smallest scales."""
    n, hkv, d, nb = 3, 2, 64, 600
    rng = np.random.default_rng(6)
    q, codes, scales, table, lens = chosen(7, [nb * 16] * n, 8, hkv, d, 16, "f32", 0, 0, 0)
    q[0, 1, 3] = float("nan")
    q[1, 2, 0] = float("inf")
    q[2, 4:] = 0.0
    scales[rng.random(scales.shape) < 0.01] = np.inf
    scales[rng.random(scales.shape) < 0.05] = 0.0
    scales[rng.random(scales.shape) < 0.05] = 1e-45
    for keep in (3, 60, 599):
        check_select(lib, q, codes, scales, table, lens, 16, keep, 1, 1)
    big = q * 3e37
    check_select(lib, big, codes, scales * 1e3, table, lens, 16, 60, 1, 1)


def test_select_many_sequences(lib):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 900, 700)
    check_select(lib, *chosen(9, lens, 4, 1, 64, 16, "bf16", 9, 1, 1), 16, 9, 1, 1)


def test_select_errors(lib):
    q, codes, scales, table, lens = chosen(10, [800, 500], 4, 2, 64, 16, "bf16", 4, 1, 1)
    P = len(scales)
    bad = table.copy()
    bad[0, 20] = P
    lists, counts = lib.pa_select_blocks(*dev(q, codes, scales, bad, lens), 800, 16, 8)
    assert lib.pa_get_status() == -7
    assert 20 not in lists[0].cpu().tolist()
    for length, cap in ((801, 800), (-1, 800), (10 ** 6, 2 ** 31 - 1)):
        l2 = lens.copy()
        l2[0] = length
        lists, counts = lib.pa_select_blocks(*dev(q, codes, scales, table, l2), cap, 16, 8)
        assert lib.pa_get_status() == -8 and lib.pa_get_status() == 0
        assert counts[0].eq(0).all() and lists[0].eq(-1).all() and counts[1].eq(8).all()


def test_select_streams_and_graph(lib):
    a = chosen(11, [3000, 100, 2500], 8, 2, 128, 16, "bf16", 20, 1, 1)
    d = dev(*a)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = lib.pa_select_blocks(*d, 3000, 16, 20, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    out = [torch.empty_like(x) for x in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.pa_select_blocks(*d, 3000, 16, 20, block_lists=out[0], list_lens=out[1])
    for seed in (12, 13):
        b = chosen(seed, [3000, 100, 2500], 8, 2, 128, 16, "bf16", 20, 1, 1)
        d[0].copy_(b[0])
        g.replay()
        ref, n = osp.select_blocks(b[0], a[1], a[2], a[3], a[4], 16, 20, 1, 1)
        assert np.array_equal(out[0].cpu().numpy(), ref) and np.array_equal(out[1].cpu().numpy(), n)
    ref, n = osp.select_blocks(a[0], a[1], a[2], a[3], a[4], 16, 20, 1, 1)
    assert np.array_equal(first[0].cpu().numpy(), ref)

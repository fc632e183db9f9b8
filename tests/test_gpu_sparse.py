"""Attention over listed blocks against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_helpers import assert_sparse_close, sparse_batch, sparse_tolerance

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 17, 100, 513, 1000, 31, 32, 33]


@pytest.mark.parametrize("dtype,kv,hq,hkv,d", [
    ("bf16", None, 8, 2, 128), ("f16", None, 8, 2, 64), ("bf16", None, 4, 4, 64), ("f16", None, 28, 4, 128),
    ("bf16", None, 12, 1, 128), ("f16", None, 33, 1, 64), ("bf16", None, 128, 1, 128), ("f16", None, 16, 1, 128),
    ("bf16", "e4m3", 8, 2, 128), ("f16", "e4m3", 12, 1, 128), ("bf16", "e5m2", 64, 8, 128), ("f16", "e5m2", 3, 3, 128),
    ("bf16", "e4m3", 20, 1, 128), ("f32", None, 8, 2, 128), ("f32", None, 9, 1, 96), ("f32", None, 2, 2, 32),
    ("f32", None, 4, 1, 256), ("f32", None, 6, 2, 224), ("f32", None, 2, 1, 192), ("f32", None, 2, 1, 160),
    ("f32", None, 20, 2, 64)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("keep", [1, 3, 40])
def test_sparse(lib, dtype, kv, hq, hkv, d, block, keep):
    b = sparse_batch(keep, dtype, LENS, keep, hq, hkv, d, block, kv)
    out = b.call(lib)
    assert lib.pa_get_status() == 0
    assert_sparse_close(b, out)
    assert (out.cpu()[(b.counts == 0).repeat(hq // hkv, 1)] == 0).all()


@pytest.mark.parametrize("dtype,kv,hq,hkv", [("bf16", None, 64, 8), ("f16", None, 8, 8), ("bf16", "e4m3", 64, 8),
                                             ("bf16", "e5m2", 16, 1)])
def test_long_lists(lib, dtype, kv, hq, hkv):
    """One sequence split over a cluster, every block listed; and many sequences."""
    b = sparse_batch(5, dtype, [9001], 600, hq, hkv, 128, 16, kv, ragged=False)
    assert_sparse_close(b, b.call(lib), "one sequence")
    b = sparse_batch(6, dtype, np.random.default_rng(1).integers(1, 700, 90), 30, hq, hkv, 128, 16, kv)
    assert_sparse_close(b, b.call(lib), "many sequences")
    assert lib.pa_get_status() == 0


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", None), ("f32", None), ("bf16", "e4m3"), ("f16", "e5m2")])
def test_all_blocks_is_decode(lib, dtype, kv):
    """A list of all blocks gives pa_decode's attention: each is within its
    roundings of the exact one, so they are within twice these of each other.
    (An output of 4 to 8, which values scaled by up to 3 reach, has bf16 steps
    of 2^-5: two outputs that are right may lie 0.03 apart.)"""
    b = sparse_batch(7, dtype, [700, 1, 333], 50, 16, 4, 128, 16, kv, ragged=False)
    got = b.call(lib).double()
    name = "pa_decode" + ({"e4m3": "_fp8", "e5m2": "_e5m2"}[kv] if kv else "")
    a = b.args()
    n = 3 if kv is None else 4
    ref = getattr(lib, name)(*a[:n], a[n], a[n + 1], 700, b.scale).double()
    tol = torch.from_numpy(sparse_tolerance(b, *b.oracle()))
    assert ((got - ref).abs().cpu() <= 2 * tol).all()
    assert_sparse_close(b, b.call(lib))


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", None), ("f32", None), ("bf16", "e4m3")])
@pytest.mark.parametrize("q_scale,scale", [(40.0, None), (1.0, -0.2), (1.0, 0.0), (0.0, 1.0), (1e-3, 1e-6)])
def test_scales(lib, dtype, kv, q_scale, scale):
    """Scores that spread over hundreds, negative and zero scales."""
    b = sparse_batch(8, dtype, [900, 40, 129], 45, 8, 2, 128, 16, kv, q_scale=q_scale, scale=scale)
    assert_sparse_close(b, b.call(lib))


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rising_scores(lib, rising, dtype):
    """Scores that rise (or fall) by a little from tile to tile: the reference
    moves seldom, weights above 1 stay exact enough."""
    b = sparse_batch(9, dtype, [4096], 256, 8, 1, 128, 16, ragged=False)
    b.q[:] = 1.0
    step = torch.linspace(0, 3.0, 256) if rising else torch.linspace(3.0, 0, 256)
    for i in range(256):
        b.k[b.table[0, i], 0] = (0.05 * b.k[b.table[0, i], 0].float() + step[i]).to(b.k.dtype)
    assert_sparse_close(b, b.call(lib))


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", None), ("f32", None), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("block", [16, 32])
def test_garbage_elsewhere(lib, dtype, kv, block):
    """NaN and infinities behind a sequence's end, in blocks not listed and in
    list entries behind the list's length reach nothing."""
    b = sparse_batch(10, dtype, [5, 37, 70, 200], 3, 8, 2, 128, block, kv)
    ref = b.call(lib)
    used = np.zeros((b.k.shape[0], 2, block), bool)
    for i, n in enumerate(b.lens):
        for h in range(2):
            for lb in b.lists[i, h, :b.counts[i, h]]:
                used[b.table[i, lb], h, :min(block, n - lb * block)] = True
            b.lists[i, h, b.counts[i, h]:] = 10 ** 6
    bad = ~torch.from_numpy(used)
    if kv is None:
        b.k[bad], b.v[bad] = float("nan"), float("inf")
    else:
        b.k[bad], b.v[bad] = 0x7F, 0x7F  # NaN in both formats
        free = ~torch.from_numpy(used.any(2))
        sc = torch.from_numpy(b.scales)
        sc[free] = float("nan")
    assert torch.equal(ref, b.call(lib))
    assert lib.pa_get_status() == 0


def test_infinities_that_count(lib):
    """An infinity or a NaN in a listed row reaches its head's output."""
    b = sparse_batch(11, "bf16", [64, 64], 4, 4, 2, 64, 16, ragged=False)
    b.v[b.table[0, 1], 0, 3, 5] = float("inf")
    b.k[b.table[1, 2], 1, 0, 0] = float("nan")
    out = b.call(lib).float().cpu()
    assert not out[0, :2, 5].isfinite().any() and out[0, :2, :5].isfinite().all() and out[0, 2:].isfinite().all()
    assert out[1, 2:].isnan().all() and out[1, :2].isfinite().all()


@pytest.mark.parametrize("exponent", [-120, -60, 0, 60, 100])
def test_scales_of_8bit_blocks(lib, exponent):
    """V scales far from 1 (and a K scale that a small query makes up for)."""
    b = sparse_batch(12, "bf16", [300, 90], 12, 8, 2, 128, 16, "e4m3")
    b.scales[..., 1] *= np.float32(2.0) ** exponent
    b.scales[..., 0] *= np.float32(2.0) ** (exponent // 2)
    b.q = (b.q.float() * 2.0 ** -(exponent // 2)).bfloat16()
    assert_sparse_close(b, b.call(lib))


def test_large_queries_over_8bit(lib):
    b = sparse_batch(13, "bf16", [200], 9, 8, 2, 128, 16, "e4m3")
    b.q = (b.q.float() * 2.0 ** 100).bfloat16()
    b.scale = b.scale * 2.0 ** -100
    assert_sparse_close(b, b.call(lib))


def test_errors(lib):
    def go(**over):
        b = sparse_batch(14, "bf16", [200, 60], 6, 4, 2, 64, 16, ragged=False)
        for name, (at, value) in over.items():
            getattr(b, name)[at] = value
        out = b.call(lib)
        assert torch.cuda.synchronize() is None
        code = lib.pa_get_status()
        assert lib.pa_get_status() == 0
        other = sparse_batch(14, "bf16", [200, 60], 6, 4, 2, 64, 16, ragged=False).call(lib)
        assert torch.equal(out[1], other[1])  # the other sequence
        return code
    assert go(lists=((0, 0, 2), 0)) == -1        # twice the same, or falling
    assert go(lists=((0, 0, 0), -3)) == -1
    assert go(lists=((0, 1, 5), 13)) == -8       # behind the end (200 tokens: blocks 0 .. 12)
    assert go(counts=((0, 0), 7)) == -8
    assert go(counts=((0, 0), -1)) == -8
    assert go(lens=(0, -5)) == -8
    assert go(lens=(0, 10 ** 6)) == -8
    assert go(table=((0, slice(None)), 10 ** 6)) == -7
    assert go(table=((0, slice(None)), -1)) == -7


def test_streams_and_graphs(lib):
    bs = [sparse_batch(20 + i, "bf16", [900, 333], 30, 32, 8, 128, 16) for i in range(3)]
    args = [b.args() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [[lib.pa_decode_sparse(*a, stream=s) for a, s in zip(args, streams)] for _ in range(4)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for b, o in zip(bs, outs[-1]):
        assert_sparse_close(b, o)
    held = [torch.empty_like(a[0]) for a in args]
    graphs = []
    for a, o in zip(args, held):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.pa_decode_sparse(*a, out=o)
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i, o in enumerate(held):
        assert torch.equal(o, outs[0][i])


def test_same_bits_again(lib):
    for kv in (None, "e4m3"):
        b = sparse_batch(30, "bf16", [5000, 700, 2], 200, 64, 8, 128, 16, kv)
        first = b.call(lib)
        for _ in range(5):
            assert torch.equal(first, b.call(lib))


def test_offsets_past_32_bits(lib):
    """Blocks whose rows lie more than 2^32 bytes into the pool."""
    P = (5 << 30) // (8 * 16 * 64 * 2)
    k = torch.zeros(P, 8, 16, 64, dtype=torch.bfloat16, device="cuda")
    b = sparse_batch(31, "bf16", [60, 100], 5, 16, 8, 64, 16)
    n = b.k.shape[0]
    k[-n:] = b.k.cuda()
    q, _, v, table, lens, lists, counts, scale = b.args()
    vv = k.clone()
    vv[-n:] = v
    got = lib.pa_decode_sparse(q, k, vv, table + (P - n), lens, lists, counts, scale)
    assert lib.pa_get_status() == 0
    assert_sparse_close(b, got)

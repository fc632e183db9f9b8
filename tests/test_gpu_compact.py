"""Compaction of the kept path, bit for bit against the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.draft_tree as ot
from tree_helpers import CODEC, DT, paged

pytestmark = pytest.mark.gpu


def case(seed, ctx, nodes, keep, block):
    rng = np.random.default_rng(seed)
    table, P = paged(rng, [c + n for c, n in zip(ctx, nodes)], block)
    width = max(max(keep), 1)
    path = np.full((len(ctx), width), -1, np.int32)
    for i, k in enumerate(keep):
        path[i, :k] = np.sort(rng.choice(nodes[i], k, replace=False))
    return rng, table, P, np.array(ctx, np.int32), path, np.array(keep, np.int32)


CTX = [0, 1, 14, 15, 16, 31, 33, 100, 60, 5]
NODES = [1, 9, 20, 40, 64, 3, 16, 64, 8, 30]
KEEP = [1, 4, 3, 9, 33, 0, 16, 40, 1, 30]


def dev(*xs):
    return [torch.as_tensor(x).cuda() for x in xs]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("hkv,d", [(1, 8), (2, 64), (8, 128), (3, 96)])
@pytest.mark.parametrize("layers", [1, 3])
def test_moves(lib, dtype, block, hkv, d, layers):
    rng, table, P, ctx, path, lens = case(1, CTX, NODES, KEEP, block)
    pools = [torch.from_numpy(rng.standard_normal((P, hkv, block, d)).astype(np.float32)).to(DT[dtype])
             for _ in range(2 * layers)]
    on = [x.cuda() for x in pools]
    lib.pa_compact_tree(on[:layers], on[layers:], *dev(table, ctx, path, lens))
    assert lib.pa_get_status() == 0
    for x, y in zip(pools, on):
        assert torch.equal(y.cpu(), ot.compact_tree(x, ctx, path, lens, table, block))


def test_many_layers(lib):
    """More layers than one launch takes, and a pool tensor as the list."""
    rng, table, P, ctx, path, lens = case(2, CTX, NODES, KEEP, 16)
    L = 150
    k = torch.from_numpy(rng.standard_normal((L, P, 1, 16, 8)).astype(np.float32))
    v = torch.from_numpy(rng.standard_normal((L, P, 1, 16, 8)).astype(np.float32))
    kd, vd = k.cuda(), v.cuda()
    lib.pa_compact_tree(kd, vd, *dev(table, ctx, path, lens))
    assert lib.pa_get_status() == 0
    for i in range(L):
        assert torch.equal(kd[i].cpu(), ot.compact_tree(k[i], ctx, path, lens, table, 16))
        assert torch.equal(vd[i].cpu(), ot.compact_tree(v[i], ctx, path, lens, table, 16))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 128)])
@pytest.mark.parametrize("scales", ["mixed", "equal", "zeros"])
def test_moves_8bit(lib, fmt, block, hkv, d, scales):
    rng, table, P, ctx, path, lens = case(3, CTX, NODES, KEEP, block)
    decode, encode = CODEC[fmt]
    layers = 2
    fine = np.arange(256, dtype=np.uint8)
    fine = fine[np.isfinite(decode(fine))]
    codes = [rng.choice(fine, size=(P, hkv, block, d)) for _ in range(2 * layers)]
    sc = [np.exp2(rng.uniform(-6, 3, (P, hkv, 2))).astype(np.float32) for _ in range(layers)]
    if scales == "equal":
        sc = [np.full((P, hkv, 2), 0.37, np.float32) for _ in range(layers)]
    if scales == "zeros":  # a block that was never written, or only with zeros, holds zero codes
        for i, s in enumerate(sc):
            s[rng.random(s.shape) < 0.4] = 0
            for w in range(2):
                codes[i + w * layers][s[..., w] == 0] = 0
    on = dev(*codes)
    onsc = dev(*sc)
    call = lib.pa_compact_tree_fp8 if fmt == "e4m3" else lib.pa_compact_tree_e5m2
    call(on[:layers], on[layers:], onsc, *dev(table, ctx, path, lens))
    assert lib.pa_get_status() == 0
    for i in range(layers):
        for w in range(2):
            ref, rs = ot.compact_tree_8bit(codes[i + w * layers], sc[i][..., w], decode, encode, ctx, path, lens,
                                           table, block)
            assert np.array_equal(onsc[i].cpu().numpy()[..., w], rs)
            # Rows that hold tokens: below ctx + kept; all other blocks whole.
            assert np.array_equal(on[i + w * layers].cpu().numpy(), ref)


def test_longest_path(lib):
    for fmt in (None, "e4m3"):
        rng, table, P, ctx, path, lens = case(4, [7, 40], [1024, 1024], [1024, 600], 16)
        if fmt is None:
            x = torch.from_numpy(rng.standard_normal((P, 2, 16, 64)).astype(np.float32))
            k, v = x.cuda(), x.cuda()
            lib.pa_compact_tree([k], [v], *dev(table, ctx, path, lens))
            assert torch.equal(k.cpu(), ot.compact_tree(x, ctx, path, lens, table, 16)) and torch.equal(k, v)
        else:
            c = rng.integers(0, 0x7E, (P, 2, 16, 64)).astype(np.uint8)
            s = np.exp2(rng.uniform(-2, 2, (P, 2, 2))).astype(np.float32)
            k, v, sc = dev(c, c, s)
            v = v.clone()
            lib.pa_compact_tree_fp8([k], [v], [sc], *dev(table, ctx, path, lens))
            ref, rs = ot.compact_tree_8bit(c, s[..., 0], *CODEC[fmt], ctx, path, lens, table, 16)
            assert np.array_equal(k.cpu().numpy(), ref) and np.array_equal(sc.cpu().numpy()[..., 0], rs)
        assert lib.pa_get_status() == 0


def test_refused_sequences_are_left_alone(lib):
    for fp8 in (False, True):
        rng, table, P, ctx, path, lens = case(5, [20, 30, 40], [9, 9, 9], [4, 5, 3], 16)
        path[:, 0] += 1
        path = np.maximum.accumulate(path + np.arange(path.shape[1]), 1).astype(np.int32)

        def run(tb=table, cx=ctx, pt=path, ln=lens):
            dt = torch.uint8 if fp8 else torch.float32
            base = torch.arange(P * 2 * 16 * 64).reshape(P, 2, 16, 64)
            k = (base % 120).to(dt).cuda()
            sc = torch.ones(P, 2, 2, device="cuda")
            v = k.clone()
            if fp8:
                lib.pa_compact_tree_fp8([k], [v], [sc], *dev(tb, cx, pt, ln))
            else:
                lib.pa_compact_tree([k], [v], *dev(tb, cx, pt, ln))
            assert torch.equal(k, v)
            return k.cpu(), lib.pa_get_status()

        good, st = run()
        assert st == 0
        mine = set(table[1, :3].tolist())
        rest = [i for i in range(P) if i not in mine]

        def bad(expect, **kw):
            got, st = run(**kw)
            assert st == expect
            assert torch.equal(got[rest], good[rest])

        def edit(x, at, val):
            y = x.copy()
            y[at] = val
            return y

        bad(-8, cx=edit(ctx, 1, -1))
        bad(-8, cx=edit(ctx, 1, table.shape[1] * 16 - 2))
        bad(-8, cx=edit(ctx, 1, 2 ** 31 - 1))
        bad(-8, ln=edit(lens, 1, path.shape[1] + 1))
        bad(-8, ln=edit(lens, 1, -1))
        bad(-1, pt=edit(path, (1, 2), path[1, 1]))  # the same node twice
        bad(-1, pt=edit(path, (1, 0), -1))
        bad(-8, pt=edit(path, (1, 4), 10 ** 6))
        bad(-7, tb=edit(table, (1, 2), P))
        bad(-7, tb=edit(table, (1, 2), -5))


def test_captured_and_replayed(lib):
    rng, table, P, ctx, path, lens = case(6, CTX, NODES, KEEP, 16)
    x = torch.from_numpy(rng.standard_normal((P, 2, 16, 64)).astype(np.float32)).to(torch.bfloat16)
    k, v = x.cuda(), x.cuda()
    args = dev(table, ctx, path, lens)
    none = torch.zeros_like(args[3])
    lib.pa_compact_tree([k], [v], args[0], args[1], args[2], none)  # nothing moves
    assert torch.equal(k.cpu(), x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.pa_compact_tree([k], [v], *args)
    k.copy_(x), v.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    ref = ot.compact_tree(x, ctx, path, lens, table, 16)
    assert torch.equal(k.cpu(), ref) and torch.equal(v.cpu(), ref)


def test_pools_beyond_32_bits(lib):
    """Rows at byte offsets beyond 2^32 of their pools."""
    rng, table, P0, ctx, path, lens = case(8, CTX, NODES, KEEP, 16)
    hkv, d = 8, 128
    P = (5 << 30) // (hkv * 16 * d * 2)
    far = P - P0
    small = [torch.from_numpy(rng.standard_normal((P0, hkv, 16, d)).astype(np.float32)).bfloat16() for _ in range(2)]
    pools = [torch.zeros(P, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, y in zip(small, pools):
        y[far:] = x.cuda()
    lib.pa_compact_tree(pools[:1], pools[1:], *dev(table + far, ctx, path, lens))
    assert lib.pa_get_status() == 0
    for x, y in zip(small, pools):
        assert torch.equal(y[far:].cpu(), ot.compact_tree(x, ctx, path, lens, table, 16))
        assert not y[:far].any()


def test_on_another_stream(lib):
    """The call runs behind what its stream holds, not beside it."""
    rng, table, P, ctx, path, lens = case(9, CTX, NODES, KEEP, 16)
    first = torch.from_numpy(rng.standard_normal((2, P, 2, 16, 64)).astype(np.float32))
    on, src = torch.zeros(first.shape, device="cuda"), first.cuda()
    args = dev(table, ctx, path, lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        on.copy_(src)
    lib.pa_compact_tree(on[:1], on[1:], *args, stream=s)
    torch.cuda.synchronize()
    assert lib.pa_get_status() == 0
    for x, y in zip(first, on):
        assert torch.equal(y.cpu(), ot.compact_tree(x, ctx, path, lens, table, 16))

"""Tree attention over the paged cache against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tree_helpers import assert_tree_close, tree_batch

pytestmark = pytest.mark.gpu


def run(lib, b, what="", **over):
    got = b.call(lib, **over)
    status = lib.pa_get_status()
    assert status == 0, lib.pa_strerror(status)
    assert_tree_close(b, got, what)
    return got


SHAPES = [
    # dtype, kv, hq, hkv, d, block
    ("f32", None, 2, 1, 64, 16),
    ("f32", None, 12, 4, 96, 32),
    ("f32", None, 4, 4, 256, 16),
    ("f32", None, 80, 2, 32, 16),
    ("bf16", None, 32, 8, 128, 16),
    ("bf16", None, 64, 8, 128, 32),
    ("f16", None, 8, 8, 64, 16),
    ("f16", None, 28, 4, 128, 32),   # group 7: a tile's last rows are unused
    ("bf16", None, 40, 2, 64, 32),   # group 20
    ("bf16", None, 128, 1, 128, 16),  # group 128: one node a tile
    ("bf16", "e4m3", 32, 8, 128, 16),
    ("f16", "e4m3", 14, 2, 128, 32),
    ("f16", "e5m2", 32, 4, 128, 16),
    ("bf16", "e5m2", 8, 8, 128, 32),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_ragged_batch(lib, shape):
    dtype, kv, hq, hkv, d, block = shape
    # Contexts and trees that end inside, at and behind tiles and blocks; no context; one node.
    ctx = [0, 1, 15, 16, 63, 64, 100, 127, 128, 200, 500]
    nodes = [1, 7, 1, 16, 1, 2, 33, 5, 64, 3, 17]
    b = tree_batch(1, dtype, ctx, nodes, hq, hkv, d, block, kv)
    run(lib, b, str(shape))


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("dtype,kv,d", [("bf16", None, 128), ("f32", None, 64), ("f16", "e4m3", 128)])
def test_tree_shapes(lib, kind, dtype, kv, d):
    b = tree_batch(2, dtype, [70, 3, 129], [40, 31, 90], 8, 2, d, 16, kv, kind)
    run(lib, b, kind)


@pytest.mark.parametrize("nodes", [130, 257, 1024])
def test_large_trees(lib, nodes):
    run(lib, tree_batch(3, "bf16", [50], [nodes], 4, 2, 64, 16), "wide")


def test_largest_chain(lib):
    run(lib, tree_batch(4, "f16", [9], [1024], 2, 2, 64, 32, kind="chain"), "chain")


@pytest.mark.parametrize("dtype,kv,d", [("bf16", None, 128), ("f16", None, 64), ("f32", None, 128),
                                        ("bf16", "e4m3", 128), ("f16", "e5m2", 128)])
def test_long_context_split_over_the_machine(lib, dtype, kv, d):
    run(lib, tree_batch(5, dtype, [9000, 20], [6, 2], 8, 2, d, 16, kv), "long")


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f32", None), ("bf16", "e4m3")])
def test_many_sequences(lib, dtype, kv):
    rng = np.random.default_rng(6)
    n = 700
    run(lib, tree_batch(6, dtype, rng.integers(0, 90, n), rng.integers(0, 6, n), 4, 2, 128, 16, kv), "many")


def test_sequences_without_nodes(lib):
    b = tree_batch(7, "bf16", [40, 30, 20, 10, 5], [0, 5, 0, 0, 3], 8, 2, 128)
    run(lib, b)
    e = tree_batch(7, "bf16", [40, 30], [0, 0], 8, 2, 128)
    assert e.call(lib).shape == (0, 8, 128)


def test_chain_equals_causal_chunk(lib):
    """A chain is a causal chunk: the chunked-prefill call is within both
    kernels' roundings of the tree call."""
    b = tree_batch(8, "bf16", [300, 17], [20, 9], 32, 8, 128, kind="chain")
    got = run(lib, b)
    a = b.device()
    other = lib.pa_chunked_prefill(a["q"], a["cu_q_lens"], a["k_cache"], a["v_cache"], a["block_tables"],
                                   a["ctx_lens"], a["max_q_len"], a["max_kv_len"], b.scale)
    assert_tree_close(b, other, "chunk")
    assert (got.float() - other.float()).abs().max() < 0.02


def _masked_garbage(b, value, which="kv"):
    """Fill every row that no node may read: the positions behind each
    sequence's tree in its last block, and spare blocks."""
    P, _, B, _ = b.k.shape
    used = np.zeros((P, B), bool)
    for i, (c, n) in enumerate(zip(b.ctx, b.counts)):
        for pos in range(int(c) + int(n)):
            used[b.table[i, pos // B], pos % B] = True
    blk, off = np.nonzero(~used)
    for x in (b.k, b.v):
        x[blk, :, off] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_behind_the_tree_do_not_matter(lib, dtype, value):
    b = tree_batch(9, dtype, [0, 3, 60, 63, 100], [2, 5, 4, 9, 40], 8, 2, 64)
    _masked_garbage(b, value)
    run(lib, b)


@pytest.mark.parametrize("kv,code", [("e4m3", 0x7F), ("e5m2", 0x7D), ("e5m2", 0x7C)])
def test_codes_behind_the_tree_do_not_matter(lib, kv, code):
    b = tree_batch(9, "bf16", [0, 3, 60, 63, 100], [2, 5, 4, 9, 40], 8, 2, 128, kv=kv)
    _masked_garbage(b, code)
    run(lib, b)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "one value"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ctx", [50, 5000])
def test_other_branches_do_not_matter(lib, dtype, where, value, ctx):
    """A node whose K or V is not finite reaches its own subtree and no other
    row: those are as if it held zeros, and rows below it are not finite where
    the definition says so."""
    nodes = 70
    b = tree_batch(10, dtype, [ctx, 20], [nodes, 8], 8, 2, 128)
    bad = [3, 40]
    below = [j for j in range(nodes) if set(bad) & set(_up(b.parents[:nodes], j))]
    at = [(b.table[0, (ctx + j) // 16], (ctx + j) % 16) for j in bad]
    clean = b.call(lib).clone()
    for blk, off in at:
        if where == "k":
            b.k[blk, :, off] = value
        elif where == "v":
            b.v[blk, :, off] = value
        else:
            b.v[blk, 1, off, 77] = value
    got = b.call(lib)
    assert lib.pa_get_status() == 0
    others = [j for j in range(nodes) if j not in below] + list(range(nodes, nodes + 8))
    assert torch.equal(got[others], clean[others])
    if where != "k":
        ref = b.oracle()[0][below]
        fine = np.isfinite(ref)
        g = got[below].double().cpu().numpy()
        assert (np.isfinite(g) == fine).all()
        assert np.array_equal(np.isnan(g), np.isnan(ref))
        assert np.array_equal(g[~fine & ~np.isnan(g)], ref[~fine & ~np.isnan(ref)])


def _up(parents, j):
    out = []
    while j >= 0:
        out.append(j)
        j = int(parents[j])
    return out


def test_scores_of_the_lowest_value(lib):
    """Keys whose scores are all far below zero still weigh 1 together."""
    b = tree_batch(11, "bf16", [0, 40], [3, 5], 4, 1, 64)
    b.q[:] = 0
    b.q[..., 0] = 200.0
    b.k[..., 0] = -200.0
    run(lib, b)


def test_steep_scores(lib):
    """Running maxima that rise from tile to tile."""
    b = tree_batch(12, "f32", [700], [9], 4, 2, 64, q_scale=6.0)
    run(lib, b)
    b = tree_batch(12, "bf16", [700, 3000], [9, 4], 4, 2, 64, q_scale=6.0)
    run(lib, b)


def test_results_repeat_and_ignore_the_neighbours(lib):
    b = tree_batch(13, "bf16", [800, 33, 470], [12, 8, 30], 32, 8, 128)
    first = b.call(lib)
    for _ in range(3):
        assert torch.equal(b.call(lib), first)


def test_captured_and_replayed(lib):
    b = tree_batch(14, "bf16", [800, 33, 470], [12, 8, 30], 16, 4, 128)
    a = b.device()
    out = torch.empty_like(a["q"])
    ws = torch.empty(lib.pa_decode_tree_workspace_size(3, 16, 4, 128, 16, 50, 64, 2000), dtype=torch.uint8,
                     device="cuda")
    a.update(max_q_len=64, max_kv_len=2000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.pa_decode_tree(**a, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.pa_decode_tree(**a, out=out, workspace=ws)
    # Other lengths and another tree within the same bounds.
    b2 = tree_batch(15, "bf16", [310, 900, 64], [20, 12, 18], 16, 4, 128)
    a2 = b2.device()
    P = a["k_cache"].shape[0]
    b2.table = b2.table % P
    for name in ("q", "cu_q_lens", "parents", "ctx_lens"):
        a[name].copy_(a2[name])
    a["block_tables"].zero_()
    w = min(a["block_tables"].shape[1], b2.table.shape[1])
    a["block_tables"][:, :w] = torch.from_numpy(b2.table[:, :w]).cuda()
    b2.table = a["block_tables"].cpu().numpy()
    b2.ctx = np.minimum(b2.ctx, w * 16 - 20).astype(np.int32)
    a["ctx_lens"].copy_(torch.from_numpy(b2.ctx))
    b2.k, b2.v = b.k, b.v
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert lib.pa_get_status() == 0
    assert_tree_close(b2, out)


def test_two_streams(lib):
    bs = [tree_batch(20 + i, "bf16", [500 * (i + 1), 44], [9, 30], 16, 4, 128) for i in range(2)]
    args = [b.device() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append([lib.pa_decode_tree(**a, stream=s) for a, s in zip(args, streams)])
    torch.cuda.synchronize()
    for pair in outs:
        for b, o in zip(bs, pair):
            assert_tree_close(b, o)


def test_sequences_beyond_the_bounds(lib):
    """A sequence beyond the given bounds is reported and left alone."""
    b = tree_batch(16, "bf16", [100, 50, 20], [4, 9, 3], 8, 2, 128)
    a = b.device()
    out = torch.full_like(a["q"], 7.0)
    a["max_q_len"] = 8
    lib.pa_decode_tree(**a, out=out)
    assert lib.pa_get_status() == -8
    assert (out[4:13] == 7.0).all()
    ref = b.call(lib)
    assert torch.equal(out[:4], ref[:4]) and torch.equal(out[13:], ref[13:])
    a["max_q_len"], a["max_kv_len"] = 9, 100
    lib.pa_decode_tree(**a, out=out.fill_(7.0))
    assert lib.pa_get_status() == -8
    assert (out[:4] == 7.0).all() and torch.equal(out[4:], ref[4:])
    for ctx in (-1, 2 ** 31 - 1):
        a = b.device()
        a["ctx_lens"][1] = ctx
        lib.pa_decode_tree(**a, out=out.fill_(7.0))
        assert lib.pa_get_status() == -8
        assert (out[4:13] == 7.0).all() and torch.equal(out[:4], ref[:4])
    a = b.device()
    a["cu_q_lens"][2] = 2  # falls
    lib.pa_decode_tree(**a, out=out)
    assert lib.pa_get_status() == -8
    a = b.device()
    a["cu_q_lens"][3] = 99
    lib.pa_decode_tree(**a, out=out)
    assert lib.pa_get_status() == -8


def test_bad_parents_and_blocks(lib):
    for dtype in ("bf16", "f32"):
        b = tree_batch(17, dtype, [100, 50], [9, 9], 8, 2, 128)
        a = b.device()
        ref = lib.pa_decode_tree(**a)
        for up in (5, 9, 10 ** 6, -2):
            a = b.device()
            a["parents"][4] = up
            got = lib.pa_decode_tree(**a)
            assert lib.pa_get_status() == -1
            assert torch.equal(got[9:], ref[9:])
        for blk in (-1, a["k_cache"].shape[0], 2 ** 30):
            a = b.device()
            a["block_tables"][0, 2] = blk
            got = lib.pa_decode_tree(**a)
            assert lib.pa_get_status() == -7
            assert torch.equal(got[9:], ref[9:])


def test_binding_refuses(lib):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    good = dict(q=z(4, 8, 128), cu_q_lens=z(2, dt=i32), parents=z(4, dt=i32), k_cache=z(3, 2, 16, 128),
                v_cache=z(3, 2, 16, 128), block_tables=z(1, 3, dt=i32), ctx_lens=z(1, dt=i32), max_q_len=4,
                max_kv_len=20, scale=0.1)
    for name, bad in (("parents", z(5, dt=i32)), ("cu_q_lens", z(3, dt=i32)), ("v_cache", z(3, 2, 16, 64)),
                      ("k_cache", z(3, 2, 16, 64)), ("ctx_lens", z(2, dt=i32)), ("out", z(3, 8, 128)),
                      ("q", z(8, 4, 128).transpose(0, 1)), ("k_cache", z(3, 16, 2, 128).transpose(1, 2)),
                      ("workspace", z(4096, 2)[:, 0])):
        with pytest.raises(ValueError, match=name):
            lib.pa_decode_tree(**dict(good, **{name: bad}))
    for name, bad in (("q", z(4, 8, 128, dt=torch.float64)), ("parents", z(4, dt=torch.int64)),
                      ("k_cache", z(3, 2, 16, 128, dt=torch.float16)), ("ctx_lens", torch.zeros(1, dtype=i32))):
        with pytest.raises(TypeError, match=name):
            lib.pa_decode_tree(**dict(good, **{name: bad}))
    with pytest.raises(lib.PagedAttnError):
        lib.pa_decode_tree(**dict(good, workspace=z(16, dt=torch.uint8)))
    pool, odd = z(3, 2, 16, 64), z(3, 2, 16, 128)
    tail = (z(1, 3, dt=i32), z(1, dt=i32), z(1, 4, dt=i32), z(1, dt=i32))
    for k, v in (([pool, odd], [pool, pool]), ([pool, pool], [pool, pool.float()]), ([odd[..., :64]], [pool])):
        with pytest.raises((ValueError, TypeError), match="_caches"):
            lib.pa_compact_tree(k, v, *tail)


def test_memory_of_another_stream(lib):
    """Outputs and workspaces made for another stream do not take memory that
    the current stream still has to read."""
    b = tree_batch(23, "bf16", [500, 44], [9, 30], 16, 4, 128)
    a = b.device()
    s = torch.cuda.Stream()
    ws = lib.pa_decode_tree_workspace_size(2, 16, 4, 128, 16, 39, a["max_q_len"], a["max_kv_len"])
    torch.cuda.synchronize()
    old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (ws, a["q"].nbytes)]
    torch.cuda._sleep(50_000_000)
    kept = [x.clone() for x in old]
    del old
    out = lib.pa_decode_tree(**a, stream=s)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in kept)
    assert_tree_close(b, out)


def test_two_graphs_on_two_streams(lib):
    """Captured calls with workspaces of their own, replayed side by side."""
    bs = [tree_batch(25 + i, dt, [700 * (i + 1), 44], [9, 30], 16, 4, 128) for i, dt in enumerate(("bf16", "f32"))]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in bs]
    for b in bs:
        a = b.device()
        b.call(lib)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lib.pa_decode_tree(**a))
        graphs.append((g, a))
    for _ in range(5):
        for (g, _a), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for b, o in zip(bs, outs):
        assert_tree_close(b, o)


@pytest.mark.parametrize("hkv", [1, 3, 4])
@pytest.mark.parametrize("nodes", [[40, 70, 33, 1, 100], [17] * 40])
@pytest.mark.parametrize("kv", [None, "e4m3"])
def test_several_query_tiles(lib, hkv, nodes, kv):
    """Even and odd numbers of query tiles and of KV heads, long and short
    trees in one batch."""
    run(lib, tree_batch(27, "bf16", [300 + 37 * i for i in range(len(nodes))], nodes, 8 * hkv, hkv, 128, kv=kv))


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("power", [-100, -118, 60])
def test_extreme_value_scales(lib, kv, power):
    """V scales near the ends of fp32: outputs scale with them."""
    b = tree_batch(29, "bf16", [200, 5, 900], [5, 9, 1], 8, 2, 128, kv=kv)
    ref = b.call(lib)
    b.scales[..., 1] *= 2.0 ** power
    got = b.call(lib)
    assert lib.pa_get_status() == 0
    # A power of two: the same sums. (fp32 loses bits below 2^-126.)
    want = ref.double() * 2.0 ** power
    assert torch.allclose(got.double(), want, rtol=2.0 ** -7, atol=2.0 ** -133)


def test_pools_beyond_32_bits(lib):
    """Blocks at element offsets beyond 2^31 (and byte offsets beyond 2^32)."""
    for dtype, d, hkv, need in (("bf16", 128, 8, 5 << 30), ("f32", 256, 8, 9 << 30)):
        b = tree_batch(31, dtype, [200, 5, 70], [5, 9, 40], 16, hkv, d)
        a = b.device()
        P0 = b.k.shape[0]
        P = (need // b.k.element_size()) // (hkv * 16 * d)
        far = P - P0
        for name in ("k_cache", "v_cache"):
            pool = torch.zeros(P, hkv, 16, d, dtype=b.k.dtype, device="cuda")
            pool[far:] = a[name]
            a[name] = pool
        a["block_tables"] = a["block_tables"] + far
        out = lib.pa_decode_tree(**a)
        assert lib.pa_get_status() == 0
        assert_tree_close(b, out, dtype)
        a.clear()
        del pool, out
        torch.cuda.empty_cache()


def _with_a_hidden_block(seed, nodes, first, size):
    """Parents of a tree whose nodes first .. first + size - 1 are leaves: no
    other node sees them."""
    rng = np.random.default_rng(seed)
    out = [-1]
    for j in range(1, nodes):
        ok = [a for a in range(max(0, j - 30), j) if not first <= a < first + size]
        out.append(int(rng.choice(ok or [0])))
    return out


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), 2.0 ** 22, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("ctx", [32, 5024])
@pytest.mark.parametrize("block", [16, 32])
def test_scales_of_other_branches_do_not_matter(lib, kv, scale, which, ctx, block):
    """The scale of a block that holds nodes of other branches alone reaches
    no row of the others, whatever it is."""
    nodes, first = 100, 32
    b = tree_batch(33, "bf16", [ctx, 20], [nodes, 8], 8, 2, 128, block, kv=kv)
    b.parents[:nodes] = _with_a_hidden_block(34, nodes, first, block)
    clean = b.call(lib).clone()
    w = "kv".index(which)
    b.scales[b.table[0, (ctx + first) // block], :, w] *= np.float32(scale)
    got = b.call(lib)
    assert lib.pa_get_status() == 0
    others = [j for j in range(nodes + 8) if not first <= j < first + block]
    assert torch.equal(got[others], clean[others])
    if w and np.isfinite(scale):
        assert_tree_close(b, got)


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
def test_a_drafted_infinity_stays_in_its_block(lib, kv):
    """The cache write gives the block of a V row that is not finite the scale
    infinity: rows that see nothing of the block are as without it."""
    nodes, ctx, first = 100, 32, 32
    b = tree_batch(35, "bf16", [ctx], [nodes], 8, 2, 128, kv=kv)
    b.parents[:] = _with_a_hidden_block(36, nodes, first, 16)
    rng = np.random.default_rng(37)
    k, v = (torch.from_numpy(rng.standard_normal((nodes, 2, 128)).astype(np.float32)).bfloat16() for _ in range(2))
    pos = ctx + np.arange(nodes)
    slots = torch.from_numpy(b.table[0, pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
    form = {"e4m3": "fp8", "e5m2": "e5m2"}[kv]
    outs = []
    for value in (1.0, float("inf")):
        a = b.device()
        v[first + 8] = value
        getattr(lib, f"pa_reshape_and_cache_{form}")(k.cuda(), v.cuda(), slots, a["k_cache"], a["v_cache"],
                                                     a["kv_scales"])
        outs.append(getattr(lib, f"pa_decode_tree_{form}")(**a))
    assert lib.pa_get_status() == 0
    others = [j for j in range(nodes) if not first <= j < first + 16]
    assert torch.equal(outs[0][others], outs[1][others])
    assert not torch.isfinite(outs[1][first + 8].float()).any()


@pytest.mark.parametrize("kv,code", [("e4m3", 0x7F), ("e4m3", 0xFF), ("e5m2", 0x7C), ("e5m2", 0xFC), ("e5m2", 0x7D)])
@pytest.mark.parametrize("where", ["k", "v", "one value"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ctx", [50, 5000])
def test_codes_of_other_branches_do_not_matter(lib, kv, code, where, dtype, ctx):
    """8-bit codes that are not finite in nodes of a tree: rows that do not see
    them are as without them, the others are what the definition says."""
    nodes = 70
    b = tree_batch(10, dtype, [ctx, 20], [nodes, 8], 8, 2, 128, kv=kv)
    bad = [3, 40]
    below = [j for j in range(nodes) if set(bad) & set(_up(b.parents[:nodes], j))]
    clean = b.call(lib).clone()
    for blk, off in [(b.table[0, (ctx + j) // 16], (ctx + j) % 16) for j in bad]:
        if where == "k":
            b.k[blk, :, off] = code
        elif where == "v":
            b.v[blk, :, off] = code
        else:
            b.v[blk, 1, off, 77] = code
    got = b.call(lib)
    assert lib.pa_get_status() == 0
    others = [j for j in range(nodes) if j not in below] + list(range(nodes, nodes + 8))
    assert torch.equal(got[others], clean[others])
    if where == "k":  # (128 infinite products of both signs are NaN too)
        assert torch.isnan(got[below]).all()
        return
    ref = b.oracle()[0][below]
    fine = np.isfinite(ref)
    g = got[below].double().cpu().numpy()
    assert (np.isfinite(g) == fine).all()
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    assert np.array_equal(g[~fine & ~np.isnan(g)], ref[~fine & ~np.isnan(ref)])


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f32", None), ("f16", "e5m2"), ("bf16", "e4m3")])
def test_what_the_neighbours_hold_does_not_matter(lib, dtype, kv):
    """Other contents in the neighbours' blocks: the same bits. Other lengths
    and trees beside it, which cut its keys elsewhere: within the tolerance."""
    b = tree_batch(39, dtype, [800, 333, 470], [12, 8, 30], 32, 8, 128, kv=kv)
    first = b.call(lib).clone()
    mine = b.table[1, :-(-341 // 16)]
    mine = mine.astype(np.int64)
    other = np.setdiff1d(np.arange(b.k.shape[0]), mine)
    for x in (b.k, b.v):
        x[other] = x[other[::-1].copy()]
    got = run(lib, b)
    assert torch.equal(got[12:20], first[12:20])
    assert not torch.equal(got[:12], first[:12])
    for ctx, nodes in (([0, 333, 5000], [1, 8, 3]), ([70, 333, 64], [100, 8, 0])):
        c = tree_batch(40, dtype, ctx, nodes, 32, 8, 128, kv=kv)
        at = [nodes[0], nodes[0] + 8]
        c.q[at[0]:at[1]], c.parents[at[0]:at[1]] = b.q[12:20], b.parents[12:20]
        hold = c.table[1, :len(mine)].astype(np.int64)
        c.k[hold], c.v[hold] = b.k[mine], b.v[mine]
        if kv:
            c.scales[hold] = b.scales[mine]
        run(lib, c)


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f32", None), ("bf16", "e4m3")])
@pytest.mark.parametrize("what", ["k", "v"])
def test_not_finite_under_a_small_weight(lib, dtype, kv, what):
    """A NaN that a row sees reaches it from wherever the context is cut, also
    from keys whose weights are 0 in fp32 beside the others'."""
    b = tree_batch(38, dtype, [9000, 20], [6, 2], 8, 2, 128, kv=kv)
    b.q[:6, :, 0] = 40.0
    large = b.table[0, 4000 // 16:5000 // 16].astype(np.int64)  # scores of some 1000
    at, nan = int(b.table[0, 100 // 16]), float("nan")
    if kv is None:
        b.k[large, :, :, 0] = 300.0
    else:
        b.scales[large, :, 0] = 2.0
        b.k[large, :, :, 0], nan = 0x77, 0x7F
    got = b.call(lib)
    assert torch.isfinite(got).all()
    (b.k if what == "k" else b.v)[at, :, 100 % 16, 5] = nan
    got = b.call(lib)
    assert lib.pa_get_status() == 0
    assert torch.isnan(got[:6] if what == "k" else got[:6, :, 5]).all()
    assert torch.isfinite(got[6:]).all()
    if what == "v":
        assert torch.isfinite(torch.cat([got[:6, :, :5], got[:6, :, 6:]], -1)).all()


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_the_default_stream(lib, handle):
    """A call on the default stream, made while another one is current, takes
    no memory that some third stream still has to read."""
    b = tree_batch(41, "bf16", [500, 44], [9, 30], 16, 4, 128)
    a = b.device()
    ws = lib.pa_decode_tree_workspace_size(2, 16, 4, 128, 16, 39, a["max_q_len"], a["max_kv_len"])
    current = torch.cuda.Stream()
    torch.cuda.synchronize()
    # Streams come from a ring of 32: the next one given out is the first again.
    # (A few are enough; with all of them the call would wait for a place on the device.)
    streams = [torch.cuda.Stream() for _ in range(32)][:3]
    for sleep in (0, 50_000_000):  # (the first time for the streams' memory, which takes longer than the sleep)
        kept = []
        for s in streams:
            with torch.cuda.stream(s):
                old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (ws, a["q"].nbytes)]
                torch.cuda._sleep(sleep)
                kept += [x.clone() for x in old]
                del old
    with torch.cuda.stream(current):
        out = lib.pa_decode_tree(**a, stream=0 if handle else torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in kept)
    assert_tree_close(b, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_beyond_32_bits(lib, dtype):
    """A sequence whose last tile would end behind position 2^31 is reported
    and left alone, also under the largest bound."""
    b = tree_batch(42, dtype, [100, 50], [4, 9], 8, 2, 64)
    a = b.device()
    ref = lib.pa_decode_tree(**a).clone()
    a["max_kv_len"] = 2 ** 31 - 1
    wide = torch.zeros(2, 2 ** 27, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = a["block_tables"]
    a["block_tables"] = wide
    out = torch.full_like(ref, 7.0)
    assert_tree_close(b, lib.pa_decode_tree(**a, out=out))
    assert lib.pa_get_status() == 0
    for ctx in (2 ** 31 - 12, 2 ** 31 - 72):
        a["ctx_lens"][1] = ctx
        lib.pa_decode_tree(**a, out=out.fill_(7.0))
        assert lib.pa_get_status() == -8
        assert (out[4:] == 7.0).all() and torch.equal(out[:4], ref[:4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_sequences_outside_the_rows(lib, dtype):
    """A cu_q_lens that leaves [0, total_q] is reported for a sequence without
    nodes too; one inside it is not, whatever its context says."""
    b = tree_batch(43, dtype, [100, 50, 70], [4, 0, 9], 8, 2, 64)
    ref = b.call(lib).clone()
    a = b.device()
    a["ctx_lens"][1] = 10 ** 6
    assert torch.equal(lib.pa_decode_tree(**a), ref)
    assert lib.pa_get_status() == 0
    a = b.device()
    for cu, status in (([0, 4, 13, 13], 0), ([13] * 4, 0), ([14] * 4, -8), ([-1] * 4, -8), ([0, 4, 13, 14], -8)):
        a["cu_q_lens"].copy_(torch.tensor(cu, dtype=torch.int32))
        lib.pa_decode_tree(**a)
        assert lib.pa_get_status() == status, cu

"""Pins of the draft-tree oracle: against the chunked-prefill oracle, sums
over all outcomes, and moves of labelled rows."""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

import oracle
import oracle.draft_tree as ot
from tree_helpers import CODEC, paged, tree_batch


def test_a_chain_is_a_causal_chunk():
    b = tree_batch(1, "f32", [0, 5, 40], [7, 20, 3], 4, 2, 32, kind="chain")
    out = b.oracle()[0]
    ref = oracle.prefill(b.q, b.cu, b.ctx, b.k, b.v, b.table, b.scale, b.block)
    assert np.abs(out - ref).max() < 1e-12


def test_a_node_is_the_end_of_its_chain():
    """Each node's output is that of a decode row whose last positions are
    its ancestors', gathered into blocks of their own."""
    b = tree_batch(2, "f32", [21], [12], 4, 2, 32)
    out = b.oracle()[0]
    for j in range(12):
        up = ot.ancestors(b.parents, j)[::-1]
        pos = list(range(21)) + [21 + a for a in up]
        rows = [(b.table[0, x // 16], x % 16) for x in pos]
        n = -(-len(pos) // 16)
        k, v = (torch.zeros(n, 2, 16, 32) for _ in range(2))
        for i, (blk, off) in enumerate(rows):
            k[i // 16, :, i % 16], v[i // 16, :, i % 16] = b.k[blk, :, off], b.v[blk, :, off]
        ref = oracle.decode(b.q[j:j + 1], k, v, np.arange(n, dtype=np.int32)[None], np.array([len(pos)]), b.scale, 16)
        assert np.abs(out[j] - ref[0]).max() < 1e-12


@pytest.mark.parametrize("children", [1, 2, 3])
@pytest.mark.parametrize("draft", [True, False])
def test_the_first_token_is_distributed_as_the_target(children, draft):
    """Summed over every choice of drafts (weighted by the draft's
    probabilities) and over each child's acceptance, by the rule's
    thresholds: P(first token = y) = p(y). The oracle keeps a child just
    below its threshold and refuses it just above."""
    rng = np.random.default_rng(children)
    V = 4
    p = rng.dirichlet(np.ones(V))
    q = rng.dirichlet(np.ones(V))
    total = np.zeros(V)
    choices = itertools.product(range(V), repeat=children) if draft else [(2, 0, 2)[:children]]
    for drawn in choices:
        weight = np.prod([q[x] for x in drawn]) if draft else 1.0
        w, mass, alive = p.copy(), 1.0, 1.0
        thresholds = []
        for x in drawn:
            keep = min(1.0, w[x] / (mass * (q[x] if draft else 1.0))) if mass > 0 else 0.0
            thresholds.append(keep)
            total[x] += weight * alive * keep
            alive *= 1 - keep
            if draft:
                w = np.maximum(0, w - mass * q)
                mass = w.sum()
            else:
                mass -= w[x]
                w[x] = 0
        if alive > 1e-15 and w.sum() > 0:
            total += weight * alive * w / w.sum()
        rows = [torch.from_numpy(np.tile(x, (1 + children, 1))) for x in (p, q)]
        for k, keep in enumerate(thresholds):
            if any(t >= 1 for t in thresholds[:k]):
                break  # an earlier child is always kept
            for u, kept in ((keep - 1e-9, True), (keep + 1e-9, False)):
                if not 0 <= u < 1:
                    continue
                ua = np.array([0.0, *[min(t + 1e-9, 1.0) for t in thresholds]])
                ua[1 + k] = u
                path, lens, _ = ot.verify_tree(rows[0], rows[1] if draft else None, [0, *drawn], [0, 1 + children],
                                               [-1] + [0] * children, ua, [0.5], 2)
                assert (lens[0] == 2 and path[0, 1] == 1 + k) == kept
    assert np.abs(total - p).max() < 1e-9


def test_sampling_takes_the_first_entry_past_the_threshold():
    p = torch.tensor([[0.0, 0.25, 0.0, 0.5, 0.25, 0.0]])
    for u, y in ((0.0, 1), (0.2499, 1), (0.25, 3), (0.7499, 3), (0.75, 4), (0.9999, 4)):
        assert ot.verify_tree(p, None, [0], [0, 1], [-1], [0.0], [u], 1)[2][0] == y


def test_a_refused_token_is_not_drawn_again():
    p = torch.tensor([[0.6, 0.4, 0.0], [0.0, 0.0, 1.0]])
    path, lens, nxt = ot.verify_tree(p, None, [0, 0], [0, 2], [-1, 0], [0.0, 0.7], [0.0], 2)
    assert lens[0] == 1 and nxt[0] == 1
    path, lens, nxt = ot.verify_tree(p, None, [0, 0], [0, 2], [-1, 0], [0.0, 0.5], [0.9], 2)
    assert lens[0] == 2 and path[0].tolist() == [0, 1] and nxt[0] == 2


def test_compaction_moves_labelled_rows():
    rng = np.random.default_rng(3)
    ctx, nodes = [5, 14, 0], [30, 20, 9]
    table, P = paged(rng, [c + n for c, n in zip(ctx, nodes)], 16)
    pool = np.zeros((P, 1, 16, 1))
    for i in range(3):
        for pos in range(ctx[i] + nodes[i]):
            pool[table[i, pos // 16], 0, pos % 16, 0] = 1000 * (i + 1) + pos
    path = np.array([[0, 3, 12, 29], [2, 5, -1, -1], [0, 1, 8, -1]])
    lens = [4, 2, 3]
    new = ot.compact_tree(pool, ctx, path, lens, table, 16)
    for i in range(3):
        line = [new[table[i, x // 16], 0, x % 16, 0] - 1000 * (i + 1) for x in range(ctx[i] + lens[i])]
        assert line == list(range(ctx[i])) + [ctx[i] + a for a in path[i][:lens[i]]]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_8bit_compaction_keeps_values_within_a_rounding(fmt):
    rng = np.random.default_rng(4)
    decode, encode = CODEC[fmt]
    ctx, nodes, path, lens = [13], [40], np.array([[0, 1, 9, 33]]), [4]
    table, P = paged(rng, [53], 16)
    sc = np.exp2(rng.uniform(-3, 3, (P, 2))).astype(np.float32)
    codes = encode(rng.standard_normal((P, 2, 16, 64)).astype(np.float32) * 50)
    new, ns = ot.compact_tree_8bit(codes, sc, decode, encode, ctx, path, lens, table, 16)
    old_v, new_v = decode(codes) * sc[:, :, None, None], decode(new) * ns[:, :, None, None].astype(float)
    half = 2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3
    tiny = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}[fmt]  # half the smallest code
    for dst, src in [(x, x) for x in range(13)] + [(13 + k, 13 + a) for k, a in enumerate(path[0])]:
        a, b = old_v[table[0, src // 16], :, src % 16], new_v[table[0, dst // 16], :, dst % 16]
        s = ns[table[0, dst // 16]][:, None]
        assert (np.abs(a - b) <= half * np.abs(a) * 1.0001 + tiny * s).all()
        assert (ns[table[0, dst // 16]] >= sc[table[0, src // 16]]).all()

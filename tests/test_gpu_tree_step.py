"""Draft-tree steps as a serving engine runs them: slots, cache writes,
attention in every layer, verification and compaction, step after step, eager
and captured. A token's K/V depends on the token alone here, so after every
step the cache must hold the kept tokens' rows in order."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.draft_tree as ot
from tree_helpers import CODEC, DT, TreeBatch, assert_tree_close, paged, random_parents

pytestmark = pytest.mark.gpu

VOCAB, LAYERS, SEQS, NODES, HQ, HKV, STEPS, BLOCK = 61, 3, 5, 9, 16, 4, 6, 16


class Engine:
    """A stand-in for a model: fixed K/V rows per token and layer, random
    probabilities and trees, and the committed tokens on the host."""

    def __init__(self, lib, seed, dtype, kv, d):
        from paged_kv_cache_14_gb300.step import TreeStep
        self.lib, self.kv, self.d, self.dt = lib, kv, d, DT[dtype]
        self.dtype = dtype
        self.rng = rng = np.random.default_rng(seed)
        self.rows = [torch.from_numpy(rng.standard_normal((2, VOCAB, HKV, d)).astype(np.float32)).to(self.dt)
                     for _ in range(LAYERS)]
        room = 60 + (STEPS + 2) * NODES
        self.table, P = paged(rng, [room] * SEQS, BLOCK)
        self.tokens = [rng.integers(0, VOCAB, n).tolist() for n in (1, 16, 31, 40, 60)]
        self.pool_dt = torch.uint8 if kv else self.dt
        zeros = lambda *s, dt=self.pool_dt: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.k = [zeros(P, HKV, BLOCK, d) for _ in range(LAYERS)]
        self.v = [zeros(P, HKV, BLOCK, d) for _ in range(LAYERS)]
        self.sc = [zeros(P, HKV, 2, dt=torch.float32) for _ in range(LAYERS)] if kv else None
        i32 = lambda *s: zeros(*s, dt=torch.int32)  # noqa: E731
        T = SEQS * NODES
        self.st = TreeStep(k_caches=self.k, v_caches=self.v, kv_scales=self.sc, kv_format=kv or "e4m3",
                           block_tables=torch.from_numpy(self.table).cuda(), ctx_lens=i32(SEQS), cu_q_lens=i32(SEQS + 1),
                           parents=i32(T), draft_tokens=i32(T), new_seq_ids=i32(T), new_positions=i32(T),
                           num_q_heads=HQ, dtype=self.dt, max_q_len=NODES, max_kv_len=room, scale=d ** -0.5)
        self.q = [zeros(T, HQ, d, dt=self.dt) for _ in range(LAYERS)]
        self.kn, self.vn = ([zeros(T, HKV, d, dt=self.dt) for _ in range(LAYERS)] for _ in range(2))
        self.target, self.draft = (zeros(T, VOCAB, dt=torch.float32) for _ in range(2))
        self.ua, self.us = zeros(T, dt=torch.float32), zeros(SEQS, dt=torch.float32)
        self.outs = [zeros(T, HQ, d, dt=self.dt) for _ in range(LAYERS)]
        self.prefill()

    def prefill(self):
        """Cache all committed tokens but the newest (its row is node 0)."""
        for i, toks in enumerate(self.tokens):
            n = len(toks) - 1
            if n == 0:
                continue
            ids = torch.full((n,), i, dtype=torch.int32, device="cuda")
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            slots = self.lib.pa_slot_mapping(self.st.block_tables, ids, pos, BLOCK, self.st.num_blocks)
            for layer in range(LAYERS):
                k, v = (x[toks[:-1]].contiguous().cuda() for x in self.rows[layer])
                if self.kv is None:
                    self.lib.pa_reshape_and_cache(k, v, slots, self.k[layer], self.v[layer])
                else:
                    self.st.call_8bit("pa_reshape_and_cache")(k, v, slots, self.k[layer], self.v[layer], self.sc[layer])

    def draw(self):
        """A step's inputs: trees of 1 .. NODES nodes (rows behind the last
        sequence's are padding), written into the fixed device tensors."""
        rng = self.rng
        counts = rng.integers(1, NODES + 1, SEQS)
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        T = SEQS * NODES
        self.par, self.tok = np.full(T, -1, np.int32), np.zeros(T, np.int32)
        ids, pos = np.zeros(T, np.int32), np.zeros(T, np.int32)
        self.ctx = np.array([len(t) - 1 for t in self.tokens], np.int32)
        for i in range(SEQS):
            lo, hi = self.cu[i], self.cu[i + 1]
            self.par[lo:hi] = random_parents(rng, hi - lo)
            self.tok[lo:hi] = rng.integers(0, VOCAB, hi - lo)
            self.tok[lo] = self.tokens[i][-1]
            ids[lo:hi], pos[lo:hi] = i, self.ctx[i] + np.arange(hi - lo)
        lg = rng.standard_normal((T, VOCAB)).astype(np.float32)
        soft = lambda x: np.exp(x) / np.exp(x).sum(1, keepdims=True)  # noqa: E731
        self.hp, self.hq = soft(lg).astype(np.float32), soft(lg + 0.3 * rng.standard_normal(lg.shape)).astype(np.float32)
        self.hua, self.hus = rng.random(T, dtype=np.float32), rng.random(SEQS, dtype=np.float32)
        # Padding rows write to the first sequence's last block, which holds no token.
        last = self.cu[-1]
        pos[last:] = (self.table.shape[1] - 2) * BLOCK + np.arange(T - last) % BLOCK
        for t, x in ((self.st.ctx_lens, self.ctx), (self.st.cu_q_lens, self.cu), (self.st.parents, self.par),
                     (self.st.draft_tokens, self.tok), (self.st.new_seq_ids, ids), (self.st.new_positions, pos),
                     (self.target, self.hp), (self.draft, self.hq), (self.ua, self.hua), (self.us, self.hus)):
            t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        for layer in range(LAYERS):
            self.kn[layer].copy_(self.rows[layer][0][self.tok])
            self.vn[layer].copy_(self.rows[layer][1][self.tok])
            self.q[layer].copy_(torch.from_numpy(rng.standard_normal((T, HQ, self.d)).astype(np.float32)))

    def run(self):
        st = self.st
        st.slots()
        for layer in range(LAYERS):
            st.write(layer, self.kn[layer], self.vn[layer])
            self.outs[layer].copy_(st.attend(layer, self.q[layer]))
        st.accept(self.target, self.draft, self.ua, self.us)

    def check(self, pools):
        """The attention on the pools as they were before compaction, the
        choice, and the cache after it."""
        live = int(self.cu[-1])
        for layer, (k, v, sc) in enumerate(pools):
            b = TreeBatch(self.dtype, self.kv, self.q[layer][:live].cpu(), k, v, sc, self.table, self.ctx, self.cu,
                          self.par[:live], self.d ** -0.5, BLOCK)
            assert_tree_close(b, self.outs[layer][:live], f"layer {layer}")
        path, lens, nxt = (x.cpu().numpy() for x in (self.st.path, self.st.path_lens, self.st.next_tokens))
        ref = ot.verify_tree(self.hp, self.hq, self.tok, self.cu, self.par, self.hua, self.hus, NODES)
        for g, r in zip((path, lens, nxt), ref):
            assert np.array_equal(g, r)
        for i in range(SEQS):
            kept = [int(self.tok[self.cu[i] + a]) for a in path[i, :lens[i]]]
            self.tokens[i] = self.tokens[i][:-1] + kept + [int(nxt[i])]
            n = len(self.tokens[i]) - 1
            pos = np.arange(n)
            blk, off = self.table[i, pos // BLOCK], pos % BLOCK
            for layer in range(LAYERS):
                for w, pool in enumerate((self.k, self.v)):
                    want = self.rows[layer][w][self.tokens[i][:-1]]
                    got = pool[layer].cpu()[blk, :, off]
                    if self.kv is None:
                        assert torch.equal(got, want)
                        continue
                    # Each rounding is at most half a step of its value and
                    # half the smallest code of the block's scale; a row is
                    # rounded anew when its block's scale grows, a few times
                    # at most (every step's write and move may each do it).
                    dec = CODEC[self.kv][0]
                    s = self.sc[layer].cpu().numpy()[blk, :, w].astype(np.float64)[..., None]
                    val = dec(got.numpy()) * s
                    half, tiny = (2.0 ** -4, 2.0 ** -10) if self.kv == "e4m3" else (2.0 ** -3, 2.0 ** -17)
                    err = np.abs(val - want.double().numpy())
                    times = 2 * (STEPS + 1)
                    assert (err <= ((1 + half) ** times - 1) * np.abs(want.double().numpy()) + times * tiny * s).all()
                    assert np.median(err / (np.abs(want.double().numpy()) + 1e-3)) < half

    def snapshot(self):
        return [(k.cpu().numpy(), v.cpu().numpy(), s.cpu().numpy()) if self.kv else (k.cpu(), v.cpu(), None)
                for k, v, s in zip(self.k, self.v, self.sc or [None] * LAYERS)]


CASES = [("bf16", None, 128), ("f16", None, 64), ("f32", None, 32), ("bf16", "e4m3", 128), ("f16", "e5m2", 128)]


@pytest.mark.parametrize("dtype,kv,d", CASES)
def test_steps(lib, dtype, kv, d):
    e = Engine(lib, 1, dtype, kv, d)
    for _ in range(STEPS):
        e.draw()
        st = e.st
        st.slots()
        for layer in range(LAYERS):
            st.write(layer, e.kn[layer], e.vn[layer])
            e.outs[layer].copy_(st.attend(layer, e.q[layer]))
        pools = e.snapshot()
        st.accept(e.target, e.draft, e.ua, e.us)
        assert lib.pa_get_status() == 0
        e.check(pools)


@pytest.mark.parametrize("dtype,kv,d", CASES[:1] + CASES[3:4])
def test_captured_steps_equal_eager_ones(lib, dtype, kv, d):
    a, b = (Engine(lib, 2, dtype, kv, d) for _ in range(2))
    b.draw()
    a.draw()
    a.run()
    b.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # (records; runs nothing)
        b.run()
    for step in range(STEPS):
        if step:
            for e in (a, b):
                path, lens, nxt = (x.cpu().numpy() for x in (e.st.path, e.st.path_lens, e.st.next_tokens))
                for i in range(SEQS):
                    kept = [int(e.tok[e.cu[i] + j]) for j in path[i, :lens[i]]]
                    e.tokens[i] = e.tokens[i][:-1] + kept + [int(nxt[i])]
                e.draw()
            a.run()
            g.replay()
        torch.cuda.synchronize()
        assert lib.pa_get_status() == 0
        for x, y in zip(a.k + a.v + (a.sc or []), b.k + b.v + (b.sc or [])):
            assert torch.equal(x, y)
        live = int(a.cu[-1])
        for x, y in zip(a.outs, b.outs):
            assert torch.equal(x[:live], y[:live])
        assert torch.equal(a.st.path, b.st.path) and torch.equal(a.st.next_tokens, b.st.next_tokens)

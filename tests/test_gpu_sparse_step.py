"""Steps over long contexts: prompts written in chunks, then decode steps over a
model's layers, each kept equal to the oracle's caches, summaries and choice of
blocks, and its attention within tolerance; eager and captured."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import oracle.sparse as osp
from sparse_helpers import SparseBatch, assert_sparse_close, dev, normal, values
from tree_helpers import DT, paged

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK, KEEP, SINK, RECENT = 8, 2, 128, 16, 6, 1, 2


class Model:
    """The oracle's side: every layer's cache and summaries on the host."""

    def __init__(self, seed, dtype, fmt, layers, lens, room):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.fmt, self.layers = dtype, fmt, layers
        self.table, self.P = paged(self.rng, [x + room for x in lens], BLOCK)
        shape = (self.P, HKV, BLOCK, D)
        dt = DT[dtype] if fmt is None else torch.uint8
        self.k = [torch.zeros(shape, dtype=dt) for _ in range(layers)]
        self.v = [torch.zeros(shape, dtype=dt) for _ in range(layers)]
        self.scales = None if fmt is None else [np.zeros((self.P, HKV, 2), np.float32) for _ in range(layers)]
        self.codes = [np.zeros((self.P, HKV, 2, D), np.int8) for _ in range(layers)]
        self.code_scales = [np.zeros((self.P, HKV), np.float32) for _ in range(layers)]
        self.cs = osp.rope_table(0, 1024, osp.rope_frequencies(D, base=500000.0)).astype(np.float32)
        self.ctx = np.zeros(len(lens), np.int32)

    def tokens(self, counts):
        seq = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
        pos = np.concatenate([np.arange(c, c + n) for c, n in zip(self.ctx, counts)]).astype(np.int32)
        rows = [tuple(normal(self.rng, len(seq), h, D).to(DT[self.dtype]) for h in (HQ, HKV, HKV))
                for _ in range(self.layers)]
        return seq, pos, rows

    def write(self, layer, seq, pos, row, lens):
        q, k, v = row
        slots = np.array([self.table[s, x // BLOCK] * BLOCK + x % BLOCK for s, x in zip(seq, pos)], np.int64)
        kr = osp.rotate(k, self.cs, pos, False)
        if self.fmt is None:
            oracle.reshape_and_cache(torch.from_numpy(kr).to(k.dtype), v, slots, self.k[layer], self.v[layer], BLOCK)
        else:
            osp.cache_write_8bit(self.fmt, kr, v.float().numpy(), slots, self.k[layer].numpy(), self.v[layer].numpy(),
                                 self.scales[layer], BLOCK)
        x = values(self.k[layer], None if self.scales is None else self.scales[layer], 0, self.fmt)
        osp.block_summaries(x, self.table, self.ctx, lens, BLOCK, self.codes[layer], self.code_scales[layer])
        return torch.from_numpy(osp.rotate(q, self.cs, pos, False)).to(q.dtype)

    def attention(self, layer, q, lens):
        lists, counts = osp.select_blocks(q, self.codes[layer], self.code_scales[layer], self.table, lens, BLOCK, KEEP,
                                          SINK, RECENT)
        return SparseBatch(self.dtype, self.fmt, q, self.k[layer], self.v[layer],
                           None if self.scales is None else self.scales[layer], self.table, lens, lists, counts,
                           D ** -0.5, BLOCK)


def make_step(lib, m, tokens, most, decode):
    from paged_kv_cache_14_gb300.step import SparseStep
    n = len(m.ctx)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return SparseStep(k_caches=[x.cuda() for x in m.k] if decode is None else decode.k_caches,
                      v_caches=[x.cuda() for x in m.v] if decode is None else decode.v_caches,
                      kv_scales=None if m.scales is None else
                      [dev(x) for x in m.scales] if decode is None else decode.kv_scales,
                      kv_format=m.fmt or "e4m3", block_tables=dev(m.table), ctx_lens=i32(n), seq_lens=i32(n),
                      new_seq_ids=i32(tokens), new_positions=i32(tokens), cos_sin=dev(m.cs), num_q_heads=HQ,
                      dtype=DT[m.dtype], max_seq_len=1024, max_new_tokens=most, max_list_len=KEEP, scale=D ** -0.5,
                      num_sink=SINK, num_recent=RECENT)


def fill(step, m, seq, pos, lens):
    step.new_seq_ids.copy_(torch.from_numpy(seq))
    step.new_positions.copy_(torch.from_numpy(pos))
    step.ctx_lens.copy_(torch.from_numpy(m.ctx))
    step.seq_lens.copy_(torch.from_numpy(lens))


def same_state(step, m):
    for layer in range(m.layers):
        assert torch.equal(step.k_caches[layer].cpu(), m.k[layer]) and torch.equal(step.v_caches[layer].cpu(), m.v[layer])
        if m.scales is not None:
            assert np.array_equal(step.kv_scales[layer].cpu().numpy(), m.scales[layer])
        assert np.array_equal(step.summaries[layer].cpu().numpy(), m.codes[layer])
        assert np.array_equal(step.summary_scales[layer].cpu().numpy(), m.code_scales[layer])


@pytest.mark.parametrize("dtype,fmt", [("bf16", None), ("f16", None), ("f32", None), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(lib, dtype, fmt, captured):
    prompt = np.array([200, 17, 1, 333, 90], np.int32)
    layers, steps = 3, 6
    m = Model(5, dtype, fmt, layers, prompt.tolist(), steps + 2)
    n = len(prompt)
    # The prompts, in two chunks.
    step = None
    for counts in (prompt // 2 + 1, prompt - prompt // 2):
        seq, pos, rows = m.tokens(counts)
        first = make_step(lib, m, len(seq), int(counts.max()), step)
        if step is not None:
            first.summaries, first.summary_scales = step.summaries, step.summary_scales
        step = first
        lens = (m.ctx + counts).astype(np.int32)
        fill(step, m, seq, pos, lens)
        step.slots()
        for layer in range(layers):
            q = step.write(layer, *(x.cuda() for x in rows[layer]))
            assert torch.equal(q.cpu(), m.write(layer, seq, pos, rows[layer], lens))
        m.ctx = lens
    same_state(step, m)
    # Decode steps.
    last = step
    step = make_step(lib, m, n, 1, last)
    step.summaries, step.summary_scales = last.summaries, last.summary_scales
    inputs = [tuple(torch.zeros(n, h, D, dtype=DT[dtype], device="cuda") for h in (HQ, HKV, HKV)) for _ in range(layers)]
    outs = [torch.zeros(n, HQ, D, dtype=DT[dtype], device="cuda") for _ in range(layers)]

    def body():
        step.slots()
        for layer in range(layers):
            step.write(layer, *inputs[layer])
            outs[layer].copy_(step.attend(layer))

    graph = None
    for k in range(steps):
        seq, pos, rows = m.tokens(np.ones(n, int))
        lens = m.ctx + 1
        fill(step, m, seq, pos, lens)
        for a, b in zip(inputs, rows):
            for x, y in zip(a, b):
                x.copy_(y)
        if captured and graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
        graph.replay() if captured else body()
        assert lib.pa_get_status() == 0
        for layer in range(layers):
            q = m.write(layer, seq, pos, rows[layer], lens)
            assert_sparse_close(m.attention(layer, q, lens), outs[layer], f"step {k}, layer {layer}")
        m.ctx = lens
    same_state(step, m)
    assert np.array_equal(step.block_lists.cpu().numpy(), m.attention(layers - 1, q, lens).lists)


def test_refusals():
    from paged_kv_cache_14_gb300.step import SparseStep
    with pytest.raises(ValueError):
        SparseStep(k_caches=[], v_caches=[], block_tables=None, ctx_lens=None, seq_lens=None, new_seq_ids=None,
                   new_positions=None, cos_sin=None, num_q_heads=1, dtype=None, max_seq_len=1, max_new_tokens=1,
                   max_list_len=1, scale=1.0, kv_format="int8")


def test_sparse_after_other_changes(lib):
    """Blocks copied on write and swapped back have their summaries made again."""
    m = Model(6, "bf16", None, 1, [100], 20)
    seq, pos, rows = m.tokens([100])
    step = make_step(lib, m, 100, 100, None)
    lens = np.array([100], np.int32)
    fill(step, m, seq, pos, lens)
    step.slots()
    step.write(0, *(x.cuda() for x in rows[0]))
    m.write(0, seq, pos, rows[0], lens)
    spare = next(b for b in range(m.P) if b not in m.table[0, :8])
    lib.pa_copy_blocks(step.k_caches[0], step.v_caches[0], [[m.table[0, 3], spare]])
    step.block_tables[0, 3] = spare
    step.summarize(0, step.ctx_lens, 100)
    m.k[0][spare], m.v[0][spare] = m.k[0][m.table[0, 3]], m.v[0][m.table[0, 3]]
    m.table[0, 3] = spare
    osp.block_summaries(values(m.k[0], None, 0, None), m.table, m.ctx, lens, BLOCK, m.codes[0], m.code_scales[0])
    same_state(step, m)
    q = normal(m.rng, 1, HQ, D).bfloat16()
    assert_sparse_close(m.attention(0, q, lens), step.attend(0, q.cuda()))
    assert lib.pa_get_status() == 0


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_offsets_past_32_bits(lib, fmt):
    """A step on the last blocks of pools of more than 2^32 elements, and a choice
    among summaries of more than 2^32 bytes, give what the first blocks give."""
    rng = np.random.default_rng(8)
    hq, hkv, d, n, near = 16, 8, 128, 300, 24
    sfx = "" if fmt is None else "_fp8"
    q, k, v = (normal(rng, n, h, d).bfloat16().cuda() for h in (hq, hkv, hkv))
    cs = lib.pa_rope_table(n, d)
    pos, lens, zero = dev(np.arange(n, dtype=np.int32), np.array([n], np.int32), np.zeros(1, np.int32))
    table = dev(rng.permutation(near)[:(n + 15) // 16].astype(np.int32)[None])
    results = []
    for P in (near, (1 << 32) // (hkv * 16 * d) + 100):
        first = P - near
        shape, dt = (P, hkv, 16, d), torch.bfloat16 if fmt is None else torch.uint8
        kc, vc = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
        sc = () if fmt is None else (torch.zeros(P, hkv, 2, device="cuda"),)
        for x in (kc, vc):
            x[first:] = 0
        t = table + first
        slots = (t[0].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:n].contiguous()
        qr = getattr(lib, "pa_rope_and_cache" + sfx)(q, k, v, pos, slots, cs, kc, vc, *sc)
        codes = torch.zeros(P, hkv, 2, d, dtype=torch.int8, device="cuda")
        scales = torch.zeros(P, hkv, device="cuda")
        getattr(lib, "pa_block_summaries" + sfx)(kc, *sc, t, zero, lens, n, codes, scales)
        last = qr[-1:].contiguous()
        lists, counts = lib.pa_select_blocks(last, codes, scales, t, lens, n, 16, 8)
        out = getattr(lib, "pa_decode_sparse" + sfx)(last, kc, vc, *sc, t, lens, lists, counts, d ** -0.5)
        assert lib.pa_get_status() == 0
        results.append([x[first:].clone() for x in (kc, vc, *sc, codes, scales)] + [qr, lists, counts, out])
        del kc, vc, sc
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][-4].float().isfinite().all() and (results[0][-2] == 8).all()
    codes, scales = results[0][-6:-4]
    P = (1 << 32) // (hkv * 2 * d) + 100
    far_codes = torch.empty(P, hkv, 2, d, dtype=torch.int8, device="cuda")
    far_scales = torch.empty(P, hkv, device="cuda")
    far_codes[P - near:], far_scales[P - near:] = codes, scales
    lists, counts = lib.pa_select_blocks(results[0][-4][-1:].contiguous(), far_codes, far_scales, table + (P - near),
                                         lens, n, 16, 8)
    assert lib.pa_get_status() == 0
    assert torch.equal(lists, results[0][-3]) and torch.equal(counts, results[0][-2])

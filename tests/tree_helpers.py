"""Seeded draft-tree batches and the tolerance of tree attention."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

import oracle.draft_tree as ot
import oracle.fp8_kv as f8

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODEC = {"e4m3": (f8.e4m3_decode, f8.e4m3_encode), "e5m2": (f8.e5m2_decode, f8.e5m2_encode)}
QUANT = {"e4m3": f8.quantize_fresh_blocks, "e5m2": f8.quantize_fresh_blocks_e5m2}


def random_parents(rng, n: int, kind: str = "random") -> list[int]:
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [int(rng.integers(-1, j)) if j else -1 for j in range(n)]
    return [int(rng.integers(max(0, j - 6), j)) if j else -1 for j in range(n)]


def paged(rng, lens, block_size: int, spare: int = 3):
    """(block tables, pool size): every sequence's blocks scattered over the pool."""
    nb = [-(-max(x, 1) // block_size) for x in lens]
    perm = rng.permutation(sum(nb) + spare).astype(np.int32)
    table = np.zeros((len(lens), max(nb) + 1), np.int32)
    at = 0
    for i, k in enumerate(nb):
        table[i, :k] = perm[at:at + k]
        at += k
    return table, sum(nb) + spare


@dataclass
class TreeBatch:
    dtype: str
    kv: str
    q: torch.Tensor
    k: object
    v: object
    scales: np.ndarray | None
    table: np.ndarray
    ctx: np.ndarray
    cu: np.ndarray
    parents: np.ndarray
    scale: float
    block: int

    @property
    def counts(self):
        return np.diff(self.cu)

    def values(self):
        """The pools' stored values (K, V) as the oracle takes them."""
        if self.scales is None:
            return self.k, self.v
        dec = CODEC[self.kv][0]
        return tuple(dec(x) * self.scales[..., w].astype(np.float64)[:, :, None, None]
                     for w, x in ((0, self.k), (1, self.v)))

    def oracle(self):
        k, v = self.values()
        return ot.decode_tree(self.q, self.cu, self.parents, self.ctx, k, v, self.table, self.scale, self.block)

    def device(self, dev="cuda"):
        t = lambda x: torch.as_tensor(x).to(dev)  # noqa: E731
        return dict(q=t(self.q), cu_q_lens=t(self.cu), parents=t(self.parents), k_cache=t(self.k), v_cache=t(self.v),
                    block_tables=t(self.table), ctx_lens=t(self.ctx), max_q_len=max(1, int(self.counts.max())),
                    max_kv_len=max(1, int((self.ctx + self.counts).max())), scale=self.scale,
                    **({} if self.scales is None else {"kv_scales": t(self.scales)}))

    def call(self, lib, **over):
        a = self.device()
        a.update(over)
        name = "pa_decode_tree" + ({"e4m3": "_fp8", "e5m2": "_e5m2"}[self.kv] if self.scales is not None else "")
        return getattr(lib, name)(**a)


def tree_batch(seed, dtype, ctx, nodes, hq, hkv, d, block=16, kv=None, kind="random", q_scale=1.0) -> TreeBatch:
    rng = np.random.default_rng(seed)
    ctx, nodes = np.asarray(ctx, np.int32), list(nodes)
    table, P = paged(rng, [int(a) + b for a, b in zip(ctx, nodes)], block)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    parents = np.array(sum((random_parents(rng, n, kind) for n in nodes), []), np.int32)
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    q = (normal(int(cu[-1]), hq, d) * q_scale).to(DT[dtype])
    k, v, sc = normal(P, hkv, block, d), normal(P, hkv, block, d), None
    if kv is None:
        k, v = k.to(DT[dtype]), v.to(DT[dtype])
    else:
        grow = rng.uniform(0.3, 3.0, size=(P, hkv, 1, 1)).astype(np.float32)
        (k, ks), (v, vs) = QUANT[kv](k.numpy() * grow), QUANT[kv](v.numpy() * grow)
        sc = np.stack([ks, vs], -1).astype(np.float32)
    return TreeBatch(dtype, kv, q, k, v, sc, table, ctx, cu, parents, d ** -0.5, block)


def tree_tolerance(b: TreeBatch, out, weighted, largest):
    """Per output: what the kernel's roundings can add up to.

    The output is rounded once (half a step of its type, relative). Every
    softmax weight is rounded to 16 bits (half a step; fp16 weights below
    2^-14 by at most 2^-25, against a row sum of at least 1), which moves the
    output by at most that share of sum w |v|. A score is a sum of D products
    in fp32, off by at most (D + 8) half steps of sum |q k| (a tensor-core
    adder may cut instead of round: whole steps, 2^-23); the exponential adds
    4 steps; a weight that is off by a share e moves numerator and
    denominator, together 2 e sum w |v|."""
    d = b.q.shape[-1]
    e16 = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[b.dtype]
    ew = 0.0 if b.dtype == "f32" else 2.0 ** -11 if b.kv else e16
    step = 2.0 ** -23
    es = largest[..., None] * (d + 8) * step + 8 * step
    tol = e16 * np.abs(out) + (ew + 2 * es) * weighted + 4 * step * np.abs(out)
    if b.dtype == "f16" or b.kv:
        n = int((b.ctx + b.counts).max())
        k, v = b.values()
        tol = tol + n * 2.0 ** -25 * float(np.nanmax(np.abs(v.double().numpy() if hasattr(v, "double") else v)))
    return tol * 1.05 + 1e-30


def assert_tree_close(b: TreeBatch, got: torch.Tensor, what: str = ""):
    out, weighted, largest = b.oracle()
    g = got.detach().double().cpu().numpy()
    assert g.shape == out.shape
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - out) / tree_tolerance(b, out, weighted, largest)
    assert over.max() <= 1.0, f"{what}: {over.max():.2f} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"

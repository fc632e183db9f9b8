"""Seeded batches of the long-context calls and the tolerance of sparse attention."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

import oracle.sparse as osp
from tree_helpers import CODEC, DT, QUANT, paged

SUFFIX = {None: "", "e4m3": "_fp8", "e5m2": "_e5m2"}


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))


def dev(*xs):
    out = [torch.as_tensor(x).cuda() for x in xs]
    return out[0] if len(out) == 1 else out


def pools(rng, P, hkv, block, d, dtype, kv=None):
    """(K, V, scales): tensors of the type, or codes and scales of an 8-bit cache."""
    k, v = normal(rng, P, hkv, block, d), normal(rng, P, hkv, block, d)
    if kv is None:
        return k.to(DT[dtype]), v.to(DT[dtype]), None
    grow = rng.uniform(0.3, 3.0, size=(P, hkv, 1, 1)).astype(np.float32)
    (k, ks), (v, vs) = QUANT[kv](k.numpy() * grow), QUANT[kv](v.numpy() * grow)
    return torch.from_numpy(k), torch.from_numpy(v), np.stack([ks, vs], -1).astype(np.float32)


def values(k, scales, which, kv):
    """An 8-bit pool's values as the library defines them: code times scale, in fp32."""
    if kv is None:
        return k.float().numpy()
    return CODEC[kv][0](k.numpy()).astype(np.float32) * scales[..., which][:, :, None, None]


@dataclass
class SparseBatch:
    dtype: str
    kv: str | None
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    scales: np.ndarray | None
    table: np.ndarray
    lens: np.ndarray
    lists: np.ndarray
    counts: np.ndarray
    scale: float
    block: int

    def args(self):
        sc = () if self.scales is None else (dev(self.scales),)
        return (dev(self.q), dev(self.k), dev(self.v), *sc, *dev(self.table, self.lens, self.lists, self.counts),
                self.scale)

    def call(self, lib, **over):
        return getattr(lib, "pa_decode_sparse" + SUFFIX[self.kv])(*self.args(), **over)

    def stored(self):
        if self.scales is None:
            return self.k, self.v
        dec = CODEC[self.kv][0]
        return tuple(dec(x.numpy()) * self.scales[..., w].astype(np.float64)[:, :, None, None]
                     for w, x in ((0, self.k), (1, self.v)))

    def oracle(self):
        k, v = self.stored()
        return osp.decode_sparse(self.q, k, v, self.table, self.lens, self.lists, self.counts, self.scale, self.block)


def random_lists(rng, lens, block, hkv, keep, ragged=True):
    n = len(lens)
    lists, counts = np.full((n, hkv, keep), -1, np.int32), np.zeros((n, hkv), np.int32)
    for i in range(n):
        nb = -(-int(lens[i]) // block)
        for h in range(hkv):
            k = min(nb, keep)
            if ragged and k > 1:
                k = int(rng.integers(0 if (i + h) % 5 == 4 else 1, k + 1))
            mine = np.sort(rng.choice(nb, k, replace=False)) if k else []
            if k and h % 2 == 0:
                mine[-1] = nb - 1  # the block that may be partly filled
                mine = np.unique(mine)
            lists[i, h, :len(mine)] = mine
            counts[i, h] = len(mine)
    return lists, counts


def sparse_batch(seed, dtype, lens, keep, hq, hkv, d, block=16, kv=None, q_scale=1.0, ragged=True, scale=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    table, P = paged(rng, [int(x) for x in lens], block)
    q = (normal(rng, len(lens), hq, d) * q_scale).to(DT[dtype])
    k, v, sc = pools(rng, P, hkv, block, d, dtype, kv)
    lists, counts = random_lists(rng, lens, block, hkv, keep, ragged)
    return SparseBatch(dtype, kv, q, k, v, sc, table, lens, lists, counts, d ** -0.5 if scale is None else scale, block)


def sparse_tolerance(b: SparseBatch, out, weighted, largest):
    """Per output: what the kernel's roundings can add up to.

    The output is rounded once (half a step of its type). Every softmax weight
    is rounded to 16 bits (half a step; fp16 weights below 2^-14 by at most
    2^-25, against a row sum of at least 1: the largest weight is 1 or more). A score is a sum of D products in fp32, off by at most
    (D + 8) steps of 2^-23 of sum |q k|; the exponential and its argument add 8
    steps; an error e of a weight's exponent moves numerator and denominator,
    together 2 e sum w |v|. Over an 8-bit cache a bf16 query goes into fp16 by
    a power of two, its largest value at 2^14 or above: an element is off by
    2^-25 at most, 2^-39 of the largest, D of them by 2^-39 D times the largest
    product, far below the other terms (D + 8 covers it)."""
    d = b.q.shape[-1]
    e16 = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[b.dtype]
    ew = 0.0 if b.dtype == "f32" else 2.0 ** -11 if b.kv else e16
    step = 2.0 ** -23
    es = largest[..., None] * (d + 8) * step + 8 * step
    n = int(b.lens.max(initial=1))
    tol = e16 * np.abs(out) + (ew + 2 * es + n * 2.0 ** -24 * (b.dtype == "f32")) * weighted + 8 * step * np.abs(out)
    if b.dtype == "f16" or b.kv:
        k, v = b.stored()
        top = float(np.nanmax(np.abs(v.double().numpy() if hasattr(v, "double") else v)))
        tol = tol + n * 2.0 ** -25 * top + 2.0 ** -25
    return tol * 1.05 + 1e-30


def assert_sparse_close(b: SparseBatch, got: torch.Tensor, what: str = ""):
    out, weighted, largest = b.oracle()
    g = got.detach().double().cpu().numpy()
    assert g.shape == out.shape
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - out) / sparse_tolerance(b, out, weighted, largest)
    assert over.max() <= 1.0, f"{what}: {over.max():.2f} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"

"""CPU oracle for the draft-tree calls: attention of tree nodes over a paged
cache, verification of drafted tokens, compaction of the kept path.

TEST INFRASTRUCTURE ONLY, in float64 and written from the definitions: no
blocking, no closed forms, one node and one child at a time.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import gather_sequence, kv_head_of, to_f64


def ancestors(parents, node: int) -> list[int]:
    """The node and its ancestors, upwards. A parent that is not below its
    node counts as none."""
    out = [int(node)]
    while True:
        up = int(parents[out[-1]])
        if up < 0 or up >= out[-1]:
            return out
        out.append(up)


def decode_tree(q, cu_q_lens, parents, ctx_lens, k_cache, v_cache, block_tables, scale: float, block_size: int):
    """Returns (out, weighted, largest), float64: the attention output, the
    softmax-weighted sum of |v| per output, and the largest scale * sum |q k|
    of a row (the two magnitudes that rounding errors scale with). A key
    that a row does not see takes no part, whatever it holds."""
    qf = to_f64(q)
    T, hq, D = qf.shape
    hkv = k_cache.shape[1]
    out, weighted, largest = np.zeros((T, hq, D)), np.zeros((T, hq, D)), np.zeros((T, hq))
    for i, ctx in enumerate(np.asarray(ctx_lens)):
        lo, hi = int(cu_q_lens[i]), int(cu_q_lens[i + 1])
        ctx = int(ctx)
        if hi == lo:
            continue
        keys = gather_sequence(k_cache, block_tables[i], ctx + hi - lo, block_size)
        vals = gather_sequence(v_cache, block_tables[i], ctx + hi - lo, block_size)
        for j in range(hi - lo):
            seen = list(range(ctx)) + sorted(ctx + a for a in ancestors(parents[lo:hi], j))
            for h in range(hq):
                g = kv_head_of(h, hq, hkv)
                k, v = keys[seen, g], vals[seen, g]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k @ qf[lo + j, h])
                    w = np.exp(s - s.max())
                    out[lo + j, h] = (w @ v) / w.sum()
                    weighted[lo + j, h] = (w @ np.abs(v)) / w.sum()
                    largest[lo + j, h] = abs(scale) * (np.abs(k) @ np.abs(qf[lo + j, h])).max()
    return out, weighted, largest


def verify_tree(target, draft, tokens, cu_q_lens, parents, u_accept, u_sample, max_path_len: int):
    """(path, path_lens, next_tokens), by the definition: weights w kept as an
    array, one refusal at a time."""
    def clean(x):
        return np.clip(np.nan_to_num(to_f64(x), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)

    n = len(u_sample)
    V = target.shape[1]
    path = np.full((n, max_path_len), -1, np.int32)
    lens, nexts = np.zeros(n, np.int32), np.full(n, -1, np.int32)
    for i in range(n):
        lo, hi = int(cu_q_lens[i]), int(cu_q_lens[i + 1])
        if hi == lo:
            continue
        kept = [0]
        while True:
            at = kept[-1]
            p = clean(target[lo + at])
            q = None if draft is None else clean(draft[lo + at])
            w, mass, step = p.copy(), 1.0, None
            for c in range(at + 1, hi - lo):
                x = int(tokens[lo + c])
                if len(kept) == max_path_len or int(parents[lo + c]) != at or not 0 <= x < V:
                    continue
                if float(u_accept[lo + c]) * (1.0 if q is None else q[x]) * mass < w[x]:
                    step = c
                    break
                if q is None:
                    mass -= w[x]
                    w[x] = 0.0
                else:
                    w = np.maximum(0.0, w - mass * q)
                    mass = w.sum()
            if step is None:
                break
            kept.append(step)
        if w.sum() <= 0:
            w = p
        c = np.cumsum(w)
        path[i, :len(kept)] = kept
        lens[i] = len(kept)
        if c[-1] > 0:
            nexts[i] = int(np.argmax(c > float(u_sample[i]) * c[-1]))
    return path, lens, nexts


def _moves(i, ctx_lens, path, path_lens, block_tables, block_size):
    """[(source block, offset, destination block, offset, position)] of a sequence."""
    out = []
    for k in range(int(path_lens[i])):
        s, d = int(ctx_lens[i]) + int(path[i][k]), int(ctx_lens[i]) + k
        out.append((int(block_tables[i][s // block_size]), s % block_size,
                    int(block_tables[i][d // block_size]), d % block_size, d))
    return out


def compact_tree(pool, ctx_lens, path, path_lens, block_tables, block_size: int):
    """A copy of one pool [P, Hkv, B, D] with the kept rows moved together."""
    new = pool.clone() if hasattr(pool, "clone") else pool.copy()
    for i in range(len(path_lens)):
        for sb, so, db, do, _ in _moves(i, ctx_lens, path, path_lens, block_tables, block_size):
            new[db, :, do] = pool[sb, :, so]
    return new


def compact_tree_8bit(codes, scales, decode, encode, ctx_lens, path, path_lens, block_tables, block_size: int):
    """(codes, scales) of one 8-bit pool (uint8 [P, Hkv, B, D], float32
    [P, Hkv]) with the kept rows moved together, every block that rows land
    in under the largest scale of the rows that stay in it. decode / encode:
    the format's codec."""
    new, ns = codes.copy(), scales.copy()

    def recode(c, s_old, s_new):
        if s_old == s_new:
            return c
        return encode((decode(c).astype(np.float32) * np.float32(s_old / s_new)).astype(np.float32))

    for i in range(len(path_lens)):
        mv = _moves(i, ctx_lens, path, path_lens, block_tables, block_size)
        for logical in sorted({m[4] // block_size for m in mv}):
            here = [m for m in mv if m[4] // block_size == logical]
            db, first = here[0][2], here[0][3]
            for h in range(codes.shape[1]):
                old = scales[db, h]
                s = max([scales[m[0], h] for m in here] + ([old] if first else []))
                s = np.float32(s)
                if first and s > old > 0:
                    new[db, h, :first] = recode(codes[db, h, :first], old, s)
                for sb, so, _, do, _ in here:
                    new[db, h, do] = recode(codes[sb, h, so], scales[sb, h], s)
                ns[db, h] = s
    return new, ns

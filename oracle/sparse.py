"""Plain oracle of a long-context decode step: rotary positions and the cache
write, block summaries, the choice of blocks, attention over listed blocks.

TEST INFRASTRUCTURE ONLY. Angles and attention are float64; what the library
defines in fp32 (a rotation's products and sums, scales, quotients, scores) is
numpy float32, one operation at a time.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import fp8_kv
from .paged_attention import to_f64

F32 = np.float32


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, low: float = 1.0, high: float | None = None) -> np.ndarray:
    """Radians a position of each pair."""
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "base":
            f = 1.0 if i == 0 else (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif scaling == "bands":
            w = (original_len * f / (2 * math.pi) - low) / (high - low)
            w = min(1.0, max(0.0, w))
            f = w * f + (1 - w) * f / factor
        elif scaling == "ramp":
            pair = lambda t: rot * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
            a, z = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            w = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f = (1 - w) * f + w * f / factor
        out.append(f)
    return np.array(out)


def rope_table(first: int, positions: int, freqs, amplitude: float = 1.0) -> np.ndarray:
    angle = np.arange(first, first + positions, dtype=np.float64)[:, None] * np.asarray(freqs)
    return amplitude * np.concatenate([np.cos(angle), np.sin(angle)], 1)


def rotate(x, cos_sin, positions, interleaved: bool) -> np.ndarray:
    """Rows x [T, H, D] turned, in float32 steps."""
    x = x.detach().to(torch.float32).cpu().numpy()
    cs = np.asarray(cos_sin, F32)[np.asarray(positions)]
    rot = cs.shape[1]
    half = rot // 2
    out = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = cs[:, i, None], cs[:, half + i, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out


def summarize(values: np.ndarray) -> tuple[np.ndarray, np.float32]:
    """One block's keys [rows, D] (float32) -> (int8 codes [2, D], scale)."""
    values = np.asarray(values, F32)
    codes = np.zeros((2, values.shape[1]), np.int8)
    if not np.isfinite(values).all():
        return codes, F32(np.inf)
    hi, lo = values.max(0), values.min(0)
    scale = F32(np.maximum(np.abs(hi), np.abs(lo)).max() / F32(127))
    if scale > 0:
        with np.errstate(over="ignore"):
            codes[0] = np.minimum(np.ceil(hi / scale), 127)
            codes[1] = np.maximum(np.floor(lo / scale), -127)
    return codes, scale


def block_summaries(values, table, first, lens, block: int, summaries, scales) -> None:
    """values: [P, Hkv, B, D] float32; summaries, scales updated in place."""
    for i in range(len(lens)):
        if lens[i] <= first[i]:
            continue
        for lb in range(first[i] // block, (lens[i] - 1) // block + 1):
            p = table[i][lb]
            rows = min(block, lens[i] - lb * block)
            for h in range(values.shape[1]):
                summaries[p, h], scales[p, h] = summarize(values[p, h, :rows])


def block_scores(q, codes, scale) -> np.ndarray:
    """q: [G, D] float32 of one group; codes [n, 2, D], scale [n]: the blocks' scores."""
    best = np.full(len(scale), -np.inf, F32)
    with np.errstate(invalid="ignore", over="ignore"):
        for row in np.asarray(q, F32):
            top = np.abs(row).max()
            sq = F32(top / F32(127)) if np.isfinite(row).all() else F32(0)
            qc = np.rint(np.clip(row / sq, -127, 127)) if sq > 0 else np.zeros_like(row)
            whole = np.maximum(qc * codes[:, 0].astype(np.float64), qc * codes[:, 1].astype(np.float64)).sum(1)
            best = np.maximum(best, sq * whole.astype(F32))
        score = np.where(scale == 0, F32(0), best * scale)
        return np.where(np.isfinite(scale), score, F32(np.inf)).astype(F32)


def select_blocks(q, summaries, scales, table, lens, block: int, keep: int, sink: int, recent: int):
    """(lists [N, Hkv, keep] padded with -1, their lengths)."""
    n, hq, d = q.shape
    hkv = summaries.shape[1]
    g = hq // hkv
    q = q.detach().to(torch.float32).cpu().numpy()
    lists = np.full((n, hkv, keep), -1, np.int32)
    counts = np.zeros((n, hkv), np.int32)
    for i in range(n):
        nb = -(-int(lens[i]) // block)
        for h in range(hkv):
            if nb <= keep:
                mine = list(range(nb))
            else:
                p = np.asarray(table[i][:nb])
                score = block_scores(q[i, h * g:(h + 1) * g], summaries[p, h], scales[p, h])
                rest = sorted(range(sink, nb - recent), key=lambda b: (-score[b], b))
                mine = sorted(list(range(sink)) + list(range(nb - recent, nb)) + rest[:keep - sink - recent])
            lists[i, h, :len(mine)] = mine
            counts[i, h] = len(mine)
    return lists, counts


def decode_sparse(q, k, v, table, lens, lists, counts, scale: float, block: int):
    """(out, sum of weights times |v|, largest sum |q k| scale) in float64,
    the last two for tolerances."""
    q, k, v = to_f64(q), to_f64(k), to_f64(v)
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out, weighted = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    largest = np.zeros((n, hq))
    for i in range(n):
        for h in range(hq):
            kv = h // g
            blocks = [int(b) for b in lists[i, kv, :counts[i, kv]]]
            if not blocks:
                continue
            take = lambda x: np.concatenate(  # noqa: E731
                [x[table[i][b], kv, :min(block, lens[i] - b * block)] for b in blocks])
            kk, vv = take(k), take(v)
            s = kk @ q[i, h] * scale
            largest[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            weighted[i, h] = w @ np.abs(vv)
    return out, weighted, largest


def cache_write_8bit(fmt: str, k, v, slots, k_codes, v_codes, scales, block: int) -> None:
    call = fp8_kv.reshape_and_cache_fp8 if fmt == "e4m3" else fp8_kv.reshape_and_cache_e5m2
    call(k, v, slots, k_codes, v_codes, scales, block)

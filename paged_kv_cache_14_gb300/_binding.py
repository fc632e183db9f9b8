"""ctypes binding of libpagedattn (argument marshalling only).

Every function here takes torch tensors, checks that they are CUDA tensors of
the expected dtype and layout, passes their data pointers and the current (or
given) CUDA stream to the C entry point of the same name, and raises
PagedAttnError on a non-zero status. All computation happens in the library's
CUDA kernels; there is no fallback of any kind: if the library is missing,
load() raises.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os

import numpy as np
import torch

from .builder import LIB_PATH

_lib: ctypes.CDLL | None = None

PA_F32, PA_F16, PA_BF16 = 0, 1, 2
_DT = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}

EXPORTS = (
    "pa_strerror", "pa_version", "pa_get_status", "pa_slot_mapping", "pa_reshape_and_cache",
    "pa_copy_blocks", "pa_decode_partition_size", "pa_decode_workspace_size", "pa_decode",
    "pa_chunked_prefill_workspace_size", "pa_chunked_prefill", "pa_decode_shared_prefix_workspace_size",
    "pa_decode_shared_prefix", "pa_decode_noalloc_scratch_limit", "pa_decode_noalloc",
    "pa_reshape_and_cache_fp8", "pa_copy_blocks_fp8", "pa_decode_fp8", "pa_swap_blocks",
    "pa_decode_step_shared_prefix", "pa_decode_step", "pa_selftest_bounded_wait", "pa_decode_shared_prefix_fp8",
    "pa_chunked_prefill_fp8", "pa_reshape_and_cache_e5m2", "pa_decode_e5m2", "pa_decode_shared_prefix_e5m2",
    "pa_chunked_prefill_e5m2", "pa_decode_tree_workspace_size", "pa_decode_tree", "pa_decode_tree_fp8",
    "pa_decode_tree_e5m2", "pa_verify_tree", "pa_compact_tree", "pa_compact_tree_fp8", "pa_compact_tree_e5m2",
)

_i32, _i64, _f32, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {pa_strerror(status)} ({status})")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libpagedattn.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(there is no fallback path)")
    lib = ctypes.CDLL(path)
    sig = {
        "pa_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "pa_version": (ctypes.c_int, []),
        "pa_get_status": (ctypes.c_int, [_vp]),
        "pa_slot_mapping": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _i64, _i32, _i32, _vp, _vp]),
        "pa_reshape_and_cache": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                                                ctypes.c_int, _vp]),
        "pa_copy_blocks": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i64, _vp]),
        "pa_decode_partition_size": (_i32, [_i32, _i32, _i32, _i32, _i32, _i32]),
        "pa_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
        "pa_decode": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _f32, _vp, _i32, _vp, _sz, ctypes.c_int, _vp]),
        "pa_chunked_prefill_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
        "pa_chunked_prefill": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                              _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, ctypes.c_int, _vp]),
        "pa_decode_shared_prefix_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
        "pa_decode_shared_prefix": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i32,
                                                   _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp, _sz, ctypes.c_int,
                                                   _vp]),
        "pa_decode_noalloc_scratch_limit": (_sz, []),
        "pa_decode_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                             _i32, _f32, _vp, _i32, ctypes.c_int, _vp]),
        "pa_reshape_and_cache_fp8": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                                    ctypes.c_int, _vp]),
        "pa_copy_blocks_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp]),
        "pa_swap_blocks": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _vp]),
        "pa_selftest_bounded_wait": (ctypes.c_int, [_i64, _vp]),
        "pa_decode_step": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                          _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp, _sz,
                                          ctypes.c_int, _vp]),
        "pa_decode_step_shared_prefix": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                                        _vp, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _i32,
                                                        _i32, _i32, _i32, _f32, _vp, _i32, _vp, _sz, ctypes.c_int,
                                                        _vp]),
        "pa_decode_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                         _i32, _f32, _vp, _i32, _vp, _sz, ctypes.c_int, _vp]),
        "pa_decode_shared_prefix_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp,
                                                       _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp,
                                                       _sz, ctypes.c_int, _vp]),
        "pa_chunked_prefill_fp8": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                                  _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, ctypes.c_int,
                                                  _vp]),
    }
    sig.update({
        "pa_decode_tree_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
        "pa_decode_tree": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                          _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, ctypes.c_int, _vp]),
        "pa_decode_tree_fp8": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                              _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, ctypes.c_int, _vp]),
        "pa_verify_tree": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                          _i32, _vp, _vp, _vp, ctypes.c_int, _vp]),
        "pa_compact_tree": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                           _i32, ctypes.c_int, _vp]),
        "pa_compact_tree_fp8": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32,
                                               _i32, _i32, _i32, _vp]),
    })
    for name in ("reshape_and_cache", "decode", "decode_shared_prefix", "chunked_prefill", "decode_tree",
                 "compact_tree"):
        sig[f"pa_{name}_e5m2"] = sig[f"pa_{name}_fp8"]  # same arguments, e5m2 codes
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols(path: str | None = None) -> dict[str, bool]:
    """Which of the header's entry points the library exports (no GPU needed)."""
    lib = ctypes.CDLL(path or LIB_PATH)
    return {name: hasattr(lib, name) for name in EXPORTS}


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise PagedAttnError(rc, where)


def pa_strerror(status: int) -> str:
    return load().pa_strerror(int(status)).decode()


def pa_version() -> int:
    return int(load().pa_version())


def pa_get_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device error word."""
    return int(load().pa_get_status(_stream(stream)))


def pa_slot_mapping(block_tables: torch.Tensor, seq_ids: torch.Tensor, positions: torch.Tensor,
                    block_size: int, num_blocks: int, slot_mapping: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    n = positions.shape[0]
    if slot_mapping is None:
        slot_mapping = torch.empty(n, dtype=torch.int64, device=positions.device)
    rc = load().pa_slot_mapping(
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1], block_tables.shape[0],
        _cuda(seq_ids, "seq_ids", torch.int32), _cuda(positions, "positions", torch.int32), n,
        block_size, num_blocks, _cuda(slot_mapping, "slot_mapping", torch.int64), _stream(stream))
    _check(rc, "pa_slot_mapping")
    return slot_mapping


def pa_reshape_and_cache(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    P, hkv, B, D = k_cache.shape
    dt = k_cache.dtype
    rc = load().pa_reshape_and_cache(
        _cuda(k, "k", dt), _cuda(v, "v", dt), _cuda(slot_mapping, "slot_mapping", torch.int64), k.shape[0],
        _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt), P, B, hkv, D, _DT[dt], _stream(stream))
    _check(rc, "pa_reshape_and_cache")


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_dst_pairs, stream=None) -> None:
    """src_dst_pairs: HOST int64 [n, 2] (numpy array, list or CPU tensor)."""
    pairs = np.ascontiguousarray(np.asarray(src_dst_pairs, dtype=np.int64).reshape(-1, 2))
    P = k_cache.shape[0]
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    rc = load().pa_copy_blocks(
        _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache", k_cache.dtype),
        pairs.ctypes.data_as(ctypes.c_void_p), pairs.shape[0], P, block_bytes, _stream(stream))
    _check(rc, "pa_copy_blocks")


def pa_decode_partition_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, block_size: int,
                             max_seq_len: int, partition_size: int = 0) -> int:
    r = int(load().pa_decode_partition_size(num_seqs, num_q_heads, num_kv_heads, block_size, max_seq_len,
                                            partition_size))
    if r < 0:
        raise PagedAttnError(r, "pa_decode_partition_size")
    return r


def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                             block_size: int, max_seq_len: int, partition_size: int = 0) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                               max_seq_len, partition_size))


def pa_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
              seq_lens: torch.Tensor, max_seq_len: int, scale: float, out: torch.Tensor | None = None,
              partition_size: int = 0, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    N, hq, D = q.shape
    P, hkv, B, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache head_dim differ")
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().pa_decode(
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len), hq, hkv, D, B, P, float(scale),
        _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt], _stream(stream))
    _check(rc, "pa_decode")
    return out


def pa_chunked_prefill_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                      block_size: int, total_q: int, max_kv_len: int) -> int:
    return int(load().pa_chunked_prefill_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                        block_size, total_q, max_kv_len))


def pa_chunked_prefill(q: torch.Tensor, cu_q_lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       block_tables: torch.Tensor, ctx_lens: torch.Tensor, max_q_len: int, max_kv_len: int,
                       scale: float, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    T, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    n = ctx_lens.shape[0]
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_chunked_prefill_workspace_size(n, hq, hkv, D, B, T, max_kv_len)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().pa_chunked_prefill(
        _cuda(q, "q", dt), T, _cuda(cu_q_lens, "cu_q_lens", torch.int32), _cuda(k_cache, "k_cache", dt),
        _cuda(v_cache, "v_cache", dt), _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(ctx_lens, "ctx_lens", torch.int32), n, int(max_q_len), int(max_kv_len), hq, hkv, D, B, P,
        float(scale), _cuda(out, "out", dt), ws_ptr, ws_bytes, _DT[dt], _stream(stream))
    _check(rc, "pa_chunked_prefill")
    return out


def pa_decode_shared_prefix_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                           block_size: int, max_seq_len: int, partition_size: int,
                                           num_groups: int) -> int:
    return int(load().pa_decode_shared_prefix_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                             block_size, max_seq_len, partition_size, num_groups))


def pa_decode_shared_prefix(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                            group_starts: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                            out: torch.Tensor | None = None, partition_size: int = 0,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    N, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    G = group_starts.shape[0] - 1
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_shared_prefix_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size, G)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().pa_decode_shared_prefix(
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len),
        _cuda(group_starts, "group_starts", torch.int32), _cuda(prefix_lens, "prefix_lens", torch.int32), G,
        hq, hkv, D, B, P, float(scale), _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt],
        _stream(stream))
    _check(rc, "pa_decode_shared_prefix")
    return out


def pa_decode_step(cow_pairs, new_seq_ids: torch.Tensor, new_positions: torch.Tensor, k_new: torch.Tensor,
                   v_new: torch.Tensor, slot_mapping: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                   scale: float, out: torch.Tensor | None = None, partition_size: int = 0,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step in one call: pa_copy_blocks(cow_pairs), pa_slot_mapping,
    pa_reshape_and_cache, pa_decode. cow_pairs: HOST int64 [n, 2]."""
    pairs = np.ascontiguousarray(np.asarray(cow_pairs, dtype=np.int64).reshape(-1, 2))
    N, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    dt = q.dtype
    T = new_seq_ids.shape[0]
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().pa_decode_step(
        pairs.ctypes.data_as(ctypes.c_void_p) if pairs.shape[0] else None, pairs.shape[0],
        _cuda(new_seq_ids, "new_seq_ids", torch.int32), _cuda(new_positions, "new_positions", torch.int32),
        _cuda(k_new, "k_new", dt), _cuda(v_new, "v_new", dt), T, _cuda(slot_mapping, "slot_mapping", torch.int64),
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len), hq, hkv, D, B, P, float(scale),
        _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt], _stream(stream))
    _check(rc, "pa_decode_step")
    return out


def pa_decode_step_shared_prefix(cow_pairs, new_seq_ids: torch.Tensor, new_positions: torch.Tensor,
                                 k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                                 q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                 group_starts: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                                 out: torch.Tensor | None = None, partition_size: int = 0,
                                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step in one call: pa_copy_blocks(cow_pairs), pa_slot_mapping,
    pa_reshape_and_cache, pa_decode_shared_prefix. cow_pairs: HOST int64
    [n, 2] (numpy array, list or CPU tensor)."""
    pairs = np.ascontiguousarray(np.asarray(cow_pairs, dtype=np.int64).reshape(-1, 2))
    N, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    G = group_starts.shape[0] - 1
    dt = q.dtype
    T = new_seq_ids.shape[0]
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_shared_prefix_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size, G)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().pa_decode_step_shared_prefix(
        pairs.ctypes.data_as(ctypes.c_void_p) if pairs.shape[0] else None, pairs.shape[0],
        _cuda(new_seq_ids, "new_seq_ids", torch.int32), _cuda(new_positions, "new_positions", torch.int32),
        _cuda(k_new, "k_new", dt), _cuda(v_new, "v_new", dt), T, _cuda(slot_mapping, "slot_mapping", torch.int64),
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len),
        _cuda(group_starts, "group_starts", torch.int32), _cuda(prefix_lens, "prefix_lens", torch.int32), G,
        hq, hkv, D, B, P, float(scale), _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt],
        _stream(stream))
    _check(rc, "pa_decode_step_shared_prefix")
    return out


def pa_selftest_bounded_wait(limit_ns: int, stream=None) -> None:
    """Launch a wait that nothing completes: it gives up after limit_ns and
    records PA_ERR_TIMEOUT (read it with pa_get_status)."""
    _check(load().pa_selftest_bounded_wait(int(limit_ns), _stream(stream)), "pa_selftest_bounded_wait")


def pa_decode_noalloc_scratch_limit() -> int:
    return int(load().pa_decode_noalloc_scratch_limit())


def pa_decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                      seq_lens: torch.Tensor, max_seq_len: int, scale: float, out: torch.Tensor,
                      partition_size: int = 0, stream=None) -> torch.Tensor:
    """pa_decode with the library's fixed scratch instead of a workspace.
    `out` must be given: this path allocates nothing."""
    N, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    dt = q.dtype
    rc = load().pa_decode_noalloc(
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", dt), _cuda(v_cache, "v_cache", dt),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len), hq, hkv, D, B, P, float(scale),
        _cuda(out, "out", dt), int(partition_size), _DT[dt], _stream(stream))
    _check(rc, "pa_decode_noalloc")
    return out


# ---------------------------------------------------------------------------
# 8-bit KV cache: uint8 code pools [P, Hkv, B, D] and float32 scales
# [P, Hkv, 2] (K, V) per (block, KV head). The *_fp8 calls hold e4m3 codes,
# the *_e5m2 calls e5m2 codes; pa_copy_blocks_fp8 serves both.
# ---------------------------------------------------------------------------

def pa_reshape_and_cache_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                             k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor,
                             stream=None) -> None:
    _reshape_and_cache_8bit("pa_reshape_and_cache_fp8", k, v, slot_mapping, k_cache, v_cache, kv_scales, stream)


def pa_reshape_and_cache_e5m2(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                              k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor,
                              stream=None) -> None:
    _reshape_and_cache_8bit("pa_reshape_and_cache_e5m2", k, v, slot_mapping, k_cache, v_cache, kv_scales, stream)


def _reshape_and_cache_8bit(sym, k, v, slot_mapping, k_cache, v_cache, kv_scales, stream) -> None:
    P, hkv, B, D = k_cache.shape
    dt = k.dtype
    rc = getattr(load(), sym)(
        _cuda(k, "k", dt), _cuda(v, "v", dt), _cuda(slot_mapping, "slot_mapping", torch.int64), k.shape[0],
        _cuda(k_cache, "k_cache", torch.uint8), _cuda(v_cache, "v_cache", torch.uint8),
        _cuda(kv_scales, "kv_scales", torch.float32), P, B, hkv, D, _DT[dt], _stream(stream))
    _check(rc, sym)


def pa_copy_blocks_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor, src_dst_pairs,
                       stream=None) -> None:
    """src_dst_pairs: HOST int64 [n, 2] (numpy array, list or CPU tensor)."""
    pairs = np.ascontiguousarray(np.asarray(src_dst_pairs, dtype=np.int64).reshape(-1, 2))
    P, hkv, B, D = k_cache.shape
    rc = load().pa_copy_blocks_fp8(
        _cuda(k_cache, "k_cache", torch.uint8), _cuda(v_cache, "v_cache", torch.uint8),
        _cuda(kv_scales, "kv_scales", torch.float32), pairs.ctypes.data_as(ctypes.c_void_p), pairs.shape[0], P, B,
        hkv, D, _stream(stream))
    _check(rc, "pa_copy_blocks_fp8")


def pa_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor,
                  block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                  out: torch.Tensor | None = None, partition_size: int = 0, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    return _decode_8bit("pa_decode_fp8", q, k_cache, v_cache, kv_scales, block_tables, seq_lens, max_seq_len, scale,
                        out, partition_size, workspace, stream)


def pa_decode_e5m2(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor,
                   block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                   out: torch.Tensor | None = None, partition_size: int = 0, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    return _decode_8bit("pa_decode_e5m2", q, k_cache, v_cache, kv_scales, block_tables, seq_lens, max_seq_len,
                        scale, out, partition_size, workspace, stream)


def _decode_8bit(sym, q, k_cache, v_cache, kv_scales, block_tables, seq_lens, max_seq_len, scale, out,
                 partition_size, workspace, stream) -> torch.Tensor:
    N, hq, D = q.shape
    P, hkv, B, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache head_dim differ")
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = getattr(load(), sym)(
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", torch.uint8), _cuda(v_cache, "v_cache", torch.uint8),
        _cuda(kv_scales, "kv_scales", torch.float32), _cuda(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len), hq, hkv, D, B, P,
        float(scale), _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt], _stream(stream))
    _check(rc, sym)
    return out


def pa_decode_shared_prefix_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                kv_scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                max_seq_len: int, group_starts: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                                out: torch.Tensor | None = None, partition_size: int = 0,
                                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    return _shared_prefix_8bit("pa_decode_shared_prefix_fp8", q, k_cache, v_cache, kv_scales, block_tables,
                               seq_lens, max_seq_len, group_starts, prefix_lens, scale, out, partition_size,
                               workspace, stream)


def pa_decode_shared_prefix_e5m2(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 kv_scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                 max_seq_len: int, group_starts: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                                 out: torch.Tensor | None = None, partition_size: int = 0,
                                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    return _shared_prefix_8bit("pa_decode_shared_prefix_e5m2", q, k_cache, v_cache, kv_scales, block_tables,
                               seq_lens, max_seq_len, group_starts, prefix_lens, scale, out, partition_size,
                               workspace, stream)


def _shared_prefix_8bit(sym, q, k_cache, v_cache, kv_scales, block_tables, seq_lens, max_seq_len, group_starts,
                        prefix_lens, scale, out, partition_size, workspace, stream) -> torch.Tensor:
    N, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    G = group_starts.shape[0] - 1
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_decode_shared_prefix_workspace_size(N, hq, hkv, D, B, max_seq_len, partition_size, G)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = getattr(load(), sym)(
        _cuda(q, "q", dt), _cuda(k_cache, "k_cache", torch.uint8), _cuda(v_cache, "v_cache", torch.uint8),
        _cuda(kv_scales, "kv_scales", torch.float32), _cuda(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _cuda(seq_lens, "seq_lens", torch.int32), N, int(max_seq_len),
        _cuda(group_starts, "group_starts", torch.int32), _cuda(prefix_lens, "prefix_lens", torch.int32), G,
        hq, hkv, D, B, P, float(scale), _cuda(out, "out", dt), int(partition_size), ws_ptr, ws_bytes, _DT[dt],
        _stream(stream))
    _check(rc, sym)
    return out


def pa_chunked_prefill_fp8(q: torch.Tensor, cu_q_lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           kv_scales: torch.Tensor, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
                           max_q_len: int, max_kv_len: int, scale: float, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    return _prefill_8bit("pa_chunked_prefill_fp8", q, cu_q_lens, k_cache, v_cache, kv_scales, block_tables, ctx_lens,
                         max_q_len, max_kv_len, scale, out, workspace, stream)


def pa_chunked_prefill_e5m2(q: torch.Tensor, cu_q_lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            kv_scales: torch.Tensor, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
                            max_q_len: int, max_kv_len: int, scale: float, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    return _prefill_8bit("pa_chunked_prefill_e5m2", q, cu_q_lens, k_cache, v_cache, kv_scales, block_tables,
                         ctx_lens, max_q_len, max_kv_len, scale, out, workspace, stream)


def _prefill_8bit(sym, q, cu_q_lens, k_cache, v_cache, kv_scales, block_tables, ctx_lens, max_q_len, max_kv_len,
                  scale, out, workspace, stream) -> torch.Tensor:
    T, hq, D = q.shape
    P, hkv, B, _ = k_cache.shape
    n = ctx_lens.shape[0]
    dt = q.dtype
    if out is None:
        out = torch.empty_like(q)
    need = pa_chunked_prefill_workspace_size(n, hq, hkv, D, B, T, max_kv_len)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _cuda(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = getattr(load(), sym)(
        _cuda(q, "q", dt), T, _cuda(cu_q_lens, "cu_q_lens", torch.int32), _cuda(k_cache, "k_cache", torch.uint8),
        _cuda(v_cache, "v_cache", torch.uint8), _cuda(kv_scales, "kv_scales", torch.float32),
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(ctx_lens, "ctx_lens", torch.int32), n, int(max_q_len), int(max_kv_len), hq, hkv, D, B, P,
        float(scale), _cuda(out, "out", dt), ws_ptr, ws_bytes, _DT[dt], _stream(stream))
    _check(rc, sym)
    return out


def _pool_ptr(t: torch.Tensor | None, name: str) -> int | None:
    """Pointer of a pool for pa_swap_blocks: a contiguous CUDA tensor or a
    pinned CPU tensor."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or t.is_pinned()):
        raise TypeError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def pa_swap_blocks(src_k: torch.Tensor, src_v: torch.Tensor | None, dst_k: torch.Tensor,
                   dst_v: torch.Tensor | None, src_dst_pairs, stream=None) -> None:
    """Whole blocks dst[dst] <- src[src] between two pools (CUDA or pinned CPU
    tensors, leading dimension = blocks). src_dst_pairs: HOST int64 [n, 2]."""
    pairs = np.ascontiguousarray(np.asarray(src_dst_pairs, dtype=np.int64).reshape(-1, 2))
    if src_k.dtype != dst_k.dtype or src_k.shape[1:] != dst_k.shape[1:]:
        raise ValueError("source and destination pools differ in block layout")
    block_bytes = src_k[0].numel() * src_k.element_size()
    rc = load().pa_swap_blocks(
        _pool_ptr(src_k, "src_k"), _pool_ptr(src_v, "src_v"), _pool_ptr(dst_k, "dst_k"), _pool_ptr(dst_v, "dst_v"),
        pairs.ctypes.data_as(ctypes.c_void_p), pairs.shape[0], src_k.shape[0], dst_k.shape[0], block_bytes,
        _stream(stream))
    _check(rc, "pa_swap_blocks")


# ---------------------------------------------------------------------------
# Draft trees: attention, verification, compaction of the kept path.
# ---------------------------------------------------------------------------

def _refuse(t, name: str, dtype, dev: int, shape) -> None:
    """Raise what is wrong with an argument that _arg does not take."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, name: str, dtype, dev: int, shape) -> int:
    """Pointer of a contiguous tensor of this type and shape on device dev
    (the current one: the calls launch there)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _refuse(t, name, dtype, dev, shape)


def _place(t, name: str, stream) -> tuple[int, int, object]:
    """The current device, the stream's handle, and the stream if it is not
    the current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = torch.cuda.current_device()
    here = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return dev, here, None
    handle = _stream(stream)
    if handle == here:
        return dev, handle, None
    # (ExternalStream makes a new stream of handle 0, which is the default one's.)
    return dev, handle, torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream(dev)


def _scratch(like: torch.Tensor, shape, dtype, side) -> torch.Tensor:
    """A new tensor for a call on the current stream or on another one (side).
    Memory comes from the stream that writes it first, so that whatever used
    it before is over by then; the caller may go on to read it on the current
    one, which is why that one is recorded. (Tensor.new_empty between kernel
    launches takes twice torch.empty's time.)"""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(here)
    return t


def pa_decode_tree_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                                  total_q: int, max_q_len: int, max_kv_len: int,
                                  dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().pa_decode_tree_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, total_q,
                                                    max_q_len, max_kv_len, _DT[dtype]))


def pa_decode_tree(q: torch.Tensor, cu_q_lens: torch.Tensor, parents: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, ctx_lens: torch.Tensor, max_q_len: int,
                   max_kv_len: int, scale: float, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of every sequence's tree nodes (rows of q) over its paged context."""
    return _decode_tree("pa_decode_tree", q, cu_q_lens, parents, k_cache, v_cache, None, block_tables, ctx_lens,
                        max_q_len, max_kv_len, scale, out, workspace, stream)


def pa_decode_tree_fp8(q: torch.Tensor, cu_q_lens: torch.Tensor, parents: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, kv_scales: torch.Tensor, block_tables: torch.Tensor,
                       ctx_lens: torch.Tensor, max_q_len: int, max_kv_len: int, scale: float,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """pa_decode_tree over e4m3 pools."""
    return _decode_tree("pa_decode_tree_fp8", q, cu_q_lens, parents, k_cache, v_cache, kv_scales, block_tables,
                        ctx_lens, max_q_len, max_kv_len, scale, out, workspace, stream)


def pa_decode_tree_e5m2(q: torch.Tensor, cu_q_lens: torch.Tensor, parents: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, kv_scales: torch.Tensor, block_tables: torch.Tensor,
                        ctx_lens: torch.Tensor, max_q_len: int, max_kv_len: int, scale: float,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """pa_decode_tree over e5m2 pools."""
    return _decode_tree("pa_decode_tree_e5m2", q, cu_q_lens, parents, k_cache, v_cache, kv_scales, block_tables,
                        ctx_lens, max_q_len, max_kv_len, scale, out, workspace, stream)


def _decode_tree(sym, q, cu_q_lens, parents, k_cache, v_cache, kv_scales, block_tables, ctx_lens, max_q_len,
                 max_kv_len, scale, out, workspace, stream) -> torch.Tensor:
    lib = load()
    dev, handle, side = _place(q, "q", stream)
    T, hq, D = q.shape
    P, hkv, B, _ = pool = k_cache.shape
    n, mb = block_tables.shape
    dt, i32 = q.dtype, torch.int32
    code = _DT.get(dt)
    if code is None:
        raise TypeError(f"q must be float32, float16 or bfloat16, got {dt}")
    if pool[3] != D:
        raise ValueError(f"k_cache has shape {tuple(pool)}, q's head_dim is {D}")
    kv = dt if kv_scales is None else torch.uint8
    qp = _arg(q, "q", dt, dev, q.shape)
    if out is None:
        out = _scratch(q, (T, hq, D), dt, side)
    if workspace is None:
        need = lib.pa_decode_tree_workspace_size(n, hq, hkv, D, B, T, max_q_len, max_kv_len, code)
        workspace = _scratch(q, (max(need, 16),), torch.uint8, side)
    pools = (_arg(k_cache, "k_cache", kv, dev, pool), _arg(v_cache, "v_cache", kv, dev, pool))
    if kv_scales is not None:
        pools += (_arg(kv_scales, "kv_scales", torch.float32, dev, (P, hkv, 2)),)
    rc = getattr(lib, sym)(
        qp, T, _arg(cu_q_lens, "cu_q_lens", i32, dev, (n + 1,)), _arg(parents, "parents", i32, dev, (T,)), *pools,
        _arg(block_tables, "block_tables", i32, dev, (n, mb)), mb, _arg(ctx_lens, "ctx_lens", i32, dev, (n,)), n,
        max_q_len, max_kv_len, hq, hkv, D, B, P, scale, _arg(out, "out", dt, dev, (T, hq, D)),
        _arg(workspace, "workspace", workspace.dtype, dev, workspace.shape), workspace.nbytes, code, handle)
    if rc:
        raise PagedAttnError(rc, sym)
    return out


def _rows(t, name: str, dtype, dev: int, shape) -> tuple[int, int]:
    """Pointer and row stride (elements) of a 2-D CUDA tensor whose rows are contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, name, dtype, dev, shape)
    step, one = t.stride()
    if shape[1] > 1 and one != 1 or shape[0] > 1 and step < shape[1]:
        raise ValueError(f"{name}'s rows must be contiguous and not overlap")
    return t.data_ptr(), max(step, shape[1])


def pa_verify_tree(target_probs: torch.Tensor, draft_probs: torch.Tensor | None, draft_tokens: torch.Tensor,
                   cu_q_lens: torch.Tensor, parents: torch.Tensor, uniform_accept: torch.Tensor,
                   uniform_sample: torch.Tensor, max_q_len: int, max_path_len: int, path: torch.Tensor | None = None,
                   path_lens: torch.Tensor | None = None, next_tokens: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Keep drafted tokens and draw the next one: (path, path_lens, next_tokens).
    target_probs, draft_probs: [total_q, vocab]; rows may be padded apart."""
    lib = load()
    dev, handle, side = _place(target_probs, "target_probs", stream)
    T, V = shape = target_probs.shape
    n = uniform_sample.shape[0]
    dt, i32, f32 = target_probs.dtype, torch.int32, torch.float32
    code = _DT.get(dt)
    if code is None:
        raise TypeError(f"target_probs must be float32, float16 or bfloat16, got {dt}")
    tp, ts = _rows(target_probs, "target_probs", dt, dev, shape)
    dp, ds = (None, 0) if draft_probs is None else _rows(draft_probs, "draft_probs", dt, dev, shape)
    rows = (T,)
    if path is None:
        path = _scratch(target_probs, (n, max_path_len), i32, side)
    if path_lens is None:
        path_lens = _scratch(target_probs, (n,), i32, side)
    if next_tokens is None:
        next_tokens = _scratch(target_probs, (n,), i32, side)
    rc = lib.pa_verify_tree(
        tp, ts, dp, ds, _arg(draft_tokens, "draft_tokens", i32, dev, rows),
        _arg(cu_q_lens, "cu_q_lens", i32, dev, (n + 1,)), _arg(parents, "parents", i32, dev, rows),
        _arg(uniform_accept, "uniform_accept", f32, dev, rows), _arg(uniform_sample, "uniform_sample", f32, dev, (n,)),
        n, T, max_q_len, V, max_path_len, _arg(path, "path", i32, dev, (n, max_path_len)),
        _arg(path_lens, "path_lens", i32, dev, (n,)), _arg(next_tokens, "next_tokens", i32, dev, (n,)), code, handle)
    if rc:
        raise PagedAttnError(rc, "pa_verify_tree")
    return path, path_lens, next_tokens


def pa_compact_tree(k_caches, v_caches, block_tables: torch.Tensor, ctx_lens: torch.Tensor, path: torch.Tensor,
                    path_lens: torch.Tensor, stream=None) -> None:
    """Move the kept nodes' K/V rows together in every layer. k_caches,
    v_caches: one pool [blocks, Hkv, B, D] per layer."""
    _compact_tree("pa_compact_tree", k_caches, v_caches, None, block_tables, ctx_lens, path, path_lens, stream)


def pa_compact_tree_fp8(k_caches, v_caches, kv_scales, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
                        path: torch.Tensor, path_lens: torch.Tensor, stream=None) -> None:
    """pa_compact_tree over e4m3 pools; kv_scales: one [blocks, Hkv, 2] per layer."""
    _compact_tree("pa_compact_tree_fp8", k_caches, v_caches, kv_scales, block_tables, ctx_lens, path, path_lens,
                  stream)


def pa_compact_tree_e5m2(k_caches, v_caches, kv_scales, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
                         path: torch.Tensor, path_lens: torch.Tensor, stream=None) -> None:
    """pa_compact_tree over e5m2 pools; kv_scales: one [blocks, Hkv, 2] per layer."""
    _compact_tree("pa_compact_tree_e5m2", k_caches, v_caches, kv_scales, block_tables, ctx_lens, path, path_lens,
                  stream)


_DTYPE, _SHAPE = operator.attrgetter("dtype"), operator.attrgetter("shape")


def _pools(pools, name: str, dtype, dev: int, shape) -> array.array:
    """Pointers of the layers' pools, as _arg. The checks run as loops in C:
    a model has dozens of layers, and this is most of a call's host time. One
    tensor of all layers' pools is one check."""
    T = torch.Tensor
    if isinstance(pools, T):
        at = _arg(pools, name, dtype, dev, (len(pools), *shape))
        step = pools[0].nbytes
        return array.array("Q", range(at, at + len(pools) * step, step) if step else [at] * len(pools))
    if not (set(map(_DTYPE, pools)) == {dtype} and list(map(_SHAPE, pools)) == [shape] * len(pools)
            and set(map(T.get_device, pools)) == {dev} and all(map(T.is_contiguous, pools))):
        for i, t in enumerate(pools):
            _arg(t, f"{name}[{i}]", dtype, dev, shape)
    return array.array("Q", map(T.data_ptr, pools))


def _compact_tree(sym, k_caches, v_caches, kv_scales, block_tables, ctx_lens, path, path_lens, stream) -> None:
    lib = load()
    layers = len(k_caches)
    if len(v_caches) != layers or (kv_scales is not None and len(kv_scales) != layers):
        raise ValueError("k_caches, v_caches and kv_scales must list the same layers")
    if layers == 0:
        return
    dev, handle, _ = _place(k_caches[0], "k_caches[0]", stream)
    P, hkv, B, D = shape = k_caches[0].shape
    n, mb = block_tables.shape
    width = path.shape[1]
    i32 = torch.int32
    if kv_scales is None:
        dt = k_caches[0].dtype
        code = (_DT.get(dt),)
        if code[0] is None:
            raise TypeError(f"k_caches must be float32, float16 or bfloat16, got {dt}")
    else:
        dt, code = torch.uint8, ()
    lists = [_pools(k_caches, "k_caches", dt, dev, shape), _pools(v_caches, "v_caches", dt, dev, shape)]
    if kv_scales is not None:
        lists.append(_pools(kv_scales, "kv_scales", torch.float32, dev, torch.Size((P, hkv, 2))))
    rc = getattr(lib, sym)(
        *(x.buffer_info()[0] for x in lists), layers, _arg(block_tables, "block_tables", i32, dev, (n, mb)), mb,
        _arg(ctx_lens, "ctx_lens", i32, dev, (n,)), _arg(path, "path", i32, dev, (n, width)),
        _arg(path_lens, "path_lens", i32, dev, (n,)), n, width, P, B, hkv, D, *code, handle)
    if rc:
        raise PagedAttnError(rc, sym)

// Compaction of a draft tree's kept path: the K/V row of node path[k] of a
// sequence (position ctx + path[k]) moves to position ctx + k, in every layer,
// as if all rows were read before any is written.
//
// A path's nodes rise strictly, so path[k] >= k and a row is never written
// before a later row has to read it as its source: for k' > k,
// path[k'] > path[k] >= k. A thread that owns the same bytes of all of a
// (layer, sequence, KV head)'s rows may therefore move them in path order,
// with no staging and no barrier between its loads and its stores. A thread
// takes 16-byte columns, and the grid covers every layer at once: 128 sequences
// of up to 24 nodes in 32 layers (151 MB read and written) take 28 us on pools
// that are not in L2, 80% of HBM's rate, and 22 us again and again on the
// same ones, part of which stays there; 4 sequences in one layer 3.3 us, a
// launch and three dependent loads (lengths, path, blocks, rows).
#include <algorithm>
#include <functional>
#include <memory>
#include <new>

#include "pa_common.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kCompactMaxPath = 1024;
constexpr int kCompactLayers = 64;  // layers of one launch: their pools travel as kernel parameters
constexpr int kCompactThreads = 128;

struct CompactLayers {
  void* k[kCompactLayers];
  void* v[kCompactLayers];
  float* scales[kCompactLayers];
};

struct CompactParams {
  const int32_t* block_tables;
  const int32_t* ctx_lens;
  const int32_t* path;
  const int32_t* path_lens;
  int32_t max_blocks_per_seq, num_seqs, max_path_len, num_blocks, block_size, num_kv_heads, row_bytes, num_layers;
  int* status;
};

// A move's source and destination: (block, offset), block -1 for none.
struct Move {
  int32_t src_block, dst_block;
  int16_t src_off, dst_off;
};

// Shared memory: the moves of one sequence. Returns their number; 0 (and an
// error) for an illegal path. Contains barriers: run by the whole CTA.
__device__ __forceinline__ int compact_moves(const CompactParams& p, int seq, Move* mv, bool report) {
  const int len = p.path_lens[seq], ctx = p.ctx_lens[seq];
  const int32_t* path = p.path + (int64_t)seq * p.max_path_len;
  const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
  bool bad_len = len < 0 || len > p.max_path_len || ctx < 0, bad_path = false, bad_block = false;
  if (!bad_len) {
    for (int k = threadIdx.x; k < len; k += blockDim.x) {
      const int a = path[k];
      if (a < 0 || (k > 0 && path[k - 1] >= a)) {
        bad_path = true;
        continue;
      }
      const int64_t src = (int64_t)ctx + a, dst = (int64_t)ctx + k;
      if (src >= (int64_t)p.max_blocks_per_seq * p.block_size) {
        bad_len = true;
        continue;
      }
      Move m;
      m.src_block = table[src / p.block_size];
      m.dst_block = table[dst / p.block_size];
      m.src_off = (int16_t)(src % p.block_size);
      m.dst_off = (int16_t)(dst % p.block_size);
      if (m.src_block < 0 || m.src_block >= p.num_blocks || m.dst_block < 0 || m.dst_block >= p.num_blocks)
        bad_block = true;
      mv[k] = m;
    }
  }
  if (!__syncthreads_or(bad_len || bad_path || bad_block)) return len;
  const int any_len = __syncthreads_or(bad_len), any_path = __syncthreads_or(bad_path);
  if (report && threadIdx.x == 0)
    record_error(p.status, any_path ? PA_ERR_ARG : any_len ? PA_ERR_SEQLEN : PA_ERR_BLOCK_OOB);
  return 0;
}

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p, const CompactLayers pools) {
  __shared__ Move mv[kCompactMaxPath];
  const int seq = blockIdx.x;
  const int n = compact_moves(p, seq, mv, blockIdx.y == 0);
  const int vecs = p.row_bytes >> 4;
  const int cols = 2 * p.num_kv_heads * vecs;  // 16-byte columns of one layer
  for (int64_t i = blockIdx.y * kCompactThreads + threadIdx.x; i < (int64_t)cols * p.num_layers;
       i += gridDim.y * kCompactThreads) {
    const int layer = (int)(i / cols);
    int c = (int)(i - (int64_t)layer * cols);
    const int half = p.num_kv_heads * vecs;
    uint8_t* pool = static_cast<uint8_t*>(c < half ? pools.k[layer] : pools.v[layer]);
    c = c < half ? c : c - half;
    const int h = c / vecs, x = c - h * vecs;
    auto place = [&](int blk, int off) {
      return reinterpret_cast<int4*>(pool + (((int64_t)blk * p.num_kv_heads + h) * p.block_size + off) * p.row_bytes) +
             x;
    };
    for (int k = 0; k < n; ++k) {
      const Move m = mv[k];
      if (m.src_block == m.dst_block && m.src_off == m.dst_off) continue;
      *place(m.dst_block, m.dst_off) = *place(m.src_block, m.src_off);
    }
  }
}

template <int VEC>
__device__ __forceinline__ void copy_codes(const uint8_t* from, uint8_t* to) {
  if constexpr (VEC == 2) *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
  else *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
}

// 8-bit cache: one warp per (layer, sequence, KV head, pool). The rows that
// land in one block are encoded under s_new = the largest scale of the rows
// that stay in it (the moved ones and, in the first block, the committed ones
// below them), each code by fl32(s_old / s_new), as the cache write does when
// a block's scale grows. A row whose scale is s_new keeps its codes. A warp
// moves one row of a block after the other (64 sequences of up to 40 nodes in
// 16 layers: 13 us for 19 MB), bound by that chain of loads and by the scales'
// before it.
template <int VEC, bool E5>
__global__ void __launch_bounds__(kCompactThreads) compact_8bit_kernel(const CompactParams p,
                                                                       const CompactLayers pools) {
  constexpr int D = VEC * 32;
  __shared__ Move mv[kCompactMaxPath];
  const int seq = blockIdx.x, lane = threadIdx.x & 31;
  const int n = compact_moves(p, seq, mv, blockIdx.y == 0);
  const int per_layer = 2 * p.num_kv_heads;
  const int warps = gridDim.y * (kCompactThreads / 32);
  for (int w = blockIdx.y * (kCompactThreads / 32) + (threadIdx.x >> 5); w < per_layer * p.num_layers; w += warps) {
    const int layer = w / per_layer, rem = w - layer * per_layer;
    const int h = rem >> 1, which = rem & 1;
    uint8_t* pool = static_cast<uint8_t*>(which ? pools.v[layer] : pools.k[layer]);
    float* scales = pools.scales[layer];
    auto scale_of = [&](int blk) -> float* { return scales + ((int64_t)blk * p.num_kv_heads + h) * 2 + which; };
    auto row = [&](int blk, int off) -> uint8_t* {
      return pool + (((int64_t)blk * p.num_kv_heads + h) * p.block_size + off) * D + lane * VEC;
    };
    for (int k0 = 0; k0 < n;) {
      // The rows k0 .. k1-1 land in one block.
      const int blk = mv[k0].dst_block, first = mv[k0].dst_off;
      const int k1 = min(n, k0 + p.block_size - first);
      const float s_dst = *scale_of(blk);
      float s_new = first > 0 ? s_dst : 0.f;
      for (int k = k0; k < k1; ++k) s_new = fmaxf(s_new, *scale_of(mv[k].src_block));
      auto recode = [&](const uint8_t* from, uint8_t* to, float s_old) {
        if (s_old == s_new) {
          if (from != to) copy_codes<VEC>(from, to);
          return;
        }
        const float r = __fdiv_rn(s_old, s_new);
        float x[VEC];
        load_codes<VEC, E5>(from, x);
        uint32_t c[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) c[i / 2] = f32x2_to_fp8x2<E5>(__fmul_rn(x[i], r), __fmul_rn(x[i + 1], r));
        store_codes<VEC>(to, c);
      };
      if (first > 0 && s_new > s_dst && s_dst > 0.f)
        for (int o = 0; o < first; ++o) recode(row(blk, o), row(blk, o), s_dst);
      for (int k = k0; k < k1; ++k) {
        const Move m = mv[k];
        recode(row(m.src_block, m.src_off), row(m.dst_block, m.dst_off), *scale_of(m.src_block));
      }
      __syncwarp();
      if (lane == 0) *scale_of(blk) = s_new;
      __syncwarp();
      k0 = k1;
    }
  }
}

// Whether a pool (or scale array) is listed twice: its rows would be moved twice,
// by CTAs that know nothing of each other.
static int listed_twice(void* const* k, void* const* v, float* const* scales, int32_t n) {
  std::unique_ptr<const void*[]> all(new (std::nothrow) const void*[2 * (size_t)n]);
  if (!all) return PA_ERR_CUDA;
  auto twice = [&](const void** end) {
    std::sort(all.get(), end, std::less<const void*>());
    return std::adjacent_find(all.get(), end) != static_cast<const void**>(end);
  };
  if (twice(std::copy(v, v + n, std::copy(k, k + n, all.get())))) return PA_ERR_ARG;
  if (scales && twice(std::copy(scales, scales + n, all.get()))) return PA_ERR_ARG;
  return PA_OK;
}

static int compact(void* const* k_caches, void* const* v_caches, float* const* kv_scales, int32_t num_layers,
                   const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                   const int32_t* path, const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len,
                   int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int elem_bytes,
                   bool kv8, bool e5, cudaStream_t stream) {
  auto aligned16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  if (num_seqs < 0 || num_layers < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || num_kv_heads < 1 || head_dim < 1 ||
      max_path_len < 1)
    return PA_ERR_ARG;
  if (block_size != 16 && block_size != 32) return PA_ERR_BLOCKSIZE;
  if (!elem_bytes) return PA_ERR_DTYPE;
  if (kv8 ? head_dim != 64 && head_dim != 128 : ((int64_t)head_dim * elem_bytes) % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (max_path_len > kCompactMaxPath) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_kv_heads * head_dim > (1 << 20)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_layers == 0) return PA_OK;
  if (!k_caches || !v_caches || (kv8 && !kv_scales) || !block_tables || !ctx_lens || !path || !path_lens)
    return PA_ERR_ARG;
  for (int32_t i = 0; i < num_layers; ++i) {
    if (!k_caches[i] || !v_caches[i] || (kv8 && !kv_scales[i])) return PA_ERR_ARG;
    if (!aligned16(k_caches[i]) || !aligned16(v_caches[i])) return PA_ERR_ALIGN;
    if (kv8 && (reinterpret_cast<uintptr_t>(kv_scales[i]) & 3u)) return PA_ERR_ALIGN;
  }
  const int twice = listed_twice(k_caches, v_caches, kv8 ? kv_scales : nullptr, num_layers);
  if (twice != PA_OK) return twice;
  int* st = device_status_ptr();
  if (!st) return PA_ERR_CUDA;
  CompactParams p{};
  p.block_tables = block_tables;
  p.ctx_lens = ctx_lens;
  p.path = path;
  p.path_lens = path_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_path_len = max_path_len;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.num_kv_heads = num_kv_heads;
  p.row_bytes = head_dim * elem_bytes;
  p.status = st;
  for (int32_t l0 = 0; l0 < num_layers; l0 += kCompactLayers) {
    CompactLayers pools{};
    p.num_layers = std::min(num_layers - l0, kCompactLayers);
    for (int32_t i = 0; i < p.num_layers; ++i) {
      pools.k[i] = k_caches[l0 + i];
      pools.v[i] = v_caches[l0 + i];
      if (kv8) pools.scales[i] = kv_scales[l0 + i];
    }
    const int64_t per_block = kv8 ? kCompactThreads / 32 : kCompactThreads;
    const int64_t items = (int64_t)p.num_layers * 2 * num_kv_heads * (kv8 ? 1 : p.row_bytes / 16);
    const dim3 grid(num_seqs, (unsigned)std::min<int64_t>((items + per_block - 1) / per_block, 65535));
    if (!kv8) compact_kernel<<<grid, kCompactThreads, 0, stream>>>(p, pools);
    else if (head_dim == 64 && e5) compact_8bit_kernel<2, true><<<grid, kCompactThreads, 0, stream>>>(p, pools);
    else if (head_dim == 64) compact_8bit_kernel<2, false><<<grid, kCompactThreads, 0, stream>>>(p, pools);
    else if (e5) compact_8bit_kernel<4, true><<<grid, kCompactThreads, 0, stream>>>(p, pools);
    else compact_8bit_kernel<4, false><<<grid, kCompactThreads, 0, stream>>>(p, pools);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

}  // namespace pa

extern "C" {

int pa_compact_tree(void* const* k_caches, void* const* v_caches, int32_t num_layers, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* ctx_lens, const int32_t* path,
                    const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len, int32_t num_blocks,
                    int32_t block_size, int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream) {
  const int eb = dtype == PA_F32 ? 4 : dtype == PA_F16 || dtype == PA_BF16 ? 2 : 0;
  return pa::compact(k_caches, v_caches, nullptr, num_layers, block_tables, max_blocks_per_seq, ctx_lens, path,
                     path_lens, num_seqs, max_path_len, num_blocks, block_size, num_kv_heads, head_dim, eb, false,
                     false, static_cast<cudaStream_t>(stream));
}

int pa_compact_tree_fp8(void* const* k_caches, void* const* v_caches, float* const* kv_scales, int32_t num_layers,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                        const int32_t* path, const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len,
                        int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                        void* stream) {
  return pa::compact(k_caches, v_caches, kv_scales, num_layers, block_tables, max_blocks_per_seq, ctx_lens, path,
                     path_lens, num_seqs, max_path_len, num_blocks, block_size, num_kv_heads, head_dim, 1, true,
                     false, static_cast<cudaStream_t>(stream));
}

int pa_compact_tree_e5m2(void* const* k_caches, void* const* v_caches, float* const* kv_scales, int32_t num_layers,
                         const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                         const int32_t* path, const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len,
                         int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                         void* stream) {
  return pa::compact(k_caches, v_caches, kv_scales, num_layers, block_tables, max_blocks_per_seq, ctx_lens, path,
                     path_lens, num_seqs, max_path_len, num_blocks, block_size, num_kv_heads, head_dim, 1, true,
                     true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

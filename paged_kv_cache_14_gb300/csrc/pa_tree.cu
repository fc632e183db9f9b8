// Tree attention over the paged cache: entry points, the CUDA-core kernel
// and the kernel that joins the pieces of a unit.
//
// One pass of a draft tree: node j of a sequence (its K/V cached at position
// ctx + j) attends to the ctx committed positions and to itself and its
// ancestors in the tree:
//   out[j] = sum_t exp(s_t - max s) v_t / sum_t exp(s_t - max s),
//   s_t = scale q[j] . k_t,  t in {0 .. ctx-1} and {ctx + a : a = j or above j}.
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pa_tree.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// fp32 I/O: exact fp32 arithmetic on CUDA cores. A query tile is 32 rows (row =
// node * group + head), a key tile 32 positions, four CTAs on an SM (two for
// head_dim above 128). 16 threads own four rows: each takes four rows x two
// keys of the scores, then four rows x every 16th float4 column of the output
// (a 16-byte shared-memory load takes four of the SM's cycles, so a thread has
// to use each for several rows). K and V arrive with cp.async in one buffer
// each: the next K flies while the values are added up, the next V while the
// scores are. Small calls are latency: 3 sequences of up to 1500, trees of 11,
// group 3, head_dim 96 give 351 CTAs about two key tiles each (the longest
// tree's 33 rows take two query tiles a KV head), 27 us from the scan of the
// lengths to the last store, and 6 us of join; one row a thread took 47.
// ---------------------------------------------------------------------------
namespace ts {
constexpr int kRows = 32;
constexpr int kPer = 16;   // threads of four rows
constexpr int kR = 4;      // rows of a thread
constexpr int kThreads = kRows / kR * kPer;
constexpr int kWs = kRows + 4;  // weights of one key
constexpr int kKeys = 32;
__host__ __device__ constexpr int per_sm(int d) { return d <= 128 ? 4 : 2; }
__host__ __device__ constexpr int smem_bytes(int d) {
  return (kRows * (d + 4) + kKeys * (d + 4) + kKeys * d + kKeys * kWs) * 4;
}
}  // namespace ts

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <int D>
__global__ void __launch_bounds__(ts::kThreads, ts::per_sm(D)) tree_simt_kernel(const TreeParams p) {
  using namespace ts;
  constexpr int kMine = kKeys / kPer, kCols = (D + 4 * kPer - 1) / (4 * kPer);
  constexpr int kGroups = kKeys / 16;  // 16-key groups of a tile: each in one block
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);  // [kRows][D + 4]
  float* ks = qs + kRows * (D + 4);             // [kKeys][D + 4]
  float* vs = ks + kKeys * (D + 4);             // [kKeys][D]
  float* ws = vs + kKeys * D;                   // [kKeys][kWs]
  __shared__ int64_t scan[kThreads / 16 + 2];
  __shared__ int blk[2][kGroups];

  pdl_trigger();
  const TreeRange range = tree_range<kThreads>(p, scan);
  if (threadIdx.x == 0) p.merge[blockIdx.x].parts = 0;
  const int row0 = threadIdx.x / kPer * kR, part = threadIdx.x % kPer;
  TreeWalk walk(p, range);
  TreePiece c;
  while (walk.next(p, c)) {
    const int32_t* parents = p.parents + c.s.q0;
    tree_check_parents<kThreads>(p, c, threadIdx.x);
    const int32_t* table = p.block_tables + (int64_t)c.seq * p.max_blocks_per_seq;
    const int rows = c.s.nodes * p.group;
    const int r0 = c.qt * kRows + row0;  // this thread's first row of the unit
    const bool live = c.qt * kRows + (threadIdx.x >> 5) * (32 / kPer * kR) < rows;  // the warp has rows
    const int kv_len = c.kv_len();
    auto load_blocks = [&](int t) {  // ids of tile t's blocks, -1 for none
      if (threadIdx.x < kGroups && t < c.t1) {
        const int pos = t * kKeys + threadIdx.x * 16;
        int id = -1;
        if (pos < kv_len) {
          id = table[pos / p.block_size];
          if (id < 0 || id >= p.num_blocks) {
            record_error(p.status, PA_ERR_BLOCK_OOB);
            id = -1;
          }
        }
        blk[t & 1][threadIdx.x] = id;
      }
    };
    auto load_tile = [&](int t, const void* pool, float* to, int stride) {
      if (t < c.t1) {
        for (int i = threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
          const int key = i / (D / 4), d4 = (i - key * (D / 4)) * 4, pos = t * kKeys + key;
          const int id = blk[t & 1][key / 16];
          const bool real = id >= 0 && pos < kv_len;  // else zeros
          const int64_t at =
              real ? (((int64_t)id * p.num_kv_heads + c.kvh) * p.block_size + pos % p.block_size) * D + d4 : 0;
          cp_async16(smem_u32(to + key * stride + d4), static_cast<const float*>(pool) + at, real);
        }
      }
      cp_async_commit();  // (an empty group behind the last tile keeps the count)
    };
    __syncthreads();  // the previous piece is done with the buffers
    load_blocks(c.t0);
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int rr = i / (D / 4), d4 = (i - rr * (D / 4)) * 4;
      const int ur = c.qt * kRows + rr;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ur < rows) {
        const int nd = ur / p.group, h = c.kvh * p.group + ur - nd * p.group;
        x = __ldg(reinterpret_cast<const float4*>(
            static_cast<const float*>(p.q) + ((int64_t)(c.s.q0 + nd) * p.num_q_heads + h) * D + d4));
      }
      *reinterpret_cast<float4*>(qs + rr * (D + 4) + d4) = x;
    }
    __syncthreads();
    load_tile(c.t0, p.k_cache, ks, D + 4);
    load_tile(c.t0, p.v_cache, vs, D);
    float m[kR], l[kR];
    float4 o[kR][kCols];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = c.t0; t < c.t1; ++t) {
      const int k0 = t * kKeys;
      cp_async_wait<1>();
      __syncthreads();  // K(t) is here
      load_blocks(t + 1);
      uint32_t seen[kR];
      const bool masked = k0 + kKeys > c.s.ctx;
      if (live) {
      float s[kR][kMine];
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int j = 0; j < kMine; ++j) s[i][j] = 0.f;
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        float4 qv[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) qv[i] = *reinterpret_cast<const float4*>(qs + (row0 + i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const float4 kv = *reinterpret_cast<const float4*>(ks + (part + kPer * j) * (D + 4) + d);
#pragma unroll
          for (int i = 0; i < kR; ++i)
            s[i][j] = fmaf(qv[i].x, kv.x, fmaf(qv[i].y, kv.y, fmaf(qv[i].z, kv.z, fmaf(qv[i].w, kv.w, s[i][j]))));
        }
      }
      // Keys that a row sees, one bit each.
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        seen[i] = 0xffffffffu;
        if (masked) {
          const int first = k0 - c.s.ctx;  // node of the tile's first key (below 0: context)
          seen[i] = tree_ancestors(parents, min((r0 + i) / p.group, c.s.nodes - 1), first);
          if (first < 0) seen[i] |= (1u << -first) - 1u;
        }
      }
      float alpha[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          s[i][j] = (seen[i] >> (part + kPer * j)) & 1u ? s[i][j] * p.scale_log2 : -CUDART_INF_F;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int x = 1; x < kPer; x *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        // A row that has seen no key yet keeps m = -inf and l = 0.
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        alpha[i] = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          s[i][j] = exp2f(s[i][j] - ref);
          sum += s[i][j];
        }
#pragma unroll
        for (int x = 1; x < kPer; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[i] = l[i] * alpha[i] + sum;
        m[i] = mx;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          o[i][j].x *= alpha[i], o[i][j].y *= alpha[i], o[i][j].z *= alpha[i], o[i][j].w *= alpha[i];
      }
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        *reinterpret_cast<float4*>(ws + (part + kPer * j) * kWs + row0) =
            make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      }
      cp_async_wait<0>();
      __syncthreads();  // V(t) and the weights are here, K(t) is read
      load_tile(t + 1, p.k_cache, ks, D + 4);
      // Weights behind the mask are 0, which takes the values there out unless
      // one is not finite: only a tile that holds such a value looks at the
      // mask again.
      bool dirty = false;
      if (masked) {
        for (int i = max(c.s.ctx - k0, 0) * (D / 4) + threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
          const float4 v = reinterpret_cast<const float4*>(vs)[i];
          dirty |= !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < CUDART_INF_F);
        }
        dirty = __syncthreads_or(dirty);
      }
      auto add = [&](int key, bool check) {
        const float4 w4 = *reinterpret_cast<const float4*>(ws + key * kWs + row0);
        const float w[kR] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int d4 = (part + kPer * j) * 4;
          if (D % (4 * kPer) != 0 && j == kCols - 1 && d4 >= D) continue;
          const float4 v = *reinterpret_cast<const float4*>(vs + key * D + d4);
#pragma unroll
          for (int i = 0; i < kR; ++i) {
            if (check && !((seen[i] >> key) & 1u)) continue;
            o[i][j].x = fmaf(w[i], v.x, o[i][j].x);
            o[i][j].y = fmaf(w[i], v.y, o[i][j].y);
            o[i][j].z = fmaf(w[i], v.z, o[i][j].z);
            o[i][j].w = fmaf(w[i], v.w, o[i][j].w);
          }
        }
      };
      if (live && !dirty) {
#pragma unroll 4
        for (int key = 0; key < kKeys; ++key) add(key, false);
      } else if (live) {
#pragma unroll 1
        for (int key = 0; key < kKeys; ++key) add(key, true);
      }
      __syncthreads();  // V(t) and the weights are read
      load_tile(t + 1, p.v_cache, vs, D);
    }
    cp_async_wait<0>();
    const bool whole = c.whole();
    if (!whole && c.t0 == 0 && threadIdx.x == 0) tree_note_merge(p, range, c);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int r = r0 + i, node = r / p.group, h = c.kvh * p.group + r - node * p.group;
      if (r >= rows) break;
      const float f = whole ? 1.f / l[i] : 1.f;
      const int64_t slot = (int64_t)tree_slot(c) * kRows + row0 + i;
      float* to = whole ? static_cast<float*>(p.out) + ((int64_t)(c.s.q0 + node) * p.num_q_heads + h) * D
                        : p.part_o + slot * D;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int d4 = (part + kPer * j) * 4;
        if (d4 < D) store4(to + d4, make_float4(o[i][j].x * f, o[i][j].y * f, o[i][j].z * f, o[i][j].w * f));
      }
      if (!whole && part == 0) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m[i], l[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Join: block (b, y) joins rows of the unit that CTA b began and did not
// finish. m in log2 units: out = sum_i 2^(m_i - M) o~_i / sum_i 2^(m_i - M) l_i.
// What it costs is latency: two rounds of dependent loads, and a thousand small
// blocks. With few pieces (where many units are split, as in any large batch)
// a warp takes four rows and four pieces of each at once; with more (few
// units, a long context), one row and 16 pieces at once. Pieces are added up
// in their order either way. After the attention's end it takes 6 us for 64
// sequences of 4096 (15 MB of partials), 7 to 11 us for 30 MB of them, 6 us for
// 4 of 131072 and 3 us for one short one.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 4;
constexpr int kJoinFew = 4;  // pieces of a unit that four rows' loads cover

// ROWS rows from r0 on; lane i * LOOK + k looks after piece k of row i.
template <typename T, int ROWS, int BATCH>
__device__ __forceinline__ void join_rows(const TreeParams& p, const TreeMerge& mg, int rows, int r0) {
  constexpr int LOOK = 32 / ROWS;  // pieces whose weights are at hand
  static_assert(LOOK % BATCH == 0, "whole batches");
  const int D = p.head_dim, lane = threadIdx.x & 31, parts = mg.parts;
  // Piece k of row r: slot 2b + 1 for the first, 2 (b + k team) for the others.
  auto slot = [&](int r, int k) -> int64_t {
    return (int64_t)(2 * (blockIdx.x + k * p.team) + (k == 0 ? 1 : 0)) * p.tile_m + r;
  };
  const int mr = min(r0 + lane / LOOK, rows - 1), mk = lane % LOOK;
  auto piece_ml = [&](int k) -> float2 {
    return k < parts ? __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot(mr, k) * 2))
                     : make_float2(-CUDART_INF_F, 0.f);
  };
  const float2 first = piece_ml(mk);
  float M = first.x;
  for (int k = LOOK + mk; k < parts; k += LOOK) M = fmaxf(M, piece_ml(k).x);
#pragma unroll
  for (int o = 1; o < LOOK; o *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  for (int d0 = 0; d0 < D; d0 += 128) {
    const int d4 = d0 + lane * 4;
    float4 acc[ROWS];
    float L = 0.f;  // of row mr
#pragma unroll
    for (int i = 0; i < ROWS; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += LOOK) {
      const float2 ml = k0 == 0 ? first : piece_ml(k0 + mk);
      // A piece whose keys the row sees none of (m = -inf, l = 0) weighs
      // nothing, whatever the row's maximum is. One that weighs next to
      // nothing still counts: 0 times an infinity or NaN that the row sees is
      // NaN, as it is within a piece.
      const float w = ml.x == -CUDART_INF_F && ml.y == 0.f ? 0.f : exp2f(ml.x - M);
      L += w * ml.y;
#pragma unroll
      for (int k1 = 0; k1 < LOOK; k1 += BATCH) {
        if (k0 + k1 >= parts) break;
        float4 v[ROWS][BATCH];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            v[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r0 + i < rows && k0 + k1 + k < parts && d4 < D)
              v[i][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot(r0 + i, k0 + k1 + k) * D + d4));
          }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const float wk = __shfl_sync(0xffffffffu, w, i * LOOK + k1 + k);
            acc[i].x = fmaf(wk, v[i][k].x, acc[i].x);
            acc[i].y = fmaf(wk, v[i][k].y, acc[i].y);
            acc[i].z = fmaf(wk, v[i][k].z, acc[i].z);
            acc[i].w = fmaf(wk, v[i][k].w, acc[i].w);
          }
      }
    }
#pragma unroll
    for (int o = 1; o < LOOK; o *= 2) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float inv = 1.f / __shfl_sync(0xffffffffu, L, i * LOOK);
      if (r0 + i < rows && d4 < D) {
        const int ur = mg.qt * p.tile_rows + r0 + i;
        const int node = ur / p.group, h = mg.kvh * p.group + ur - node * p.group;
        store4(static_cast<T*>(p.out) + ((int64_t)(mg.q0 + node) * p.num_q_heads + h) * D + d4,
               make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const TreeParams p) {
  pdl_wait();
  const TreeMerge mg = p.merge[blockIdx.x];
  if (mg.parts == 0) return;
  const int rows = min(p.tile_rows, mg.nodes * p.group - mg.qt * p.tile_rows);
  const int w = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (mg.parts <= kJoinFew) {
    if (w * 4 < rows) join_rows<T, 4, kJoinFew>(p, mg, rows, w * 4);
  } else {
    for (int r = w; r < rows; r += gridDim.y * kJoinWarps) join_rows<T, 1, 16>(p, mg, rows, r);
  }
}

template <int D>
static int run_simt(const TreeParams& p, int ctas, cudaStream_t stream) {
  auto kern = tree_simt_kernel<D>;
  constexpr int smem = ts::smem_bytes(D);
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem) != PA_OK) return PA_ERR_CUDA;
  kern<<<ctas, ts::kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

static int launch_tree_simt(const TreeParams& p, int ctas, cudaStream_t stream) {
  switch (p.head_dim) {
    case 32: return run_simt<32>(p, ctas, stream);
    case 64: return run_simt<64>(p, ctas, stream);
    case 96: return run_simt<96>(p, ctas, stream);
    case 128: return run_simt<128>(p, ctas, stream);
    case 160: return run_simt<160>(p, ctas, stream);
    case 192: return run_simt<192>(p, ctas, stream);
    case 224: return run_simt<224>(p, ctas, stream);
    case 256: return run_simt<256>(p, ctas, stream);
  }
  return PA_ERR_UNSUPPORTED;
}

static int launch_tree_join(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream) {
  // Enough warps for four rows each where units are split into few pieces on
  // average, for one row each otherwise (10^4 blocks that mostly find nothing
  // to do cost 3 us more than a quarter of them).
  const int64_t units = (int64_t)std::min(p.num_seqs, p.total_q) * p.num_kv_heads;
  const int per_block = units * kJoinFew >= ctas ? 4 * kJoinWarps : kJoinWarps;
  const dim3 grid(ctas, (p.tile_rows + per_block - 1) / per_block), block(32 * kJoinWarps);
  cudaError_t e;
  if (dt == PA_F32) e = launch_dependent(tree_join_kernel<float>, grid, block, 0, stream, p);
  else if (dt == PA_F16) e = launch_dependent(tree_join_kernel<__half>, grid, block, 0, stream, p);
  else e = launch_dependent(tree_join_kernel<__nv_bfloat16>, grid, block, 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

namespace {

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// Tiles, grid and workspace of a call; what the size query and the launch share.
struct TreeLayout {
  int rc = PA_OK;
  int ctas = 0, tile_rows = 0, tile_m = 0, tile_keys = 0, team = 1, piece_cost = 1;
  size_t merge = 0, part_o = 0, part_ml = 0, total = 0;
};

TreeLayout tree_layout(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int32_t total_q, int32_t max_q_len, int32_t max_kv_len, pa_dtype dt) {
  TreeLayout w;
  auto fail = [&](int rc) {
    w.rc = rc;
    return w;
  };
  if (num_seqs < 0 || total_q < 0 || head_dim < 1 || num_q_heads < 1 || num_kv_heads < 1) return fail(PA_ERR_ARG);
  if (num_q_heads % num_kv_heads) return fail(PA_ERR_HEADS);
  if (block_size != 16 && block_size != 32) return fail(PA_ERR_BLOCKSIZE);
  if (dt != PA_F32 && dt != PA_F16 && dt != PA_BF16) return fail(PA_ERR_DTYPE);
  const int group = num_q_heads / num_kv_heads;
  if (dt == PA_F32) {
    if (head_dim < 32 || head_dim > 256 || head_dim % 32) return fail(PA_ERR_UNSUPPORTED);
  } else if ((head_dim != 64 && head_dim != 128) || group > 128) {
    return fail(PA_ERR_UNSUPPORTED);
  }
  if (num_seqs == 0 || total_q == 0) return w;
  if (max_q_len < 1 || max_kv_len < 1) return fail(PA_ERR_ARG);
  if (num_seqs > 65535 || max_q_len > kMaxTreeNodes) return fail(PA_ERR_UNSUPPORTED);
  int per_sm;
  if (dt == PA_F32) {
    w.tile_rows = w.tile_m = ts::kRows;
    w.tile_keys = ts::kKeys;
    w.piece_cost = 12;
    per_sm = ts::per_sm(head_dim);
  } else {
    w.tile_m = kTreeTcRows;
    w.tile_rows = kTreeTcRows / group * group;
    w.tile_keys = kTreeTcKeys;
    w.piece_cost = 3;
    per_sm = 2;
    // Teams of two where trees may fill several query tiles, of an even number of
    // KV heads (an odd one would leave a member idle at every odd last tile).
    if ((int64_t)max_q_len * group > w.tile_rows && num_kv_heads % 2 == 0) w.team = 2;
  }
  // Most key tiles there can be: one more query tile than its rows fill for every sequence.
  const double units = ((double)total_q * group / w.tile_rows + std::min(num_seqs, total_q)) * num_kv_heads;
  const double most = units * (((int64_t)max_kv_len + w.tile_keys - 1) / w.tile_keys) + 1;
  w.ctas = (int)std::max(1.0, std::min(most, (double)per_sm * num_sms_current_device()));
  w.ctas = (w.ctas + w.team - 1) / w.team * w.team;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.part_o = up((size_t)w.ctas * sizeof(TreeMerge));
  w.part_ml = up(w.part_o + (size_t)2 * w.ctas * w.tile_m * head_dim * 4);
  w.total = up(w.part_ml + (size_t)2 * w.ctas * w.tile_m * 2 * 4);
  return w;
}

int decode_tree(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents, const void* k_cache,
                const void* v_cache, const float* kv_scales, int32_t kv_fmt, const int32_t* block_tables,
                int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype,
                bool kv8, cudaStream_t stream) {
  const TreeLayout w = tree_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, total_q, max_q_len,
                                   max_kv_len, dtype);
  if (w.rc != PA_OK) return w.rc;
  if (max_blocks_per_seq < 1 || num_blocks < 1 || !std::isfinite(scale)) return PA_ERR_ARG;
  if (dtype != PA_F32 && !(scale > 0.f)) return PA_ERR_ARG;
  if (kv8 && dtype == PA_F32) return PA_ERR_DTYPE;
  if (kv8 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  // (Rows are 32-bit coordinates of a tensor map there.)
  if (dtype != PA_F32 && (int64_t)num_blocks * num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (!q || !cu_q_lens || !parents || !k_cache || !v_cache || !block_tables || !ctx_lens || !out) return PA_ERR_ARG;
  if (kv8 && !kv_scales) return PA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(kv_scales))
    return PA_ERR_ALIGN;
  if (!workspace || workspace_bytes < w.total) return PA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PA_ERR_ALIGN;
  int* st = device_status_ptr();
  if (!st) return PA_ERR_CUDA;
  TreeParams p{};
  p.q = q;
  p.out = out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_scales = kv_scales;
  p.kv_fmt = kv_fmt;
  p.block_tables = block_tables;
  p.cu_q_lens = cu_q_lens;
  p.parents = parents;
  p.ctx_lens = ctx_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  // Positions are 32-bit, also that behind a last tile.
  p.max_kv_len = std::min(max_kv_len, INT32_MAX - 63);
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.group = num_q_heads / num_kv_heads;
  p.tile_rows = w.tile_rows;
  p.tile_m = w.tile_m;
  p.tile_keys = w.tile_keys;
  p.team = w.team;
  p.piece_cost = w.piece_cost;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.merge = reinterpret_cast<TreeMerge*>(ws + w.merge);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  p.status = st;
  const int rc = dtype == PA_F32 ? launch_tree_simt(p, w.ctas, stream) : launch_tree_tc(p, w.ctas, dtype, stream);
  if (rc != PA_OK) return rc;
  return launch_tree_join(p, w.ctas, dtype, stream);
}
}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_tree_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t block_size, int32_t total_q, int32_t max_q_len, int32_t max_kv_len,
                                     pa_dtype dtype) {
  const pa::TreeLayout w = pa::tree_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, total_q,
                                           max_q_len, max_kv_len, dtype);
  return w.rc == PA_OK ? w.total : 0;
}

int pa_decode_tree(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                   const void* k_cache, const void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                   const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes,
                   pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, nullptr, 0, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, false,
                         static_cast<cudaStream_t>(stream));
}

int pa_decode_tree_fp8(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                       const void* k_cache, const void* v_cache, const float* kv_scales, const int32_t* block_tables,
                       int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                       int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int32_t num_blocks, float scale, void* out, void* workspace,
                       size_t workspace_bytes, pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, kv_scales, pa::PA_KV_E4M3, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, true,
                         static_cast<cudaStream_t>(stream));
}

int pa_decode_tree_e5m2(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                        const void* k_cache, const void* v_cache, const float* kv_scales,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                        int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                        void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, kv_scales, pa::PA_KV_E5M2, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, true,
                         static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// Block summaries, and the choice of the blocks that a decode query attends
// to.
//
// A summary is the range of every key dimension over a block's tokens, in 8
// bits: with s = max |k| / 127, hi = ceil(max_t k / s) and lo =
// floor(min_t k / s). For a query in 8 bits, q = s_q * code, no key of the
// block has a larger product with it than
//   s_q s  sum_d max(code_d hi_d, code_d lo_d),
// whose sum is a whole number below 2^22. Scores are therefore exact up to two
// fp32 products in a fixed order: the choice does not depend on the order in
// which the device runs, and a tie goes to the lower block.
#include <algorithm>
#include <climits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// ---------------------------------------------------------------------------
// Summaries
// ---------------------------------------------------------------------------

struct SummaryParams {
  const void* k_cache;
  const float* kv_scales;
  const int32_t* block_tables;
  const int32_t* first_tokens;
  const int32_t* seq_lens;
  int8_t* summaries;
  float* scales;
  int32_t max_blocks_per_seq, num_seqs, max_new_tokens, num_blocks, block_size, num_kv_heads, head_dim;
  int32_t seq_blocks;  // blocks of a sequence that a call may summarise
  int64_t items;
  int* status;
};

constexpr int kSummaryThreads = 256;

// A warp's item: the block to summarise, its rows and KV head; false if there
// is nothing to do.
__device__ __forceinline__ bool summary_item(const SummaryParams& p, int64_t item, bool report, int64_t& blk,
                                             int& rows, int& head) {
  head = (int)(item % p.num_kv_heads);
  const int64_t rest = item / p.num_kv_heads;
  const int seq = (int)(rest / p.seq_blocks), j = (int)(rest - (int64_t)seq * p.seq_blocks);
  const int first = p.first_tokens[seq], len = p.seq_lens[seq];
  report = report && head == 0;
  if (first < 0 || len < first || len - first > p.max_new_tokens) {
    if (report && j == 0) record_error(p.status, PA_ERR_SEQLEN);
    return false;
  }
  if (len == first) return false;
  const int lb = first / p.block_size + j;
  if (lb > (len - 1) / p.block_size) return false;
  if (lb >= p.max_blocks_per_seq) {
    if (report) record_error(p.status, PA_ERR_SEQLEN);
    return false;
  }
  blk = p.block_tables[(int64_t)seq * p.max_blocks_per_seq + lb];
  if (blk < 0 || blk >= p.num_blocks) {
    if (report) record_error(p.status, PA_ERR_BLOCK_OOB);
    return false;
  }
  rows = min(p.block_size, len - lb * p.block_size);
  return true;
}

// The scale of values of at most `top` in size: infinite where they are not
// all finite.
__device__ __forceinline__ float summary_scale(float top) {
  return top <= 3.402823466e38f ? __fdiv_rn(top, 127.f) : __int_as_float(0x7f800000);
}
__device__ __forceinline__ int code_up(float x, float scale) {
  return scale > 0.f && scale <= 3.402823466e38f ? (int)fminf(ceilf(__fdiv_rn(x, scale)), 127.f) : 0;
}
__device__ __forceinline__ int code_down(float x, float scale) {
  return scale > 0.f && scale <= 3.402823466e38f ? (int)fmaxf(floorf(__fdiv_rn(x, scale)), -127.f) : 0;
}
// Maximum and minimum that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct HalfRange {
  using T2 = __half2;
  __device__ __forceinline__ static uint32_t top(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ static uint32_t low(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ static float2 wide(uint32_t a) {
    return __half22float2(*reinterpret_cast<const __half2*>(&a));
  }
};
struct Bf16Range {
  __device__ __forceinline__ static uint32_t top(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ static uint32_t low(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ static float2 wide(uint32_t a) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&a));
  }
};

// 16-bit rows, or 8-bit codes (KV8: 1 e4m3, 2 e5m2) widened to fp16. A warp
// per (block, KV head): a lane takes 16 bytes of a row, RPP rows at a time.
template <typename R, int D, int KV8>
__global__ void __launch_bounds__(kSummaryThreads) summary_kernel(const __grid_constant__ SummaryParams p) {
  constexpr int E = KV8 ? 16 : 8;      // elements of a lane
  constexpr int VPR = D / E;           // lanes of a row
  constexpr int RPP = 32 / VPR;        // rows of a pass
  constexpr int W = E / 2;             // packed pairs of a lane
  constexpr int NR = 16 / RPP;         // passes of 16 rows
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * (int64_t)(kSummaryThreads / 32) + (threadIdx.x >> 5);
  if (item >= p.items) return;
  int64_t blk;
  int rows, head;
  if (!summary_item(p, item, lane == 0, blk, rows, head)) return;
  const int64_t at = blk * p.num_kv_heads + head;
  const uint8_t* src = static_cast<const uint8_t*>(p.k_cache) + at * p.block_size * D * (KV8 ? 1 : 2) +
                       (lane % VPR) * 16;
  uint32_t hi[W], lo[W];
  bool started = false;
  for (int r0 = 0; r0 < rows; r0 += 16) {
    uint4 raw[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      // Behind the last row: the last once more.
      const int r = min(r0 + i * RPP + lane / VPR, rows - 1);
      raw[i] = *reinterpret_cast<const uint4*>(src + r * (D * (KV8 ? 1 : 2)));
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t x[W];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (KV8 == 0) x[j] = w[j];
        else fp8x4_to_f16x4<KV8 == 2>(w[j], x[2 * j], x[2 * j + 1]);
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        hi[j] = started || i ? R::top(hi[j], x[j]) : x[j];
        lo[j] = started || i ? R::low(lo[j], x[j]) : x[j];
      }
    }
    started = true;
  }
#pragma unroll
  for (int o = VPR; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      hi[j] = R::top(hi[j], __shfl_xor_sync(kAll, hi[j], o));
      lo[j] = R::low(lo[j], __shfl_xor_sync(kAll, lo[j], o));
    }
  }
  const float mul = KV8 ? p.kv_scales[at * 2] : 1.f;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const float2 a = R::wide(hi[j]), b = R::wide(lo[j]);
    top = max_nan(top, max_nan(max_nan(fabsf(a.x), fabsf(a.y)), max_nan(fabsf(b.x), fabsf(b.y))));
  }
#pragma unroll
  for (int o = 1; o < VPR; o <<= 1) top = max_nan(top, __shfl_xor_sync(kAll, top, o));
  const float scale = summary_scale(KV8 ? fabsf(__fmul_rn(top, mul)) : top);
  // The first lanes of a row's write the upper ends, the next ones the lower.
  const int part = lane / VPR;
  if (part < 2) {
    uint32_t out[E / 4];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 v = R::wide(part ? lo[j] : hi[j]);
      const float x = KV8 ? __fmul_rn(v.x, mul) : v.x, y = KV8 ? __fmul_rn(v.y, mul) : v.y;
      const int c0 = part ? code_down(x, scale) : code_up(x, scale);
      const int c1 = part ? code_down(y, scale) : code_up(y, scale);
      const uint32_t two = (c0 & 255) | (c1 & 255) << 8;
      if (j & 1) out[j / 2] |= two << 16;
      else out[j / 2] = two;
    }
    int8_t* dst = p.summaries + (at * 2 + part) * D + (lane % VPR) * E;
    if constexpr (KV8 != 0) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  }
  if (lane == 0) p.scales[at] = scale;
}

// fp32 rows of 32 N elements, a lane taking every 32nd.
template <int N>
__global__ void __launch_bounds__(kSummaryThreads) summary_f32_kernel(const __grid_constant__ SummaryParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * (int64_t)(kSummaryThreads / 32) + (threadIdx.x >> 5);
  if (item >= p.items) return;
  int64_t blk;
  int rows, head;
  if (!summary_item(p, item, lane == 0, blk, rows, head)) return;
  const int64_t at = blk * p.num_kv_heads + head;
  const float* src = static_cast<const float*>(p.k_cache) + at * p.block_size * (32 * N) + lane;
  float hi[N], lo[N], top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) hi[i] = lo[i] = src[32 * i];
  for (int r = 1; r < rows; ++r) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = src[r * (32 * N) + 32 * i];
      hi[i] = max_nan(hi[i], x);
      lo[i] = min_nan(lo[i], x);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) top = max_nan(top, max_nan(fabsf(hi[i]), fabsf(lo[i])));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float scale = summary_scale(top);
  int8_t* dst = p.summaries + at * 2 * (32 * N) + lane;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    dst[32 * i] = (int8_t)code_up(hi[i], scale);
    dst[32 * N + 32 * i] = (int8_t)code_down(lo[i], scale);
  }
  if (lane == 0) p.scales[at] = scale;
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------

struct SelectParams {
  const void* q;
  const int8_t* summaries;
  const float* scales;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int32_t* lists;
  int32_t* list_lens;
  int32_t max_blocks_per_seq, num_seqs, max_seq_len, num_q_heads, num_kv_heads, num_blocks, block_size, group;
  int32_t max_list_len, num_sink, num_recent, head_tiles;
  int* status;
};

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectMaxCluster = 8;
constexpr int kSelectTile = 16;  // blocks of one matrix product

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ int remote_int(const void* local, int rank) {
  uint32_t a;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Scores as unsigned numbers of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // one zero
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Four signed bytes to two pairs of fp16, exactly: with the sign bit flipped
// a byte is code + 128, and behind the byte 0x64 it is the mantissa of
// 1024 + 128 + code.
__device__ __forceinline__ void s8x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const uint32_t bias = 0xe480e480u;  // -1152
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

// Exclusive prefix sum over the CTA's threads; `scratch` is kSelectWarps + 1
// ints. Contains barriers.
__device__ __forceinline__ int select_scan(int v, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) scratch[w] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSelectWarps; ++i) {
    const int s = scratch[i];
    before += i < w ? s : 0;
    total += s;
  }
  return before + x - v;
}

// One cluster per (sequence, KV head). Its CTAs split the row's blocks, score
// them 16 at a time on the tensor cores (codes up to 127 are exact in fp16,
// their products' sums exact in fp32), keep the scores in shared memory, and
// find the score of the last block to take by counting digits of 8 bits from
// the top, a cluster-wide histogram each.
template <typename T, int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int Q2 = 2 * D + 4;  // fp16 of a query row in shared memory: 8 bytes on, so that rows take other banks
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int hist[4][256];
  __shared__ int scratch[kSelectWarps];
  __shared__ int range[2], totals[2], found[3];
  __half* qs = reinterpret_cast<__half*>(smem);
  float* q_scale = reinterpret_cast<float*>(smem + p.head_tiles * 8 * Q2 * 2);
  uint32_t* keys = reinterpret_cast<uint32_t*>(q_scale + p.head_tiles * 8);
  int ranks, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int row = blockIdx.x / ranks, seq = row / p.num_kv_heads, head = row - seq * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  int32_t* list = p.lists + (int64_t)row * p.max_list_len;
  const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
  const int len = p.seq_lens[seq];
  int nb = len > 0 ? (len - 1) / p.block_size + 1 : 0;
  if (len < 0 || len > p.max_seq_len || nb > p.max_blocks_per_seq) {
    if (rank == 0 && tid == 0 && head == 0) record_error(p.status, PA_ERR_SEQLEN);
    nb = 0;
  }
  if (nb <= p.max_list_len) {  // all of them (the same for the whole cluster)
    for (int i = rank * kSelectThreads + tid; i < p.max_list_len; i += ranks * kSelectThreads)
      list[i] = i < nb ? i : -1;
    if (rank == 0 && tid == 0) p.list_lens[row] = nb;
    return;
  }
  for (int i = tid; i < 4 * 256; i += kSelectThreads) (&hist[0][0])[i] = 0;
  // The queries' codes, their positive and their negative part.
  for (int h = warp; h < p.head_tiles * 8; h += kSelectWarps) {
    float x[D / 32], top = 0.f;
    const bool there = h < p.group;
    const T* q = static_cast<const T*>(p.q) + ((int64_t)seq * p.num_q_heads + head * p.group + (there ? h : 0)) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[i] = there ? to_f32(q[lane + 32 * i]) : 0.f;
      top = fabsf(x[i]) <= 3.402823466e38f ? fmaxf(top, fabsf(x[i])) : __int_as_float(0x7f800000);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    // (A row that is not all finite counts as zeros.)
    const float scale = top <= 3.402823466e38f ? __fdiv_rn(top, 127.f) : 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float code = scale > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], scale)), -127.f), 127.f) : 0.f;
      qs[h * Q2 + lane + 32 * i] = __float2half_rn(fmaxf(code, 0.f));
      qs[h * Q2 + D + lane + 32 * i] = __float2half_rn(fminf(code, 0.f));
    }
    if (lane == 0) q_scale[h] = scale;
  }
  __syncthreads();
  const int sink = p.num_sink, some = nb - sink - p.num_recent;  // blocks that compete
  int need = p.max_list_len - sink - p.num_recent;               // of which so many are taken
  const int chunk = ((some + ranks - 1) / ranks + kSelectTile - 1) / kSelectTile * kSelectTile;
  const int lo = min(rank * chunk, some), mine = min(chunk, some - lo);
  uint32_t kmin = 0xffffffffu, kmax = 0;
  for (int b0 = warp * kSelectTile; b0 < mine; b0 += kSelectWarps * kSelectTile) {
    // Lane (r, c) reads 16 bytes of each 64 of the rows of blocks r and r + 8.
    uint4 a[2][D / 32];
    float mul[2];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = b0 + r + 8 * i;
      const int32_t blk = b < mine ? table[sink + lo + b] : 0;
      ok[i] = blk >= 0 && blk < p.num_blocks;
      const int64_t at = (int64_t)(ok[i] ? blk : 0) * p.num_kv_heads + head;
      mul[i] = p.scales[at];
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        a[i][j] = *reinterpret_cast<const uint4*>(p.summaries + at * 2 * D + 64 * j + 16 * c);
    }
    float best[2] = {__int_as_float(0xff800000), __int_as_float(0xff800000)};
    for (int n = 0; n < p.head_tiles; ++n) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const __half* qn = qs + (n * 8 + r) * Q2 + 16 * c;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint32_t w0[4] = {a[0][j].x, a[0][j].y, a[0][j].z, a[0][j].w};
        const uint32_t w1[4] = {a[1][j].x, a[1][j].y, a[1][j].z, a[1][j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t f[4];
          s8x4_to_f16x4(w0[k], f[0], f[2]);
          s8x4_to_f16x4(w1[k], f[1], f[3]);
          const uint2 b = *reinterpret_cast<const uint2*>(qn + 64 * j + 4 * k);
          MmaOp<__half>::run(acc, f, b.x, b.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = n * 8 + 2 * c + i;
        if (h < p.group) {
          best[0] = fmaxf(best[0], __fmul_rn(acc[i], q_scale[h]));
          best[1] = fmaxf(best[1], __fmul_rn(acc[2 + i], q_scale[h]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      best[i] = fmaxf(best[i], __shfl_xor_sync(kAll, best[i], 1));
      best[i] = fmaxf(best[i], __shfl_xor_sync(kAll, best[i], 2));
      const int b = b0 + r + 8 * i;
      if (c == 0 && b < mine) {
        // A block with keys that are not finite comes before all others.
        // (Scale 0: all its keys are 0, whatever else overflows.)
        uint32_t key = !(mul[i] <= 3.402823466e38f) ? 0xff800000u
                                                    : ordered(mul[i] == 0.f ? 0.f : __fmul_rn(best[i], mul[i]));
        if (!ok[i]) {
          record_error(p.status, PA_ERR_BLOCK_OOB);
          key = 0;
        }
        keys[b] = key;
        kmin = min(kmin, key);
        kmax = max(kmax, key);
      }
    }
  }
  // The row's range: digits are counted of key - kmin, from its top bit down.
  if (tid == 0) {
    range[0] = (int)0xffffffffu;
    range[1] = 0;
  }
  __syncthreads();
  kmin = __reduce_min_sync(kAll, kmin);
  kmax = __reduce_max_sync(kAll, kmax);
  if (lane == 0) {
    atomicMin(reinterpret_cast<uint32_t*>(&range[0]), kmin);
    atomicMax(reinterpret_cast<uint32_t*>(&range[1]), kmax);
  }
  cluster_sync_all();
  for (int i = 0; i < ranks; ++i) {
    kmin = min(kmin, (uint32_t)remote_int(&range[0], i));
    kmax = max(kmax, (uint32_t)remote_int(&range[1], i));
  }
  // Keys from `base` on are still in question; those above `over` are taken.
  int bits = 32 - __clz(kmax - kmin);
  uint32_t base = kmin, width = kmax - kmin;  // keys base .. base + width
  int pass = 0;
  bool whole = false;  // all keys in question are taken
  while (need > 0 && bits > 0 && !whole) {
    const int shift = max(bits - 8, 0);
    for (int i = tid; i < mine; i += kSelectThreads) {
      const uint32_t x = keys[i] - base;
      if (keys[i] >= base && x <= width) atomicAdd(&hist[pass][x >> shift], 1);
    }
    cluster_sync_all();
    // Thread t counts digit 255 - t; the first digits from the top that make
    // up `need` end in the one looked for.
    int count = 0, total;
    for (int i = 0; i < ranks; ++i) count += remote_int(&hist[pass][255 - tid], i);
    const int above = select_scan(count, scratch, total);
    if (above < need && above + count >= need) {
      found[0] = 255 - tid;
      found[1] = above;
      found[2] = count;
    }
    __syncthreads();
    need -= found[1];
    base += (uint32_t)found[0] << shift;
    width = min((1u << shift) - 1u, kmax - base);
    whole = need == found[2];
    bits = shift;
    ++pass;
    __syncthreads();
  }
  // Taken: keys above base + width, those of [base, base + width] if `whole`,
  // or else (all equal then) the first `need` of them.
  const uint32_t over = base + width;
  const int seg = (mine + kSelectThreads - 1) / kSelectThreads | 1;  // odd: other banks
  const int s0 = min(tid * seg, mine), s1 = min(s0 + seg, mine);
  int more = 0, same = 0;
  for (int i = s0; i < s1; ++i) {
    more += keys[i] > over;
    same += keys[i] >= base && keys[i] <= over;
  }
  int all_more, all_same;
  int more_before = select_scan(more, scratch, all_more), same_before = select_scan(same, scratch, all_same);
  if (tid == 0) {
    totals[0] = all_more;
    totals[1] = all_same;
  }
  cluster_sync_all();
  for (int i = 0; i < rank; ++i) {
    more_before += remote_int(&totals[0], i);
    same_before += remote_int(&totals[1], i);
  }
  int out = sink + more_before + min(same_before, need);
  for (int i = s0; i < s1; ++i) {
    const bool tie = keys[i] >= base && keys[i] <= over;
    if (keys[i] > over || (tie && same_before < need)) list[out++] = sink + lo + i;
    same_before += tie;
  }
  if (rank == 0) {
    for (int i = tid; i < sink; i += kSelectThreads) list[i] = i;
    for (int i = tid; i < p.num_recent; i += kSelectThreads)
      list[p.max_list_len - p.num_recent + i] = nb - p.num_recent + i;
    if (tid == 0) p.list_lens[row] = p.max_list_len;
  }
  cluster_sync_all();  // no CTA leaves while another reads its totals
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int D>
int launch_select(const SelectParams& p0, cudaStream_t stream) {
  SelectParams p = p0;
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
  const int blocks = (p.max_seq_len - 1) / p.block_size + 1;
  // CTAs of a row: as many as keep the batch within three per SM and leave
  // each 128 blocks.
  int ranks = 1;
  while (ranks < kSelectMaxCluster && rows * ranks * 2 <= 3 * num_sms_current_device() && blocks >= ranks * 2 * 128)
    ranks *= 2;
  const int fixed = p.head_tiles * 8 * ((2 * D + 4) * 2 + 4), most = 200 * 1024;
  auto bytes = [&] { return fixed + (((blocks + ranks - 1) / ranks + kSelectTile - 1) / kSelectTile * kSelectTile) * 4; };
  while (ranks < kSelectMaxCluster && bytes() > most) ranks *= 2;
  const int smem = bytes();
  if (smem > most) return PA_ERR_UNSUPPORTED;
  const auto kernel = select_kernel<T, D>;
  if (smem > 32 * 1024 && set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), most) != PA_OK)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// kv8: 0, or 1 + the format of an 8-bit cache.
int block_summaries(const void* k_cache, const float* kv_scales, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* first_tokens, const int32_t* seq_lens,
                    int32_t num_seqs, int32_t max_new_tokens, int32_t num_blocks, int32_t block_size,
                    int32_t num_kv_heads, int32_t head_dim, int8_t* summaries, float* summary_scales, pa_dtype dtype,
                    int kv8, cudaStream_t stream) {
  if (num_seqs < 0 || max_new_tokens < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || num_kv_heads < 1)
    return PA_ERR_ARG;
  if (!kv8 && dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (block_size != 16 && block_size != 32) return PA_ERR_BLOCKSIZE;
  const bool wide = !kv8 && dtype == PA_F32;
  if (wide ? head_dim < 32 || head_dim > 256 || head_dim % 32 : head_dim != 64 && head_dim != 128)
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_new_tokens == 0) return PA_OK;
  if (!k_cache || !block_tables || !first_tokens || !seq_lens || !summaries || !summary_scales || (kv8 && !kv_scales))
    return PA_ERR_ARG;
  if (!aligned16(k_cache) || !aligned16(summaries) || !aligned16(summary_scales) || (kv8 && !aligned16(kv_scales)))
    return PA_ERR_ALIGN;
  SummaryParams p{};
  p.k_cache = k_cache;
  p.kv_scales = kv_scales;
  p.block_tables = block_tables;
  p.first_tokens = first_tokens;
  p.seq_lens = seq_lens;
  p.summaries = summaries;
  p.scales = summary_scales;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_new_tokens = max_new_tokens;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  // New tokens may start at the end of a block; a sequence has no more blocks than its table.
  p.seq_blocks = (int32_t)std::min<int64_t>(((int64_t)max_new_tokens + block_size - 2) / block_size + 1,
                                            (int64_t)max_blocks_per_seq + 1);
  p.items = (int64_t)num_seqs * p.seq_blocks * num_kv_heads;
  const int64_t ctas = (p.items + kSummaryThreads / 32 - 1) / (kSummaryThreads / 32);
  if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
  const unsigned n = (unsigned)ctas;
#define PA_SUM(R, KV8)                                                                       \
  (head_dim == 64 ? (summary_kernel<R, 64, KV8><<<n, kSummaryThreads, 0, stream>>>(p), 0)    \
                  : (summary_kernel<R, 128, KV8><<<n, kSummaryThreads, 0, stream>>>(p), 0))
  if (kv8 == 1 + PA_KV_E4M3) {
    PA_SUM(HalfRange, 1);
  } else if (kv8) {
    PA_SUM(HalfRange, 2);
  } else if (dtype == PA_F16) {
    PA_SUM(HalfRange, 0);
  } else if (dtype == PA_BF16) {
    PA_SUM(Bf16Range, 0);
  } else {
    switch (head_dim / 32) {
      case 1: summary_f32_kernel<1><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 2: summary_f32_kernel<2><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 3: summary_f32_kernel<3><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 4: summary_f32_kernel<4><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 5: summary_f32_kernel<5><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 6: summary_f32_kernel<6><<<n, kSummaryThreads, 0, stream>>>(p); break;
      case 7: summary_f32_kernel<7><<<n, kSummaryThreads, 0, stream>>>(p); break;
      default: summary_f32_kernel<8><<<n, kSummaryThreads, 0, stream>>>(p); break;
    }
  }
#undef PA_SUM
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_block_summaries(const void* k_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* first_tokens, const int32_t* seq_lens, int32_t num_seqs,
                       int32_t max_new_tokens, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                       int32_t head_dim, int8_t* summaries, float* summary_scales, pa_dtype dtype, void* stream) {
  return pa::block_summaries(k_cache, nullptr, block_tables, max_blocks_per_seq, first_tokens, seq_lens, num_seqs,
                             max_new_tokens, num_blocks, block_size, num_kv_heads, head_dim, summaries,
                             summary_scales, dtype, 0, static_cast<cudaStream_t>(stream));
}

int pa_block_summaries_fp8(const void* k_cache, const float* kv_scales, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* first_tokens, const int32_t* seq_lens,
                           int32_t num_seqs, int32_t max_new_tokens, int32_t num_blocks, int32_t block_size,
                           int32_t num_kv_heads, int32_t head_dim, int8_t* summaries, float* summary_scales,
                           void* stream) {
  return pa::block_summaries(k_cache, kv_scales, block_tables, max_blocks_per_seq, first_tokens, seq_lens, num_seqs,
                             max_new_tokens, num_blocks, block_size, num_kv_heads, head_dim, summaries,
                             summary_scales, PA_F16, 1 + pa::PA_KV_E4M3, static_cast<cudaStream_t>(stream));
}

int pa_block_summaries_e5m2(const void* k_cache, const float* kv_scales, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* first_tokens, const int32_t* seq_lens,
                            int32_t num_seqs, int32_t max_new_tokens, int32_t num_blocks, int32_t block_size,
                            int32_t num_kv_heads, int32_t head_dim, int8_t* summaries, float* summary_scales,
                            void* stream) {
  return pa::block_summaries(k_cache, kv_scales, block_tables, max_blocks_per_seq, first_tokens, seq_lens, num_seqs,
                             max_new_tokens, num_blocks, block_size, num_kv_heads, head_dim, summaries,
                             summary_scales, PA_F16, 1 + pa::PA_KV_E5M2, static_cast<cudaStream_t>(stream));
}

int pa_select_blocks(const void* q, const int8_t* summaries, const float* summary_scales, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t num_blocks, int32_t max_list_len, int32_t num_sink, int32_t num_recent,
                     int32_t* block_lists, int32_t* list_lens, pa_dtype dtype, void* stream) {
  using namespace pa;
  if (num_seqs < 0 || max_seq_len < 1 || max_blocks_per_seq < 1 || num_blocks < 1 || num_q_heads < 1 ||
      num_kv_heads < 1 || max_list_len < 1 || num_sink < 0 || num_recent < 0 ||
      (int64_t)num_sink + num_recent > max_list_len)
    return PA_ERR_ARG;
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (num_q_heads % num_kv_heads) return PA_ERR_HEADS;
  if (block_size != 16 && block_size != 32) return PA_ERR_BLOCKSIZE;
  if (head_dim < 32 || head_dim > 256 || head_dim % 32 || num_q_heads / num_kv_heads > 128) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || (int64_t)num_seqs * num_kv_heads > (1 << 26)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!q || !summaries || !summary_scales || !block_tables || !seq_lens || !block_lists || !list_lens)
    return PA_ERR_ARG;
  if (!aligned16(q) || !aligned16(summaries) || !aligned16(summary_scales) || !aligned16(block_lists) ||
      !aligned16(list_lens))
    return PA_ERR_ALIGN;
  SelectParams p{};
  p.q = q;
  p.summaries = summaries;
  p.scales = summary_scales;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.lists = block_lists;
  p.list_lens = list_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  // No sequence is longer than its table.
  p.max_seq_len = (int32_t)std::min<int64_t>(max_seq_len, (int64_t)max_blocks_per_seq * block_size);
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.group = num_q_heads / num_kv_heads;
  p.max_list_len = max_list_len;
  p.num_sink = num_sink;
  p.num_recent = num_recent;
  p.head_tiles = (p.group + 7) / 8;
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
#define PA_SEL_D(D)                                                                          \
  (dtype == PA_F32   ? launch_select<float, D>(p, s)                                         \
   : dtype == PA_F16 ? launch_select<__half, D>(p, s)                                        \
                     : launch_select<__nv_bfloat16, D>(p, s))
  switch (head_dim) {
    case 32: return PA_SEL_D(32);
    case 64: return PA_SEL_D(64);
    case 96: return PA_SEL_D(96);
    case 128: return PA_SEL_D(128);
    case 160: return PA_SEL_D(160);
    case 192: return PA_SEL_D(192);
    case 224: return PA_SEL_D(224);
    default: return PA_SEL_D(256);
  }
#undef PA_SEL_D
}

}  // extern "C"

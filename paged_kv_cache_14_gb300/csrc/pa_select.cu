// Block summaries, and the choice of the blocks that a decode query attends
// to.
//
// A summary is the range of every key dimension over a block's tokens, in 8
// bits: with s = max |k| / 127, hi = ceil(max_t k / s) and lo =
// floor(min_t k / s). For a query in 8 bits, q = s_q * code, no key of the
// block has a larger product with it than
//   s_q s  sum_d max(code_d hi_d, code_d lo_d),
// whose sum is a whole number below 2^23. Scores are therefore exact up to two
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
  int64_t items;       // (sequence, block, KV head)
  int32_t stages;      // tiles that a warp has on their way
  int* status;
};

constexpr int kSummaryWarps = 8;
constexpr int kSummaryThreads = 32 * kSummaryWarps;

// Item x of the call, a (block, KV head): whether there is anything to do, the
// tile's number and its rows.
__device__ __forceinline__ bool summary_item(const SummaryParams& p, int64_t x, int64_t& at, int& rows) {
  const int item = (int)(x / p.num_kv_heads), head = (int)(x - (int64_t)item * p.num_kv_heads);
  const int seq = item / p.seq_blocks, j = item - seq * p.seq_blocks;
  const int first = p.first_tokens[seq], len = p.seq_lens[seq];
  const bool report = head == 0;
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
  const int blk = p.block_tables[(int64_t)seq * p.max_blocks_per_seq + lb];
  if (blk < 0 || blk >= p.num_blocks) {
    if (report) record_error(p.status, PA_ERR_BLOCK_OOB);
    return false;
  }
  at = (int64_t)blk * p.num_kv_heads + head;
  rows = min(p.block_size, len - lb * p.block_size);
  return true;
}

// The scale of values of at most `top` in size: infinite where they are not
// all finite.
__device__ __forceinline__ float summary_scale(float top) {
  return top <= 3.402823466e38f ? __fdiv_rn(top, 127.f) : __int_as_float(0x7f800000);
}
// ceil(x / scale), at most 127. The lower ends go through it with their signs
// changed: floor(x / s) = -ceil(-x / s).
__device__ __forceinline__ int code_up(float x, const Divisor& scale) {
  return scale.by > 0.f && scale.by <= 3.402823466e38f ? (int)fminf(ceilf(quotient(x, scale)), 127.f) : 0;
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

// 16-bit rows, or 8-bit codes (KV8: 1 e4m3, 2 e5m2) widened to fp16, of one
// tile in shared memory: a lane takes 16 bytes of a row, RPP rows at a time.
template <typename R, int D, int KV8>
__device__ __forceinline__ void summary_of(const SummaryParams& p, const uint8_t* tile, int64_t at, int rows,
                                           float mul) {
  constexpr int E = KV8 ? 16 : 8;  // elements of a lane
  constexpr int VPR = D / E;       // lanes of a row
  constexpr int RPP = 32 / VPR;    // rows of a pass
  constexpr int W = E / 2;         // packed pairs of a lane
  constexpr int NR = 16 / RPP;     // passes of 16 rows
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const uint8_t* src = tile + (lane % VPR) * 16;
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
  // The RPP lanes that hold the same elements share the rest: half of them
  // take the upper ends, the others the lower (with their signs changed, so
  // that both are maxima), and each a part of the words. What a lane gives
  // away goes to the lane that keeps it.
  const bool low = lane & 16;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const uint32_t l = lo[j] ^ 0x80008000u, keep = low ? l : hi[j];
    hi[j] = R::top(keep, __shfl_xor_sync(kAll, low ? hi[j] : l, 16));
  }
  int part = 0;  // first of the lane's words
#pragma unroll
  for (int o = 8, n = W / 2; o >= VPR; o >>= 1, n >>= 1) {
    const bool up = lane & o;
    part += up ? n : 0;
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      if (j >= n) break;
      const uint32_t keep = up ? hi[j + n] : hi[j];
      hi[j] = R::top(keep, __shfl_xor_sync(kAll, up ? hi[j] : hi[j + n], o));
    }
  }
  constexpr int C = 2 * E / RPP;  // elements that a lane has now: 8 or 4
  uint32_t most = hi[0];
#pragma unroll
  for (int j = 1; j < C / 2; ++j) most = R::top(most, hi[j]);
  const float2 two = R::wide(most);
  float top = max_nan(two.x, two.y);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = max_nan(top, __shfl_xor_sync(kAll, top, o));
  const float scale = summary_scale(KV8 ? __fmul_rn(top, mul) : top);
  const Divisor div = divisor(scale);
  uint32_t out[C / 4] = {};
#pragma unroll
  for (int j = 0; j < C / 2; ++j) {
    const float2 v = R::wide(hi[j]);
    int c0 = code_up(KV8 ? __fmul_rn(v.x, mul) : v.x, div), c1 = code_up(KV8 ? __fmul_rn(v.y, mul) : v.y, div);
    if (low) c0 = -c0, c1 = -c1;
    out[j / 2] |= ((c0 & 255) | (c1 & 255) << 8) << (j & 1) * 16;
  }
  int8_t* dst = p.summaries + (at * 2 + low) * D + (lane % VPR) * E + 2 * part;
  if constexpr (C == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (lane == 0) p.scales[at] = scale;
}

// fp32 rows of 32 N elements, a lane taking every 32nd: 4 x 32768 tokens of 128
// (554 MB with what is written) in 100 us, 5.6 TB/s, 104 in blocks of 32.
template <int N>
__device__ __forceinline__ void summary_of_f32(const SummaryParams& p, int64_t at, int rows) {
  const int lane = threadIdx.x & 31;
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
  const Divisor div = divisor(scale);
  int8_t* dst = p.summaries + at * 2 * (32 * N) + lane;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    dst[32 * i] = (int8_t)code_up(hi[i], div);
    dst[32 * N + 32 * i] = (int8_t)-code_up(-lo[i], div);
  }
  if (lane == 0) p.scales[at] = scale;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

constexpr int kSummaryMaxStages = 8;

// Each warp for itself: it finds 32 items at a time, a lane each, keeps the
// next tiles on their way into shared memory and takes them in order. Bound by
// HBM: the blocks of 4 x 65536 tokens (428 MB with what is written) in 74 us,
// 5.8 TB/s, 32 rows a block 88 us for 554 MB (6.3); over e4m3 pools by the
// widening and encoding (61 us for half the bytes). One tile a warp from global memory into registers took 92 us. A decode
// step's call (64 sequences, a block each) is a chain of latencies, 3 us.
template <typename R, int D, int KV8>
__global__ void __launch_bounds__(kSummaryThreads) summary_kernel(const __grid_constant__ SummaryParams p) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int RB = D * (KV8 ? 1 : 2);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kSummaryWarps][kSummaryMaxStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile_bytes = p.block_size * RB;
  uint8_t* ring = smem + warp * p.stages * tile_bytes;
  if (lane == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    fence_barrier_init();
  }
  __syncwarp();
  const int64_t step = (int64_t)gridDim.x * kSummaryWarps;
  int put = 0, put_turn = 0, got = 0, got_turn = 0;  // stage and round of the next tile to ask for, to take
  for (int64_t base = (int64_t)blockIdx.x * kSummaryWarps + warp; base < p.items; base += 32 * step) {
    int64_t at = 0;
    int rows = 0;
    float mul = 1.f;
    if (base + lane * step < p.items && summary_item(p, base + lane * step, at, rows)) {
      if constexpr (KV8 != 0) mul = p.kv_scales[at * 2];
    }
    unsigned ask = __ballot_sync(kAll, rows > 0), take = ask;
    auto next = [&] {
      if (!ask) return;
      const int l = __ffs(ask) - 1;
      ask &= ask - 1;
      if (lane == l) {
        const uint32_t bar = smem_u32(&bars[warp][put]);
        mbar_arrive_expect_tx(bar, rows * RB);
        bulk_load(smem_u32(ring + put * tile_bytes), static_cast<const uint8_t*>(p.k_cache) + at * tile_bytes,
                  rows * RB, bar);
      }
      if (++put == p.stages) put = 0, put_turn ^= 1;
    };
    for (int i = 0; i < p.stages; ++i) next();
    while (take) {
      const int l = __ffs(take) - 1;
      take &= take - 1;
      if (!__all_sync(kAll, mbar_wait(smem_u32(&bars[warp][got]), got_turn, p.status))) {
        // Not in time: what is on its way still has to arrive.
        for (; got != put || got_turn != put_turn;) {
          mbar_wait(smem_u32(&bars[warp][got]), got_turn, p.status);
          if (++got == p.stages) got = 0, got_turn ^= 1;
        }
        return;
      }
      summary_of<R, D, KV8>(p, ring + got * tile_bytes, __shfl_sync(kAll, at, l), __shfl_sync(kAll, rows, l),
                            __shfl_sync(kAll, mul, l));
      __syncwarp();  // the tile has been read
      if (++got == p.stages) got = 0, got_turn ^= 1;
      next();
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kSummaryThreads) summary_f32_kernel(const __grid_constant__ SummaryParams p) {
  const int64_t step = (int64_t)gridDim.x * kSummaryWarps;
  for (int64_t x = (int64_t)blockIdx.x * kSummaryWarps + (threadIdx.x >> 5); x < p.items; x += step) {
    int64_t at;
    int rows;
    if (summary_item(p, x, at, rows)) summary_of_f32<N>(p, at, rows);
  }
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
  pa_dtype dtype;
  int* status;
};

// Warps of a CTA, and of an SM: 128 registers each. (24 of 80 registers, which
// spill: 41 us for 8 x 131072 tokens where 16 take 37.)
constexpr int kSelectMaxWarps = 16;
constexpr int kSelectMaxCluster = 8;
constexpr int kSelectTile = 16;    // blocks of one matrix product
constexpr int kSelectStages = 2;   // tiles of a warp in shared memory: in use, on its way
constexpr int kDigit = 9;          // bits of a digit
constexpr int kBins = 1 << kDigit; // its values, a 32nd of them to a lane
constexpr int kPasses = 4;         // digits of a score
constexpr int kLaneBins = kBins / 32 + 4;  // a lane's bins are apart by 16 bytes more, in other banks
constexpr uint32_t kNoBlock = 0xffc00001u; // a scale (a NaN) that marks a block outside the pool

// A query row's codes, 64 bytes on where rows would lie in the same banks.
constexpr int select_query_bytes(int d) { return 2 * d + (d % 64 == 0 ? 64 : 0); }
// Shared memory of the tiles on their way, which the counts take over.
constexpr int select_ring_bytes(int d, int warps) {
  const int ring = warps * kSelectStages * (kSelectTile * 2 * d + kSelectTile * 4);
  const int counts = (kPasses + 1) * 32 * kLaneBins * 4;
  return ring > counts ? ring : counts;
}

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
__device__ __forceinline__ uint2 remote_pair(const void* local, int rank) {
  uint32_t a;
  uint2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int4 remote_int4(const void* local, int rank) {
  uint32_t a;
  int4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ int bin_at(uint32_t digit) { return digit + digit / (kBins / 32) * 4; }

// Scores as unsigned numbers of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // one zero
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// 16 x 8 sums of 32 products of signed bytes.
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One cluster (with CL; else one CTA) per (sequence, KV head). Its CTAs split
// the row's blocks, score them 16 at a time by matrix products of bytes and keep
// the scores in shared memory. The score of the last block to take is found by
// counting: digits of 9 bits from the top of the range that the row's scores
// span, so that the first splits them well whatever their size, and the
// search ends when a digit's blocks are all taken (after two digits, mostly).
//
// What bounds it is the chain of its phases: for 64 sequences of up to 8192
// tokens 4 us to the first tile (lengths, table, summaries), 8 to score all
// (53 MB at HBM's rate), 1 for the digits and 1 for the list, in a call of 22;
// for 8 of up to 131072 (cluster barriers between the phases) 4, 19 (102 MB;
// an SM takes 40 GB/s), 5 and 2 in a call of 35. The byte products keep the
// tensor pipe 64 cycles each where fp16's (m16n8k16, half as deep) take 9, but
// widening the codes costs what that saves.
//
// The summaries come by asynchronous copies, a tile ahead of each warp: 16
// blocks' rows as they lie, but for the halves of 128 bytes of every other
// row, which change places so that a fragment's rows take all banks. ONE: the
// group's heads fit one tile of 8, whose codes then stay in registers.
template <int D, bool CL, bool ONE>
__global__ void __launch_bounds__(32 * kSelectMaxWarps)
    select_kernel(const __grid_constant__ SelectParams p) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kRow = 2 * D, kPieces = kRow / 16, kTile = kSelectTile * kRow + kSelectTile * 4;
  constexpr int kQuery = select_query_bytes(D);
  constexpr bool kSwap = kRow % 128 == 0;  // (other rows start 64 bytes apart by themselves)
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t scratch[kSelectMaxWarps], total;
  __shared__ __align__(8) uint32_t range[2];
  const int threads = blockDim.x, warps = threads >> 5;
  // The tiles' ring, later the counts; the queries; the scores.
  int(*hist)[32 * kLaneBins] = reinterpret_cast<int(*)[32 * kLaneBins]>(smem);
  int* sum = hist[kPasses];
  uint8_t* qs = smem + select_ring_bytes(D, warps);
  float* q_scale = reinterpret_cast<float*>(qs + p.head_tiles * 8 * kQuery);
  uint32_t* keys = reinterpret_cast<uint32_t*>(q_scale + p.head_tiles * 8);
  int ranks = 1, rank = 0;
  if constexpr (CL) {
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  }
  const int row = blockIdx.x / ranks, seq = row / p.num_kv_heads, head = row - seq * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  int32_t* list = p.lists + (int64_t)row * p.max_list_len;
  const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
  const int len = p.seq_lens[seq];
  float x[D / 32];  // the first query row of this warp, asked for before anything waits
  auto query = [&](int h) {
    const int64_t at = ((int64_t)seq * p.num_q_heads + head * p.group + h) * D + lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      x[i] = h >= p.group         ? 0.f
             : p.dtype == PA_F32 ? static_cast<const float*>(p.q)[at + 32 * i]
             : p.dtype == PA_F16 ? to_f32(static_cast<const __half*>(p.q)[at + 32 * i])
                                 : to_f32(static_cast<const __nv_bfloat16*>(p.q)[at + 32 * i]);
  };
  query(warp);
  int nb = len > 0 ? (len - 1) / p.block_size + 1 : 0;
  if (len < 0 || len > p.max_seq_len || nb > p.max_blocks_per_seq) {
    if (rank == 0 && tid == 0 && head == 0) record_error(p.status, PA_ERR_SEQLEN);
    nb = 0;
  }
  if (nb <= p.max_list_len) {  // all of them (the same for the whole cluster)
    for (int i = rank * threads + tid; i < p.max_list_len; i += ranks * threads)
      list[i] = i < nb ? i : -1;
    if (rank == 0 && tid == 0) p.list_lens[row] = nb;
    return;
  }
  const int sink = p.num_sink, some = nb - sink - p.num_recent;  // blocks that compete
  int need = p.max_list_len - sink - p.num_recent;               // of which so many are taken
  const int chunk = ((some + ranks - 1) / ranks + kSelectTile - 1) / kSelectTile * kSelectTile;
  const int lo = min(rank * chunk, some), mine = min(chunk, some - lo);

  // The first tile's blocks from the table (behind the end: the last block).
  // All blocks' numbers lie where their scores will be, by copies of their own,
  // so that no other tile waits for the table.
  const int32_t* from_table = table + sink + lo;
  const uint32_t first_id =
      mine > warp * kSelectTile && lane < kSelectTile ? from_table[min(warp * kSelectTile + lane, mine - 1)] : 0u;
  for (int i = tid; i < (mine + kSelectTile - 1) / kSelectTile * kSelectTile; i += threads)
    copy_async4(smem_u32(&keys[i]), from_table + min(i, mine - 1));
  copy_async_commit();
  if (tid == 0) {
    range[0] = 0xffffffffu;
    range[1] = 0;
  }
  const int step = warps * kSelectTile;
  uint8_t* ring = smem + warp * kSelectStages * kTile;
  // The tile at b0 into a stage.
  const uint32_t block_bytes = p.num_kv_heads * kRow;
  const int8_t* summaries = p.summaries + (int64_t)head * kRow;
  auto fetch = [&](int b0, int stage, bool first) {
    if (b0 < mine) {
      const uint32_t to = smem_u32(ring + stage * kTile);
      // Instruction i takes whole rows, and a lane its neighbours in the next
      // ones, so that four of its blocks' numbers are one load.
      constexpr int kCopies = kSelectTile * kPieces / 32;
      const uint32_t most = p.num_blocks - 1;
      if constexpr (kCopies % 4 == 0 && 32 % kPieces == 0) {
        const int row0 = lane / kPieces * kCopies, piece = lane % kPieces;
        const int8_t* from = summaries + piece * 16;
#pragma unroll
        for (int i = 0; i < kCopies; i += 4) {
          uint32_t ids[4];
          if (first) {
#pragma unroll
            for (int k = 0; k < 4; ++k) ids[k] = __shfl_sync(kAll, first_id, row0 + i + k);
          } else {
            const uint4 id = *reinterpret_cast<const uint4*>(keys + b0 + row0 + i);
            ids[0] = id.x;
            ids[1] = id.y;
            ids[2] = id.z;
            ids[3] = id.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            copy_async16(to + (row0 + i + k) * kRow + (kSwap ? piece ^ (i + k & 1) << 2 : piece) * 16,
                         from + (uint64_t)min(ids[k], most) * block_bytes);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int x = i * 32 + lane, row = x / kPieces, piece = x - row * kPieces;
          copy_async16(to + row * kRow + (kSwap ? piece ^ (row & 1) << 2 : piece) * 16,
                       summaries + (uint64_t)min(first ? __shfl_sync(kAll, first_id, row) : keys[b0 + row], most) *
                                       block_bytes + piece * 16);
        }
      }
      if (lane < kSelectTile) {
        const uint32_t s = to + kSelectTile * kRow + lane * 4;
        const uint32_t id = first ? first_id : keys[b0 + lane];
        if (id < (uint32_t)p.num_blocks) {
          copy_async4(s, p.scales + (int64_t)id * p.num_kv_heads + head);
        } else {
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(s), "r"(kNoBlock) : "memory");
          record_error(p.status, PA_ERR_BLOCK_OOB);
        }
      }
    }
    copy_async_commit();
  };
  fetch(warp * kSelectTile, 0, true);
  // The queries' codes, their positive and their negative part.
  for (int h = warp; h < p.head_tiles * 8; h += warps) {
    if (h != warp) query(h);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      top = fabsf(x[i]) <= 3.402823466e38f ? fmaxf(top, fabsf(x[i])) : __int_as_float(0x7f800000);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    // (A row that is not all finite counts as zeros.)
    const float scale = top <= 3.402823466e38f ? __fdiv_rn(top, 127.f) : 0.f;
    const Divisor div = divisor(scale);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float code = scale > 0.f ? fminf(fmaxf(rintf(quotient(x[i], div)), -127.f), 127.f) : 0.f;
      qs[h * kQuery + lane + 32 * i] = (uint8_t)(int)fmaxf(code, 0.f);
      qs[h * kQuery + D + lane + 32 * i] = (uint8_t)(int)fminf(code, 0.f);
    }
    if (lane == 0) q_scale[h] = scale;
  }
  copy_async_wait<1>();  // the table's entries (the first tile may still be on its way)
  __syncthreads();
  uint4 qf[ONE ? D / 32 : 1];
  float qs0 = 0.f, qs1 = 0.f;
  if constexpr (ONE) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) qf[j] = *reinterpret_cast<const uint4*>(qs + r * kQuery + 16 * c + 64 * j);
    qs0 = q_scale[2 * c];
    qs1 = q_scale[2 * c + 1];
  }
  const float none = __int_as_float(0xff800000);
  const bool odd = c & 1, upper = c & 2;

  uint32_t kmin = 0xffffffffu, kmax = 0;
  for (int b0 = warp * kSelectTile; b0 < mine; b0 += 2 * step) {
    float best[2][2], scale = 0.f;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // Lane (r, c): 16 bytes of each 64 of the rows of blocks r and r + 8.
      best[t][0] = best[t][1] = none;
      fetch(b0 + (t + 1) * step, t ^ 1, false);
      copy_async_wait<1>();
      __syncwarp();
      if (b0 + t * step < mine) {
        const uint8_t* tile = ring + t * kTile;
        const uint8_t* at = tile + r * kRow;
        const int swap = kSwap ? (r & 1) << 2 : 0;
        for (int n = 0; n < (ONE ? 1 : p.head_tiles); ++n) {
          int part[4][4] = {};  // (four sums, so that a product need not wait for the one before)
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const int piece = (4 * j + c ^ swap) * 16;
            const uint4 x0 = *reinterpret_cast<const uint4*>(at + piece);
            const uint4 x1 = *reinterpret_cast<const uint4*>(at + 8 * kRow + piece);
            const uint4 y = ONE ? qf[ONE ? j : 0]
                                : *reinterpret_cast<const uint4*>(qs + (n * 8 + r) * kQuery + 16 * c + 64 * j);
            mma_s8(part[2 * j & 3], x0.x, x1.x, x0.y, x1.y, y.x, y.y);
            mma_s8(part[2 * j + 1 & 3], x0.z, x1.z, x0.w, x1.w, y.z, y.w);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = n * 8 + 2 * c + i;
            const float s = ONE ? i ? qs1 : qs0 : q_scale[h];
            if (h < p.group) {
              best[t][0] = fmaxf(best[t][0], __fmul_rn((float)(part[0][i] + part[1][i] + (part[2][i] + part[3][i])), s));
              best[t][1] =
                  fmaxf(best[t][1],
                        __fmul_rn((float)(part[0][2 + i] + part[1][2 + i] + (part[2][2 + i] + part[3][2 + i])), s));
            }
          }
        }
        if (odd == (t == 1)) scale = reinterpret_cast<const float*>(tile + kSelectTile * kRow)[r + (upper ? 8 : 0)];
      }
      __syncwarp();  // the tile has been read
    }
    // The maximum over the group's heads, which four lanes share: each gives
    // the others what they keep, and keeps one block of the two tiles' 32.
    float m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m[i] = fmaxf(odd ? best[1][i] : best[0][i], __shfl_xor_sync(kAll, odd ? best[0][i] : best[1][i], 1));
    const float top = fmaxf(upper ? m[1] : m[0], __shfl_xor_sync(kAll, upper ? m[0] : m[1], 2));
    const int b = b0 + (odd ? step : 0) + r + (upper ? 8 : 0);
    if (b < mine) {
      // A block with keys that are not finite comes before all others, one
      // outside the pool behind. (Scale 0: all its keys are 0, whatever else
      // overflows.)
      const uint32_t key = __float_as_uint(scale) == kNoBlock ? 0u
                           : !(scale <= 3.402823466e38f)         ? 0xff800000u
                                                         : ordered(scale == 0.f ? 0.f : __fmul_rn(top, scale));
      keys[b] = key;
      kmin = min(kmin, key);
      kmax = max(kmax, key);
    }
  }
  copy_async_wait<0>();
  __syncthreads();
  for (int i = tid; i < kPasses * 32 * kLaneBins / 4; i += threads)
    reinterpret_cast<int4*>(smem)[i] = make_int4(0, 0, 0, 0);
  kmin = __reduce_min_sync(kAll, kmin);
  kmax = __reduce_max_sync(kAll, kmax);
  if (lane == 0) {
    atomicMin(&range[0], kmin);
    atomicMax(&range[1], kmax);
  }
  if constexpr (CL) {
    cluster_sync_all();
    const uint2 x = remote_pair(range, lane % ranks);
    kmin = __reduce_min_sync(kAll, x.x);
    kmax = __reduce_max_sync(kAll, x.y);
  } else {
    __syncthreads();
    kmin = range[0];
    kmax = range[1];
  }
  // Keys from `base` to base + width are in question; those above are taken.
  int bits = 32 - __clz(kmax - kmin);
  uint32_t base = kmin, width = kmax - kmin;
  int pass = 0;
  bool whole = false;  // all keys in question are taken
  while (need > 0 && bits > 0 && !whole) {
    const int shift = max(bits - kDigit, 0);
    for (int i = tid; i < mine; i += threads) {
      const uint32_t key = keys[i];
      if (key >= base && key - base <= width) atomicAdd(&hist[pass][bin_at((key - base) >> shift)], 1);
    }
    const int* bins = hist[pass];
    if constexpr (CL) {
      cluster_sync_all();
      // (A thread has four digits' counts, all CTAs' at once.)
      for (int i = 4 * tid; i < kBins; i += 4 * threads) {
        int4 y[kSelectMaxCluster];
#pragma unroll
        for (int j = 0; j < kSelectMaxCluster; ++j)
          y[j] = j < ranks ? remote_int4(&hist[pass][bin_at(i)], j) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int j = 1; j < kSelectMaxCluster; ++j) {
          y[0].x += y[j].x;
          y[0].y += y[j].y;
          y[0].z += y[j].z;
          y[0].w += y[j].w;
        }
        *reinterpret_cast<int4*>(&sum[bin_at(i)]) = y[0];
      }
      bins = sum;
    }
    __syncthreads();
    // Every warp counts for itself: lane 31 has the lowest digits, and the
    // lanes' sums from the top tell whose digit makes up `need`.
    int v[kBins / 32], count = 0;
#pragma unroll
    for (int i = 0; i < kBins / 128; ++i) {
      const int4 x = *reinterpret_cast<const int4*>(bins + (31 - lane) * kLaneBins + 4 * i);
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
      count += x.x + x.y + x.z + x.w;
    }
    int above = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, above, o);
      if (lane >= o) above += y;
    }
    const int who = __ffs(__ballot_sync(kAll, above >= need)) - 1;
    above -= count;
    int digit = 0, here = 0;
#pragma unroll
    for (int i = kBins / 32 - 1; i >= 0; --i) {  // from the top to the first that makes up `need`
      if (above + here < need) {
        above += here;
        here = v[i];
        digit = i;
      }
    }
    digit = __shfl_sync(kAll, (31 - lane) * (kBins / 32) + digit, who);
    need -= __shfl_sync(kAll, above, who);
    here = __shfl_sync(kAll, here, who);
    base += (uint32_t)digit << shift;
    width = min((1u << shift) - 1u, kmax - base);
    whole = need == here;
    bits = shift;
    ++pass;
    if constexpr (CL) __syncthreads();  // `sum` is read
  }
  // Taken: keys above base + width, those of [base, base + width] if `whole`,
  // or else (all equal then) the first `need` of them.
  const uint32_t over = base + width;
  const int seg = (mine + threads - 1) / threads | 1;  // odd: other banks
  const int s0 = min(tid * seg, mine), s1 = min(s0 + seg, mine);
  // Taken for certain, and in question (upper half), in the segments before.
  uint32_t before = 0;
  for (int i = s0; i < s1; ++i) before += keys[i] > over ? 1u : keys[i] >= base ? 1u << 16 : 0u;
  {
    const uint32_t own = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) scratch[warp] = before;
    before -= own;
  }
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < kSelectMaxWarps; ++i) {
    if (i >= warps) break;
    before += i < warp ? scratch[i] : 0u;
    all += scratch[i];
  }
  int more_before = before & 0xffff, same_before = before >> 16;
  if constexpr (CL) {
    if (tid == 0) total = all;
    cluster_sync_all();
    const uint32_t x = lane < rank ? remote_int(&total, lane) : 0u;
    more_before += __reduce_add_sync(kAll, x & 0xffff);
    same_before += __reduce_add_sync(kAll, x >> 16);
  }
  int out = sink + more_before + min(same_before, need);
  for (int i = s0; i < s1; ++i) {
    const bool tie = keys[i] >= base && keys[i] <= over;
    if (keys[i] > over || (tie && same_before < need)) list[out++] = sink + lo + i;
    same_before += tie;
  }
  if (rank == 0) {
    for (int i = tid; i < sink; i += threads) list[i] = i;
    for (int i = tid; i < p.num_recent; i += threads)
      list[p.max_list_len - p.num_recent + i] = nb - p.num_recent + i;
    if (tid == 0) p.list_lens[row] = p.max_list_len;
  }
  if constexpr (CL) cluster_sync_all();  // no CTA leaves while another reads its totals
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared memory of a CTA of `warps` warps with `scores` scores, and the most that
// it may be.
int select_bytes(int d, int head_tiles, int warps, int scores) {
  return select_ring_bytes(d, warps) + head_tiles * 8 * (select_query_bytes(d) + 4) + scores * 4;
}
constexpr int kSelectMostBytes = 220 * 1024;
// Blocks whose scores the largest cluster holds.
int64_t select_max_blocks(int d, int head_tiles) {
  const int scores = (kSelectMostBytes - select_bytes(d, head_tiles, 4, 0)) / 4;
  return (int64_t)kSelectMaxCluster * (scores / kSelectTile * kSelectTile);
}

template <int D>
int launch_select(const SelectParams& p0, cudaStream_t stream) {
  SelectParams p = p0;
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
  const int blocks = (p.max_seq_len - 1) / p.block_size + 1;
  // CTAs of a row: of 128 blocks at least, or as many as shared memory takes to
  // hold the scores; then the warps of each so that all CTAs run at once.
  const int sms = num_sms_current_device(), most = kSelectMostBytes;
  int ranks = cluster_ranks(rows, sms, blocks / 128);
  auto scores = [&] { return ((blocks + ranks - 1) / ranks + kSelectTile - 1) / kSelectTile * kSelectTile; };
  auto bytes = [&](int warps) { return select_bytes(D, p.head_tiles, warps, scores()); };
  while (ranks < kSelectMaxCluster && bytes(4) > most) ranks *= 2;
  const int64_t per_sm = (rows * ranks + sms - 1) / sms;
  int warps = (int)std::min<int64_t>(std::min(kSelectMaxWarps, scores() / kSelectTile), kSelectMaxWarps / per_sm);
  while (warps > 4 && bytes(warps) > most / std::min<int64_t>(per_sm, kSelectMaxWarps / 4)) --warps;
  warps = std::max(warps, 4);
  const int smem = bytes(warps);
  const bool one = p.head_tiles == 1;
  const auto kernel = ranks > 1 ? one ? select_kernel<D, true, true> : select_kernel<D, true, false>
                      : one    ? select_kernel<D, false, true>
                               : select_kernel<D, false, false>;
  if (smem > 47 * 1024 && set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), most) != PA_OK)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
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
  if ((int64_t)num_seqs * p.seq_blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
  p.items = (int64_t)num_seqs * p.seq_blocks * num_kv_heads;
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
  // Three CTAs an SM with 64 KB of tiles each, or one with 128 KB where a warp's
  // two tiles take that (16-bit blocks of 32 rows of 128): as many as run at once,
  // since they go on from tile to tile.
  const int tile = block_size * head_dim * (kv8 ? 1 : 2);
  p.stages = std::max(2, std::min(kSummaryMaxStages, 64 * 1024 / (kSummaryWarps * tile)));
  const int smem = kSummaryWarps * p.stages * tile;
  const int resident = wide ? 8 : smem > 64 * 1024 ? 1 : 3;
  const unsigned n = (unsigned)std::min<int64_t>((p.items + kSummaryWarps - 1) / kSummaryWarps,
                                                 resident * num_sms_current_device());
#define PA_SUM_D(R, D, KV8)                                                                                  \
  {                                                                                                          \
    const auto kernel = summary_kernel<R, D, KV8>;                                                           \
    if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), 128 * 1024) != PA_OK) return PA_ERR_CUDA;\
    kernel<<<n, kSummaryThreads, smem, stream>>>(p);                                                         \
  }
#define PA_SUM(R, KV8)                        \
  if (head_dim == 64) PA_SUM_D(R, 64, KV8)    \
  else PA_SUM_D(R, 128, KV8)
  if (wide) {
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
  } else if (kv8 == 1 + PA_KV_E4M3) {
    PA_SUM(HalfRange, 1)
  } else if (kv8) {
    PA_SUM(HalfRange, 2)
  } else if (dtype == PA_F16) {
    PA_SUM(HalfRange, 0)
  } else {
    PA_SUM(Bf16Range, 0)
  }
#undef PA_SUM_D
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
  if (num_seqs > 65535 || num_kv_heads > (1 << 20) || (int64_t)num_seqs * num_kv_heads > (1 << 26))
    return PA_ERR_UNSUPPORTED;
  const int head_tiles = (num_q_heads / num_kv_heads + 7) / 8;
  // No sequence is longer than its table.
  const int64_t longest = std::min<int64_t>(max_seq_len, (int64_t)max_blocks_per_seq * block_size);
  if ((longest - 1) / block_size + 1 > select_max_blocks(head_dim, head_tiles)) return PA_ERR_UNSUPPORTED;
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
  p.max_seq_len = (int32_t)longest;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.group = num_q_heads / num_kv_heads;
  p.max_list_len = max_list_len;
  p.num_sink = num_sink;
  p.num_recent = num_recent;
  p.head_tiles = head_tiles;
  p.dtype = dtype;
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 32: return launch_select<32>(p, s);
    case 64: return launch_select<64>(p, s);
    case 96: return launch_select<96>(p, s);
    case 128: return launch_select<128>(p, s);
    case 160: return launch_select<160>(p, s);
    case 192: return launch_select<192>(p, s);
    case 224: return launch_select<224>(p, s);
    default: return launch_select<256>(p, s);
  }
}

}  // extern "C"

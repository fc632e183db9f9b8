// Decode attention over listed blocks: softmax(q K^T scale) V over the tokens
// of the blocks that each (sequence, KV head) lists.
//
// The bytes of the listed K and V rows bound it: a block's keys meet the
// query heads of one group only (4 G operations for 2 x 2 bytes). One cluster
// works on a (sequence, KV head), its warps on 16 tokens at a time. Asynchronous
// copies bring the next tiles into each warp's part of shared memory, and
// fragments are read from there 16 bytes a lane, which the products' free order
// of k (the head's dimensions) and of m (the output's) allows:
//   scores S[16 tokens][8 heads] = K q^T, lane (r, c) holding 8 dimensions
//     from 32 j + 8 c on of tokens r and r + 8;
//   output O^T[D][8 heads] += V^T P^T, lane (r, c) holding 8 dimensions from
//     8 r on (and 64 + 8 r) of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9, paired
//     by byte permutes; P goes from one layout to the other by a transpose of
//     8 x 8 matrices.
// Each warp keeps a running reference m and a sum l of each head. The
// reference moves only when a score passes it by 2^8 (weights stay below 2^8,
// far from the largest fp16), so that most tiles need no maximum over the
// warp. Warps, then the cluster's CTAs, are joined in a fixed order.
//
// 64 sequences of 8 KV heads with 128 listed blocks each (bf16, 533 MB) take 91
// us, 5.9 TB/s (90 with weights of one bf16, whose error is that of the output's
// rounding once more). 8 sequences with 256 blocks (e4m3, 67 MB) take 20: 3 to the
// first tile (lists, table, tiles), 10 for the tiles at HBM's rate, 3 for the
// joins, and the launch. One user's 64 blocks take 6, nearly all of it such
// latencies.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

struct SparseParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* kv_scales;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* lists;
  const int32_t* list_lens;
  void* out;
  int32_t max_blocks_per_seq, max_list_len, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  int32_t group, row_groups;
  float scale_log2;
  int* status;
};

constexpr int kSparseMaxWarps = 12;
constexpr int kSparseMaxCluster = 8;
constexpr int kSparseF32Threads = 128;
// Tiles (K and V) of a warp in shared memory, the one in use among them.
constexpr int sparse_stages(int tile_bytes) { return 8192 / tile_bytes; }
constexpr float kMoveAt = 8.f;  // log2 of the weight that moves the reference

namespace {

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ float remote_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// A pair of weights in two parts: the largest numbers of the type below them (0
// of 0), and what is left, times kUp, the type's smallest number at least. Both
// are above 0 where the first is, so that they make of an infinite value the same
// infinity. fp16 has room for few sizes: its weights are 2^kLift times as large (up
// to 2^15 then, where what is left is at most 2^5), and so are their sums; the
// smallest have a first part from 2^-31 on, and are off by 2^-41.
__device__ __forceinline__ float next_below(float e) { return __int_as_float(max(__float_as_int(e), 1) - 1); }
template <typename M>
struct TwoParts;
template <>
struct TwoParts<__nv_bfloat16> {
  static constexpr float kUp = 1.f, kLift = 0.f;
  __device__ __forceinline__ static void split(float x, float y, uint32_t& first, uint32_t& rest) {
    const uint32_t a = __float_as_uint(next_below(x)), b = __float_as_uint(next_below(y));
    first = __byte_perm(a, b, 0x7632);
    rest = MmaOp<__nv_bfloat16>::pack(x - __uint_as_float(a & 0xffff0000u), y - __uint_as_float(b & 0xffff0000u));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(rest) : "r"(0x00010001u));
  }
};
template <>
struct TwoParts<__half> {
  static constexpr float kUp = 1024.f, kLift = 7.f;
  __device__ __forceinline__ static void split(float x, float y, uint32_t& first, uint32_t& rest) {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(first) : "f"(next_below(y)), "f"(next_below(x)));
    const float2 held = __half22float2(*reinterpret_cast<const __half2*>(&first));
    rest = MmaOp<__half>::pack((x - held.x) * kUp, (y - held.y) * kUp);
    asm("max.f16x2 %0, %0, %1;" : "+r"(rest) : "r"(0x00010001u));
  }
};

// The cluster's row: its sequence, KV head and query heads, and its list.
struct SparseRow {
  int ranks, rank, row, seq, head, first_head, heads, len, entries;
  const int32_t* list;
  const int32_t* table;
};
__device__ __forceinline__ SparseRow sparse_row(const SparseParams& p, int heads_per_row) {
  SparseRow w;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(w.ranks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(w.rank));
  const int x = blockIdx.x / w.ranks;
  w.row = x / p.row_groups;
  const int rg = x - w.row * p.row_groups;
  w.seq = w.row / p.num_kv_heads;
  w.head = w.row - w.seq * p.num_kv_heads;
  w.first_head = w.head * p.group + rg * heads_per_row;
  w.heads = min(heads_per_row, p.group - rg * heads_per_row);
  w.len = p.seq_lens[w.seq];
  w.entries = p.list_lens[w.row];
  w.list = p.lists + (int64_t)w.row * p.max_list_len;
  w.table = p.block_tables + (int64_t)w.seq * p.max_blocks_per_seq;
  return w;
}
// Its lengths, once they are there: entries 0 if they are refused.
__device__ __forceinline__ void sparse_check(const SparseParams& p, SparseRow& w) {
  if (w.entries < 0 || w.entries > p.max_list_len || w.len < 0 ||
      (w.len > 0 && (w.len - 1) / p.block_size >= p.max_blocks_per_seq)) {
    if (threadIdx.x == 0) record_error(p.status, PA_ERR_SEQLEN);
    w.entries = 0;
  }
}

// List entry i and the one before it, wherever the list ends (asked for before
// its length is known).
__device__ __forceinline__ int2 sparse_entry(const SparseParams& p, const SparseRow& w, int i) {
  return i < p.max_list_len ? make_int2(i > 0 ? w.list[i - 1] : -1, w.list[i]) : make_int2(-1, -1);
}
// Tokens `16 sub ..` of an entry: (block, tokens there); no tokens for an
// entry that is refused.
__device__ __forceinline__ int2 sparse_item(const SparseParams& p, const SparseRow& w, int2 entry, int sub) {
  const int lb = entry.y;
  if (lb <= entry.x || lb < 0 || w.len <= 0 || lb > (w.len - 1) / p.block_size) {
    record_error(p.status, lb <= entry.x || lb < 0 ? PA_ERR_ARG : PA_ERR_SEQLEN);
    return make_int2(0, 0);
  }
  const int blk = w.table[lb];
  if (blk < 0 || blk >= p.num_blocks) {
    record_error(p.status, PA_ERR_BLOCK_OOB);
    return make_int2(0, 0);
  }
  return make_int2(blk, min(16, max(0, w.len - lb * p.block_size - 16 * sub)));
}

// One output of four dimensions: a row without blocks is zeros.
template <typename T, int D>
__device__ __forceinline__ void sparse_store(const SparseParams& p, const SparseRow& w, int h, int d, float4 acc,
                                             float sum) {
  const float inv = w.entries > 0 ? 1.f / sum : 0.f;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  store4(static_cast<T*>(p.out) + ((int64_t)w.seq * p.num_q_heads + w.first_head + h) * D + d, acc);
}

// A part's weight in a join where `top` is the largest reference. (A part that
// saw no score has zeros, or a NaN to keep.)
__device__ __forceinline__ float part_weight(float m, float top) { return m == neg_inf() ? 1.f : exp2f(m - top); }

// Joins a cluster's CTAs: o [heads][D], m and l in every CTA's shared memory
// (o relative to m); each CTA writes its share of the output. Ends with a
// cluster barrier, after which shared memory may go.
template <typename T, int D>
__device__ __forceinline__ void sparse_join(const SparseParams& p, const SparseRow& w, const float* o, const float* m,
                                            const float* l) {
  cluster_sync();
  const int quads = w.heads * (D / 4);
  for (int x = w.rank * blockDim.x + threadIdx.x; x < quads; x += w.ranks * blockDim.x) {
    const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
    // All CTAs' parts at once.
    float mi[kSparseMaxCluster], li[kSparseMaxCluster];
    float4 v[kSparseMaxCluster];
#pragma unroll
    for (int i = 0; i < kSparseMaxCluster; ++i) {
      if (i >= w.ranks) break;
      mi[i] = remote_f32(remote(m + h, i));
      li[i] = remote_f32(remote(l + h, i));
      v[i] = remote_f32x4(remote(o + h * D + d, i));
    }
    float top = neg_inf(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kSparseMaxCluster; ++i)
      if (i < w.ranks) top = fmaxf(top, mi[i]);
#pragma unroll
    for (int i = 0; i < kSparseMaxCluster; ++i) {
      if (i >= w.ranks) break;
      const float f = part_weight(mi[i], top);
      sum += f * li[i];
      acc.x += f * v[i].x;
      acc.y += f * v[i].y;
      acc.z += f * v[i].z;
      acc.w += f * v[i].w;
    }
    sparse_store<T, D>(p, w, h, d, acc, sum);
  }
  cluster_sync();
}

}  // namespace

// KV8: 0 (the pools hold T), 1 e4m3, 2 e5m2 (codes widened to fp16 exactly;
// a bf16 query row goes into fp16 by a power of two that its scores take
// back; a block's V scale multiplies the block's product, so that no weight
// carries it). NT: tiles of 8 query heads.
template <typename T, int KV8, int D, int NT>
__global__ void __launch_bounds__(NT == 1 ? 384 : 256) sparse_kernel(const __grid_constant__ SparseParams p) {
  using M = typename std::conditional<KV8 != 0, __half, T>::type;  // the products' type
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int H = 8 * NT;
  constexpr int KP = KV8 ? D / 64 : D / 32;   // 16-byte pieces of a K row for a lane
  constexpr int VP = KV8 ? D / 128 : D / 64;  // 16-byte pieces of a V row for a lane
  constexpr int MT = D / 16;                  // tiles of 16 output dimensions
  constexpr int KS = D / 16;                  // steps of the score product
  // Weights in two parts where one of the products' type would be no more exact
  // than the output's: all but fp16 weights for bf16 outputs, which lose 2^-11 of
  // the output's 2^-8 (two parts there: 8 sequences of 256 blocks, 64/8 heads, e4m3
  // 17.7 -> 18.1 us, 32/2 heads 13.6 -> 15.1).
  constexpr bool kTwoParts = std::is_same<M, T>::value;
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' tiles, later their outputs
  float(*so)[H][D] = reinterpret_cast<float(*)[H][D]>(smem);
  __shared__ float sm[kSparseMaxWarps][H], sl[kSparseMaxWarps][H], cta_m[H], cta_l[H];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  SparseRow w = sparse_row(p, H);
  const int halves = p.block_size >> 4;  // items of a block
  const int cta_warps = blockDim.x >> 5, warps = w.ranks * cta_warps, me = w.rank * cta_warps + warp;
  int2 entry = sparse_entry(p, w, (me + lane * warps) / halves);  // of the first items

  // The queries' fragments: head r (and r + 8), 16 bytes as the keys lie.
  uint32_t qf[NT][KS][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = n * 8 + r;
    const T* q = static_cast<const T*>(p.q) + ((int64_t)w.seq * p.num_q_heads + w.first_head + (h < w.heads ? h : 0)) * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      // (Two 16-byte pieces of an 8-bit row's 16 dimensions, or one of 8.)
      const uint4 x = *reinterpret_cast<const uint4*>(KV8 ? q + 64 * (j / 2) + 16 * c + 8 * (j & 1) : q + 32 * j + 8 * c);
      qf[n][2 * j][0] = x.x;
      qf[n][2 * j][1] = x.y;
      qf[n][2 * j + 1][0] = x.z;
      qf[n][2 * j + 1][1] = x.w;
    }
  }
  float mul[NT][2];  // of the scores of heads 2 c, 2 c + 1
  // (Done when the first tiles are on their way.)
  auto scale_queries = [&] {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mul[n][0] = mul[n][1] = p.scale_log2;
      if constexpr (KV8 != 0 && std::is_same<T, __nv_bfloat16>::value) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[n][k][i]));
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        // The row's largest value goes to [2^14, 2^15): what that puts below
        // fp16's normal numbers is 2^28 times smaller.
        const int e = top > 0.f ? min(max((__float_as_int(top) >> 23) - 127 - 14, -126), 113) : 0;
        const float down = __int_as_float((127 - e) << 23), up = __int_as_float((127 + e) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[n][k][i]));
            qf[n][k][i] = MmaOp<__half>::pack(v.x * down, v.y * down);
          }
        mul[n][0] *= __shfl_sync(kAll, up, 8 * c);
        mul[n][1] *= __shfl_sync(kAll, up, 8 * c + 4);
      }
    }
  };

  float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int t = 0; t < MT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
    m[n][0] = m[n][1] = neg_inf();
    l[n][0] = l[n][1] = 0.f;
  }

  sparse_check(p, w);
  const int items = w.entries * halves;
  constexpr int RB = KV8 ? D : 2 * D;  // bytes of a row
  constexpr int kTile = 16 * RB, kStages = sparse_stages(kTile);
  uint8_t* ring = smem + warp * kStages * 2 * kTile;
  for (int base = me; base < items; base += 32 * warps) {
    // 32 items ahead, one a lane.
    const int mine = base + lane * warps;
    int2 it = make_int2(0, 0);
    float ks = 1.f, vs = 1.f;
    if (mine < items) {
      if (base != me) entry = sparse_entry(p, w, mine / halves);
      it = sparse_item(p, w, entry, halves == 2 ? mine & 1 : 0);
      if constexpr (KV8 != 0) {
        const float2 s = *reinterpret_cast<const float2*>(p.kv_scales + ((int64_t)it.x * p.num_kv_heads + w.head) * 2);
        ks = s.x;
        vs = s.y;
      }
    }
    const int count = min(32, (items - base + warps - 1) / warps);
    // Item x's K and V rows into a stage (rows behind its last: that row once
    // more; an item without tokens: the pool's first row, which weighs nothing).
    // The 16-byte pieces of a row change places by its number, so that those
    // that eight lanes read together lie in different banks.
    auto fetch = [&](int x, int stage) {
      if (x < count) {
        const int blk = __shfl_sync(kAll, it.x, x), last = max(__shfl_sync(kAll, it.y, x) - 1, 0);
        const int sub = halves == 2 ? (base + x * warps) & 1 : 0;
        const int64_t at = (((int64_t)blk * p.num_kv_heads + w.head) * p.block_size + 16 * sub) * RB;
        const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache) + at;
        const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache) + at;
        const uint32_t to = smem_u32(ring + stage * 2 * kTile);
#pragma unroll
        for (int i = 0; i < kTile / 512; ++i) {
          const int y = i * 32 + lane, row = y / (RB / 16), piece = y % (RB / 16), from = min(row, last) * RB + piece * 16;
          copy_async16(to + row * RB + (piece ^ (row & 1) << 2) * 16, kc + from);
          copy_async16(to + kTile + row * RB + (piece ^ (row & 6)) * 16, vc + from);
        }
      }
      copy_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i, i);
    if (base == me) scale_queries();
    int stage = 0;
    for (int x = 0; x < count; ++x) {
      fetch(x + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      copy_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* kt = ring + stage * 2 * kTile + r * RB;
      const uint8_t* vt = ring + stage * 2 * kTile + kTile + 2 * c * RB;
      const int n_tok = __shfl_sync(kAll, it.y, x);
      const float k_scale = KV8 ? __shfl_sync(kAll, ks, x) : 1.f, v_scale = KV8 ? __shfl_sync(kAll, vs, x) : 1.f;
      // Scores.
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        const int piece = (4 * j + c ^ (r & 1) << 2) * 16;
        const uint4 x0 = *reinterpret_cast<const uint4*>(kt + piece);
        const uint4 x1 = *reinterpret_cast<const uint4*>(kt + 8 * RB + piece);
        const uint32_t a0[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
        if constexpr (KV8 == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a[4] = {a0[2 * k], a1[2 * k], a0[2 * k + 1], a1[2 * k + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) MmaOp<M>::run(s[n], a, qf[n][2 * j + k][0], qf[n][2 * j + k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a[4];
            fp8x4_to_f16x4<KV8 == 2>(a0[k], a[0], a[2]);
            fp8x4_to_f16x4<KV8 == 2>(a1[k], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) MmaOp<M>::run(s[n], a, qf[n][4 * j + k][0], qf[n][4 * j + k][1]);
          }
        }
      }
      bool move = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[n][i] = r + 8 * (i >> 1) < n_tok ? s[n][i] * (KV8 ? mul[n][i & 1] * k_scale : mul[n][i & 1]) : neg_inf();
          move |= s[n][i] > m[n][i & 1] + kMoveAt;
        }
      }
      if (__any_sync(kAll, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(s[n][i], s[n][2 + i]);
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
            top = fmaxf(top, m[n][i]);
            if (top > m[n][i]) {
              const float f = fast_exp2(m[n][i] - top);
              m[n][i] = top;
              l[n][i] *= f;
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                o[n][t][i] *= f;
                o[n][t][2 + i] *= f;
              }
            }
          }
        }
      }
      // Weights in the products' type (their sums are taken before).
      uint32_t pf[NT][2], rest[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = m[n][i & 1];
          e[i] = fast_exp2(s[n][i] - (ref == neg_inf() ? 0.f : ref - (kTwoParts ? TwoParts<M>::kLift : 0.f)));
          l[n][i & 1] += e[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (kTwoParts) {
            TwoParts<M>::split(e[2 * i], e[2 * i + 1], pf[n][i], rest[n][i]);
            pf[n][i] = transposed(pf[n][i]);
            rest[n][i] = transposed(rest[n][i]);
          } else {
            pf[n][i] = transposed(MmaOp<M>::pack(e[2 * i], e[2 * i + 1]));
          }
        }
      }
      // Lane elements: word 2 i, 2 i + 1 of token i's dimensions.
      uint32_t v[4][MT];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = 2 * c + (i & 1) + 8 * (i >> 1) < n_tok;
#pragma unroll
        for (int j = 0; j < VP; ++j) {
          const uint4 y = *reinterpret_cast<const uint4*>(vt + ((i & 1) + 8 * (i >> 1)) * RB + (8 * j + r ^ 2 * c) * 16);
          const uint32_t x4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t word = there ? x4[k] : 0u;
            if constexpr (KV8 == 0) v[i][4 * j + k] = word;
            else fp8x4_to_f16x4<KV8 == 2>(word, v[i][8 * j + 2 * k], v[i][8 * j + 2 * k + 1]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        // Elements t and t + MT of every token's list.
        const int e0 = t, e1 = t + MT;
        const uint32_t a[4] = {__byte_perm(v[0][e0 / 2], v[1][e0 / 2], e0 & 1 ? 0x7632 : 0x5410),
                               __byte_perm(v[0][e1 / 2], v[1][e1 / 2], e1 & 1 ? 0x7632 : 0x5410),
                               __byte_perm(v[2][e0 / 2], v[3][e0 / 2], e0 & 1 ? 0x7632 : 0x5410),
                               __byte_perm(v[2][e1 / 2], v[3][e1 / 2], e1 & 1 ? 0x7632 : 0x5410)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          constexpr bool kScaled = kTwoParts && TwoParts<M>::kUp != 1.f;
          float left[4] = {0.f, 0.f, 0.f, 0.f};  // the rests' product, times kUp
          if constexpr (kScaled) MmaOp<M>::run(left, a, rest[n][0], rest[n][1]);
          if constexpr (KV8 == 0) {
            MmaOp<M>::run(o[n][t], a, pf[n][0], pf[n][1]);
            if constexpr (kTwoParts && !kScaled) MmaOp<M>::run(o[n][t], a, rest[n][0], rest[n][1]);
            if constexpr (kScaled) {
#pragma unroll
              for (int i = 0; i < 4; ++i) o[n][t][i] = fmaf(left[i], 1.f / TwoParts<M>::kUp, o[n][t][i]);
            }
          } else {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            MmaOp<M>::run(part, a, pf[n][0], pf[n][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (kScaled) part[i] = fmaf(left[i], 1.f / TwoParts<M>::kUp, part[i]);
              o[n][t][i] = fmaf(v_scale, part[i], o[n][t][i]);
            }
          }
        }
      }
      __syncwarp();  // the tiles have been read
      if (++stage == kStages) stage = 0;
    }
  }

  // Join the warps. Element e of a lane's list is dimension e of 16-byte
  // piece e / per, `per` elements each, its pieces 8 lanes apart.
  constexpr int PER = KV8 ? 16 : 8;
  copy_async_wait<0>();
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = n * 8 + 2 * c + i;
      float sum = l[n][i];
      sum += __shfl_xor_sync(kAll, sum, 4);
      sum += __shfl_xor_sync(kAll, sum, 8);
      sum += __shfl_xor_sync(kAll, sum, 16);
      if (r == 0) {
        sm[warp][h] = m[n][i];
        sl[warp][h] = sum;
      }
#pragma unroll
      for (int e = 0; e < 2 * MT; ++e) {
        const int d = e / PER * (8 * PER) + r * PER + e % PER;
        so[warp][h][d] = o[n][e % MT][i + 2 * (e / MT)];
      }
    }
  }
  __syncthreads();
  // A thread takes four dimensions of a head; a CTA alone writes them out.
  for (int x = tid; x < H * D / 4; x += blockDim.x) {
    const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
    float top = neg_inf(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < cta_warps; ++i) top = fmaxf(top, sm[i][h]);
    for (int i = 0; i < cta_warps; ++i) {
      const float f = part_weight(sm[i][h], top);
      const float4 v = reinterpret_cast<const float4*>(so[i])[x];
      sum += f * sl[i][h];
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if (w.ranks == 1) {
      if (h < w.heads) sparse_store<T, D>(p, w, h, d, acc, sum);
    } else {
      reinterpret_cast<float4*>(so[0])[x] = acc;
      if (d == 0) {
        cta_m[h] = top;
        cta_l[h] = sum;
      }
    }
  }
  if (w.ranks > 1) sparse_join<T, D>(p, w, &so[0][0][0], cta_m, cta_l);
}

// fp32 on CUDA cores, exact fp32 arithmetic, for 8 query heads: a CTA scores 16
// tokens at a time, a (head, token) pair a thread, and adds their values, a
// dimension (or two) a thread, while copies bring the next 16 tokens.
constexpr int sparse_f32_smem(int d) { return (8 * d + 8 * (d + 4) + 2 * 16 * (d + 4) + 2 * 16 * d) * 4; }

template <int D>
__global__ void __launch_bounds__(kSparseF32Threads) sparse_f32_kernel(const __grid_constant__ SparseParams p) {
  constexpr int H = 8, TOK = 16, ST = D + 4;
  constexpr int DT = (D + kSparseF32Threads - 1) / kSparseF32Threads;  // dimensions of a thread
  extern __shared__ __align__(16) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);  // [H][D]
  float* sq = so + H * D;                      // [H][ST]
  float* sk = sq + H * ST;                     // [2][TOK][ST]
  float* sv = sk + 2 * TOK * ST;               // [2][TOK][D]
  __shared__ __align__(16) float ss[TOK][H];
  __shared__ float sm[H], sl[H], sf[H];
  const int tid = threadIdx.x;
  SparseRow w = sparse_row(p, H);
  sparse_check(p, w);
  const int halves = p.block_size >> 4, items = w.entries * halves;
  const float* q = static_cast<const float*>(p.q) + ((int64_t)w.seq * p.num_q_heads + w.first_head) * D;
  for (int x = tid; x < w.heads * D; x += kSparseF32Threads) sq[x / D * ST + x % D] = q[x];
  if (tid < H) {
    sm[tid] = neg_inf();
    sl[tid] = 0.f;
  }
  float acc[H][DT];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[h][i] = 0.f;
  // Item x's tokens into a half of the buffers (every thread asks what it is:
  // the answer is the same); the number of them.
  auto fetch = [&](int x, int half) {
    int tokens = 0;
    if (x < items) {
      const int sub = halves == 2 ? x & 1 : 0;
      const int2 it = sparse_item(p, w, sparse_entry(p, w, x / halves), sub);
      tokens = it.y;
      const int64_t at = (((int64_t)it.x * p.num_kv_heads + w.head) * p.block_size + 16 * sub) * D;
      for (int y = tid; y < tokens * (D / 4); y += kSparseF32Threads) {
        const int t = y / (D / 4), d = (y - t * (D / 4)) * 4;
        copy_async16(smem_u32(sk + (half * TOK + t) * ST + d), static_cast<const float*>(p.k_cache) + at + t * D + d);
        copy_async16(smem_u32(sv + (half * TOK + t) * D + d), static_cast<const float*>(p.v_cache) + at + t * D + d);
      }
    }
    copy_async_commit();
    return tokens;
  };
  int half = 0, tokens = fetch(w.rank, 0);
  for (int x = w.rank; x < items; x += w.ranks, half ^= 1) {
    const int next = fetch(x + w.ranks, half ^ 1);
    copy_async_wait<1>();
    __syncthreads();
    const float *kt = sk + half * TOK * ST, *vt = sv + half * TOK * D;
    {
      const int t = tid % TOK, h = tid / TOK;  // 16 tokens x 8 heads
      float s = neg_inf();
      if (t < tokens && h < w.heads) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
          const float4 x4 = *reinterpret_cast<const float4*>(kt + t * ST + d);
          const float4 y4 = *reinterpret_cast<const float4*>(sq + h * ST + d);
          a.x = fmaf(x4.x, y4.x, a.x);
          a.y = fmaf(x4.y, y4.y, a.y);
          a.z = fmaf(x4.z, y4.z, a.z);
          a.w = fmaf(x4.w, y4.w, a.w);
        }
        s = ((a.x + a.y) + (a.z + a.w)) * p.scale_log2;
      }
      float top = s;
#pragma unroll
      for (int i = 1; i < TOK; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      const float old = sm[h], now = fmaxf(old, top);
      const float ref = now == neg_inf() ? 0.f : now;
      const float e = exp2f(s - ref);
      float sum = e;
#pragma unroll
      for (int i = 1; i < TOK; i <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
      ss[t][h] = e;
      __syncwarp();
      if (t == 0) {
        const float f = old == neg_inf() ? 1.f : exp2f(old - ref);
        sf[h] = f;
        sl[h] = sl[h] * f + sum;
        sm[h] = now;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float f = sf[h];
#pragma unroll
      for (int i = 0; i < DT; ++i) acc[h][i] *= f;
    }
    for (int t = 0; t < tokens; ++t) {
      const float4 e0 = *reinterpret_cast<const float4*>(&ss[t][0]), e1 = *reinterpret_cast<const float4*>(&ss[t][4]);
      const float e[H] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const int d = tid + i * kSparseF32Threads;
        const float v = d < D ? vt[t * D + d] : 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h][i] = fmaf(e[h], v, acc[h][i]);
      }
    }
    tokens = next;
    __syncthreads();  // the buffers' half and the weights have been read
  }
  copy_async_wait<0>();
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < DT; ++i)
      if (tid + i * kSparseF32Threads < D) so[h * D + tid + i * kSparseF32Threads] = acc[h][i];
  sparse_join<float, D>(p, w, so, sm, sl);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int launch_sparse(void (*kernel)(SparseParams), const SparseParams& p, int ranks, int warps, int smem,
                  cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.num_seqs * p.num_kv_heads * p.row_groups * ranks));
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

template <int D>
int launch_sparse_f32(const SparseParams& p, cudaStream_t stream) {
  constexpr int smem = sparse_f32_smem(D);
  if (smem > 40 * 1024 &&
      set_max_dynamic_smem(reinterpret_cast<const void*>(sparse_f32_kernel<D>), smem) != PA_OK)
    return PA_ERR_CUDA;
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads * p.row_groups;
  const int64_t items = (int64_t)p.max_list_len * (p.block_size / 16);
  const int sms = num_sms_current_device();
  const int ranks = cluster_ranks(rows, 4 * sms, items / 4);  // (four CTAs an SM)
  return launch_sparse(sparse_f32_kernel<D>, p, ranks, kSparseF32Threads / 32, smem, stream);
}

template <typename T, int KV8, int D, int NT>
int launch_sparse_tc(const SparseParams& p, cudaStream_t stream) {
  constexpr int tile = 16 * D * (KV8 ? 1 : 2), warp_smem = sparse_stages(tile) * 2 * tile;
  constexpr int kRoom = NT == 1 ? 12 : 8;  // warps that an SM's registers (and shared memory) hold
  static_assert(warp_smem >= 8 * NT * D * 4, "a warp's output fits into its tiles");
  // All CTAs at once, if an SM's warps suffice: the CTAs of a row (of 8 items at
  // least) and the warps of each, no warp with less than two items.
  const int sms = num_sms_current_device();
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads * p.row_groups;
  const int64_t items = (int64_t)p.max_list_len * (p.block_size / 16);
  const int ranks = cluster_ranks(rows, sms, items / 8);
  const int64_t per_sm = (rows * ranks + sms - 1) / sms;
  int warps = (int)std::min<int64_t>(kRoom, per_sm * 2 <= kRoom ? kRoom / per_sm : 4);
  warps = (int)std::min<int64_t>(warps, std::max<int64_t>(2, (items + 2 * ranks - 1) / (2 * ranks)));
  const auto kernel = sparse_kernel<T, KV8, D, NT>;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kRoom * warp_smem) != PA_OK)
    return PA_ERR_CUDA;
  return launch_sparse(kernel, p, ranks, warps, warps * warp_smem, stream);
}

template <typename T, int KV8, int D>
int launch_sparse_tc(const SparseParams& p, cudaStream_t stream) {
  return p.group <= 8 ? launch_sparse_tc<T, KV8, D, 1>(p, stream) : launch_sparse_tc<T, KV8, D, 2>(p, stream);
}

// kv8: 0, or 1 + the format of an 8-bit cache.
int decode_sparse(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                  const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                  const int32_t* block_lists, const int32_t* list_lens, int32_t max_list_len, int32_t num_seqs,
                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int32_t num_blocks, float scale, void* out, pa_dtype dtype, int kv8, cudaStream_t stream) {
  if (num_seqs < 0 || max_blocks_per_seq < 1 || max_list_len < 1 || num_q_heads < 1 || num_kv_heads < 1 ||
      num_blocks < 1 || !std::isfinite(scale))
    return PA_ERR_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16 && (kv8 || dtype != PA_F32)) return PA_ERR_DTYPE;
  if (num_q_heads % num_kv_heads) return PA_ERR_HEADS;
  if (block_size != 16 && block_size != 32) return PA_ERR_BLOCKSIZE;
  const int group = num_q_heads / num_kv_heads;
  if (kv8 ? head_dim != 128
          : dtype == PA_F32 ? head_dim < 32 || head_dim > 256 || head_dim % 32 : head_dim != 64 && head_dim != 128)
    return PA_ERR_UNSUPPORTED;
  if (group > 128 || num_seqs > 65535 || max_list_len > (1 << 26)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !block_lists || !list_lens || !out ||
      (kv8 && !kv_scales))
    return PA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || (kv8 && !aligned16(kv_scales)))
    return PA_ERR_ALIGN;
  SparseParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_scales = kv_scales;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.lists = block_lists;
  p.list_lens = list_lens;
  p.out = out;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_list_len = max_list_len;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.group = group;
  const int per_row = dtype == PA_F32 || group <= 8 ? 8 : 16;
  p.row_groups = (group + per_row - 1) / per_row;
  p.scale_log2 = scale * 1.4426950408889634f;
  if ((int64_t)num_seqs * num_kv_heads * p.row_groups > (1 << 27)) return PA_ERR_UNSUPPORTED;
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
  if (dtype == PA_F32) {
    switch (head_dim / 32) {
      case 1: return launch_sparse_f32<32>(p, stream);
      case 2: return launch_sparse_f32<64>(p, stream);
      case 3: return launch_sparse_f32<96>(p, stream);
      case 4: return launch_sparse_f32<128>(p, stream);
      case 5: return launch_sparse_f32<160>(p, stream);
      case 6: return launch_sparse_f32<192>(p, stream);
      case 7: return launch_sparse_f32<224>(p, stream);
      default: return launch_sparse_f32<256>(p, stream);
    }
  }
  const bool half = dtype == PA_F16;
  if (kv8 == 1 + PA_KV_E4M3)
    return half ? launch_sparse_tc<__half, 1, 128>(p, stream) : launch_sparse_tc<__nv_bfloat16, 1, 128>(p, stream);
  if (kv8)
    return half ? launch_sparse_tc<__half, 2, 128>(p, stream) : launch_sparse_tc<__nv_bfloat16, 2, 128>(p, stream);
  if (head_dim == 64)
    return half ? launch_sparse_tc<__half, 0, 64>(p, stream) : launch_sparse_tc<__nv_bfloat16, 0, 64>(p, stream);
  return half ? launch_sparse_tc<__half, 0, 128>(p, stream) : launch_sparse_tc<__nv_bfloat16, 0, 128>(p, stream);
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_decode_sparse(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const int32_t* block_lists,
                     const int32_t* list_lens, int32_t max_list_len, int32_t num_seqs, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                     void* out, pa_dtype dtype, void* stream) {
  return pa::decode_sparse(q, k_cache, v_cache, nullptr, block_tables, max_blocks_per_seq, seq_lens, block_lists,
                           list_lens, max_list_len, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           num_blocks, scale, out, dtype, 0, static_cast<cudaStream_t>(stream));
}

int pa_decode_sparse_fp8(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                         const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* block_lists, const int32_t* list_lens, int32_t max_list_len,
                         int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int32_t num_blocks, float scale, void* out, pa_dtype dtype,
                         void* stream) {
  return pa::decode_sparse(q, k_cache, v_cache, kv_scales, block_tables, max_blocks_per_seq, seq_lens, block_lists,
                           list_lens, max_list_len, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           num_blocks, scale, out, dtype, 1 + pa::PA_KV_E4M3, static_cast<cudaStream_t>(stream));
}

int pa_decode_sparse_e5m2(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                          const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                          const int32_t* block_lists, const int32_t* list_lens, int32_t max_list_len,
                          int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                          int32_t block_size, int32_t num_blocks, float scale, void* out, pa_dtype dtype,
                          void* stream) {
  return pa::decode_sparse(q, k_cache, v_cache, kv_scales, block_tables, max_blocks_per_seq, seq_lens, block_lists,
                           list_lens, max_list_len, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           num_blocks, scale, out, dtype, 1 + pa::PA_KV_E5M2, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

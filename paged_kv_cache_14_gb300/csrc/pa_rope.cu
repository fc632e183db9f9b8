// Rotary positions: the table of cosines and sines, and the rotation of new
// queries and keys with the cache write on the way.
//
// A pair (x1, x2) of a row at position p turns by the angle p f_i:
//   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin.
// Every product, sum and difference is one IEEE fp32 operation (no fused
// multiply-add), so results can be reproduced bit for bit from the table.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kRopeMaxDim = 256;
constexpr int kRopeThreads = 128;

// ---------------------------------------------------------------------------
// The table
// ---------------------------------------------------------------------------

// Turns a position of each pair, as fractions of 2^64: p * step mod 2^64 is
// the position's angle without its whole turns, exact to 2^-64 of a turn a
// position, where fp32 would lose an angle of 2^17 radians by 2^-7. (The GPU's
// 64-bit floating point has a sixtieth of its fp32 rate; integers have not.)
struct RopeSteps {
  unsigned long long step[kRopeMaxDim / 2];
};

// cos and sin of position p: the upper 32 bits of its angle (2^-32 of a turn is
// 1.5e-9) less the nearest quarter turn, and the rest, at most pi/4, through
// the Taylor polynomials of degree 9 and 10 (their next terms are below 2^-28).
__device__ __forceinline__ void turn(uint32_t p, unsigned long long step, float& c, float& s) {
  const uint32_t t = p * (uint32_t)(step >> 32) + __umulhi(p, (uint32_t)step);
  const uint32_t quarter = (t + (1u << 29)) >> 30;
  const float x = __int2float_rn((int)(t << 2)) * (float)(1.5707963267948966 / 4294967296.0);
  const float y = x * x;
  const float sn =
      x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
  const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
  const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
  c = (quarter + 1) & 2 ? -a : a;
  s = quarter & 2 ? -b : b;
}

// A thread keeps N pairs (4 where the halves are whole float4) and goes from
// position to position. Bound by instruction issue, about as long as the
// stores take: 131072 positions of 128 (67 MB) in 11.3 us of a graph's replay, 5.9
// TB/s, where a fill of the same memory takes 10.2; a call by itself 13.7.
template <int N>
__global__ void __launch_bounds__(kRopeThreads) rope_table_kernel(float* __restrict__ out, uint32_t first,
                                                                   uint32_t positions, int32_t half, float amplitude,
                                                                   const __grid_constant__ RopeSteps steps) {
  const int groups = half / N, rows = kRopeThreads / groups;  // positions that a CTA does at a time
  const int row = threadIdx.x / groups, i = (threadIdx.x - row * groups) * N;
  if (row >= rows) return;
  unsigned long long step[N];
#pragma unroll
  for (int k = 0; k < N; ++k) step[k] = steps.step[i + k];
  for (int64_t p = (int64_t)blockIdx.x * rows + row; p < positions; p += (int64_t)gridDim.x * rows) {
    float c[N], s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      turn(first + (uint32_t)p, step[k], c[k], s[k]);
      c[k] *= amplitude;
      s[k] *= amplitude;
    }
    float* dst = out + p * 2 * half + i;
    if constexpr (N == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(dst + half) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      dst[0] = c[0];
      dst[half] = s[0];
    }
  }
}

// ---------------------------------------------------------------------------
// Rotation and cache write
// ---------------------------------------------------------------------------

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements from a token to the next
  const int32_t* positions;
  const int64_t* slots;
  const float* table;
  int32_t num_positions, rot;
  int64_t num_tokens;
  void* q_out;
  void* k_cache;
  void* v_cache;
  float* kv_scales;
  int32_t num_blocks, block_size, num_q_heads, num_kv_heads, head_dim;
  int32_t row_units;    // work units of a row
  int32_t rows;         // rows of a token: queries, and keys and values of a 16- or 32-bit cache
  int32_t pass_rows;    // rows that a CTA does at a time
  int32_t chunks;       // CTAs of a token
  uint32_t cache_ctas;  // 8-bit caches: CTAs that write them
  int32_t group;        // 8-bit caches: tokens of a warp
  int* status;
};

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// A token's slot (-1: it is skipped) and position. (Both are asked for at once.)
struct RopePlace {
  int64_t slot;
  int32_t pos;
};
__device__ __forceinline__ RopePlace rope_place(const RopeParams& p, int64_t t, bool report) {
  RopePlace at{p.slots[t], p.positions[t]};
  if (at.slot < 0) {  // padding
    at.slot = -1;
  } else if (at.slot >= (int64_t)p.num_blocks * p.block_size) {
    if (report) record_error(p.status, PA_ERR_BLOCK_OOB);
    at.slot = -1;
  } else if (at.pos < 0 || at.pos >= p.num_positions) {
    if (report) record_error(p.status, PA_ERR_SEQLEN);
    at.slot = -1;
  }
  return at;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes of elements.
template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  union {
    int4 raw;
    T e[N];
  };
  __device__ __forceinline__ Vec16() {}
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const int4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<int4*>(p) = raw; }
};

// One element.
template <typename T>
struct Vec1 {
  T e[1];
  __device__ __forceinline__ void load(const T* p) { e[0] = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = e[0]; }
};

enum RopeLayout { kRopePairs, kRopeHalves, kRopeHalvesOdd };

// Where row `row` of a token lies, and where it goes: queries first, then keys
// and values.
template <typename T>
__device__ __forceinline__ const T* rope_source(const RopeParams& p, int64_t t, int row) {
  const int h = row - p.num_q_heads;
  return h < 0 ? static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)row * p.head_dim
         : h < p.num_kv_heads
             ? static_cast<const T*>(p.k) + t * p.k_stride + (int64_t)h * p.head_dim
             : static_cast<const T*>(p.v) + t * p.v_stride + (int64_t)(h - p.num_kv_heads) * p.head_dim;
}
template <typename T>
__device__ __forceinline__ T* rope_target(const RopeParams& p, int64_t t, int64_t blk, int off, int row) {
  const int h = row - p.num_q_heads;
  if (h < 0) return static_cast<T*>(p.q_out) + (t * p.num_q_heads + row) * p.head_dim;
  const bool is_v = h >= p.num_kv_heads;
  return static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
         ((blk * p.num_kv_heads + (is_v ? h - p.num_kv_heads : h)) * p.block_size + off) * p.head_dim;
}

// A CTA takes a token's rows, or a part of them, `pass_rows` at a time; a
// thread keeps its place in the row and with it its cosines and sines. Its
// place is a vector of each half, or a vector that stays (kRopeHalves); a
// vector of pairs (kRopePairs); an element of each half, or one that stays
// (kRopeHalvesOdd: a half that is no whole number of vectors). Rows are read
// once and written once, rope_batch of them in flight; a query may be rotated
// in place, because the thread that writes an element is the one that reads it.
//
// Bound by HBM: 13504 tokens of 64 + 8 + 8 heads (fp16, half of each head, side
// by side) in 92 us, 6.0 TB/s read and written; of 32 + 8 + 8 (bf16 halves) in
// 57, 6.0 TB/s; 12000 of 32 + 8 + 8 fp32 rows in 88, 6.8 TB/s. Halves that are no
// whole vectors take an element a thread: 12000 such tokens (bf16, 90 of 128
// dimensions) 164, 1.8 TB/s. More rows in flight need registers that warps
// would have (halves: 2, 3, 4 rows 62, 57, 67 us; pairs: 4, 5 rows 94, 92).
constexpr int rope_batch(int layout) { return layout == kRopePairs ? 5 : 3; }

template <typename T, int LAYOUT>
__device__ __forceinline__ void rope_token(const RopeParams& p, int64_t t, int chunk) {
  constexpr int N = LAYOUT == kRopeHalvesOdd ? 1 : Vec16<T>::N;
  constexpr int PAIRS = LAYOUT == kRopePairs ? N / 2 : N;
  constexpr int B = rope_batch(LAYOUT);
  using V = typename std::conditional<LAYOUT == kRopeHalvesOdd, Vec1<T>, Vec16<T>>::type;
  const int places = min(p.row_units, kRopeThreads), row0 = threadIdx.x / places;
  const int half = p.rot >> 1, rotated = p.num_q_heads + p.num_kv_heads, step = p.chunks * p.pass_rows;
  const RopePlace place = rope_place(p, t, chunk == 0 && threadIdx.x == 0);
  if (row0 >= p.pass_rows) return;
  for (int u = threadIdx.x - row0 * places; u < p.row_units; u += places) {
    const int d = u * N;
    // Pairs of this place: all of them turn, or (pairs) those below rot.
    const bool two = LAYOUT != kRopePairs && d < half;
    const int at = LAYOUT == kRopePairs || two ? d : half + d;  // a place behind the halves
    const int turning = LAYOUT == kRopePairs ? max(0, min(PAIRS, (p.rot - d) >> 1)) : two ? PAIRS : 0;
    int r0 = chunk * p.pass_rows + row0;
    V x[B], y[B];
    auto load = [&] {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (r0 + k * step >= p.rows) break;
        const T* src = rope_source<T>(p, t, r0 + k * step);
        x[k].load(src + at);
        if (two) y[k].load(src + half + d);
      }
    };
    load();  // (before the token's place is known: its rows are there in any case)
    if (place.slot < 0) return;
    const float* cs = p.table + (int64_t)place.pos * p.rot;
    const int64_t blk = place.slot / p.block_size;
    const int off = (int)(place.slot - blk * p.block_size);
    float c[PAIRS], s[PAIRS];
    const float* from = cs + (LAYOUT == kRopePairs ? d >> 1 : d);
    if (turning == PAIRS && PAIRS % 4 == 0 && (half & 3) == 0) {
#pragma unroll
      for (int i = 0; i < PAIRS / 4; ++i) {
        reinterpret_cast<float4*>(c)[i] = reinterpret_cast<const float4*>(from)[i];
        reinterpret_cast<float4*>(s)[i] = reinterpret_cast<const float4*>(from + half)[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        c[i] = i < turning ? from[i] : 1.f;
        s[i] = i < turning ? from[half + i] : 0.f;
      }
    }
    while (true) {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int row = r0 + k * step;
        if (row >= p.rows) break;
        if (row < rotated) {
          if constexpr (LAYOUT == kRopePairs) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
              if (i < turning) {
                float a = to_f32(x[k].e[2 * i]), b = to_f32(x[k].e[2 * i + 1]);
                rotate(a, b, c[i], s[i]);
                x[k].e[2 * i] = from_f32<T>(a);
                x[k].e[2 * i + 1] = from_f32<T>(b);
              }
            }
          } else if (two) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
              float a = to_f32(x[k].e[i]), b = to_f32(y[k].e[i]);
              rotate(a, b, c[i], s[i]);
              x[k].e[i] = from_f32<T>(a);
              y[k].e[i] = from_f32<T>(b);
            }
          }
        }
        T* dst = rope_target<T>(p, t, blk, off, row);
        x[k].store(dst + at);
        if (two) y[k].store(dst + half + d);
      }
      r0 += B * step;
      if (r0 >= p.rows) break;
      load();
    }
  }
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const unsigned t = blockIdx.x / p.chunks;
  rope_token<T, LAYOUT>(p, t, blockIdx.x - t * p.chunks);
}

// ---------------------------------------------------------------------------
// 8-bit caches. The queries' units as above; keys and values as
// pa_reshape_and_cache_fp8 writes them, a warp per (run of tokens in one
// block, KV head, pool), the keys rotated in fp32 and encoded from there (one
// rounding, not two).
// ---------------------------------------------------------------------------

// Elements d .. d + VEC - 1 of a row as they lie.
template <typename T, int VEC>
__device__ __forceinline__ void row_values(const T* row, int d, float (&x)[VEC]) {
  struct alignas(VEC * sizeof(T)) Part {
    T e[VEC];
  };
  const Part v = *reinterpret_cast<const Part*>(row + d);
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = to_f32(v.e[i]);
}

// The same, rotated if cs is given. `whole`: the halves are whole numbers of
// VEC.
template <typename T, int VEC>
__device__ __forceinline__ void rope_values(const T* row, const float* cs, int d, int rot, bool inter, bool whole,
                                            float (&x)[VEC]) {
  row_values<T, VEC>(row, d, x);
  if (!cs || d >= rot) return;
  const int half = rot >> 1;
  if (inter) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
      if (d + i < rot) rotate(x[i], x[i + 1], cs[(d + i) >> 1], cs[half + ((d + i) >> 1)]);
    return;
  }
  if (whole) {
    const bool upper = d >= half;
    const int lo = upper ? d - half : d;
    float y[VEC], c[VEC], s[VEC];
    row_values<T, VEC>(row, upper ? lo : d + half, y);
    row_values<float, VEC>(cs, lo, c);
    row_values<float, VEC>(cs + half, lo, s);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      // (Half of the pair, with the operations of rotate().)
      x[i] = upper ? __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]))
                   : __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int e = d + i;
    if (e >= rot) continue;
    const bool upper = e >= half;
    const int lo = upper ? e - half : e;
    float a = to_f32(row[lo]), b = to_f32(row[lo + half]);
    rotate(a, b, cs[lo], cs[half + lo]);
    x[i] = upper ? b : a;
  }
}

// The place of token j, which need not exist.
__device__ __forceinline__ RopePlace rope_place_or_none(const RopeParams& p, int64_t j) {
  return j >= 0 && j < p.num_tokens ? rope_place(p, j, false) : RopePlace{-1, 0};
}

constexpr int kRunBatch = 2;

// The run of tokens that starts with token t (its place: slot): one KV head of
// one pool. Rows are loaded kRunBatch at a time; the rows of a run that is no
// longer are kept from the search for the largest value to their encoding.
template <typename T, int VEC, bool E5>
__device__ __forceinline__ void rope_run_8bit(const RopeParams& p, bool inter, int64_t t, int64_t slot, int h,
                                              int pool) {
  constexpr int D = VEC * 32;
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, bs = p.block_size;
  const int64_t blk = slot / bs, tile = blk * p.num_kv_heads + h;
  const T* src = static_cast<const T*>(pool == 0 ? p.k : p.v) + h * D;
  const int64_t stride = pool == 0 ? p.k_stride : p.v_stride;
  const bool whole = (p.rot >> 1) % VEC == 0;
  uint8_t* codes = static_cast<uint8_t*>(pool == 0 ? p.k_cache : p.v_cache) + tile * bs * D + lane * VEC;
  float* sp = p.kv_scales + tile * 2 + pool;
  const float stored = *sp;
  float x[kRunBatch][VEC];
  int off[kRunBatch];
  // The next rows of `mem` (tokens base + its bits; lanes have their places).
  auto take = [&](int64_t base, const RopePlace& at, unsigned& mem) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kRunBatch; ++k) {
      if (!mem) break;
      const int ln = __ffs(mem) - 1;
      mem &= mem - 1;
      off[k] = (int)(__shfl_sync(kFull, at.slot, ln) - blk * bs);
      const float* cs = pool == 0 ? p.table + (int64_t)__shfl_sync(kFull, at.pos, ln) * p.rot : nullptr;
      rope_values<T, VEC>(src + (base + ln) * stride, cs, lane * VEC, p.rot, inter, whole, x[k]);
      n = k + 1;
    }
    return n;
  };
  float amax = 0.f;
  int omin = bs, rows = 0, kept = 0;
  int64_t end = p.num_tokens;
  for (int64_t base = t; base < p.num_tokens; base += 32) {
    const RopePlace at = rope_place_or_none(p, base + lane);
    const unsigned other = __ballot_sync(kFull, at.slot >= 0 && at.slot / bs != blk);
    const int lim = other ? __ffs(other) - 1 : 32;
    unsigned mem = __ballot_sync(kFull, at.slot >= 0 && lane < lim);
    while (mem) {
      kept = take(base, at, mem);
      rows += kept;
#pragma unroll
      for (int k = 0; k < kRunBatch; ++k) {
        if (k >= kept) break;
        omin = min(omin, off[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[k][i]));
      }
    }
    if (other) {
      end = base + lim;
      break;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  const float s_old = omin == 0 ? 0.f : stored;
  const float s_new = fmaxf(s_old, __fdiv_rn(amax, E5 ? 57344.f : 448.f));
  if (s_new > s_old && s_old > 0.f) {
    const float r = __fdiv_rn(s_old, s_new);
    constexpr int kAgain = 8;  // rows in flight
    for (int o0 = 0; o0 < omin; o0 += kAgain) {
      float y[kAgain][VEC];
#pragma unroll
      for (int k = 0; k < kAgain; ++k) load_codes<VEC, E5>(codes + min(o0 + k, omin - 1) * D, y[k]);
#pragma unroll
      for (int k = 0; k < kAgain; ++k) {
        uint32_t c[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
          c[i / 2] = f32x2_to_fp8x2<E5>(__fmul_rn(y[k][i], r), __fmul_rn(y[k][i + 1], r));
        if (o0 + k < omin) store_codes<VEC>(codes + (o0 + k) * D, c);
      }
    }
  }
  const Divisor div = divisor(s_new);
  auto encode = [&](int n) {
#pragma unroll
    for (int k = 0; k < kRunBatch; ++k) {
      if (k >= n) break;
      uint32_t c[VEC / 2];
#pragma unroll
      for (int i = 0; i < VEC; i += 2)
        c[i / 2] = s_new > 0.f ? f32x2_to_fp8x2<E5>(quotient(x[k][i], div), quotient(x[k][i + 1], div)) : 0u;
      store_codes<VEC>(codes + off[k] * D, c);
    }
  };
  if (rows == kept) {
    encode(kept);
  } else {
    for (int64_t base = t; base < end; base += 32) {
      const RopePlace at = rope_place_or_none(p, base + lane < end ? base + lane : -1);
      unsigned mem = __ballot_sync(kFull, at.slot >= 0);
      while (mem) encode(take(base, at, mem));
    }
  }
  if (lane == 0) *sp = s_new;
}

// A warp per (group of tokens, KV head, pool): the runs that start in the
// group. A token starts a run if the nearest one before it that counts lies in
// another block; lanes look at the 16 tokens before the group and at the
// group's.
template <typename T, int VEC, bool E5>
__device__ __forceinline__ void rope_cache_8bit(const RopeParams& p, bool inter, int64_t w) {
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, hkv = p.num_kv_heads, bs = p.block_size;
  const int64_t g = w / (hkv * 2), t0 = g * p.group;
  const int rem = (int)(w - g * hkv * 2), h = rem >> 1, pool = rem & 1;
  const int64_t t = t0 - 16 + lane;
  const bool mine = lane >= 16 && lane < 16 + p.group && t < p.num_tokens;
  const int64_t slot = rope_place_or_none(p, t).slot;
  if (mine && slot < 0 && rem == 0) rope_place(p, t, true);  // (what is wrong with it)
  const unsigned ok = __ballot_sync(kFull, slot >= 0);
  const unsigned below = ok & ((1u << lane) - 1u);
  const int64_t before = __shfl_sync(kFull, slot, below ? 31 - __clz(below) : 0);
  unsigned starts = __ballot_sync(kFull, mine && slot >= 0 && (!below || before / bs != slot / bs));
  const unsigned unsure = __ballot_sync(kFull, mine && slot >= 0 && !below && t0 > 16);
  if (unsure) {
    // Nothing but padding in the window: look further back.
    const int ln = __ffs(unsure) - 1;
    const int64_t blk = __shfl_sync(kFull, slot, ln) / bs;
    for (int64_t base = t0 - 17; base >= 0; base -= 32) {
      const int64_t sj = rope_place_or_none(p, base - lane).slot;
      const unsigned found = __ballot_sync(kFull, sj >= 0);
      if (found) {
        const int64_t near = __shfl_sync(kFull, sj, __ffs(found) - 1);  // lowest lane = latest token
        if (near / bs == blk) starts &= ~(1u << ln);
        break;
      }
    }
  }
  while (starts) {
    const int ln = __ffs(starts) - 1;
    starts &= starts - 1;
    rope_run_8bit<T, VEC, E5>(p, inter, t0 - 16 + ln, __shfl_sync(kFull, slot, ln), h, pool);
  }
}

// The caches' CTAs come first: they take longer than the queries'. 64 registers
// (8 CTAs an SM) for what is a chain of loads: 256 tokens of 64 + 8 + 8 heads,
// each in a block under way, take 7 us (10 with 96), 6100 prompt tokens 74 (88),
// of which the rows of the 8-bit caches are two thirds: a block of 16 a warp, two
// rows in flight, read, rotated and looked up once for the largest value and once
// more to be encoded. (Half of the variants spill 36 to 80 bytes to get by with 64
// registers.) A chunk of 32 tokens is that chain alone, 18 us.
template <typename T, int VEC, bool E5, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_8bit_kernel(const __grid_constant__ RopeParams p) {
  if (blockIdx.x < p.cache_ctas) {
    const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (w < (p.num_tokens + p.group - 1) / p.group * p.num_kv_heads * 2)
      rope_cache_8bit<T, VEC, E5>(p, LAYOUT == kRopePairs, w);
    return;
  }
  const unsigned x = blockIdx.x - p.cache_ctas, t = x / p.chunks;
  rope_token<T, LAYOUT>(p, t, x - t * p.chunks);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Numbers of some 104 bits as sums of two doubles (Dekker, "A floating-point
// technique for extending the available precision", 1971), with the fused
// multiply-add for a product's remainder. A frequency of 53 bits is off by
// 2^-22 of a radian at position 2^31, as far as an entry may be.
struct Twice {
  double hi, lo;
};
Twice plus(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Twice operator+(Twice a, Twice b) {
  const Twice s = plus(a.hi, b.hi);
  return plus(s.hi, s.lo + (a.lo + b.lo));
}
Twice operator-(Twice a, Twice b) { return a + Twice{-b.hi, -b.lo}; }
Twice operator*(Twice a, Twice b) {
  const double p = a.hi * b.hi;
  return plus(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Twice operator/(Twice a, Twice b) {
  const double q = a.hi / b.hi;
  const Twice rest = a - b * Twice{q, 0.0};
  return plus(q, rest.hi / b.hi);
}
// x^(-1/n), by Newton's steps from the double.
Twice inverse_root(double x, int n) {
  Twice r{std::pow(x, -1.0 / n), 0.0};
  for (int step = 0; step < 2; ++step) {
    Twice product{x, 0.0}, square = r;
    for (int k = n; k; k >>= 1, square = square * square)
      if (k & 1) product = product * square;
    r = r + r * (Twice{1.0, 0.0} - product) / Twice{(double)n, 0.0};
  }
  return r;
}
// x without its whole part, in units of 2^-64.
unsigned long long fraction(double x) {
  const double part = std::fabs(x) - std::floor(std::fabs(x));
  const unsigned long long units = (unsigned long long)(part * 18446744073709551616.0);
  return x < 0 ? 0 - units : units;
}

template <typename T, int LAYOUT>
int launch_rope(const RopeParams& p, int kv8, cudaStream_t stream) {
  if (!kv8) {
    rope_kernel<T, LAYOUT><<<(unsigned)(p.num_tokens * p.chunks), kRopeThreads, 0, stream>>>(p);
  } else {
    const unsigned ctas = p.cache_ctas + (p.num_q_heads > 0 ? (unsigned)(p.num_tokens * p.chunks) : 0u);
    const bool e5 = kv8 == 1 + PA_KV_E5M2;
    if (p.head_dim == 64 && e5) rope_8bit_kernel<T, 2, true, LAYOUT><<<ctas, kRopeThreads, 0, stream>>>(p);
    else if (p.head_dim == 64) rope_8bit_kernel<T, 2, false, LAYOUT><<<ctas, kRopeThreads, 0, stream>>>(p);
    else if (e5) rope_8bit_kernel<T, 4, true, LAYOUT><<<ctas, kRopeThreads, 0, stream>>>(p);
    else rope_8bit_kernel<T, 4, false, LAYOUT><<<ctas, kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// kv8: 0, or 1 + the format of an 8-bit cache.
int rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                   const int32_t* positions, const int64_t* slot_mapping, const float* cos_sin,
                   int32_t num_positions, int32_t rot_dim, int32_t interleaved, int64_t num_tokens, void* q_out,
                   void* k_cache, void* v_cache, float* kv_scales, int32_t num_blocks, int32_t block_size,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, int kv8,
                   cudaStream_t stream) {
  const int size = dtype == PA_F32 ? 4 : dtype == PA_F16 || dtype == PA_BF16 ? 2 : 0;
  if (!size) return PA_ERR_DTYPE;
  if (num_tokens < 0 || num_blocks < 1 || num_q_heads < 0 || num_kv_heads < 1 || head_dim < 1 || num_positions < 1)
    return PA_ERR_ARG;
  if (block_size != 16 && block_size != 32) return PA_ERR_BLOCKSIZE;
  if (kv8 ? head_dim != 64 && head_dim != 128 : head_dim * size % 16 != 0 || head_dim > 1024)
    return PA_ERR_UNSUPPORTED;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim || rot_dim > kRopeMaxDim) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !positions || !slot_mapping || !cos_sin || !k_cache || !v_cache || (kv8 && !kv_scales))
    return PA_ERR_ARG;
  if (num_q_heads > 0 && (!q || !q_out)) return PA_ERR_ARG;
  const int64_t kv_row = (int64_t)num_kv_heads * head_dim, q_row = (int64_t)num_q_heads * head_dim;
  if (k_stride < kv_row || v_stride < kv_row || (num_q_heads > 0 && q_stride < q_row)) return PA_ERR_ARG;
  // In place the rows have to be where q's are.
  if (num_q_heads > 0 && q == q_out && q_stride != q_row) return PA_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cos_sin) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (kv8 && !aligned16(kv_scales)) || (num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))))
    return PA_ERR_ALIGN;
  if (k_stride * size % 16 || v_stride * size % 16 || (num_q_heads > 0 && q_stride * size % 16)) return PA_ERR_ALIGN;
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slot_mapping;
  p.table = cos_sin;
  p.num_positions = num_positions;
  p.rot = rot_dim;
  p.num_tokens = num_tokens;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_scales = kv_scales;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  const int vec = 16 / size, half = rot_dim / 2;
  const int layout = interleaved ? kRopePairs : half % vec == 0 ? kRopeHalves : kRopeHalvesOdd;
  p.row_units = layout == kRopePairs    ? head_dim / vec
                : layout == kRopeHalves ? (head_dim - half) / vec
                                        : head_dim - half;
  p.rows = kv8 ? num_q_heads : num_q_heads + 2 * num_kv_heads;
  if (num_q_heads > (1 << 20) || num_kv_heads > (1 << 20)) return PA_ERR_UNSUPPORTED;
  p.pass_rows = std::max(1, kRopeThreads / p.row_units);
  // CTAs of a token: one for each pass over its rows, as long as the machine
  // has room for them all at once (16 an SM); then as few as fill it.
  const int passes = std::max(1, (p.rows + p.pass_rows - 1) / p.pass_rows);
  const int64_t room = 16 * num_sms_current_device();
  p.chunks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(passes, room / num_tokens));
  // Tokens of a warp (8-bit caches): more than one when that leaves each SM 32 warps.
  const int64_t warps = num_tokens * num_kv_heads * 2;
  p.group = (int32_t)std::max<int64_t>(1, std::min<int64_t>(16, warps / (32 * num_sms_current_device())));
  if (num_tokens > (1ll << 30) || num_tokens * num_kv_heads > (1ll << 30)) return PA_ERR_UNSUPPORTED;
  p.cache_ctas = (uint32_t)(((num_tokens + p.group - 1) / p.group * num_kv_heads * 2 + kRopeThreads / 32 - 1) /
                            (kRopeThreads / 32));
  if ((p.status = device_status_ptr()) == nullptr) return PA_ERR_CUDA;
#define PA_ROPE(T)                                                       \
  (layout == kRopePairs    ? launch_rope<T, kRopePairs>(p, kv8, stream)  \
   : layout == kRopeHalves ? launch_rope<T, kRopeHalves>(p, kv8, stream) \
                           : launch_rope<T, kRopeHalvesOdd>(p, kv8, stream))
  return dtype == PA_F32 ? PA_ROPE(float) : dtype == PA_F16 ? PA_ROPE(__half) : PA_ROPE(__nv_bfloat16);
#undef PA_ROPE
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_rope_table(float* cos_sin, int64_t first_position, int64_t num_positions, int32_t rot_dim, double base,
                  int32_t scaling, double factor, int32_t original_len, double low, double high, double amplitude,
                  void* stream) {
  using namespace pa;
  if (first_position < 0 || num_positions < 0 || first_position > INT32_MAX || num_positions > INT32_MAX ||
      first_position + num_positions > (1ll << 31))
    return PA_ERR_ARG;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > kRopeMaxDim) return PA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base) || !(std::fabs(amplitude) <= FLT_MAX)) return PA_ERR_ARG;
  if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_RAMP) return PA_ERR_ARG;
  if (scaling != PA_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor))) return PA_ERR_ARG;
  if ((scaling == PA_ROPE_BANDS || scaling == PA_ROPE_RAMP) &&
      (original_len < 1 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return PA_ERR_ARG;
  const double kTwoPi = 6.283185307179586476925;
  const Twice one{1.0, 0.0}, per_turn{0.15915494309189535, -9.839338337591243e-18};  // 1, 1 / (2 pi)
  const Twice per_factor = scaling == PA_ROPE_NONE ? one : one / Twice{factor, 0.0};
  // (A band narrower than normal numbers is a step.)
  const Twice per_band = one / plus(std::max(high, low + 1e-300), -low), positions{(double)original_len, 0.0};
  const int half = rot_dim / 2;
  Twice ratio = half > 1 ? inverse_root(base, half) : one;  // from a frequency to the next
  if (scaling == PA_ROPE_BASE && half > 1) {
    // base * factor^(half / (half - 1)): factor's part of it is factor^(-1 / (half - 1)).
    if (!(base * std::pow(factor, half / (half - 1.0)) > 0.0)) return PA_ERR_ARG;
    ratio = ratio * inverse_root(factor, half - 1);
  }
  auto pair_of = [&](double turns) {  // the pair that makes so many turns in original_len
    return rot_dim * std::log(original_len / (kTwoPi * turns)) / (2 * std::log(base));
  };
  const double first = std::max(std::floor(pair_of(high)), 0.0),
               last = std::min(std::ceil(pair_of(low)), rot_dim - 1.0);
  const Twice per_pair = one / Twice{std::max(last - first, 0.001), 0.0};
  RopeSteps steps{};
  Twice plain = one;
  for (int i = 0; i < half; ++i, plain = plain * ratio) {
    Twice f = plain;
    if (scaling == PA_ROPE_LINEAR) f = f * per_factor;
    if (scaling >= PA_ROPE_BANDS) {
      // The share of the frequency that the factor divides.
      const Twice share = scaling == PA_ROPE_BANDS
                              ? one - (f * per_turn * positions - Twice{low, 0.0}) * per_band
                              : Twice{i - first, 0.0} * per_pair;
      if ((one - share).hi <= 0.0) f = f * per_factor;
      else if (share.hi > 0.0) f = (one - share) * f + share * f * per_factor;
    }
    if (!std::isfinite(f.hi)) return PA_ERR_ARG;  // (a factor that leaves the doubles' range)
    const Twice turns = f * per_turn;
    steps.step[i] = fraction(turns.hi) + fraction(turns.lo);
  }
  if (num_positions == 0) return PA_OK;
  if (!cos_sin) return PA_ERR_ARG;
  if (!aligned16(cos_sin)) return PA_ERR_ALIGN;
  const int n = half % 4 == 0 ? 4 : 1, rows = kRopeThreads / (half / n);
  // Eight CTAs an SM: a thread reads its steps from the constant bank, one
  // address a lane, which takes as long as several positions do (131072 of 128:
  // 12 us, 13 with 16 CTAs an SM, 14 with 32, 32 with 100).
  const unsigned ctas = (unsigned)std::min<int64_t>((num_positions + rows - 1) / rows, 8 * num_sms_current_device());
  const auto kernel = n == 4 ? rope_table_kernel<4> : rope_table_kernel<1>;
  kernel<<<ctas, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      cos_sin, (uint32_t)first_position, (uint32_t)num_positions, half, (float)amplitude, steps);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping, const float* cos_sin,
                      int32_t num_positions, int32_t rot_dim, int32_t interleaved, int64_t num_tokens, void* q_out,
                      void* k_cache, void* v_cache, int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream) {
  return pa::rope_and_cache(q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, cos_sin, num_positions,
                            rot_dim, interleaved, num_tokens, q_out, k_cache, v_cache, nullptr, num_blocks,
                            block_size, num_q_heads, num_kv_heads, head_dim, dtype, 0,
                            static_cast<cudaStream_t>(stream));
}

int pa_rope_and_cache_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                          const float* cos_sin, int32_t num_positions, int32_t rot_dim, int32_t interleaved,
                          int64_t num_tokens, void* q_out, void* k_cache, void* v_cache, float* kv_scales,
                          int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, pa_dtype dtype, void* stream) {
  return pa::rope_and_cache(q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, cos_sin, num_positions,
                            rot_dim, interleaved, num_tokens, q_out, k_cache, v_cache, kv_scales, num_blocks,
                            block_size, num_q_heads, num_kv_heads, head_dim, dtype, 1 + pa::PA_KV_E4M3,
                            static_cast<cudaStream_t>(stream));
}

int pa_rope_and_cache_e5m2(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                           const float* cos_sin, int32_t num_positions, int32_t rot_dim, int32_t interleaved,
                           int64_t num_tokens, void* q_out, void* k_cache, void* v_cache, float* kv_scales,
                           int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_dim, pa_dtype dtype, void* stream) {
  return pa::rope_and_cache(q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, cos_sin, num_positions,
                            rot_dim, interleaved, num_tokens, q_out, k_cache, v_cache, kv_scales, num_blocks,
                            block_size, num_q_heads, num_kv_heads, head_dim, dtype, 1 + pa::PA_KV_E5M2,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// Rotary positions: the table of cosines and sines, and the rotation of new
// queries and keys with the cache write on the way.
//
// A pair (x1, x2) of a row at position p turns by the angle p f_i:
//   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin.
// Every product, sum and difference is one IEEE fp32 operation (no fused
// multiply-add), so results can be reproduced bit for bit from the table.
#include <algorithm>
#include <cmath>

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

// cos and sin of t / 2^64 turns: the nearest quarter turn is taken out, and
// the rest, at most pi/4, goes through the Taylor polynomials of degree 9 and
// 10 (their next terms are below 2^-28).
__device__ __forceinline__ void turn(unsigned long long t, float& c, float& s) {
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);
  const float x = __ll2float_rn((long long)(t << 2)) * (float)(1.5707963267948966 / 18446744073709551616.0);
  const float y = x * x;
  const float sn =
      x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
  const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
  const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
  c = (quarter + 1) & 2 ? -a : a;
  s = quarter & 2 ? -b : b;
}

__global__ void __launch_bounds__(kRopeThreads) rope_table_kernel(float* __restrict__ out, uint32_t first,
                                                                   int64_t positions, int32_t half, float amplitude,
                                                                   const __grid_constant__ RopeSteps steps) {
  const int64_t total = positions * half;
  for (int64_t x = blockIdx.x * (int64_t)kRopeThreads + threadIdx.x; x < total;
       x += (int64_t)gridDim.x * kRopeThreads) {
    const int64_t p = x / half;
    const int i = (int)(x - p * half);
    float c, s;
    turn((first + (unsigned long long)p) * steps.step[i], c, s);
    float* row = out + p * 2 * half;
    row[i] = c * amplitude;
    row[half + i] = s * amplitude;
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
  int32_t row_units;    // work units of a rotated row
  int32_t token_units;  // work units of a token
  int32_t chunks;       // CTAs of a token
  int64_t q_ctas;       // 8-bit caches: CTAs that rotate queries
  int* status;
};

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Where a token goes: its table row, or nullptr if it is skipped.
__device__ __forceinline__ const float* rope_row(const RopeParams& p, int64_t t, int64_t slot, bool report) {
  if (slot < 0) return nullptr;  // padding
  if (slot >= (int64_t)p.num_blocks * p.block_size) {
    if (report) record_error(p.status, PA_ERR_BLOCK_OOB);
    return nullptr;
  }
  const int32_t pos = p.positions[t];
  if (pos < 0 || pos >= p.num_positions) {
    if (report) record_error(p.status, PA_ERR_SEQLEN);
    return nullptr;
  }
  return p.table + (int64_t)pos * p.rot;
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

enum RopeLayout { kRopePairs, kRopeHalves, kRopeHalvesOdd };

// Source and destination of row `row` of a token: queries first, then keys
// and values.
template <typename T>
__device__ __forceinline__ void rope_ends(const RopeParams& p, int64_t t, int64_t slot, int row, const T*& src,
                                          T*& dst) {
  const int d = p.head_dim;
  if (row < p.num_q_heads) {
    src = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)row * d;
    dst = static_cast<T*>(p.q_out) + (t * p.num_q_heads + row) * d;
    return;
  }
  const bool is_v = row >= p.num_q_heads + p.num_kv_heads;
  const int h = row - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
  const int64_t blk = slot / p.block_size;
  const int off = (int)(slot - blk * p.block_size);
  const int64_t to = ((blk * p.num_kv_heads + h) * p.block_size + off) * d;
  src = static_cast<const T*>(is_v ? p.v : p.k) + t * (is_v ? p.v_stride : p.k_stride) + (int64_t)h * d;
  dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + to;
}

// One thread per unit of a token: with halves a vector of each half or a
// vector that stays, with pairs a vector of pairs; a vector of a value row.
// (kRopeHalvesOdd, a half that is no whole number of vectors: an element of
// each half, or one that stays.) Rows are read once and written once; a
// query may be rotated in place, because the thread that writes an element is
// the one that reads it.
template <typename T, int LAYOUT>
__device__ __forceinline__ void rope_unit(const RopeParams& p, int64_t t, int unit) {
  constexpr int N = Vec16<T>::N;
  const int64_t slot = p.slots[t];
  const float* cs = rope_row(p, t, slot, unit == 0);
  if (!cs) return;
  const int half = p.rot >> 1, rotated = (p.num_q_heads + p.num_kv_heads) * p.row_units;
  const T* src;
  T* dst;
  if (unit >= rotated) {
    const int u = unit - rotated, per = p.head_dim / N, row = u / per;
    rope_ends(p, t, slot, p.num_q_heads + p.num_kv_heads + row, src, dst);
    Vec16<T> x;
    x.load(src + (u - row * per) * N);
    x.store(dst + (u - row * per) * N);
    return;
  }
  const int row = unit / p.row_units, u = unit - row * p.row_units;
  rope_ends(p, t, slot, row, src, dst);
  if constexpr (LAYOUT == kRopePairs) {
    const int d = u * N;
    Vec16<T> x;
    x.load(src + d);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if (d + i < p.rot) {
        float a = to_f32(x.e[i]), b = to_f32(x.e[i + 1]);
        rotate(a, b, cs[(d + i) >> 1], cs[half + ((d + i) >> 1)]);
        x.e[i] = from_f32<T>(a);
        x.e[i + 1] = from_f32<T>(b);
      }
    }
    x.store(dst + d);
  } else if constexpr (LAYOUT == kRopeHalves) {
    const int d = u * N;
    Vec16<T> x, y;
    if (d >= half) {  // behind the rotated part
      x.load(src + half + d);
      x.store(dst + half + d);
      return;
    }
    x.load(src + d);
    y.load(src + half + d);
    float c[N], s[N];
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + d + i);
      *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + half + d + i);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float a = to_f32(x.e[i]), b = to_f32(y.e[i]);
      rotate(a, b, c[i], s[i]);
      x.e[i] = from_f32<T>(a);
      y.e[i] = from_f32<T>(b);
    }
    x.store(dst + d);
    y.store(dst + half + d);
  } else {
    if (u >= half) {
      dst[half + u] = src[half + u];
      return;
    }
    float a = to_f32(src[u]), b = to_f32(src[half + u]);
    rotate(a, b, cs[u], cs[half + u]);
    dst[u] = from_f32<T>(a);
    dst[half + u] = from_f32<T>(b);
  }
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const int64_t t = blockIdx.x / p.chunks;
  const int unit = (int)(blockIdx.x - t * p.chunks) * kRopeThreads + threadIdx.x;
  if (unit < p.token_units) rope_unit<T, LAYOUT>(p, t, unit);
}

// ---------------------------------------------------------------------------
// 8-bit caches. The queries' units as above; keys and values as
// pa_reshape_and_cache_fp8 writes them, a warp per (run of tokens in one
// block, KV head, pool), the keys rotated in fp32 and encoded from there (one
// rounding, not two).
// ---------------------------------------------------------------------------

// Elements d .. d + VEC - 1 of a row, rotated if cs is given. `whole`: the
// halves are whole numbers of vectors.
template <typename T, int VEC>
__device__ __forceinline__ void rope_values(const T* row, const float* cs, int d, int rot, bool inter, bool whole,
                                            float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = to_f32(row[d + i]);
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
    const int lo = upper ? d - half : d, other = upper ? d - half : d + half;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float a = x[i], b = to_f32(row[other + i]);
      if (upper) {
        rotate(b, a, cs[lo + i], cs[half + lo + i]);
      } else {
        rotate(a, b, cs[lo + i], cs[half + lo + i]);
      }
      x[i] = a;
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

template <typename T, int VEC, bool E5>
__device__ __forceinline__ void rope_cache_8bit(const RopeParams& p, bool inter, int64_t w) {
  constexpr int D = VEC * 32;
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, hkv = p.num_kv_heads, bs = p.block_size;
  const int64_t cap = (int64_t)p.num_blocks * bs;
  const int64_t t = w / (hkv * 2);
  const int rem = (int)(w - t * hkv * 2), h = rem >> 1, pool = rem & 1;
  // A token counts if it has a place and a position (those that have not are
  // skipped as padding is).
  auto place = [&](int64_t j) -> int64_t {
    if (j < 0 || j >= p.num_tokens) return -1;
    const int64_t s = p.slots[j];
    if (s < 0 || s >= cap) return -1;
    const int32_t pos = p.positions[j];
    return pos >= 0 && pos < p.num_positions ? s : -1;
  };
  const int64_t slot = place(t);
  if (slot < 0) {
    if (lane == 0 && rem == 0) rope_row(p, t, p.slots[t], true);
    return;
  }
  const int64_t blk = slot / bs;
  // The first token of a run leads: the nearest one before it that counts
  // lies in another block.
  for (int64_t base = t - 1; base >= 0; base -= 32) {
    const int64_t sj = place(base - lane);
    const unsigned ok = __ballot_sync(kFull, sj >= 0);
    if (ok) {
      const int64_t near = __shfl_sync(kFull, sj, __ffs(ok) - 1);  // lowest lane = latest token
      if (near / bs == blk) return;
      break;
    }
  }
  const T* src = static_cast<const T*>(pool == 0 ? p.k : p.v) + h * D;
  const int64_t stride = pool == 0 ? p.k_stride : p.v_stride;
  const bool whole = (p.rot >> 1) % VEC == 0;
  uint8_t* codes =
      static_cast<uint8_t*>(pool == 0 ? p.k_cache : p.v_cache) + (blk * hkv + h) * (int64_t)bs * D + lane * VEC;
  auto values = [&](int64_t j, float (&x)[VEC]) {
    const float* cs = pool == 0 ? p.table + (int64_t)p.positions[j] * p.rot : nullptr;
    rope_values<T, VEC>(src + j * stride, cs, lane * VEC, p.rot, inter, whole, x);
  };
  // The run's rows: their largest value, the lowest offset, one past the end.
  float amax = 0.f;
  int omin = bs;
  int64_t end = p.num_tokens;
  for (int64_t base = t; base < p.num_tokens; base += 32) {
    const int64_t sj = place(base + lane);
    const unsigned other = __ballot_sync(kFull, sj >= 0 && sj / bs != blk);
    const int lim = other ? __ffs(other) - 1 : 32;
    unsigned mem = __ballot_sync(kFull, sj >= 0 && lane < lim);
    while (mem) {
      const int ln = __ffs(mem) - 1;
      mem &= mem - 1;
      const int64_t sm = __shfl_sync(kFull, sj, ln);
      omin = min(omin, (int)(sm - blk * bs));
      float x[VEC];
      values(base + ln, x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[i]));
    }
    if (other) {
      end = base + lim;
      break;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, off));
  float* sp = p.kv_scales + (blk * hkv + h) * 2 + pool;
  const float s_old = omin == 0 ? 0.f : *sp;
  const float s_new = fmaxf(s_old, __fdiv_rn(amax, E5 ? 57344.f : 448.f));
  if (s_new > s_old && s_old > 0.f) {
    const float r = __fdiv_rn(s_old, s_new);
    for (int o = 0; o < omin; ++o) {
      float x[VEC];
      load_codes<VEC, E5>(codes + o * D, x);
      uint32_t c[VEC / 2];
#pragma unroll
      for (int i = 0; i < VEC; i += 2) c[i / 2] = f32x2_to_fp8x2<E5>(__fmul_rn(x[i], r), __fmul_rn(x[i + 1], r));
      store_codes<VEC>(codes + o * D, c);
    }
  }
  for (int64_t base = t; base < end; base += 32) {
    const int64_t sj = base + lane < end ? place(base + lane) : -1;
    unsigned mem = __ballot_sync(kFull, sj >= 0);
    while (mem) {
      const int ln = __ffs(mem) - 1;
      mem &= mem - 1;
      const int64_t sm = __shfl_sync(kFull, sj, ln);
      float x[VEC];
      values(base + ln, x);
      uint32_t c[VEC / 2];
#pragma unroll
      for (int i = 0; i < VEC; i += 2)
        c[i / 2] = s_new > 0.f ? f32x2_to_fp8x2<E5>(__fdiv_rn(x[i], s_new), __fdiv_rn(x[i + 1], s_new)) : 0u;
      store_codes<VEC>(codes + (sm - blk * bs) * D, c);
    }
  }
  if (lane == 0) *sp = s_new;
}

template <typename T, int VEC, bool E5, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_8bit_kernel(const __grid_constant__ RopeParams p) {
  if (blockIdx.x >= p.q_ctas) {
    const int64_t w = (blockIdx.x - p.q_ctas) * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (w < p.num_tokens * p.num_kv_heads * 2) rope_cache_8bit<T, VEC, E5>(p, LAYOUT == kRopePairs, w);
    return;
  }
  const int64_t t = blockIdx.x / p.chunks;
  const int unit = (int)(blockIdx.x - t * p.chunks) * kRopeThreads + threadIdx.x;
  if (unit < p.num_q_heads * p.row_units) rope_unit<T, LAYOUT>(p, t, unit);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int LAYOUT>
int launch_rope(const RopeParams& p, int kv8, cudaStream_t stream) {
  if (!kv8) {
    rope_kernel<T, LAYOUT><<<(unsigned)(p.num_tokens * p.chunks), kRopeThreads, 0, stream>>>(p);
  } else {
    const int64_t warps = p.num_tokens * p.num_kv_heads * 2;
    const unsigned ctas = (unsigned)(p.q_ctas + (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
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
  p.row_units = layout == kRopePairs ? head_dim / vec
                : layout == kRopeHalves ? (head_dim - half) / vec
                                        : head_dim - half;
  const int64_t units = kv8 ? (int64_t)num_q_heads * p.row_units
                            : (int64_t)(num_q_heads + num_kv_heads) * p.row_units + kv_row / vec;
  if (units > (1 << 24)) return PA_ERR_UNSUPPORTED;
  p.token_units = (int32_t)units;
  p.chunks = std::max<int32_t>(1, (p.token_units + kRopeThreads - 1) / kRopeThreads);
  p.q_ctas = num_q_heads > 0 ? num_tokens * p.chunks : 0;
  if (num_tokens > (1ll << 31) / p.chunks - 1 || num_tokens * num_kv_heads > (1ll << 30)) return PA_ERR_UNSUPPORTED;
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
  if (!(base > 1.0) || !std::isfinite(base) || !std::isfinite(amplitude)) return PA_ERR_ARG;
  if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_RAMP) return PA_ERR_ARG;
  if (scaling != PA_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor))) return PA_ERR_ARG;
  if ((scaling == PA_ROPE_BANDS || scaling == PA_ROPE_RAMP) &&
      (original_len < 1 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return PA_ERR_ARG;
  if (num_positions == 0) return PA_OK;
  if (!cos_sin) return PA_ERR_ARG;
  if (!aligned16(cos_sin)) return PA_ERR_ALIGN;
  const double kTwoPi = 6.283185307179586476925;
  const int half = rot_dim / 2;
  if (scaling == PA_ROPE_BASE && rot_dim > 2) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  auto pair_of = [&](double turns) {  // the pair that makes so many turns in original_len
    return rot_dim * std::log(original_len / (kTwoPi * turns)) / (2 * std::log(base));
  };
  const double first = std::max(std::floor(pair_of(high)), 0.0),
               last = std::min(std::ceil(pair_of(low)), rot_dim - 1.0);
  RopeSteps steps{};
  for (int i = 0; i < half; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim), stretched = 0.0;
    if (scaling == PA_ROPE_LINEAR) f /= factor;
    if (scaling == PA_ROPE_BANDS)
      stretched = 1.0 - std::min(1.0, std::max(0.0, (original_len * f / kTwoPi - low) / (high - low)));
    if (scaling == PA_ROPE_RAMP)
      stretched = std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 0.001)));
    f = (1.0 - stretched) * f + stretched * f / factor;
    double turns = f / kTwoPi;
    turns -= std::floor(turns);
    steps.step[i] = turns >= 1.0 ? 0 : (unsigned long long)(turns * 18446744073709551616.0);
  }
  const int64_t total = num_positions * half;
  const int64_t ctas = std::min<int64_t>((total + kRopeThreads - 1) / kRopeThreads, 1 << 24);
  rope_table_kernel<<<(unsigned)ctas, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      cos_sin, (uint32_t)first_position, num_positions, half, (float)amplitude, steps);
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

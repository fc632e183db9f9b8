// 8-bit cache codes (e4m3, or e5m2 with E5) to and from fp32, for the kernels
// that write an 8-bit cache. Each conversion is one rounding to nearest even,
// saturating, so codes are reproducible bit for bit.
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_c(uint16_t c) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}

__device__ __forceinline__ uint32_t e5m2x2_to_f16x2_c(uint16_t c) {
  uint32_t d;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}

// Two floats to two 8-bit codes (e4m3, or e5m2 with E5): lo in the low byte.
template <bool E5>
__device__ __forceinline__ uint32_t f32x2_to_fp8x2(float lo, float hi) {
  uint16_t r;
  if constexpr (E5)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint32_t (&c)[VEC / 2]) {
  if constexpr (VEC == 2) {
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(c[0]);
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint32_t*>(dst) = c[0] | (c[1] << 16);
  }
}

template <int VEC, bool E5>
__device__ __forceinline__ void load_codes(const uint8_t* src, float (&x)[VEC]) {
  uint32_t w;
  if constexpr (VEC == 2) w = *reinterpret_cast<const uint16_t*>(src);
  else w = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
  for (int i = 0; i < VEC; i += 2) {
    const uint16_t c2 = static_cast<uint16_t>(w >> (8 * i));
    const uint32_t h2 = E5 ? e5m2x2_to_f16x2_c(c2) : e4m3x2_to_f16x2_c(c2);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    x[i] = f.x;
    x[i + 1] = f.y;
  }
}

}  // namespace pa

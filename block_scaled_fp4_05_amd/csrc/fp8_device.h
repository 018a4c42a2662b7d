// Device-side helpers for FP8 (E4M3) operands in blocks of 128 with FP32 scales.
//
// Element format E4M3 (OCP OFP8 v1.0, no infinity, 0x7F / 0xFF are NaN).  A block of 128
// consecutive elements of a row (activations) or of 128 x 128 (weights) has one FP32 scale
// s; an element stands for its E4M3 value times s.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_device.h"

namespace moe_fp4 {

constexpr int kFp8Block = 128;
constexpr float kE4m3Max = 448.0f;

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// The scale of a block whose largest magnitude is amax: amax / 448 (an IEEE division), at
// least 2^-126, so that it is never zero or subnormal; rounded up to a power of two on
// request.  An infinite amax keeps an infinite scale.
__device__ __forceinline__ float fp8_scale(float amax, bool pow2) {
  float s = fmaxf(amax, kE4m3Max * 0x1p-126f) / kE4m3Max;
  if (pow2) {
    const uint32_t u = __builtin_bit_cast(uint32_t, s);
    s = __builtin_bit_cast(float, (u + 0x7FFFFFu) & 0xFF800000u);
  }
  return s;
}

// x / s, rounded once.  rs = RN(1/s).  q = RN(x rs) is corrected with the residual x - q s,
// Markstein's correction, which gives RN(x / s) while the residual is exact: its last bit is
// about 2^-48 of x, above 2^-149 for every quotient that is not below half the smallest E4M3
// magnitude (2^-10) when s >= 2^-91.  Smaller s, and infinite ones, divide.
// The sign of a zero is x's.
__device__ __forceinline__ float fp8_quotient(float x, float s, float rs) {
  const float q = x * rs;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), rs, q), x);
}

__device__ __forceinline__ bool fp8_fast(float s) { return s >= 0x1p-91f && s <= 0x1p120f; }

// Eight values over their scale as E4M3 codes (nearest even; |x / s| is at most 448 up to
// rounding; NaN stays NaN).
__device__ __forceinline__ u32x2_t fp8_encode8(const float (&v)[8], float s) {
  float y[8];
  if (fp8_fast(s)) {
    const float rs = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fp8_quotient(v[i], s, rs);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] / s;
  }
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], w, true);
    c[h] = (uint32_t)w;
  }
  return u32x2_t{c[0], c[1]};
}

}  // namespace moe_fp4

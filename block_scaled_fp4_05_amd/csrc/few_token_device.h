// Device pieces of the few-token products (linear.hip, ffn.hip): 16-bit rows times
// NVFP4 weights, on the 16 x 16 x 32 matrix instruction.
//
// The weights are the A operand (16 weight rows), the tokens the B operand (up to
// 16 columns), so lane l holds weight row l % 16 and token l % 16, both at the K
// slice of lane group g = l / 16, and the result's four values are four
// consecutive weight rows of one token.  The order of K inside a product is free
// as long as both operands agree: a wavefront takes 256 elements of K per step
// and lane group g the 64 consecutive ones at 64 g, so that a lane's codes are two
// 16-byte loads, its four block scales one dword and its activations eight
// 16-byte loads, and the four lanes of a row read 128 consecutive bytes.
//
// Any K that is a multiple of 16 and at least 64 runs without a narrow path: a
// lane whose 64 elements would pass the end of the row reads the row's last 64
// instead and drops the blocks that other lanes own (scale and activations 0).
#pragma once

#include "fp4_device.h"
#include "gemm_common.h"

namespace moe_fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kFewStep = 256;  // elements of K per wavefront step
constexpr int kFewRows = 16;   // weight rows, and tokens, of one matrix product

// Eight codes (one dword) times one block scale as eight exact 16-bit values: the
// product has at most 6 significant bits and lies in [2^-10, 2688], inside both
// types' normal range.  A NaN scale stays NaN.  FP16: packed multiply.  BF16 has
// no packed multiply on gfx950, so the product is taken in FP32 and its upper half
// kept (exact, the lower half being zero).
template <bool F16>
__device__ __forceinline__ u32x4_t dequant8_16bit(uint32_t codes, float scale) {
  if (F16) {
    const _Float16 h = (_Float16)scale;
    const half2_t s2 = {h, h};
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s2;
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s2;
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s2;
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s2;
    return u32x4_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                   __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
  }
  auto pair = [&](auto v) {
    const float lo = v[0] * scale, hi = v[1] * scale;
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo),
                                 0x07060302u);
  };
  return u32x4_t{pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3))};
}

template <bool F16>
__device__ __forceinline__ float4_t mfma16(u32x4_t a, u32x4_t b, float4_t c) {
  if (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Where a lane's 64 elements of a step start, and how many of their four blocks
// (the first ones) belong to other lanes.
struct LaneK {
  int32_t k;
  int32_t skip;  // 0..4
};

__device__ __forceinline__ LaneK lane_k(int32_t step, int32_t g, int32_t k) {
  const int32_t k0 = step * kFewStep + 64 * g;
  const int32_t last = k - 64;
  LaneK r;
  r.k = k0 < last ? k0 : last;
  const int32_t over = (k0 - r.k) >> 4;
  r.skip = over < 4 ? over : 4;
  return r;
}

// One step of NT x 16 weight rows in registers.
template <int NT>
struct WeightStep {
  u32x4_t q[NT][2];
  uint32_t s[NT];
};

template <int NT>
__device__ __forceinline__ void load_weights(WeightStep<NT>& w, rsrc_t q_rs, rsrc_t s_rs,
                                             const uint32_t (&row)[NT], int32_t k, int32_t kk) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t off = row[t] * (uint32_t)(k / 2) + (uint32_t)(kk / 2);
    w.q[t][0] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, off, 0, kLoadStreamOnce);
    w.q[t][1] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, off + 16u, 0, kLoadStreamOnce);
    w.s[t] = __builtin_amdgcn_raw_buffer_load_b32(
        s_rs, row[t] * (uint32_t)(k / 16) + (uint32_t)(kk / 16), 0, 0);
  }
}

template <int NT>
__device__ __forceinline__ void drop_scales(WeightStep<NT>& w, int32_t skip) {
  const uint32_t keep = skip >= 4 ? 0u : 0xFFFFFFFFu << (8 * skip);
#pragma unroll
  for (int t = 0; t < NT; ++t) w.s[t] &= keep;
}

// Block scale J (0..3) of a lane's dword.
template <int J>
__device__ __forceinline__ float block_scale(uint32_t s) {
  return __builtin_amdgcn_cvt_f32_fp8((int)s, J);
}

// Eight matrix products of a step: operand j covers elements 8j .. 8j+7 of each
// lane's 64.  f(j, t, a): consume weight operand a of tile t.
template <bool F16, int NT, int J, typename F>
__device__ __forceinline__ void for_operands(const WeightStep<NT>& w, F&& f) {
  if constexpr (J < 8) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t codes = w.q[t][J / 4][J % 4];
      f(J, t, dequant8_16bit<F16>(codes, block_scale<J / 2>(w.s[t])));
    }
    for_operands<F16, NT, J + 1>(w, f);
  }
}

__device__ __forceinline__ float bf16_value(uint16_t b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// A 16-bit input element as FP32.
template <bool F16>
__device__ __forceinline__ float value16(uint16_t b) {
  return F16 ? (float)__builtin_bit_cast(_Float16, b) : bf16_value(b);
}

// Store one result in the output's type (rounded to nearest even).
__device__ __forceinline__ void store_as(void* out, int64_t i, float v, int32_t dtype) {
  if (dtype == kFewOutF32)
    static_cast<float*>(out)[i] = v;
  else if (dtype == kFewOutF16)
    static_cast<_Float16*>(out)[i] = (_Float16)v;
  else
    static_cast<__bf16*>(out)[i] = (__bf16)v;
}

// x / (1 + e^-x): exactly 0 or the identity where e^-x overflows or vanishes.
__device__ __forceinline__ float silu(float x) { return x / (1.0f + __expf(-x)); }

// The running sums of NT x 16 weight rows times MT x 16 tokens over a wavefront's
// steps [s0, s1), s0 < s1.  Token t's row starts at byte xoff[t] of x (kOutOfRange:
// no token, reads as zeros); groups (<= MT) of 16 tokens hold any.
// The loads of the next step are in flight while a step is computed; the loop is
// unrolled by two so that both steps keep their registers.
template <bool F16, int NT, int MT>
struct FewLoop {
  struct Regs {
    WeightStep<NT> w;
    u32x4_t x[MT][8];
  };

  rsrc_t q_rs, s_rs, x_rs;
  int32_t k, g;

  __device__ __forceinline__ void load(Regs& r, const uint32_t (&row)[NT],
                                       const uint32_t (&xoff)[MT], int32_t step) const {
    const LaneK lk = lane_k(step, g, k);
    load_weights<NT>(r.w, q_rs, s_rs, row, k, lk.k);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        r.x[m][j] = __builtin_amdgcn_raw_buffer_load_b128(
            x_rs, xoff[m] + (uint32_t)(2 * lk.k + 16 * j), 0, 0);
  }

  __device__ __forceinline__ void compute(Regs& r, float4_t (&acc)[NT][MT], int32_t step) const {
    if ((step + 1) * kFewStep > k) {  // uniform: only a row's last step
      const LaneK lk = lane_k(step, g, k);
      drop_scales<NT>(r.w, lk.skip);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < 2 * lk.skip) r.x[m][j] = u32x4_t{0, 0, 0, 0};
    }
    for_operands<F16, NT, 0>(r.w, [&](int j, int t, u32x4_t a) {
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[t][m] = mfma16<F16>(a, r.x[m][j], acc[t][m]);
    });
  }

  __device__ __forceinline__ void run(const uint32_t (&row)[NT], const uint32_t (&xoff)[MT],
                                      float4_t (&acc)[NT][MT], int32_t s0, int32_t s1) const {
    Regs a, b;
    load(a, row, xoff, s0);
    int32_t s = s0;
    for (; s + 2 < s1; s += 2) {
      load(b, row, xoff, s + 1);
      compute(a, acc, s);
      load(a, row, xoff, s + 2);
      compute(b, acc, s + 1);
    }
    if (s + 1 < s1) {
      load(b, row, xoff, s + 1);
      compute(a, acc, s);
      compute(b, acc, s + 1);
    } else {
      compute(a, acc, s);
    }
  }
};

// Leave a wavefront's sums in LDS: red[wave][tile][lane], four values each.
template <int NT, int MT>
__device__ __forceinline__ void put_sums(float4_t* red, const float4_t (&acc)[NT][MT], int wave,
                                         int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[((wave * NT + t) * MT + m) * 64 + lane] = acc[t][m];
}

// The sum over the wavefronts, in wavefront order, of one lane's values of a tile.
__device__ __forceinline__ float4_t take_sum(const float4_t* red, int tiles, int tile, int lane,
                                             int waves) {
  float4_t v = red[tile * 64 + lane];
  for (int w = 1; w < waves; ++w) v += red[(w * tiles + tile) * 64 + lane];
  return v;
}

}  // namespace moe_fp4

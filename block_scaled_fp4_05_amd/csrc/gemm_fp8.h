// What the FP8 block-scaled products (gemm_fp8.hip, gemm_fp8_tiled.hip) share: where a
// workgroup works, and how a result is stored.
//
// Products of two 16-row operands over one block of 128, which the block's two scales then
// multiply: acc += d * (sa * sw), one multiply-add an element (rows whose sa * sw is no normal
// number go another way, fp8_add_far).  Weights are the first operand:
// lane l of the result then holds activation row l % 16, whose scale is one value a lane, and
// weight rows 4 (l / 16) .. +3; the weight scale is uniform, since 16 rows at a multiple of
// 16 lie in one block of 128.  Lane l gives 32 bytes of row l % 16 of each operand; which 32
// of the 128 does not matter as long as both operands agree: the 16-byte pieces l / 16 and
// 4 + l / 16.
//
// Two ways.  The FP8 matrix cores take the bytes as they are, at twice the rate of the
// FP16 ones, but not their sums: of eight consecutive products the smaller ones are cut
// off 13 bits below the leading bit of the largest (measured bit by bit; groups of eight meet in
// FP32).  On Gaussian data a result is off by 1.5e-5 of itself, far below the rounding to 16
// bits (2^-9 or 2^-12 of it), so the compute-bound tiles use them for 16-bit results; at worst,
// where one product of every eight outweighs the rest, they lose 7 x 2^-13 of the sum of
// those, less than BF16's half step and three and a half of FP16's.  An FP32
// result, and every result of the few-row kernel, whose time is the weight stream, is computed on
// the FP16 cores from exactly converted operands, good to FP32's own roundings: which of the two a
// 16-bit result takes goes by the launch rules, so by the other rows of its call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_token_device.h"
#include "fp8_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {

__device__ __forceinline__ float4_t fp8_block_product(const i32x8_t& w, const i32x8_t& a) {
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// A lane's 32 bytes as FP16 values (exact: E4M3 is 2^-9 to 448 with four significant bits).
struct Half32 {
  half8_t v[4];
};

__device__ __forceinline__ Half32 fp8_widen(const i32x8_t& x) {
  Half32 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i], 1.0f, false);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i], 1.0f, true);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i + 1], 1.0f, false);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i + 1], 1.0f, true);
    h.v[i] = half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  return h;
}

__device__ __forceinline__ float4_t fp8_block_product(const Half32& w, const Half32& a) {
  float4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[i], a.v[i], d, 0, 0, 0);
  return d;
}

// What the matrix cores are given.
template <bool EXACT>
struct Operand {
  typedef i32x8_t type;
  static __device__ __forceinline__ const i32x8_t& of(const i32x8_t& x) { return x; }
};
template <>
struct Operand<true> {
  typedef Half32 type;
  static __device__ __forceinline__ Half32 of(const i32x8_t& x) { return fp8_widen(x); }
};

// Where sa * sw is no normal FP32 number the result may be one all the same (blocks whose largest
// magnitudes are near 2^-60 have scales near 2^-69 each).  Such "far" rows of a stage are added
// apart, the scales' exponents with the block's products and only their mantissas multiplied, and
// the usual way multiplies them with 0.  (For all rows it would make 8192^3 3% slower, 4096
// tokens of 256 experts with an FP32 result 11%; a stage without far rows is checked for
// them and no more.)

// A scale as m 2^(e - 127): 1 <= |m| < 2 and 1 <= e <= 254, but for zeros, subnormal numbers,
// infinities and NaN, which m keeps.
struct Fp8Scale {
  float m;
  int32_t e;
};

__device__ __forceinline__ Fp8Scale fp8_split(float s) {
  const uint32_t field = __builtin_bit_cast(uint32_t, s) >> 23 & 255u;
  const int32_t e = (int32_t)min(max(field, 1u), 254u);
  return Fp8Scale{__builtin_amdgcn_ldexpf(s, 127 - e), e};
}

__device__ __forceinline__ bool fp8_far(float scale) { return !__builtin_amdgcn_classf(scale, 0x108); }  // -, + normal

// 2^(ea + ew - 254) times the block's products.  (The FP8 instruction takes an exponent for each row
// of both operands, one for 32 elements, here all four of a row alike.)
__device__ __forceinline__ float4_t fp8_far_product(const i32x8_t& w, const i32x8_t& a, int32_t ew, int32_t ea) {
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, ew, 0, ea);
}
__device__ __forceinline__ float4_t fp8_far_product(const Half32& w, const Half32& a, int32_t ew, int32_t ea) {
  float4_t d = fp8_block_product(w, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_ldexpf(d[i], ea + ew - 254);
  return d;
}

// Whether one of the 32 codes is not a zero.
__device__ __forceinline__ bool fp8_any(const i32x8_t& x) {
  int bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bits |= x[i];
  return (bits & 0x7F7F7F7F) != 0;
}

// Adds a stage's far rows; scale: sa * sw, weights(t): the lane's 32 bytes of tile t.  Blocks of
// zeros, whose scale is the least there is, and scales of zero give nothing and are passed over.
// (No branch by lane: the matrix cores write the results of all lanes.)
template <int NT, int MT, bool EXACT, bool PASS_ZEROS, typename W>
__device__ __forceinline__ void fp8_add_far(float4_t (&acc)[NT][MT], const i32x8_t (&a)[MT], const float (&sa)[MT], float sw,
                                            const float (&scale)[MT], W weights) {
  bool small = false, large = false;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const bool far = fp8_far(scale[m]), below = fabsf(scale[m]) < 1.0f;
    small |= far && below && sa[m] != 0.0f && sw != 0.0f && fp8_any(a[m]);
    large |= far && !below;
  }
  const bool some_large = __builtin_amdgcn_ballot_w64(large) != 0;
  if (!some_large && __builtin_amdgcn_ballot_w64(small) == 0) return;
  const Fp8Scale by_w = fp8_split(sw);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const i32x8_t codes = weights(t);
    if (PASS_ZEROS && !some_large && __builtin_amdgcn_ballot_w64(fp8_any(codes)) == 0) continue;
    const auto w = Operand<EXACT>::of(codes);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const Fp8Scale by_a = fp8_far(scale[m]) ? fp8_split(sa[m]) : Fp8Scale{0.0f, 1};  // (keeps d finite)
      const float4_t d = fp8_far_product(w, Operand<EXACT>::of(a[m]), by_w.e, by_a.e);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][m][i] = __builtin_fmaf(d[i], by_a.m * by_w.m, acc[t][m][i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// 0 instead of the scales of far rows.
template <int MT>
__device__ __forceinline__ void fp8_drop_far(float (&scale)[MT]) {
#pragma unroll
  for (int m = 0; m < MT; ++m) scale[m] = fp8_far(scale[m]) ? 0.0f : scale[m];
}

// Whether the wavefront has far rows.
template <int MT>
__device__ __forceinline__ bool fp8_some_far(const float (&scale)[MT]) {
  bool far = false;
#pragma unroll
  for (int m = 0; m < MT; ++m) far |= fp8_far(scale[m]);
  return __builtin_expect(__builtin_amdgcn_ballot_w64(far) != 0, 0);
}

// Where a workgroup works (uniform).
struct Fp8Item {
  int32_t e;     // expert
  int32_t row0;  // first result row
  int32_t rows;  // valid rows of the tile
  int32_t n0;    // first result column
  int32_t once;  // whether these are all rows of the expert, so that its weights are read once
};

// Items of an expert of cnt rows (none for a decreasing pair of offsets).
__device__ __forceinline__ int32_t fp8_items(const Fp8GemmArgs& p, int32_t cnt, int32_t bm) {
  return cnt > 0 ? (cnt + bm - 1) / bm * p.n_tiles : 0;
}

// At most so many items of tiles of bm rows: every expert has at most one that is not full.
inline int64_t fp8_most_items(const Fp8GemmArgs& p, int64_t bm) {
  const int64_t most = p.offsets ? p.m_total / bm + (p.m_total < p.experts ? p.m_total : p.experts)
                                 : (p.m_total + bm - 1) / bm;
  return most * p.n_tiles;
}

// A workgroup's item, one of no rows if it has none.  Every thread counts the items of a run of
// experts; the one whose run holds the item names it.  Items are numbered so that an XCD
// (workgroup b runs on b % 8) gets consecutive ones, which share weight tiles (M-tiles first) or
// activation rows.  band: M-tiles that are walked together with all N-tiles.  Every thread of the
// workgroup calls it (barriers inside), on a grid of at least as many workgroups as there can be
// items, a multiple of 8.  (Offsets that go back and forth can make more: those are left out.)
template <int NTHR>
__device__ __forceinline__ Fp8Item fp8_item(const Fp8GemmArgs& p, int32_t bm, int32_t bn, int32_t band) {
  constexpr int WAVES = NTHR / 64;
  __shared__ int32_t sums[WAVES];
  __shared__ Fp8Item place;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t m_total = (int32_t)p.m_total;
  if (tid == 0) place = Fp8Item{};
  int32_t lo = tid, hi = tid == 0 ? 1 : tid;  // this thread's experts
  int32_t start = 0, second = m_total;        // first rows of its first expert and of the next
  int32_t run = 0;                            // the items before them
  int32_t total = fp8_items(p, m_total, bm);
  if (p.offsets) {
    const int32_t E = p.experts, per = (E + NTHR - 1) / NTHR;
    lo = min(tid * per, E);
    hi = min(lo + per, E);
    const int32_t first = p.offsets[lo], next0 = p.offsets[min(lo + 1, E)];  // (both on their way at once)
    start = clamp_off(first, m_total);
    second = clamp_off(next0, m_total);
    int32_t own = lo < hi ? fp8_items(p, second - start, bm) : 0;
    int32_t at = second;
    for (int32_t e = lo + 1; e < hi; ++e) {
      const int32_t next = clamp_off(p.offsets[e + 1], m_total);
      own += fp8_items(p, next - at, bm);
      at = next;
    }
    int32_t incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t t = __shfl_up(incl, d, 64);
      if (lane >= d) incl += t;
    }
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) run += sums[w];
      total += sums[w];
    }
    run += incl - own;
    total = uniform(total);
  }
  // (Two axes, since one holds fewer than 2^32 threads.)
  const int32_t blocks = gridDim.x * gridDim.y;
  const int32_t item = logical_block(blockIdx.y * gridDim.x + blockIdx.x, blocks, total);
  if (item >= total) return Fp8Item{};
  for (int32_t e = lo, at = start; e < hi; ++e) {
    const int32_t next = e == lo ? second : clamp_off(p.offsets[e + 1], m_total);
    const int32_t rows = next - at, local = item - run, items = fp8_items(p, rows, bm);
    if (local >= 0 && local < items) {
      const int32_t mts = (rows + bm - 1) / bm;
      int32_t mt, nt;
      if (mts <= band) {
        nt = local / mts;
        mt = local - nt * mts;
      } else {
        const int32_t per_band = band * p.n_tiles, b = local / per_band, within = local - b * per_band;
        const int32_t tall = min(band, mts - b * band);
        nt = within / tall;
        mt = b * band + within - nt * tall;
      }
      place = Fp8Item{e, at + mt * bm, min(bm, rows - mt * bm), nt * bn, mts == 1};
    }
    run += items;
    at = next;
  }
  __syncthreads();
  return Fp8Item{uniform(place.e), uniform(place.row0), uniform(place.rows), uniform(place.n0), uniform(place.once)};
}

// Four consecutive columns of a result row, rounded to nearest even.
__device__ __forceinline__ void fp8_store4(const Fp8GemmArgs& p, int64_t row, int32_t col, const float4_t& v) {
  const int64_t at = row * p.ldo + col;
  if (p.vec4 && col + 4 <= p.n) {
    if (p.out_dtype == kFewOutF32) {
      *reinterpret_cast<float4_t*>(static_cast<float*>(p.out) + at) = v;
    } else if (p.out_dtype == kFewOutF16) {
      typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
      *reinterpret_cast<half4_t*>(static_cast<_Float16*>(p.out) + at) =
          half4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    } else {
      typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4_t*>(static_cast<__bf16*>(p.out) + at) =
          bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < p.n) store_as(p.out, at + i, v[i], p.out_dtype);
}

// Eight consecutive results as 16-bit values, rounded to nearest even.
__device__ __forceinline__ u32x4_t fp8_round8(const float4_t& lo, const float4_t& hi, int32_t dtype) {
  if (dtype == kFewOutF16)
    return __builtin_bit_cast(u32x4_t, half8_t{(_Float16)lo[0], (_Float16)lo[1], (_Float16)lo[2], (_Float16)lo[3],
                                               (_Float16)hi[0], (_Float16)hi[1], (_Float16)hi[2], (_Float16)hi[3]});
  typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(u32x4_t, bf16x8_t{(__bf16)lo[0], (__bf16)lo[1], (__bf16)lo[2], (__bf16)lo[3],
                                              (__bf16)hi[0], (__bf16)hi[1], (__bf16)hi[2], (__bf16)hi[3]});
}

}  // namespace moe_fp4

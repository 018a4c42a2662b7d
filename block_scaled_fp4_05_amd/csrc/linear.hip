// Few-token linear layer with NVFP4 weights (moe_fp4_linear):
//
//   y[t][j] = w_scale * sum_k x[t][k] W[j][k]  (+ residual[t][j])
//   or, with the SwiGLU epilogue on n = 2I rows,  silu(y[t][i]) * y[t][I + i]
//
// x is BF16 or FP16 and stays so; the weights become exact values of the same type
// in registers and are multiplied on the matrix cores with FP32 accumulation.
//
// Bound: the weight stream, n * k * 9/16 bytes (a few tokens give a few operations a
// byte).  A workgroup owns NT x 16 weight rows and its wavefronts split K, so that
// even a 16-row tile keeps several wavefronts loading; their sums meet in LDS in
// wavefront order (no atomics: the same inputs give the same bits).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "few_token_device.h"

namespace moe_fp4 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kWaves = 8;

template <bool F16, int NT, int MT, bool SWIGLU>
__global__ __launch_bounds__(kMaxThreads) void k_linear(LinearArgs a) {
  extern __shared__ __align__(16) char smem[];
  float4_t* red = reinterpret_cast<float4_t*>(smem);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int32_t half = a.n / 2;
  const int32_t n0 = blockIdx.x * (SWIGLU ? 8 : 16) * NT;
  const int32_t m0 = blockIdx.y * 16 * MT;
  const float scale = ((sconst_f32)a.w_scale)[0];

  // Item of the epilogue: four consecutive weight rows of one token.
  const int tile = threadIdx.x >> 6;  // (nt, mt)
  const int32_t tok = m0 + (tile % MT) * 16 + (lane & 15);
  const int32_t j0 = SWIGLU ? n0 + (tile / MT) * 8 + 4 * ((lane >> 4) & 1)
                            : n0 + (tile / MT) * 16 + 4 * (lane >> 4);
  const int32_t cols = SWIGLU ? half : a.n;
  const bool mine = tile < NT * MT && tok < a.m && (!SWIGLU || lane < 32);
  float res[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (!SWIGLU && a.residual && mine) {
    const uint16_t* rp = static_cast<const uint16_t*>(a.residual) + tok * a.ld_res;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < cols) res[i] = value16<F16>(rp[j0 + i]);
  }

  uint32_t row[NT], xoff[MT];
  const int r = lane & 15;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (SWIGLU) {  // rows 0-7 of a tile: gate; 8-15: the same columns of up
      const int32_t c = n0 + 8 * t + (r & 7);
      row[t] = (uint32_t)((r >> 3) * half + (c < half ? c : half - 1));
    } else {
      const int32_t c = n0 + 16 * t + r;
      row[t] = (uint32_t)(c < a.n ? c : a.n - 1);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int32_t t = m0 + 16 * m + r;
    xoff[m] = t < a.m ? (uint32_t)(t * a.ld_x * 2) : kOutOfRange;
  }
  FewLoop<F16, NT, MT> loop;
  loop.q_rs = make_rsrc(a.w_q, (uint32_t)((int64_t)a.n * (a.k / 2)));
  loop.s_rs = make_rsrc(a.w_sf, (uint32_t)((int64_t)a.n * (a.k / 16)));
  loop.x_rs = make_rsrc(a.x, (uint32_t)(((a.m - 1) * a.ld_x + a.k) * 2));
  loop.k = a.k;
  loop.g = lane >> 4;
  float4_t acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int32_t steps = (a.k + kFewStep - 1) / kFewStep;
  const int32_t s0 = uniform(wave * steps / waves), s1 = uniform((wave + 1) * steps / waves);
  if (s0 < s1) loop.run(row, xoff, acc, s0, s1);
  put_sums<NT, MT>(red, acc, wave, lane);
  __syncthreads();
  if (!mine) return;

  const float4_t v = take_sum(red, NT * MT, tile, lane, waves);
  const int64_t o = tok * a.ldo + j0;
  if (SWIGLU) {
    const float4_t u = take_sum(red, NT * MT, tile, lane + 32, waves);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < cols) store_as(a.out, o + i, silu(v[i] * scale) * (u[i] * scale), a.out_dtype);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < cols) store_as(a.out, o + i, v[i] * scale + res[i], a.out_dtype);
  }
}

template <bool F16, int NT, int MT>
hipError_t launch(const LinearArgs& a, int waves, hipStream_t stream) {
  const int cols = a.swiglu ? a.n / 2 : a.n, width = (a.swiglu ? 8 : 16) * NT;
  const dim3 grid((cols + width - 1) / width, (a.m + 16 * MT - 1) / (16 * MT));
  const size_t lds = (size_t)waves * NT * MT * 64 * 16;
  if (a.swiglu)
    hipLaunchKernelGGL((k_linear<F16, NT, MT, true>), grid, dim3(waves * 64), lds, stream, a);
  else
    hipLaunchKernelGGL((k_linear<F16, NT, MT, false>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_typed(const LinearArgs& a, hipStream_t stream) {
  const int mt = a.m > 16 ? 2 : 1;
  return mt == 1 ? launch<F16, 1, 1>(a, kWaves, stream) : launch<F16, 1, 2>(a, kWaves, stream);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  return a.x_f16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace moe_fp4

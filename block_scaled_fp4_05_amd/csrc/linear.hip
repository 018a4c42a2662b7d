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
//
// Measured, kernel time on weights that are in no cache: 65536 x 6144, four BF16 tokens, FP32
// out: 47.4 us, 4.8 TB/s (a large copy reaches 5.05).  8192 x 6144 with SwiGLU, 16
// FP16 tokens: 12.0 us, 2.4 TB/s.  6144 x 6144, one token: 8.6 us, 2.5 TB/s: one or two
// workgroups a CU, whose start, first loads and final sum nothing covers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "few_token_device.h"

namespace moe_fp4 {
namespace {

constexpr int kMaxThreads = 512;

// XR: loads of two tokens (see FewLoop), all of them kept in flight: with four of eight
// 8192 x 6144, 16 tokens take 21.7 us instead of 13.7.
template <bool F16, int NT, int XR>
using LinearLoop = FewLoop<F16, NT, XR, XR, (NT > 1 && XR <= 4)>;

template <bool F16, int NT, int XR>
__global__ __launch_bounds__(kMaxThreads) void k_linear(LinearArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef LinearLoop<F16, NT, XR> Loop;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6, r = lane & 15;
  const bool swiglu = a.swiglu != 0;
  const int32_t half = a.n / 2, cols = swiglu ? half : a.n;
  const int32_t n0 = blockIdx.x * (swiglu ? 8 : 16) * NT;
  const int32_t m0 = blockIdx.y * 16;
  const float scale = ((sconst_f32)a.w_scale)[0];
  Loop loop;
  loop.q_rs = make_rsrc(a.w_q, (uint32_t)((int64_t)a.n * (a.k / 2)));
  loop.s_rs = make_rsrc(a.w_sf, (uint32_t)((int64_t)a.n * (a.k / 16)));
  loop.x_rs = make_rsrc(a.x, (uint32_t)(((a.m - 1) * a.ld_x + a.k) * 2));
  loop.lds = smem + wave * Loop::kLdsBytes;
  loop.k = a.k;
  loop.tokens = a.m - m0 < 16 ? a.m - m0 : 16;
  loop.lane = lane;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int lr = Loop::row_of(lane);
    int32_t row;
    if (swiglu) {  // rows 0-7 of a tile: gate; 8-15: the same columns of up
      const int32_t c = n0 + 8 * t + (lr & 7);
      row = (lr >> 3) * half + (c < half ? c : half - 1);
    } else {
      const int32_t c = n0 + 16 * t + lr;
      row = c < a.n ? c : a.n - 1;
    }
    loop.q_off[t] = (uint32_t)row * (uint32_t)(a.k / 2);
    loop.s_off[t] = (uint32_t)row * (uint32_t)(a.k / 16);
  }
#pragma unroll
  for (int i = 0; i < XR; ++i) {
    const int32_t t = 2 * i + (lane >> 5);
    loop.x_off[i] = t < loop.tokens ? (uint32_t)((m0 + t) * a.ld_x * 2 + 16 * (lane & 31)) : kOutOfRange;
  }
  float4_t acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int32_t steps = (a.k + kFewStep - 1) / kFewStep;
  loop.run(acc, uniform(wave * steps / waves), uniform((wave + 1) * steps / waves));

  // A thread's share of the result: four consecutive weight rows of one token.
  const int tile = threadIdx.x >> 6;
  const int32_t tok = m0 + r;
  const int32_t j0 = swiglu ? n0 + tile * 8 + 4 * ((lane >> 4) & 1) : n0 + tile * 16 + 4 * (lane >> 4);
  const bool mine = tile < NT && tok < a.m && j0 < cols && (!swiglu || lane < 32);
  float res[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.residual && mine) {  // its latency passes under the barrier
    const uint16_t* rp = static_cast<const uint16_t*>(a.residual) + tok * a.ld_res + j0;
    uint16_t raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = rp[j0 + i < cols ? i : 0];
#pragma unroll
    for (int i = 0; i < 4; ++i) res[i] = value16<F16>(raw[i]);
  }
  put_sums<NT>(loop.lds, acc, lane);
  __syncthreads();
  if (!mine) return;
  float4_t v = take_sum(smem, Loop::kLdsBytes, tile, lane, waves) * scale;
  if (swiglu) {
    const float4_t u = take_sum(smem, Loop::kLdsBytes, tile, lane + 32, waves) * scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
  }
  const int64_t o = tok * a.ldo + j0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j0 + i < cols) store_as(a.out, o + i, a.residual ? v[i] + res[i] : v[i], a.out_dtype);
}

template <bool F16, int NT, int XR>
hipError_t launch(const LinearArgs& a, int items, int waves, hipStream_t stream) {
  if (waves < NT) waves = NT;  // a wavefront finishes one tile of the result
  const dim3 grid(items, (a.m + 15) / 16);
  const size_t lds = (size_t)waves * LinearLoop<F16, NT, XR>::kLdsBytes;
  hipLaunchKernelGGL((k_linear<F16, NT, XR>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

// Room for 2, 4, 8 or 16 tokens: registers, and with them the wavefronts on a CU, depend on
// it (eight tokens with room for 8 against 16: 65536 x 6144 59 us against 71, 6144 x
// 6144 11.9 against 13.3, 1001 x 784 4.0 against 4.4).  More tokens take several workgroups
// an item, whose codes then come from the caches: with room for 32, 32 tokens took 35.4 us against
// 19.9 on 8192 x 6144 and 132 against 123 on 65536 x 6144; 20 on 6144 x 6144 19.5 against 20.2.
template <bool F16, int NT>
hipError_t launch_rows(const LinearArgs& a, int items, int waves, hipStream_t stream) {
  if (a.m <= 2) return launch<F16, NT, 1>(a, items, waves, stream);
  if (a.m <= 4) return launch<F16, NT, 2>(a, items, waves, stream);
  if (a.m <= 8) return launch<F16, NT, 4>(a, items, waves, stream);
  return launch<F16, NT, 8>(a, items, waves, stream);
}

// Two tiles an item (half the activation reads and half the wavefronts) once that
// leaves an item for every CU: 8192 x 6144, 16 tokens 13.6 us against 14.8; 65536 x 6144,
// 4 tokens 54 against 56 (before the codes were turned in LDS); but 6144 x 6144, one
// token 9.8 against 9.7.  Four wavefronts an item, eight where there are too few items to fill
// the CUs (one or two wavefronts on 6144 x 6144: 17.9 and 13.1 us; eight on 65536 x
// 6144: 63 us).  With more than 256 tiles eight are slower again: one token of 4352 x 6144
// 8.5 us against 7.9, of 6144 x 6144 9.0 against 8.7, 16 tokens of the latter 15.5 against 12.1;
// two-tile items of 8192 x 6144 with 16 tokens and SwiGLU 12.4 against 11.5.
template <bool F16>
hipError_t launch_typed(const LinearArgs& a, hipStream_t stream) {
  const int steps = (a.k + kFewStep - 1) / kFewStep;
  const int tiles = a.swiglu ? (a.n / 2 + 7) / 8 : (a.n + 15) / 16;
  const bool pair = tiles >= 512;
  const int items = pair ? (tiles + 1) / 2 : tiles;
  int waves = tiles <= 256 ? 8 : 4;
  if (waves > steps) waves = steps;
  return pair ? launch_rows<F16, 2>(a, items, waves, stream) : launch_rows<F16, 1>(a, items, waves, stream);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  return a.x_f16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace moe_fp4

// Gradient of the router's weights with respect to its logits (moe_fp4_route_backward).
// With d[s] the gradient of the weight of slot s, e_s its expert, x_s that expert's logit:
//
//   softmax, renormalised   w = softmax of the chosen logits;  dx[e_s] = w_s (d_s - sum w d)
//   softmax                 p over all experts;  dx[e] = p_e (sum_{e_s = e} d_s - sum_s p_s d_s)
//   sigmoid, renormalised   w = p / sum p;  dx[e_s] = w_s (1 - p_s)(d_s - sum w d)
//   sigmoid                 dx[e_s] = p_s (1 - p_s) d_s
//
// and 0 everywhere else.  All in FP32: a sigmoid is e^min(x,0) / (1 + e^-|x|) and its
// complement the same of -x, so neither loses its small end, and the quotients of w are
// taken with the largest e^min(x,0) divided out, so that tiny scores keep their proportions.
//
// A token takes 16 lanes (up to 256 experts and 16 slots) or 64, each with 16 consecutive
// experts.  Its first lanes are its slots, which compute the slots' terms and put them into a row
// of LDS (slots that name the same expert add up there, in slot order); every lane takes its
// experts' terms from it and writes each element of the dense result once.  Four tokens a
// wavefront share every instruction, and a reduction over 16 lanes needs no LDS.  Bound: the
// logits (softmax only) and the result, 2 to 8 bytes an expert, in one pass of dependent steps
// with five barriers of the workgroup around the terms (16384 tokens of 256 experts, softmax over
// all: 8 us; with 64 lanes a token 32), and for short calls the launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "few_token_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;  // experts of a lane

// 16 consecutive elements, whole (from a 16-byte aligned address) or those below `have`.
template <typename T>
__device__ __forceinline__ void load16(const void* p, int64_t at, int32_t have, bool wide, float (&v)[kPer]) {
  constexpr int N = 16 / sizeof(T);
  typedef T vec_t __attribute__((ext_vector_type(N)));
  const T* q = static_cast<const T*>(p) + at;
  if (wide && have >= kPer) {
#pragma unroll
    for (int i = 0; i < kPer; i += N) {
      const vec_t x = *reinterpret_cast<const vec_t*>(q + i);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i + j] = (float)x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = i < have ? (float)q[i] : -INFINITY;
  }
}

template <typename T>
__device__ __forceinline__ void store16(void* p, int64_t at, int32_t have, bool wide, const float (&v)[kPer]) {
  constexpr int N = 16 / sizeof(T);
  typedef T vec_t __attribute__((ext_vector_type(N)));
  T* q = static_cast<T*>(p) + at;
  if (wide && have >= kPer) {
#pragma unroll
    for (int i = 0; i < kPer; i += N) {
      vec_t x;
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = (T)v[i + j];
      *reinterpret_cast<vec_t*>(q + i) = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < have) q[i] = (T)v[i];
  }
}

__device__ __forceinline__ float add(float a, float b) { return a + b; }
// The larger one, or NaN if one is.
__device__ __forceinline__ float larger(float a, float b) { return a != a ? a : (b != b || b > a) ? b : a; }

// Over the L lanes of a token, the same bits in each: rotations within 16 lanes give every lane
// the same pairs in some order, and a sum or maximum of two does not depend on theirs.
template <int L, typename F>
__device__ __forceinline__ float reduce(float v, F f) {
  auto turned = [](float x, auto n) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + decltype(n)::value, 0xf, 0xf, false));
  };
  v = f(v, turned(v, std::integral_constant<int, 8>{}));  // row_ror
  v = f(v, turned(v, std::integral_constant<int, 4>{}));
  v = f(v, turned(v, std::integral_constant<int, 2>{}));
  v = f(v, turned(v, std::integral_constant<int, 1>{}));
  if constexpr (L == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int L, typename T, bool DENSE>
__global__ __launch_bounds__(kThreads) void k_route_backward(RouteBackwardArgs a) {
  const int lane = threadIdx.x & 63, me = lane & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool here = t < a.tokens;
  const int64_t row = here ? t : 0;
  const int32_t first = kPer * me, have = here ? a.experts - first : 0;
  float x[kPer];
  if (DENSE) load16<T>(a.logits, row * a.ld + first, have, a.wide != 0, x);

  // Lane `me` of a token is its slot `me`.
  const int32_t e = here && me < a.topk ? a.ids[row * a.topk + me] : -1;
  const bool valid = e >= 0 && e < a.experts;
  const float d = valid ? a.dweights[row * a.topk + me] : 0.0f;
  float term = d;
  if (!DENSE) {
    const float l = valid ? (float)static_cast<const T*>(a.logits)[row * a.ld + e] : -INFINITY;
    if (a.sigmoid) {
      const float low = fminf(l, 0.0f), small = expf(-fabsf(l)), whole = 1.0f + small;
      // 1 - p = e^min(-x,0) / (1 + e^-|x|): one of the two exponents is 0.
      const float left = (l > 0.0f ? small : 1.0f) / whole;
      if (a.renormalize) {
        const float m = reduce<L>(valid ? low : -INFINITY, larger);
        const float p = valid ? expf(low - m) / whole : 0.0f;
        const float w = p / reduce<L>(p, add);
        term = w * left * (d - reduce<L>(valid ? w * d : 0.0f, add));
      } else {
        term = (l > 0.0f ? 1.0f : small) / whole * left * d;
      }
    } else {
      const float m = reduce<L>(l, larger);
      const float p = valid ? expf(l - m) : 0.0f;
      const float w = p / reduce<L>(p, add);
      term = w * (d - reduce<L>(valid ? w * d : 0.0f, add));
    }
  }
  if (!valid) term = 0.0f;

  // The token's row of terms.  Whether two slots name one expert: then one of them does not find its
  // own number where it wrote it.
  __shared__ __align__(16) float rows[kThreads * kPer];
  float* const mine = rows + (threadIdx.x - me) * kPer;
  int32_t* const names = reinterpret_cast<int32_t*>(mine);
  if (valid) names[e] = me;
  __syncthreads();
  const bool twice = valid && names[e] != me;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; j += 4) *reinterpret_cast<float4_t*>(mine + first + j) = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  if (__syncthreads_or(twice)) {
    for (int k = 0; k < a.topk; ++k) {
      if (valid && me == k) mine[e] += term;
      __syncthreads();
    }
  } else if (valid) {
    mine[e] = term;
  }
  __syncthreads();
  float v[kPer];
#pragma unroll
  for (int j = 0; j < kPer; j += 4) {
    const float4_t f = *reinterpret_cast<const float4_t*>(mine + first + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j + i] = f[i];
  }
  if (DENSE) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) m = larger(m, x[j]);
    if (have <= 0) m = -INFINITY;
    m = reduce<L>(m, larger);
    float sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      x[j] = j < have ? expf(x[j] - m) : 0.0f;
      sum += x[j];
    }
    sum = 1.0f / reduce<L>(sum, add);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      x[j] = j < have ? x[j] * sum : 0.0f;
      mean += x[j] * v[j];
    }
    mean = reduce<L>(mean, add);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = x[j] * (v[j] - mean);
  }
  store16<T>(a.dlogits, row * a.ld_out + first, have, a.wide != 0, v);
}

template <int L, typename T>
hipError_t launch(const RouteBackwardArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.tokens + kThreads / L - 1) / (kThreads / L)));
  if (!a.sigmoid && !a.renormalize)
    hipLaunchKernelGGL((k_route_backward<L, T, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((k_route_backward<L, T, false>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(RouteBackwardArgs a, hipStream_t stream) {
  a.wide = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0 &&
           a.ld * sizeof(T) % 16 == 0 && a.ld_out * sizeof(T) % 16 == 0;
  return a.experts <= 256 && a.topk <= 16 ? launch<16, T>(a, stream) : launch<64, T>(a, stream);
}

}  // namespace

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream) {
  if (a.dtype == kInF32) return launch_typed<float>(a, stream);
  return a.dtype == kInF16 ? launch_typed<_Float16>(a, stream) : launch_typed<__bf16>(a, stream);
}

}  // namespace moe_fp4

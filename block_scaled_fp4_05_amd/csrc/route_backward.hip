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
// A wavefront takes G tokens: first its lanes are (token, slot) pairs, which compute the
// slots' terms; then all 64 lanes write each token's row of the dense result, every element
// once, adding the slots that name its expert in slot order.  Bound: the logits (softmax only)
// and the result, 2 to 8 bytes an expert, and for short calls the launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_token_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPerLane = 16;  // experts of a lane: 1024 / 64

__device__ __forceinline__ float load_in(const void* p, int64_t i, int32_t dtype) {
  if (dtype == kInF32) return static_cast<const float*>(p)[i];
  if (dtype == kInF16) return (float)static_cast<const _Float16*>(p)[i];
  return (float)static_cast<const __bf16*>(p)[i];
}

__device__ __forceinline__ void store_in(void* p, int64_t i, float v, int32_t dtype) {
  if (dtype == kInF32) static_cast<float*>(p)[i] = v;
  else if (dtype == kInF16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

template <typename F>
__device__ __forceinline__ float reduce(float v, int width, F f) {
  for (int d = 1; d < width; d <<= 1) v = f(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
// The larger one, or NaN if one is.
__device__ __forceinline__ float larger_nan(float a, float b) { return a != a ? a : (b != b || b > a) ? b : a; }

__global__ __launch_bounds__(kThreads) void k_route_backward(RouteBackwardArgs a) {
  const int lane = threadIdx.x & 63;
  const int width = a.slot_lanes;  // lanes of one token in the first part, a power of two
  const int64_t group = (int64_t)blockIdx.x * kWaves + uniform(threadIdx.x >> 6);
  const int64_t t0 = group * a.group_tokens;
  if (t0 >= a.tokens) return;
  const bool dense = a.sigmoid == 0 && a.renormalize == 0;

  // (token, slot) pairs.
  const int64_t t = t0 + lane / width;
  const int s = lane & (width - 1);
  const bool pair = lane / width < a.group_tokens && t < a.tokens && s < a.topk;
  const int32_t e = pair ? a.ids[t * a.topk + s] : -1;
  const bool valid = e >= 0 && e < a.experts;
  const float d = valid ? a.dweights[t * a.topk + s] : 0.0f;
  float term = d;
  if (!dense) {
    const float x = valid ? load_in(a.logits, t * a.ld + e, a.dtype) : -INFINITY;
    if (a.sigmoid) {
      const float low = fminf(x, 0.0f), left = expf(fminf(-x, 0.0f)) / (1.0f + expf(-fabsf(x)));
      if (a.renormalize) {
        const float m = reduce(valid ? low : -INFINITY, width, larger_nan);
        const float p = valid ? expf(low - m) / (1.0f + expf(-fabsf(x))) : 0.0f;
        const float sum = reduce(p, width, add);
        const float w = p / sum;
        const float mean = reduce(valid ? w * d : 0.0f, width, add);
        term = w * left * (d - mean);
      } else {
        term = expf(low) / (1.0f + expf(-fabsf(x))) * left * d;
      }
    } else {
      const float m = reduce(x, width, larger_nan);
      const float p = valid ? expf(x - m) : 0.0f;
      const float sum = reduce(p, width, add);
      const float w = p / sum;
      const float mean = reduce(valid ? w * d : 0.0f, width, add);
      term = w * (d - mean);
    }
    if (!valid) term = 0.0f;
  }

  // Rows of the result.
  for (int g = 0; g < a.group_tokens && t0 + g < a.tokens; ++g) {
    const int64_t row = t0 + g;
    float v[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) v[j] = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
      const int at = g * width + k;
      const int32_t ek = uniform(__shfl(e, at, 64));
      const float tk = __shfl(term, at, 64);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (64 * j < a.experts && 64 * j + lane == ek) v[j] += tk;
    }
    if (dense) {
      float x[kPerLane];
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        x[j] = -INFINITY;
        if (64 * j + lane < a.experts) x[j] = load_in(a.logits, row * a.ld + 64 * j + lane, a.dtype);
        if (64 * j < a.experts) m = larger_nan(m, x[j]);
      }
      m = reduce(m, 64, larger_nan);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (64 * j < a.experts) {
          x[j] = 64 * j + lane < a.experts ? expf(x[j] - m) : 0.0f;
          sum += x[j];
        }
      sum = reduce(sum, 64, add);
      float mean = 0.0f;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (64 * j < a.experts) {
          x[j] = x[j] / sum;
          mean += 64 * j + lane < a.experts ? x[j] * v[j] : 0.0f;
        }
      mean = reduce(mean, 64, add);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) v[j] = x[j] * (v[j] - mean);
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
      if (64 * j + lane < a.experts) store_in(a.dlogits, row * a.ld_out + 64 * j + lane, v[j], a.dtype);
  }
}

}  // namespace

hipError_t launch_route_backward(const RouteBackwardArgs& args, hipStream_t stream) {
  RouteBackwardArgs a = args;
  a.slot_lanes = 1;
  while (a.slot_lanes < a.topk) a.slot_lanes *= 2;
  // Tokens of a wavefront: as many as its lanes hold slots for, once there are several
  // wavefronts for every SIMD (1024 of them).
  a.group_tokens = 1;
  while (a.group_tokens * 2 * a.slot_lanes <= 64 && a.tokens >= (int64_t)a.group_tokens * 2 * 4096)
    a.group_tokens *= 2;
  const int64_t groups = (a.tokens + a.group_tokens - 1) / a.group_tokens;
  hipLaunchKernelGGL(k_route_backward, dim3((unsigned)((groups + kWaves - 1) / kWaves)), dim3(kThreads), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace moe_fp4

// The Mixture-of-Experts router (moe_fp4_route): each token's best topk experts and
// their weights, and the routed rows grouped by expert as the grouped GEMM and the
// token-order combine take them (offsets, row -> token, token -> rows).
//
//   scores    softmax:  p = e^x / sum e^x, ranked by the logit x itself
//             sigmoid:  p = 1 / (1 + e^-x), ranked by p + bias
//   groups    with num_groups > 1 only the best topk_groups runs of experts stay
//             open; a group's score is its best rank value (softmax) or the sum of its
//             two best (sigmoid)
//   ties      go to the lower index, in groups and experts
//
// A wavefront ranks one token: lane l holds consecutive experts of one group, so the
// order of lanes is the order of experts and the first lane that holds the maximum
// wins a tie.  Sigmoid values are ranked in FP64: neighbouring scores of a few hundred
// experts come closer than an FP32 step often enough to swap experts.
//
// Grouping is a counting sort by expert, stable in token order and without a
// scatter order that could vary: a block of tokens marks each expert's tokens in an
// LDS bitmap, so the row of (token, expert) is the expert's offset, plus its rows in
// earlier blocks, plus the marks before the token.  Up to kOneBlock tokens take one
// launch; more take two, the second reading the first's per-block counts.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
// Ranking values below every score: a NaN (below -inf), and an expert that is taken,
// closed or no expert at all.
constexpr double kKeyMinusInf = -1.0e308, kKeyNaN = -1.5e308;

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}

// Ranking keys: FP32 logits as integers of the same order, FP64 scores as they are.
struct Key32 {
  typedef uint32_t T;
  static __device__ __forceinline__ T none() { return 0u; }
  static __device__ __forceinline__ T of(float x) {
    if (x != x) return 1u;
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 ranks as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  static __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ T moved(T v) {
    return dpp<CTRL, ROWS>(0u, v);
  }
  static __device__ __forceinline__ T lane(T v, int l) {
    return (T)__builtin_amdgcn_readlane((int)v, l);
  }
};

struct Key64 {
  typedef double T;
  static __device__ __forceinline__ T none() { return -__builtin_inf(); }
  static __device__ __forceinline__ T of(double s) {
    return s != s ? kKeyNaN : s < kKeyMinusInf ? kKeyMinusInf : s;
  }
  static __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ T moved(T v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL, ROWS>(0u, (uint32_t)b);
    const uint32_t hi = dpp<CTRL, ROWS>(0xFFF00000u, (uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
  static __device__ __forceinline__ T lane(T v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
};

// The largest key of the wavefront, in every lane.
template <typename K>
__device__ __forceinline__ typename K::T wave_max(typename K::T v) {
  v = K::larger(v, K::template moved<0x111, 0xf>(v));
  v = K::larger(v, K::template moved<0x112, 0xf>(v));
  v = K::larger(v, K::template moved<0x114, 0xf>(v));
  v = K::larger(v, K::template moved<0x118, 0xf>(v));
  v = K::larger(v, K::template moved<0x142, 0xf>(v));
  v = K::larger(v, K::template moved<0x143, 0xf>(v));
  return K::lane(v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.dtype == kRouteF32) return static_cast<const float*>(a.logits)[i];
  const uint16_t b = static_cast<const uint16_t*>(a.logits)[i];
  return a.dtype == kRouteF16 ? (float)__builtin_bit_cast(_Float16, b)
                              : __builtin_bit_cast(float, (uint32_t)b << 16);
}

// Rank one token: lane s < topk returns the expert and weight of slot s.
template <bool SIGMOID, int VPL>
__device__ __forceinline__ void rank_token(const RouteArgs& a, int32_t t, int lane, int32_t* id,
                                           float* weight) {
  typedef typename std::conditional<SIGMOID, Key64, Key32>::type K;
  typedef typename K::T KeyT;
  const int32_t size = a.experts / a.num_groups;  // experts of a group
  const int32_t group = lane / a.group_lanes, in = lane % a.group_lanes;
  const int32_t first = in * a.per_lane;
  const int32_t expert0 = group * size + first;
  KeyT key[VPL];
  float val[VPL];  // logit (softmax) or score (sigmoid)
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const bool ok = group < a.num_groups && j < a.per_lane && first + j < size;
    float x = -__builtin_inff();
    if (ok) x = load_logit(a, (int64_t)t * a.ld + expert0 + j);
    if (SIGMOID) {
      const double p = 1.0 / (1.0 + exp(-(double)x));
      val[j] = (float)p;
      key[j] = ok ? K::of(a.bias ? p + (double)a.bias[expert0 + j] : p) : K::none();
    } else {
      val[j] = x;
      key[j] = ok ? K::of(x) : K::none();
    }
  }
  float top = 0.0f, sum = 0.0f;
  if (!SIGMOID && !a.renormalize) {
    float m = val[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = fmaxf(m, val[j]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    top = m;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] != K::none()) sum += expf(val[j] - top);
    sum = wave_sum(sum);
  }
  if (a.topk_groups < a.num_groups) {
    KeyT best = K::none(), second = K::none();
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (key[j] > best) second = best, best = key[j];
      else if (key[j] > second) second = key[j];
    }
    for (int d = 1; d < a.group_lanes; d <<= 1) {
      const KeyT b = __shfl_xor(best, d, 64), s = __shfl_xor(second, d, 64);
      const KeyT low = best > b ? b : best;
      best = K::larger(best, b);
      second = K::larger(low, K::larger(second, s));
    }
    const KeyT score = SIGMOID && size > 1 ? best + second : best;
    int32_t ahead = 0;
    for (int32_t o = 0; o < a.num_groups; ++o) {
      const KeyT other = K::lane(score, o * a.group_lanes);
      ahead += other > score || (other == score && o < group) ? 1 : 0;
    }
    if (ahead >= a.topk_groups) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = K::none();
    }
  }
  int32_t my_id = 0;
  float my_val = 0.0f;
  for (int32_t s = 0; s < a.topk; ++s) {
    KeyT best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = K::larger(best, key[j]);
    const KeyT m = wave_max<K>(best);
    const int win = __ffsll((unsigned long long)__ballot(best == m)) - 1;
    int32_t at = 0;
    float v = val[0];
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j)
      if (key[j] == m) at = j, v = val[j];
    const int32_t chosen = __builtin_amdgcn_readlane(expert0 + at, win);
    const float value = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, v), win));
    if (lane == s) my_id = chosen, my_val = value;
    if (lane == win) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j == at) key[j] = K::none();
    }
  }
  const bool mine = lane < a.topk;
  float w = my_val;
  if (SIGMOID) {
    if (a.renormalize) w = my_val / wave_sum(mine ? my_val : 0.0f);
  } else if (a.renormalize) {
    // The full softmax's denominator cancels: only the chosen experts' terms are needed.
    float m = mine ? my_val : -__builtin_inff();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    const float e = expf(my_val - m);
    w = e / wave_sum(mine ? e : 0.0f);
  } else {
    w = expf(my_val - top) / sum;
  }
  *id = my_id;
  *weight = w;
}

// Exclusive scan of total[0 .. experts) in LDS into base, plus `before` (rows of
// earlier blocks); block 0 also writes the offsets.  All threads; barriers inside.
__device__ __forceinline__ void scan_offsets(const RouteArgs& a, const int32_t* total,
                                             int32_t* before, int32_t* wave_sums, bool write) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  int32_t carry = 0;
  for (int32_t e0 = 0; e0 < a.experts; e0 += blockDim.x) {
    const int32_t e = e0 + tid;
    const int32_t c = e < a.experts ? total[e] : 0;
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sums[wave] = incl;
    __syncthreads();
    int32_t base = carry;
    for (int w = 0; w < waves; ++w) {
      const int32_t v = wave_sums[w];
      if (w < wave) base += v;
      carry += v;
    }
    if (e < a.experts) {
      const int32_t off = base + incl - c;
      if (write) a.offsets[e] = off;
      before[e] += off;
    }
    __syncthreads();
  }
  if (write && tid == 0) a.offsets[a.experts] = carry;
}

// Rows of a block's pairs: the marks before each token in its expert's bitmap.
__device__ __forceinline__ void place_rows(const RouteArgs& a, const int32_t* ids,
                                           const uint32_t* marks, const int32_t* base, int32_t t0,
                                           int32_t count, int words) {
  for (int32_t p = threadIdx.x; p < count * a.topk; p += blockDim.x) {
    const int32_t e = ids[p], tl = p / a.topk;
    const uint32_t* m = marks + e * words;
    int32_t r = base[e];
    for (int w = 0; w < tl >> 5; ++w) r += __popc(m[w]);
    r += __popc(m[tl >> 5] & ((1u << (tl & 31)) - 1));
    a.token_rows[(int64_t)t0 * a.topk + p] = r;
    a.row_token[r] = t0 + tl;
  }
}

__device__ __forceinline__ void mark(uint32_t* marks, int32_t e, int32_t tl, int words) {
  atomicOr(&marks[e * words + (tl >> 5)], 1u << (tl & 31));
}

// Ranks a block of tokens; leaves the block's rows per expert (16-bit) in counts.
template <bool SIGMOID, int VPL>
__global__ __launch_bounds__(kThreads) void k_rank(RouteArgs a) {
  extern __shared__ __align__(16) int32_t count[];  // [experts]
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int32_t t0 = blockIdx.x * a.block_tokens;
  const int32_t here = a.tokens - t0 < a.block_tokens ? a.tokens - t0 : a.block_tokens;
  for (int i = tid; i < a.counts_pitch; i += kThreads) count[i] = 0;
  __syncthreads();
  for (int32_t tl = wave; tl < here; tl += kWaves) {
    int32_t id;
    float w;
    rank_token<SIGMOID, VPL>(a, t0 + tl, lane, &id, &w);
    if (lane < a.topk) {
      const int64_t o = (int64_t)(t0 + tl) * a.topk + lane;
      a.ids[o] = id;
      a.weights[o] = w;
      atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  uint16_t* out = a.counts + (int64_t)blockIdx.x * a.counts_pitch;
  for (int i = tid; i < a.counts_pitch; i += kThreads) out[i] = (uint16_t)count[i];
}

// Places a block's rows: offsets from every block's counts, then the marks.
__global__ __launch_bounds__(kThreads) void k_place(RouteArgs a) {
  extern __shared__ __align__(16) int32_t lds[];
  const int words = a.block_tokens / 32 > 1 ? a.block_tokens / 32 : 1;
  int32_t* total = lds;
  int32_t* before = total + a.counts_pitch;
  int32_t* wave_sums = before + a.counts_pitch;
  uint32_t* marks = reinterpret_cast<uint32_t*>(wave_sums + kWaves);
  const int tid = threadIdx.x;
  const int32_t t0 = blockIdx.x * a.block_tokens;
  const int32_t here = a.tokens - t0 < a.block_tokens ? a.tokens - t0 : a.block_tokens;
  const int32_t* ids = a.ids + (int64_t)t0 * a.topk;
  for (int i = tid; i < 2 * a.counts_pitch; i += kThreads) total[i] = 0;
  for (int i = tid; i < a.experts * words; i += kThreads) marks[i] = 0;
  __syncthreads();
  for (int32_t p = tid; p < here * a.topk; p += kThreads) mark(marks, ids[p], p / a.topk, words);
  // A thread sums eight experts (16 bytes of counts) over every `stride`-th block.
  const int cols = a.counts_pitch / 8, stride = kThreads / cols;
  const int col = tid % cols, row = tid / cols;
  if (row < stride) {
    int32_t all[8] = {}, low[8] = {};
    for (int32_t b = row; b < (int32_t)gridDim.x; b += stride) {
      const uint4 v = *reinterpret_cast<const uint4*>(a.counts + (int64_t)b * a.counts_pitch + 8 * col);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      const bool earlier = b < (int32_t)blockIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t c = (int32_t)(u[i / 2] >> (16 * (i % 2)) & 0xFFFFu);
        all[i] += c;
        low[i] += earlier ? c : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (all[i]) atomicAdd(&total[8 * col + i], all[i]);
      if (low[i]) atomicAdd(&before[8 * col + i], low[i]);
    }
  }
  __syncthreads();
  scan_offsets(a, total, before, wave_sums, blockIdx.x == 0);
  place_rows(a, ids, marks, before, t0, here, words);
}

// Both steps of at most kRouteOneBlock tokens in one workgroup.
template <bool SIGMOID, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_small(RouteArgs a) {
  extern __shared__ __align__(16) int32_t lds[];
  int32_t* total = lds;
  int32_t* before = total + a.experts;
  int32_t* wave_sums = before + a.experts;
  uint32_t* marks = reinterpret_cast<uint32_t*>(wave_sums + kWaves);
  int32_t* ids = reinterpret_cast<int32_t*>(marks + a.experts);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  for (int i = tid; i < a.experts; i += blockDim.x) before[i] = 0, marks[i] = 0;
  __syncthreads();
  for (int32_t t = wave; t < a.tokens; t += blockDim.x >> 6) {
    int32_t id;
    float w;
    rank_token<SIGMOID, VPL>(a, t, lane, &id, &w);
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = id;
      a.weights[t * a.topk + lane] = w;
      ids[t * a.topk + lane] = id;
      mark(marks, id, t, 1);
    }
  }
  __syncthreads();
  for (int i = tid; i < a.experts; i += blockDim.x) total[i] = __popc(marks[i]);
  __syncthreads();
  scan_offsets(a, total, before, wave_sums, true);
  place_rows(a, ids, marks, before, 0, a.tokens, 1);
}

template <bool SIGMOID, int VPL>
hipError_t launch(const RouteArgs& a, hipStream_t stream) {
  if (a.tokens <= kRouteOneBlock) {
    const int waves = a.tokens < 4 ? 4 : a.tokens < kWaves ? (int)a.tokens : kWaves;
    const size_t lds = (size_t)(3 * a.experts + kWaves + a.tokens * a.topk) * 4;
    hipLaunchKernelGGL((k_route_small<SIGMOID, VPL>), dim3(1), dim3(waves * 64), lds, stream, a);
    return hipGetLastError();
  }
  const int blocks = (int)((a.tokens + a.block_tokens - 1) / a.block_tokens);
  hipLaunchKernelGGL((k_rank<SIGMOID, VPL>), dim3(blocks), dim3(kThreads), (size_t)a.counts_pitch * 4,
                     stream, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int words = a.block_tokens / 32 > 1 ? a.block_tokens / 32 : 1;
  const size_t lds = (size_t)(2 * a.counts_pitch + kWaves + a.experts * words) * 4;
  hipLaunchKernelGGL(k_place, dim3(blocks), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

template <bool SIGMOID>
hipError_t launch_sized(const RouteArgs& a, hipStream_t stream) {
  if (a.per_lane <= 1) return launch<SIGMOID, 1>(a, stream);
  if (a.per_lane <= 2) return launch<SIGMOID, 2>(a, stream);
  if (a.per_lane <= 4) return launch<SIGMOID, 4>(a, stream);
  if (a.per_lane <= 8) return launch<SIGMOID, 8>(a, stream);
  return launch<SIGMOID, 16>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  return a.sigmoid ? launch_sized<true>(a, stream) : launch_sized<false>(a, stream);
}

}  // namespace moe_fp4

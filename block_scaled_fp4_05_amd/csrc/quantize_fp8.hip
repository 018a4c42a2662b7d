// FP8 (E4M3) quantisers in blocks of 128 (moe_fp8_quantize, moe_fp8_quantize_weights).
//
//   rows     s = max(amax, 448 * 2^-126) / 448 of each row's 128 columns, code = E4M3(x / s);
//            the values may be the input itself, SwiGLU of its two halves, silu(g) * u,
//            or SwiGLU's gradient, [dh u s(g) (1 + g (1 - s(g))) | dh g s(g)] with
//            s the sigmoid, computed in FP32 and never written
//   weights  the same for 128 x 128 blocks, and on request the codes and scales of the
//            transposed matrix, whose blocks are the same ones
//
// Bound: bytes (a BF16 row is read once at 2 bytes and written at 1 and a bit: 16384 x 6144 in 58
// us, 5.2 TB/s; SwiGLU of 16384 x 2 x 2048 in 35 us, 4.8 TB/s; FP32 weights 4 x 6144 x 2048
// with the transposed copy 56 us, 5.4 TB/s).  A
// block of 128 is held by 16 lanes of 8 values each, so its largest magnitude is four
// exchanges away and every access is 16 bytes (two for FP32) in, 8 out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_token_device.h"
#include "fp8_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values of a row as FP32, from a 16-byte aligned address.
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float (&v)[8]) {
  if (DT == kInF32) {
    const float* p = static_cast<const float*>(base) + elem;
    const float4_t lo = *reinterpret_cast<const float4_t*>(p), hi = *reinterpret_cast<const float4_t*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
  } else if (DT == kInF16) {
    const half8_t h = *reinterpret_cast<const half8_t*>(static_cast<const _Float16*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
    typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
    const bf16x8_t h = *reinterpret_cast<const bf16x8_t*>(static_cast<const __bf16*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// 1 / (1 + e^-x) to a few FP32 steps in eight instructions (the library's exponential and a division
// take thirty, and these modes are bound by instructions: the gradient of 5003 rows of 2 x 1424
// took 24 us, with these 18 in the same kernel).  e^-x = 2^t (1 + r ln 2) with t = RN(-x log2 e) and r what t lost: the
// product's rounding and the constant's.  x is kept within +-88, where 2^t neither overflows nor
// vanishes; beyond, the sigmoid is within 6e-39 of 0 or 1, and the reciprocal instruction gives 0
// for one below 2^-126.  A NaN is the caller's to keep: its other factor is x.
__device__ __forceinline__ float sigmoid(float x) {
  const float c = __builtin_amdgcn_fmed3f(x, -88.0f, 88.0f);
  const float t = c * -0x1.715476p+0f;
  const float r = __builtin_fmaf(c, -0x1.4ae0c0p-26f, __builtin_fmaf(c, -0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, r * 0x1.62e430p-1f, e));
}

enum { kPlain = 0, kSwiglu = 1, kSwigluGrad = 2 };

// The eight values that a lane quantises.  A gradient's columns are those of [dg | du]; k
// is a multiple of 16, so eight of them lie in one half.
template <int DT, int MODE>
__device__ __forceinline__ void values8(const Fp8QuantArgs& a, int64_t row, int32_t c, float (&v)[8]) {
  if (MODE == kPlain) {
    load8<DT>(a.x, row * a.ld_x + c, v);
    return;
  }
  const int32_t half = MODE == kSwiglu ? a.k : a.k / 2;
  const bool up_half = MODE == kSwigluGrad && c >= half;
  const int32_t h = up_half ? c - half : c;
  float g[8], u[8];
  load8<DT>(a.x, row * a.ld_x + h, g);
  if (MODE == kSwiglu) {
    load8<DT>(a.x, row * a.ld_x + half + h, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g[i] * sigmoid(g[i]) * u[i];
    return;
  }
  float d[8];
  load8<DT>(a.grad, row * a.ld_grad + h, d);
  if (up_half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d[i] * (g[i] * sigmoid(g[i]));
  } else {
    load8<DT>(a.x, row * a.ld_x + half + h, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      v[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    }
  }
}

// B blocks of 128 for every 16 lanes, all loads first.
template <int DT, int MODE, int B>
__global__ __launch_bounds__(kThreads) void k_quantize_fp8(Fp8QuantArgs a) {
  const int sub = threadIdx.x & 15;
  const uint32_t total = a.blocks;
  const uint32_t first = blockIdx.x * (kThreads / 16 * B) + (threadIdx.x >> 4);
  float v[B][8];
  uint32_t row[B], kb[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const uint32_t i = first + b * (kThreads / 16);
    row[b] = a.per_row.div(i);
    kb[b] = i - row[b] * a.per_row.d;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[b][j] = 0.0f;
    const int32_t c = (int32_t)kb[b] * kFp8Block + 8 * sub;
    if (i < total && c < a.k) values8<DT, MODE>(a, row[b], c, v[b]);
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const uint32_t i = first + b * (kThreads / 16);
    float m = amax8(v[b]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    const float s = fp8_scale(m, a.pow2 != 0);
    const u32x2_t c = fp8_encode8(v[b], s);
    const int32_t col = (int32_t)kb[b] * kFp8Block + 8 * sub;
    if (i < total) {
      if (col < a.k) *reinterpret_cast<u32x2_t*>(a.q + (int64_t)row[b] * a.k + col) = c;
      if (sub == 0) a.sf[i] = s;
    }
  }
}

// SwiGLU's gradient for rows of up to 8192 gate columns: a thread computes eight columns of both halves,
// whose loads, sigmoid and conversions they share, and the blocks' maxima meet in LDS, since
// a half need not end with a block (maxima of magnitudes as integers: the order does not
// matter).  5003 rows of 2 x 1424 BF16: 12.1 us, against 18 with a block for every 16 lanes.
constexpr int kPairThreads = 1024, kPairBlocks = 160;
constexpr int64_t kPairGrid = 1 << 21;  // workgroups (of fewer than 2^32 threads in all)

template <int DT>
__global__ __launch_bounds__(kPairThreads) void k_quantize_fp8_swiglu_grad(Fp8QuantArgs a) {
  __shared__ uint32_t top[kPairBlocks];
  const int32_t half = a.k / 2, pieces = half / 8, rows = a.group_rows;
  const int32_t kbs = (int32_t)a.per_row.d, entries = rows * kbs;
  for (int32_t i = threadIdx.x; i < entries; i += blockDim.x) top[i] = 0;
  const int32_t r = (int32_t)a.per_piece.div(threadIdx.x), c = 8 * ((int32_t)threadIdx.x - r * pieces);
  const int64_t row = (int64_t)blockIdx.x * rows + r;
  const bool in = r < rows && row < a.rows;
  float dg[8], du[8];
  if (in) {
    float g[8], u[8], d[8];
    load8<DT>(a.x, row * a.ld_x + c, g);
    load8<DT>(a.x, row * a.ld_x + half + c, u);
    load8<DT>(a.grad, row * a.ld_grad + c, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      dg[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
      du[i] = d[i] * (g[i] * s);
    }
  }
  __syncthreads();
  uint32_t* const low = top + r * kbs + c / kFp8Block;
  uint32_t* const high = top + r * kbs + (half + c) / kFp8Block;
  if (in) {
    // (Eight NaN have a NaN for their largest, above every number as an integer: it counts as 0.)
    atomicMax(low, __builtin_bit_cast(uint32_t, fmaxf(amax8(dg), 0.0f)));
    atomicMax(high, __builtin_bit_cast(uint32_t, fmaxf(amax8(du), 0.0f)));
  }
  __syncthreads();
  if (in) {
    uint8_t* const q = a.q + row * a.k + c;
    *reinterpret_cast<u32x2_t*>(q) = fp8_encode8(dg, fp8_scale(__builtin_bit_cast(float, *low), a.pow2 != 0));
    *reinterpret_cast<u32x2_t*>(q + half) = fp8_encode8(du, fp8_scale(__builtin_bit_cast(float, *high), a.pow2 != 0));
  }
  for (int32_t i = threadIdx.x; i < entries; i += blockDim.x) {
    const int64_t at = (int64_t)blockIdx.x * entries + i;
    if (at < (int64_t)a.blocks) a.sf[at] = fp8_scale(__builtin_bit_cast(float, top[i]), a.pow2 != 0);
  }
}

// One 128 x 128 block a workgroup: thread t holds columns 8 (t % 16) .. +7 of rows
// t / 16 + 16 i, so 16 lanes read a row's 128 columns.  The transposed codes leave through
// LDS in pieces of 4 x 4 bytes.
constexpr int kTilePitch = kFp8Block + 4;

template <int DT, bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void k_quantize_fp8_weights(Fp8WeightArgs a) {
  __shared__ float wave_max[kThreads / 64];
  __shared__ __align__(16) uint8_t tile[TRANSPOSED ? kFp8Block * kTilePitch : 4];
  const int tid = threadIdx.x, sub = tid & 15, r0 = tid >> 4;
  const int32_t kb = blockIdx.x, nb = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int32_t n0 = nb * kFp8Block, c = kb * kFp8Block + 8 * sub;
  float v[8][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int32_t r = n0 + r0 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < a.n && c < a.k) load8<DT>(a.w, (e * a.n + r) * (int64_t)a.k + c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  if ((tid & 63) == 0) wave_max[tid >> 6] = m;
  __syncthreads();
  m = wave_max[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) m = fmaxf(m, wave_max[w]);
  const float s = fp8_scale(m, a.pow2 != 0);
  const int64_t nbs = gridDim.y, kbs = gridDim.x;
  if (tid == 0) {
    a.sf[(e * nbs + nb) * kbs + kb] = s;
    if (TRANSPOSED) a.sft[(e * kbs + kb) * nbs + nb] = s;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int32_t r = n0 + r0 + 16 * i;
    const u32x2_t q = fp8_encode8(v[i], s);
    if (r < a.n && c < a.k) *reinterpret_cast<u32x2_t*>(a.q + (e * a.n + r) * (int64_t)a.k + c) = q;
    if (TRANSPOSED) {
      uint32_t* p = reinterpret_cast<uint32_t*>(tile + (r0 + 16 * i) * kTilePitch + 8 * sub);
      p[0] = q[0];
      p[1] = q[1];
    }
  }
  if (!TRANSPOSED) return;
  __syncthreads();
  // Thread t: rows 4 (t % 32) .. +3 of the block, columns 4 (t / 32 + 8 i) .. +3.
  const int n4 = tid & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k4 = (tid >> 5) + 8 * i;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(tile + (4 * n4 + j) * kTilePitch + 4 * k4);
    // Bytes (row j, column c) -> word c, byte j.
    const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);  // columns 0, 1 of rows 0, 1
    const uint32_t hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);  // columns 2, 3
    const uint32_t lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
    const uint32_t hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    const uint32_t o[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                           __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
    const int32_t n = n0 + 4 * n4;
    if (n < a.n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t kk = kb * kFp8Block + 4 * k4 + j;
        if (kk < a.k) *reinterpret_cast<uint32_t*>(a.qt + (e * a.k + kk) * (int64_t)a.n + n) = o[j];
      }
    }
  }
}

template <int DT, int MODE>
hipError_t rows(const Fp8QuantArgs& a, hipStream_t stream) {
  constexpr int B = MODE == kSwigluGrad || DT == kInF32 ? 2 : 4;
  constexpr uint32_t per_group = kThreads / 16 * B;
  const uint32_t grid = (a.blocks + per_group - 1) / per_group;
  hipLaunchKernelGGL((k_quantize_fp8<DT, MODE, B>), dim3(grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int DT>
hipError_t rows_dt(const Fp8QuantArgs& args, hipStream_t stream) {
  Fp8QuantArgs a = args;
  const int32_t pieces = a.k / 16;  // of a half
  if (a.grad && pieces <= kPairThreads) {
    // Whole rows a workgroup: as many as 256 threads hold, or one.
    a.per_piece = FastDiv::of((uint32_t)pieces);
    a.group_rows = pieces <= 128 ? 256 / pieces : 1;
    const int threads = (a.group_rows * pieces + 63) / 64 * 64;
    const int64_t grid = (a.rows + a.group_rows - 1) / a.group_rows;
    if (grid <= kPairGrid) {
      hipLaunchKernelGGL((k_quantize_fp8_swiglu_grad<DT>), dim3((unsigned)grid), dim3(threads), 0, stream, a);
      return hipGetLastError();
    }
  }
  if (a.grad) return rows<DT, kSwigluGrad>(a, stream);
  return a.swiglu ? rows<DT, kSwiglu>(a, stream) : rows<DT, kPlain>(a, stream);
}

template <int DT>
hipError_t weights_dt(const Fp8WeightArgs& a, hipStream_t stream) {
  const dim3 grid((a.k + kFp8Block - 1) / kFp8Block, (a.n + kFp8Block - 1) / kFp8Block, a.experts);
  if (a.qt)
    hipLaunchKernelGGL((k_quantize_fp8_weights<DT, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((k_quantize_fp8_weights<DT, false>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const Fp8QuantArgs& a, hipStream_t stream) {
  if (a.dtype == kInF32) return rows_dt<kInF32>(a, stream);
  return a.dtype == kInF16 ? rows_dt<kInF16>(a, stream) : rows_dt<kInBF16>(a, stream);
}

hipError_t launch_quantize_fp8_weights(const Fp8WeightArgs& a, hipStream_t stream) {
  if (a.dtype == kInF32) return weights_dt<kInF32>(a, stream);
  return a.dtype == kInF16 ? weights_dt<kInF16>(a, stream) : weights_dt<kInBF16>(a, stream);
}

}  // namespace moe_fp4

// Token rows in expert order and the gradients of the way there and back:
//
//   moe_fp4_dispatch           out[r] = x[row_token[r]]          (0 where there is no such token)
//   moe_fp4_dispatch_backward  dx[t] = sum_s dy[token_rows[t][s]]
//   moe_fp4_combine_backward   drows[token_rows[t][s]] = w[t][s] * dout[t]
//                              dw[t][s] = sum_j rows[token_rows[t][s]][j] * dout[t][j]
//
// Bound: bytes (4096 tokens x 8 rows of 12 KB: dispatch 77 us, 5.9 TB/s, its gradient 89 us, 5.1 TB/s;
// combine's gradient 172 us, 5.0 TB/s, into the same results pass after pass 157).  Every result is written once by one thread in a fixed order (a token gathers
// its rows; nothing is scattered with atomics), so the same inputs give the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_token_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// A row is copied in pieces of 16 bytes wherever it starts (the memory takes any alignment of
// whole bytes; 4096 x 8 rows of 12 282 bytes: 105 us, in pieces of two bytes 241), its last
// piece ending with it; rows under 16 bytes go byte by byte.
//
// What the copies cost is the way of the tokens into the XCDs' L2s, as many bytes again as
// the rows written: the slots of a token are far apart.  So a workgroup takes a slice of
// a.lanes pieces of some rows, the XCDs (workgroup b runs on b % 8) have slices of their own,
// and a slice of all tokens stays in an L2 while it is used: 4096 x 8 rows of 12 KB take 77
// us, row by row 106.  With one row a token nothing is read twice, and rows go whole.
typedef u32x4_t any16_t __attribute__((aligned(1)));

__global__ __launch_bounds__(kThreads) void k_dispatch(RowsArgs a) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int side = 64 / a.lanes;  // rows side by side in a wavefront
  const int64_t share = (a.items + kXcds - 1) / kXcds;
  const int64_t first = (blockIdx.x % kXcds) * share, last = min(first + share, a.items);
  for (int64_t item = first + blockIdx.x / kXcds; item < last; item += gridDim.x / kXcds) {
    const int64_t q = a.items <= INT32_MAX ? a.per_segment.div((uint32_t)item) : item / a.segments;
    const int64_t rest = item - q * a.segments;
    const int64_t slice = a.by_slice ? q : rest;
    const int64_t row = ((a.by_slice ? rest : q) * kWaves + wave) * side + lane / a.lanes;
    int64_t c = (slice * a.lanes + (lane & (a.lanes - 1))) * 16;
    if (row >= a.rows || c >= a.row_bytes) continue;
    const int32_t t = a.map[row];
    const bool ok = t >= 0 && t < a.source_rows;
    const char* src = static_cast<const char*>(a.x) + (ok ? t * a.ld_x : 0);
    char* dst = static_cast<char*>(a.out) + row * a.ld_out;
    if (a.row_bytes >= 16) {
      c = min(c, a.row_bytes - 16);
      u32x4_t v = u32x4_t{0, 0, 0, 0};
      if (ok) v = *reinterpret_cast<const any16_t*>(src + c);
      __builtin_nontemporal_store(v, reinterpret_cast<any16_t*>(dst + c));
    } else {
      for (int64_t b = 0; b < a.row_bytes; ++b) dst[b] = ok ? src[b] : (char)0;
    }
  }
}

// Elements of a piece as FP32 and back (rounded to nearest even).
template <int DT> struct Element;
template <> struct Element<kInF32> {
  static constexpr int size = 4;
  typedef float type;
};
template <> struct Element<kInBF16> {
  static constexpr int size = 2;
  typedef __bf16 type;
};
template <> struct Element<kInF16> {
  static constexpr int size = 2;
  typedef _Float16 type;
};

// A wavefront takes 64 pieces of 16 bytes of a row or, where rows have fewer than 33, 64 / lanes
// rows side by side (lanes a power of two); up to kSlots rows of the token are in flight
// together.  A row's last piece ends with it: what two lanes both have they write alike.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_dispatch_backward(RowsArgs a) {
  typedef typename Element<DT>::type elem_t;
  constexpr int N = 16 / Element<DT>::size;  // elements of a piece
  constexpr int kSlots = 8;
  typedef elem_t vec_t __attribute__((ext_vector_type(N)));
  typedef vec_t any_t __attribute__((aligned(sizeof(elem_t))));
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kWaves;
  for (int64_t item = (int64_t)blockIdx.x * kWaves + uniform(threadIdx.x >> 6); item < a.items;
       item += waves) {
    int64_t row, c;  // c: the piece's first element
    if (a.segments > 1) {
      row = a.items <= INT32_MAX ? a.per_segment.div((uint32_t)item) : item / a.segments;
      c = ((item - row * a.segments) * 64 + lane) * N;
    } else {
      row = item * (64 / a.lanes) + lane / a.lanes;
      c = (lane & (a.lanes - 1)) * N;
    }
    if (row >= a.rows || c >= a.cols) continue;
    const bool whole = a.cols >= N;
    if (whole) c = min(c, a.cols - N);
    const int32_t* slots = a.map + row * a.topk;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    for (int32_t s0 = 0; s0 < a.topk; s0 += kSlots) {
      vec_t v[kSlots];
      bool ok[kSlots];
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        const int32_t r = s0 + s < a.topk ? slots[s0 + s] : -1;
        ok[s] = r >= 0 && r < a.source_rows;
        if (!ok[s]) continue;
        const elem_t* src = reinterpret_cast<const elem_t*>(static_cast<const char*>(a.x) + r * a.ld_x);
        if (whole) {
          v[s] = *reinterpret_cast<const any_t*>(src + c);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) v[s][i] = i < a.cols ? src[i] : (elem_t)0.0f;
        }
      }
      // A slot without a row is passed over (no other row is read in its place, whose NaN would
      // count).
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        if (ok[s]) {
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] += (float)v[s][i];
        }
    }
    elem_t* dst = reinterpret_cast<elem_t*>(static_cast<char*>(a.out) + row * a.ld_out);
    vec_t o;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (elem_t)acc[i];
    if (whole) {
      *reinterpret_cast<any_t*>(dst + c) = o;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < a.cols) dst[i] = o[i];
    }
  }
}

// Rows that no slot of their token names: zeroed (64 rows a wavefront).
__device__ __forceinline__ void zero_unnamed(const CombineBackwardArgs& a, int64_t first, int lane) {
  const int64_t r = first + lane;
  bool unnamed = false;
  if (r < a.m_total) {
    const int32_t t = a.row_token[r];
    unnamed = true;
    if (t >= 0 && t < a.num_tokens)
      for (int32_t s = 0; s < a.topk; ++s)
        if (a.token_rows[(int64_t)t * a.topk + s] == r) unnamed = false;
  }
  uint64_t left = __ballot(unnamed);
  while (left) {
    const int64_t row = first + __builtin_ctzll(left);
    left &= left - 1;
    for (int64_t c = 8 * lane; c < a.n; c += 512)
      *reinterpret_cast<u32x4_t*>(a.drows + row * a.ld_drows + c) = u32x4_t{0, 0, 0, 0};
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// One token a workgroup: lane l of wavefront w of W holds U pieces of 8 columns of the token's
// gradient, 8 * (64 * (w + W * u) + l) and on (longer rows take several passes), and G groups
// of W wavefronts share the token's rows, two in flight in each.
template <bool F32, int W, int U, int G, bool HINT>
__global__ __launch_bounds__(W * G * 64) void k_combine_backward(CombineBackwardArgs a) {
  extern __shared__ float part[];  // [W][topk] sums of the wavefronts
  constexpr int S = 2;  // rows of a group in flight together
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6) % W, group = uniform(threadIdx.x >> 6) / W;
  if (blockIdx.x >= a.num_tokens) {
    const int64_t b = (int64_t)blockIdx.x - a.num_tokens;
    zero_unnamed(a, ((b * G + group) * W + wave) * 64, lane);
    return;
  }
  const int64_t t = blockIdx.x;
  const int32_t* slots = a.token_rows + t * a.topk;
  const float* weights = a.token_weights + t * a.topk;
  const __bf16* rows = reinterpret_cast<const __bf16*>(a.rows);
  __bf16* drows = reinterpret_cast<__bf16*>(a.drows);
  for (int64_t base = 0; base < a.n; base += 512 * W * U) {
    float g[U][8];
    bool in[U];
    const auto column = [&](int u) { return base + 8 * (64 * (wave + W * u) + lane); };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = column(u);
      in[u] = c < a.n;  // n % 16 == 0: a lane's 8 columns are all in or all out
#pragma unroll
      for (int i = 0; i < 8; ++i) g[u][i] = 0.0f;
      if (!in[u]) continue;
      if (F32) {
        const float* p = static_cast<const float*>(a.dout) + t * a.ld_dout + c;
        const float4_t lo = *reinterpret_cast<const float4_t*>(p), hi = *reinterpret_cast<const float4_t*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[u][i] = lo[i], g[u][4 + i] = hi[i];
      } else {
        const bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(static_cast<const __bf16*>(a.dout) + t * a.ld_dout + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[u][i] = (float)v[i];
      }
    }
    for (int32_t s0 = S * group; s0 < a.topk; s0 += S * G) {
      bf16x8_t v[S][U];
      int32_t r[S];
      float w[S], dot[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        r[s] = s0 + s < a.topk ? slots[s0 + s] : -1;
        w[s] = s0 + s < a.topk ? weights[s0 + s] : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        r[s] = r[s] < a.m_total ? r[s] : -1;
        if (r[s] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!in[u]) continue;
          const bf16x8_t* p = reinterpret_cast<const bf16x8_t*>(rows + r[s] * a.ld_rows + column(u));
          v[s][u] = HINT ? __builtin_nontemporal_load(p) : *p;
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        dot[s] = 0.0f;
        if (r[s] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!in[u]) continue;
          bf16x8_t o;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[s] += (float)v[s][u][i] * g[u][i];
            o[i] = (__bf16)(w[s] * g[u][i]);
          }
          *reinterpret_cast<bf16x8_t*>(drows + r[s] * a.ld_drows + column(u)) = o;
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s) dot[s] = wave_sum(dot[s]);
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (lane == 0 && s0 + s < a.topk) {
          float* sum = part + wave * a.topk + s0 + s;
          *sum = base == 0 ? dot[s] : *sum + dot[s];
        }
    }
  }
  __syncthreads();
  for (int32_t s = threadIdx.x; s < a.topk; s += W * G * 64) {
    float sum = part[s];
    for (int w = 1; w < W; ++w) sum += part[w * a.topk + s];
    a.dweights[t * a.topk + s] = sum;
  }
}

template <int DT>
hipError_t dispatch_backward_dt(RowsArgs a, hipStream_t stream) {
  const int64_t pieces = (a.row_bytes + 15) / 16;
  a.lanes = 64;
  while (a.lanes > 1 && a.lanes / 2 >= pieces) a.lanes /= 2;
  a.segments = (pieces + 63) / 64;
  if (a.segments <= INT32_MAX) a.per_segment = FastDiv::of((uint32_t)a.segments);
  const int64_t side = 64 / a.lanes;  // rows side by side in a wavefront
  a.items = a.segments > 1 ? a.rows * a.segments : (a.rows + side - 1) / side;
  const int64_t grid = (a.items + kWaves - 1) / kWaves;
  hipLaunchKernelGGL((k_dispatch_backward<DT>), dim3((unsigned)(grid < (1 << 20) ? grid : (1 << 20))),
                     dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <bool F32, int G, bool HINT>
hipError_t combine_backward_dt(const CombineBackwardArgs& a, hipStream_t stream) {
  // One wavefront holds rows of up to 1024 columns.
  const bool one = a.n <= 1024;
  const int w = one ? 1 : 4, waves = w * G;
  const int64_t extra = a.row_token ? (a.m_total + 64 * waves - 1) / (64 * waves) : 0;
  const dim3 grid((unsigned)(a.num_tokens + extra));
  const size_t lds = (size_t)w * a.topk * sizeof(float);
  if (one)
    hipLaunchKernelGGL((k_combine_backward<F32, 1, 2, G, HINT>), grid, dim3(waves * 64), lds, stream, a);
  else
    hipLaunchKernelGGL((k_combine_backward<F32, 4, 3, G, HINT>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

template <bool F32>
hipError_t combine_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  // Four groups a token where one would leave SIMDs without a wavefront (4 tokens, 8 rows of
  // 12 KB: 6.2 us instead of 9.0; 256: 12.4 instead of 13.3; 512: 20.4 instead of 18.5).
  if (a.num_tokens * (a.n <= 1024 ? 1 : 4) <= 1024) return combine_backward_dt<F32, 4, false>(a, stream);
  // Rows beyond half of the last-level cache's 256 MB are read past it: they are read once, and
  // what is written stays for its reader (pass after pass into the same results: 402 MB 157 us
  // instead of 169, 268 MB 94 instead of 112; into new ones 172 and 116 both ways; but 25 MB,
  // still there when they are read, 16.6 us instead of 13.4).
  return a.m_total * a.n * 2 >= 128 << 20 ? combine_backward_dt<F32, 1, true>(a, stream)
                                    : combine_backward_dt<F32, 1, false>(a, stream);
}

}  // namespace

hipError_t launch_dispatch(const RowsArgs& args, hipStream_t stream) {
  RowsArgs a = args;
  const int64_t pieces = (a.row_bytes + 15) / 16;
  a.lanes = 64;
  while (a.lanes > 1 && a.lanes / 2 >= pieces) a.lanes /= 2;
  // By slices where a token has four rows or more (with three, 8192 x 3 of 12 KB, 95 us instead
  // of 93, in another session 95 of 102): slices of which all tokens take half an L2 (4096 x 8 of
  // 12 KB: 77 us, with a whole L2 82), but of two lines at least (16384 x 8 of 2 KB: 57 us, 55
  // with one, 72 with four), and of 1 KB where rows start inside lines, whose halves are written
  // apart (4096 x 8 of 12 282 bytes: 152 us in slices of 512 bytes, 105 of 1 KB).
  a.by_slice = a.rows >= 4 * a.source_rows;
  const uint64_t starts = (uint64_t)reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.ld_out;
  if (a.by_slice && starts % 128 == 0)
    while (a.lanes > 16 && a.source_rows * a.lanes * 16 > 2 << 20) a.lanes /= 2;
  const int64_t slices = (pieces + a.lanes - 1) / a.lanes;
  const int64_t rows = (int64_t)kWaves * (64 / a.lanes);
  const int64_t groups = (a.rows + rows - 1) / rows;
  a.items = slices * groups;
  a.segments = a.by_slice ? groups : slices;
  if (a.items <= INT32_MAX) a.per_segment = FastDiv::of((uint32_t)a.segments);
  const int64_t share = (a.items + kXcds - 1) / kXcds;
  const unsigned grid = kXcds * (unsigned)(share < (1 << 17) ? share : (1 << 17));
  hipLaunchKernelGGL(k_dispatch, dim3(grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const RowsArgs& a, hipStream_t stream) {
  if (a.dtype == kInF32) return dispatch_backward_dt<kInF32>(a, stream);
  if (a.dtype == kInF16) return dispatch_backward_dt<kInF16>(a, stream);
  return dispatch_backward_dt<kInBF16>(a, stream);
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  return a.f32_dout ? combine_backward<true>(a, stream) : combine_backward<false>(a, stream);
}

}  // namespace moe_fp4

// Token rows in expert order and the gradients of the way there and back:
//
//   moe_fp4_dispatch           out[r] = x[row_token[r]]          (0 where there is no such token)
//   moe_fp4_dispatch_backward  dx[t] = sum_s dy[token_rows[t][s]]
//   moe_fp4_combine_backward   drows[token_rows[t][s]] = w[t][s] * dout[t]
//                              dw[t][s] = sum_j rows[token_rows[t][s]][j] * dout[t][j]
//
// Bound: bytes.  Every result is written once by one thread in a fixed order (a token gathers
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

// V bytes of a row.
template <int V> struct Piece;
template <> struct Piece<16> { typedef u32x4_t type; };
template <> struct Piece<8> { typedef u32x2_t type; };
template <> struct Piece<4> { typedef uint32_t type; };
template <> struct Piece<2> { typedef uint16_t type; };
template <> struct Piece<1> { typedef uint8_t type; };

// Where a lane works: a wavefront takes one segment of 64 * U pieces of one row or, where rows
// have fewer than 33 pieces, 64 / lanes rows side by side (lanes a power of two).
struct Place {
  int64_t row;
  int64_t piece;  // first piece; the next ones follow at distance 64
  bool in;
};

template <int U>
__device__ __forceinline__ Place place(int64_t item, const RowsArgs& a, int lane) {
  Place p;
  if (a.segments > 1) {
    const int64_t r = a.items <= INT32_MAX ? a.per_segment.div((uint32_t)item) : item / a.segments;
    p.row = r;
    p.piece = (item - r * a.segments) * (64 * U) + lane;
  } else {
    p.row = item * (64 / a.lanes) + lane / a.lanes;
    p.piece = lane & (a.lanes - 1);
  }
  p.in = p.row < a.rows;
  return p;
}

// Pieces of a row that are V bytes whole; what is left (fewer than V bytes, only with V
// above an element) is copied element by element by the lane whose piece it is.
template <int V, int U>
__global__ __launch_bounds__(kThreads) void k_dispatch(RowsArgs a) {
  typedef typename Piece<V>::type piece_t;
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kWaves;
  const int64_t whole = a.row_bytes / V, all = (a.row_bytes + V - 1) / V;
  for (int64_t item = (int64_t)blockIdx.x * kWaves + uniform(threadIdx.x >> 6); item < a.items;
       item += waves) {
    const Place p = place<U>(item, a, lane);
    if (!p.in) continue;
    const int32_t t = a.map[p.row];
    const bool ok = t >= 0 && t < a.source_rows;
    const char* src = static_cast<const char*>(a.x) + (ok ? t * a.ld_x : 0);
    char* dst = static_cast<char*>(a.out) + p.row * a.ld_out;
    piece_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = p.piece + 64 * u;
      v[u] = piece_t{};
      if (ok && c < whole) v[u] = *reinterpret_cast<const piece_t*>(src + c * V);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = p.piece + 64 * u;
      if (c < whole) {
        __builtin_nontemporal_store(v[u], reinterpret_cast<piece_t*>(dst + c * V));
      } else if (c < all) {
        if (a.esize == 4)
          for (int64_t b = c * V; b < a.row_bytes; b += 4)
            *reinterpret_cast<uint32_t*>(dst + b) = ok ? *reinterpret_cast<const uint32_t*>(src + b) : 0u;
        else if (a.esize == 2)
          for (int64_t b = c * V; b < a.row_bytes; b += 2)
            *reinterpret_cast<uint16_t*>(dst + b) = ok ? *reinterpret_cast<const uint16_t*>(src + b) : (uint16_t)0;
        else
          for (int64_t b = c * V; b < a.row_bytes; ++b) dst[b] = ok ? src[b] : (char)0;
      }
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

template <int DT, int V, int U>
__global__ __launch_bounds__(kThreads) void k_dispatch_backward(RowsArgs a) {
  typedef typename Element<DT>::type elem_t;
  constexpr int N = V / Element<DT>::size;  // elements of a piece
  typedef elem_t vec_t __attribute__((ext_vector_type(N)));
  constexpr int S = 4;  // slots whose rows are in flight together
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kWaves;
  const int64_t whole = a.row_bytes / V, all = (a.row_bytes + V - 1) / V;
  for (int64_t item = (int64_t)blockIdx.x * kWaves + uniform(threadIdx.x >> 6); item < a.items;
       item += waves) {
    const Place p = place<U>(item, a, lane);
    if (!p.in) continue;
    const int32_t* slots = a.map + p.row * a.topk;
    float acc[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = 0.0f;
    for (int32_t s0 = 0; s0 < a.topk; s0 += S) {
      vec_t v[S][U];
      bool ok[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int32_t r = s0 + s < a.topk ? slots[s0 + s] : -1;
        ok[s] = r >= 0 && r < a.source_rows;
        const char* src = static_cast<const char*>(a.x) + (ok[s] ? r * a.ld_x : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = p.piece + 64 * u;
          if (ok[s] && c < whole) v[s][u] = *reinterpret_cast<const vec_t*>(src + c * V);
          else if (ok[s] && c < all) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              v[s][u][i] = c * N + i < a.cols ? reinterpret_cast<const elem_t*>(src)[c * N + i] : (elem_t)0.0f;
          }
        }
      }
      // A slot without a row is passed over (not added as 0: -0 stays -0, and what another row
      // holds plays no part).
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (ok[s]) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (p.piece + 64 * u < all) {
#pragma unroll
              for (int i = 0; i < N; ++i) acc[u][i] += (float)v[s][u][i];
            }
        }
    }
    char* dst = static_cast<char*>(a.out) + p.row * a.ld_out;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = p.piece + 64 * u;
      if (c < whole) {
        vec_t o;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = (elem_t)acc[u][i];
        *reinterpret_cast<vec_t*>(dst + c * V) = o;
      } else if (c < all) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c * N + i < a.cols) reinterpret_cast<elem_t*>(dst)[c * N + i] = (elem_t)acc[u][i];
      }
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

// One token a workgroup of W wavefronts: lane l of wavefront w holds U pieces of 8 columns of
// the token's gradient, 8 * (64 * (w + W * u) + l) and on; longer rows take several passes.
template <bool F32, int W, int U>
__global__ __launch_bounds__(W * 64) void k_combine_backward(CombineBackwardArgs a) {
  extern __shared__ float part[];  // [W][topk] sums of the wavefronts
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  if (blockIdx.x >= a.num_tokens) {
    const int64_t b = (int64_t)blockIdx.x - a.num_tokens;
    zero_unnamed(a, (b * W + wave) * 64, lane);
    return;
  }
  const int64_t t = blockIdx.x;
  const int32_t* slots = a.token_rows + t * a.topk;
  const float* weights = a.token_weights + t * a.topk;
  for (int64_t base = 0; base < a.n; base += 512 * W * U) {
    float g[U][8];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = base + 8 * (64 * (wave + W * u) + lane);
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
        typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
        const bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(static_cast<const __bf16*>(a.dout) + t * a.ld_dout + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[u][i] = (float)v[i];
      }
    }
    for (int32_t s = 0; s < a.topk; ++s) {
      const int32_t r = uniform(slots[s]);
      const bool ok = r >= 0 && r < a.m_total;
      const float w = weights[s];
      float dot = 0.0f;
      if (ok) {
        typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
        bf16x8_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = base + 8 * (64 * (wave + W * u) + lane);
          if (in[u]) v[u] = *reinterpret_cast<const bf16x8_t*>(reinterpret_cast<const __bf16*>(a.rows) + (int64_t)r * a.ld_rows + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!in[u]) continue;
          const int64_t c = base + 8 * (64 * (wave + W * u) + lane);
          bf16x8_t o;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot += (float)v[u][i] * g[u][i];
            o[i] = (__bf16)(w * g[u][i]);
          }
          *reinterpret_cast<bf16x8_t*>(reinterpret_cast<__bf16*>(a.drows) + (int64_t)r * a.ld_drows + c) = o;
        }
      }
      dot = wave_sum(dot);
      if (lane == 0) part[wave * a.topk + s] = base == 0 ? dot : part[wave * a.topk + s] + dot;
    }
  }
  __syncthreads();
  for (int32_t s = threadIdx.x; s < a.topk; s += W * 64) {
    float sum = part[s];
    for (int w = 1; w < W; ++w) sum += part[w * a.topk + s];
    a.dweights[t * a.topk + s] = sum;
  }
}

// The widest piece that every row of both matrices starts at a multiple of.
int piece_bytes(const RowsArgs& a) {
  const uint64_t all = (uint64_t)reinterpret_cast<uintptr_t>(a.x) | (uint64_t)reinterpret_cast<uintptr_t>(a.out) |
                       (uint64_t)a.ld_x | (uint64_t)a.ld_out;
  int v = 16;
  while (v > a.esize && all % v != 0) v /= 2;
  return v;
}

template <int U>
unsigned lay_out(RowsArgs& a, int v) {
  const int64_t pieces = (a.row_bytes + v - 1) / v;
  a.lanes = 64;
  while (a.lanes > 1 && a.lanes / 2 >= pieces) a.lanes /= 2;
  a.segments = (pieces + 64 * U - 1) / (64 * U);
  if (a.segments <= INT32_MAX) a.per_segment = FastDiv::of((uint32_t)a.segments);
  const int64_t side = 64 / a.lanes;  // rows side by side in a wavefront
  a.items = a.segments > 1 ? a.rows * a.segments : (a.rows + side - 1) / side;
  int64_t grid = (a.items + kWaves - 1) / kWaves;
  return (unsigned)(grid < (1 << 20) ? grid : (1 << 20));
}

template <int V>
hipError_t dispatch_v(RowsArgs a, hipStream_t stream) {
  constexpr int U = V == 16 ? 1 : 4;  // 4096 x 8 rows of 12 KB: 108 us; with 2 110, with 4 113
  const unsigned grid = lay_out<U>(a, V);
  hipLaunchKernelGGL((k_dispatch<V, U>), dim3(grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int DT, int V>
hipError_t backward_v(RowsArgs a, hipStream_t stream) {
  constexpr int U = 2;
  const unsigned grid = lay_out<U>(a, V);
  hipLaunchKernelGGL((k_dispatch_backward<DT, V, U>), dim3(grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_dt(const RowsArgs& a, hipStream_t stream) {
  switch (piece_bytes(a)) {
    case 16: return backward_v<DT, 16>(a, stream);
    case 8: return backward_v<DT, 8>(a, stream);
    case 4: return backward_v<DT, 4>(a, stream);
    default: return backward_v<DT, Element<DT>::size>(a, stream);
  }
}

template <bool F32>
hipError_t combine_backward_dt(const CombineBackwardArgs& a, hipStream_t stream) {
  // One wavefront holds rows of up to 1024 columns.
  const bool one = a.n <= 1024;
  const int w = one ? 1 : 4;
  const int64_t extra = a.row_token ? (a.m_total + 64 * w - 1) / (64 * w) : 0;
  const dim3 grid((unsigned)(a.num_tokens + extra));
  const size_t lds = (size_t)w * a.topk * sizeof(float);
  if (one)
    hipLaunchKernelGGL((k_combine_backward<F32, 1, 2>), grid, dim3(64), lds, stream, a);
  else
    hipLaunchKernelGGL((k_combine_backward<F32, 4, 3>), grid, dim3(256), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(const RowsArgs& a, hipStream_t stream) {
  switch (piece_bytes(a)) {
    case 16: return dispatch_v<16>(a, stream);
    case 8: return dispatch_v<8>(a, stream);
    case 4: return dispatch_v<4>(a, stream);
    case 2: return dispatch_v<2>(a, stream);
    default: return dispatch_v<1>(a, stream);
  }
}

hipError_t launch_dispatch_backward(const RowsArgs& a, hipStream_t stream) {
  if (a.dtype == kInF32) return backward_dt<kInF32>(a, stream);
  if (a.dtype == kInF16) return backward_dt<kInF16>(a, stream);
  return backward_dt<kInBF16>(a, stream);
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  return a.f32_dout ? combine_backward_dt<true>(a, stream) : combine_backward_dt<false>(a, stream);
}

}  // namespace moe_fp4

// A whole Mixture-of-Experts feed-forward layer for a few tokens (moe_fp4_ffn), two
// kernels:
//
//   k_ffn_up    h[t, e] = silu(g) * u,  (g, u) = w13_scale[e] * W13[e] x[t]
//   k_ffn_down  out[t]  = residual[t] + sum_e W2[e] (c[t, e] h[t, e]),
//               c[t, e] = w2_scale[e] * (sum of t's routing weights for e)
//
// Every routed expert's weights are read once; experts no token is routed to are not
// read.  Each kernel is bound by its weight stream (2/3 and 1/3 of the layer's
// bytes); with one token, by the chain launch - ids - weights - sum, twice.
//
// Experts in use are found on the device: every workgroup marks the ids in an LDS
// bitmap and takes the r-th marked expert (ascending), so the grid needs only
// min(experts, pairs) ranks and no host knowledge of the routing.  k_ffn_up leaves one record
// per rank (expert, its first row of h, its tokens as a 64-bit mask) for k_ffn_down.
//
// h is kept as the sum of two BF16 values (the first holds h rounded, the second
// the rest rounded: 2^-17 relative), already times c.  BF16 has FP32's range, so no
// activation overflows on the way whatever the layer's type, and the matrix cores
// take both parts as they are.
//
// The sum over a token's experts: every wavefront of k_ffn_down adds its experts'
// results, in ascending order, into a token array of its own in LDS, and the
// wavefronts' arrays are added in wavefront order: no atomics, and the same inputs give the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "few_token_device.h"

namespace moe_fp4 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kWaves = 8;

// What k_ffn_up tells k_ffn_down about one rank.
struct __align__(16) RankRecord {
  int32_t expert;
  int32_t row0;  // first row of h of this expert
  uint32_t tokens_lo, tokens_hi;
};
typedef const RankRecord __attribute__((address_space(4)))* sconst_record;

// Dynamic LDS of k_ffn_up before the sums: ids and weights of every pair, the
// bitmap, and the expert's token list and coefficients.
__host__ __device__ constexpr size_t up_table_bytes(int pairs, int experts) {
  return ((size_t)pairs * 8 + (size_t)((experts + 31) / 32) * 4 + 64 * 8 + 15) / 16 * 16;
}

template <bool F16, int NT, int MT>
__global__ __launch_bounds__(kMaxThreads) void k_ffn_up(FfnArgs a) {
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int pairs = a.tokens * a.topk, words = (a.experts + 31) / 32;
  int32_t* ids = reinterpret_cast<int32_t*>(smem);
  float* wts = reinterpret_cast<float*>(ids + pairs);
  uint32_t* used = reinterpret_cast<uint32_t*>(wts + pairs);
  int32_t* list = reinterpret_cast<int32_t*>(used + words);
  float* coef = reinterpret_cast<float*>(list + 64);
  float4_t* red = reinterpret_cast<float4_t*>(smem + up_table_bytes(pairs, a.experts));

  for (int i = tid; i < words; i += blockDim.x) used[i] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += blockDim.x) {
    const int32_t id = a.ids[p];
    ids[p] = id;
    wts[p] = a.weights[p];
    if (id >= 0 && id < a.experts) atomicOr(&used[id >> 5], 1u << (id & 31));
  }
  __syncthreads();

  // The rank's expert, and the number of experts in use.
  const int32_t rank = blockIdx.y;
  int32_t expert = -1, in_use = 0;
  for (int w0 = 0; w0 < words; w0 += 64) {
    const uint32_t v = w0 + lane < words ? used[w0 + lane] : 0u;
    const int32_t c = __popc(v);
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    const int32_t before = in_use + incl - c;
    const uint64_t hit = __ballot(rank >= before && rank < before + c);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)v, src);
      for (int32_t i = __builtin_amdgcn_readlane(before, src); i < rank; ++i) bits &= bits - 1;
      expert = (w0 + src) * 32 + __ffs((int)bits) - 1;
    }
    in_use += __builtin_amdgcn_readlane(incl, 63);
  }
  if (rank == 0 && blockIdx.x == 0 && tid == 0) *a.ranks = in_use;
  if (expert < 0) return;
  expert = uniform(expert);

  // Its tokens (lane = token; every wavefront finds and writes the same), each with
  // the sum of the token's weights for it, and the first row of h: one row a pair of a
  // lower expert.
  float c = 0.0f;
  bool has = false;
  if (lane < a.tokens)
    for (int s = 0; s < a.topk; ++s)
      if (ids[lane * a.topk + s] == expert) c += wts[lane * a.topk + s], has = true;
  const uint64_t tokens = __ballot(has);
  const int32_t rows = __popcll(tokens);
  int32_t row0 = 0;
  for (int p0 = 0; p0 < pairs; p0 += 64) {
    const int32_t id = p0 + lane < pairs ? ids[p0 + lane] : -1;
    row0 += __popcll(__ballot(id >= 0 && id < expert));
  }
  if (has) {
    const int at = __popcll(tokens & ((1ull << lane) - 1));
    list[at] = lane;
    coef[at] = c * ((sconst_f32)a.w2_scale)[expert];
  }
  if (blockIdx.x == 0 && tid == 0) {
    RankRecord rec;
    rec.expert = expert;
    rec.row0 = row0;
    rec.tokens_lo = (uint32_t)tokens;
    rec.tokens_hi = (uint32_t)(tokens >> 32);
    a.records[rank] = *reinterpret_cast<int4*>(&rec);
  }
  __syncthreads();

  const int32_t inter = a.inter, k = a.hidden;
  const int32_t c0 = blockIdx.x * 8 * NT;  // first intermediate column
  const float scale = ((sconst_f32)a.w13_scale)[expert];
  FewLoop<F16, NT, MT> loop;
  const int64_t wrow = (int64_t)expert * 2 * inter;
  loop.q_rs = make_rsrc(a.w13_q + wrow * (k / 2), (uint32_t)(2 * inter) * (uint32_t)(k / 2));
  loop.s_rs = make_rsrc(a.w13_sf + wrow * (k / 16), (uint32_t)(2 * inter) * (uint32_t)(k / 16));
  loop.x_rs = make_rsrc(a.x, (uint32_t)(((a.tokens - 1) * a.ld_x + k) * 2));
  loop.k = k;
  loop.g = lane >> 4;
  const int r = lane & 15;
  uint32_t row[NT], xoff[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {  // rows 0-7 of a tile: gate; 8-15: the same columns of up
    const int32_t col = c0 + 8 * t + (r & 7);
    row[t] = (uint32_t)((r >> 3) * inter + (col < inter ? col : inter - 1));
  }
  const int32_t steps = (k + kFewStep - 1) / kFewStep;
  const int32_t s0 = uniform(wave * steps / waves), s1 = uniform((wave + 1) * steps / waves);
  const int tile = tid >> 6;
  for (int32_t first = 0; first < rows; first += 16 * MT) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int32_t j = first + 16 * m + r;
      xoff[m] = j < rows ? (uint32_t)(list[j] * a.ld_x * 2) : kOutOfRange;
    }
    float4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (s0 < s1) loop.run(row, xoff, acc, s0, s1);
    if (first > 0) __syncthreads();  // the previous sums have been taken
    put_sums<NT, MT>(red, acc, wave, lane);
    __syncthreads();
    const int32_t j = first + (tile % MT) * 16 + r;
    const int32_t col = c0 + (tile / MT) * 8 + 4 * ((lane >> 4) & 1);
    if (tile < NT * MT && lane < 32 && j < rows && col < inter) {
      const float4_t gate = take_sum(red, NT * MT, tile, lane, waves);
      const float4_t up = take_sum(red, NT * MT, tile, lane + 32, waves);
      const float cf = coef[j];
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = silu(gate[i] * scale) * (up[i] * scale) * cf;
        hi[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
        // A value that is not finite has no rest.
        const float rest = v - bf16_value(hi[i]);
        lo[i] = __builtin_bit_cast(uint16_t, (__bf16)(rest - rest == 0.0f ? rest : 0.0f));
      }
      // Row layout: per 8 columns, 16 bytes of first parts, then 16 of rests.
      char* p = a.h + ((int64_t)(row0 + j) * inter + (col & ~7)) * 4 + (col & 4) * 2;
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
      *reinterpret_cast<u32x2_t*>(p + 16) = u32x2_t{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
    }
  }
}

// One wavefront's unit: 256 elements of K of one expert.
template <int NT>
struct DownRegs {
  WeightStep<NT> w;
  u32x4_t h[16];  // (first parts, rests) of elements 8j .. 8j+7
};

template <bool F16, int NT>
__global__ __launch_bounds__(kMaxThreads) void k_ffn_down(FfnArgs a) {
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  constexpr int kCols = 16 * NT;
  float* sums = reinterpret_cast<float*>(smem);  // [wave][token][kCols]
  int32_t* list = reinterpret_cast<int32_t*>(sums + (size_t)waves * a.tokens * kCols) + wave * 64;
  float* mysum = sums + (size_t)wave * a.tokens * kCols;
  const int32_t k = a.inter;
  const int32_t n0 = blockIdx.x * kCols;
  for (int i = lane; i < a.tokens * kCols; i += 64) mysum[i] = 0.0f;

  uint32_t row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int32_t c = n0 + 16 * t + r;
    row[t] = (uint32_t)(c < a.hidden ? c : a.hidden - 1);
  }
  const rsrc_t h_rs = make_rsrc(a.h, (uint32_t)(a.tokens * a.topk) * (uint32_t)k * 4u);
  const int32_t steps = (k + kFewStep - 1) / kFewStep;
  const int32_t units = ((sconst_i32)a.ranks)[0] * steps;
  const int32_t u0 = uniform((int32_t)((int64_t)wave * units / waves));
  const int32_t u1 = uniform((int32_t)((int64_t)(wave + 1) * units / waves));

  auto load_h = [&](u32x4_t (&h)[16], const RankRecord& rec, int32_t step, int32_t first) {
    const LaneK lk = lane_k(step, g, k);
    const int32_t rows = __popc(rec.tokens_lo) + __popc(rec.tokens_hi);
    const int32_t j = first + r;
    const uint32_t off = j < rows ? (uint32_t)(rec.row0 + j) * (uint32_t)k * 4u : kOutOfRange;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      h[i] = __builtin_amdgcn_raw_buffer_load_b128(h_rs, off + (uint32_t)(4 * lk.k + 16 * i), 0, 0);
  };
  auto record = [&](int32_t u) {
    const int32_t rank = u / steps;
    const sconst_i32 p = (sconst_i32)(const void*)(a.records + rank);
    RankRecord rec;
    rec.expert = p[0], rec.row0 = p[1], rec.tokens_lo = (uint32_t)p[2], rec.tokens_hi = (uint32_t)p[3];
    return rec;
  };
  auto load = [&](DownRegs<NT>& d, int32_t u) {
    const RankRecord rec = record(u);
    const int32_t step = u % steps;
    const int64_t wrow = (int64_t)rec.expert * a.hidden;
    const rsrc_t q_rs = make_rsrc(a.w2_q + wrow * (k / 2), (uint32_t)a.hidden * (uint32_t)(k / 2));
    const rsrc_t s_rs = make_rsrc(a.w2_sf + wrow * (k / 16), (uint32_t)a.hidden * (uint32_t)(k / 16));
    load_weights<NT>(d.w, q_rs, s_rs, row, k, lane_k(step, g, k).k);
    load_h(d.h, rec, step, 0);
  };
  auto compute = [&](DownRegs<NT>& d, int32_t u) {
    const RankRecord rec = record(u);
    const int32_t step = u % steps;
    const uint64_t tokens = (uint64_t)rec.tokens_hi << 32 | rec.tokens_lo;
    const int32_t rows = __popcll(tokens);
    const int32_t skip = lane_k(step, g, k).skip;
    const bool tail = (step + 1) * kFewStep > k;
    if (tokens >> lane & 1) list[__popcll(tokens & ((1ull << lane) - 1))] = lane;
    __builtin_amdgcn_wave_barrier();
    if (tail) drop_scales<NT>(d.w, skip);
    for (int32_t first = 0; first < rows; first += 16) {
      if (first > 0) load_h(d.h, rec, step, first);
      if (tail) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < 4 * skip) d.h[i] = u32x4_t{0, 0, 0, 0};
      }
      float4_t acc[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      for_operands<false, NT, 0>(d.w, [&](int j, int t, u32x4_t w) {
        acc[t] = mfma16<false>(w, d.h[2 * j], acc[t]);
        acc[t] = mfma16<false>(w, d.h[2 * j + 1], acc[t]);
      });
      if (first + r < rows) {
        float* p = mysum + list[first + r] * kCols + 4 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<float4_t*>(p + 16 * t) += acc[t];
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  if (u0 < u1) {
    DownRegs<NT> da, db;
    load(da, u0);
    int32_t u = u0;
    for (; u + 2 < u1; u += 2) {
      load(db, u + 1);
      compute(da, u);
      load(da, u + 2);
      compute(db, u + 1);
    }
    if (u + 1 < u1) {
      load(db, u + 1);
      compute(da, u);
      compute(db, u + 1);
    } else {
      compute(da, u);
    }
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * kCols; i += blockDim.x) {
    const int32_t t = i / kCols, col = n0 + i % kCols;
    if (col >= a.hidden) continue;
    float v = sums[i];
    for (int w = 1; w < waves; ++w) v += sums[(size_t)w * a.tokens * kCols + i];
    if (a.residual)
      v += value16<F16>(static_cast<const uint16_t*>(a.residual)[t * a.ld_res + col]);
    store_as(a.out, t * a.ldo + col, v, a.out_dtype);
  }
}

template <bool F16, int NT, int MT>
hipError_t launch_up(const FfnArgs& a, int waves, hipStream_t stream) {
  const int pairs = a.tokens * a.topk;
  const dim3 grid((a.inter + 8 * NT - 1) / (8 * NT), pairs < a.experts ? pairs : a.experts);
  const size_t lds = up_table_bytes(pairs, a.experts) + (size_t)waves * NT * MT * 64 * 16;
  hipLaunchKernelGGL((k_ffn_up<F16, NT, MT>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

template <bool F16, int NT>
hipError_t launch_down(const FfnArgs& a, int waves, hipStream_t stream) {
  const size_t lds = (size_t)waves * (a.tokens * 16 * NT + 64) * 4;
  const dim3 grid((a.hidden + 16 * NT - 1) / (16 * NT));
  hipLaunchKernelGGL((k_ffn_down<F16, NT>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_typed(const FfnArgs& a, hipStream_t stream) {
  hipError_t err = a.tokens > 16 ? launch_up<F16, 1, 2>(a, kWaves, stream)
                                 : launch_up<F16, 1, 1>(a, kWaves, stream);
  if (err != hipSuccess) return err;
  return launch_down<F16, 1>(a, kWaves, stream);
}

}  // namespace

hipError_t launch_ffn(const FfnArgs& a, hipStream_t stream) {
  return a.x_f16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace moe_fp4

// FP8 block-scaled grouped product for few rows (moe_grouped_gemm_fp8):
//
//   out[r][j] = sum_b sa[src(r)][b] sw[e][j / 128][b] sum_{k in block b} A[src(r)][k] W[e][j][k]
//
// Bound: the weight stream, one byte an element (up to some 64 rows give few operations a
// byte; one token of 256 experts of 512 x 6144, top-8: 8.2 to 8.4 us, most of it latency: the offsets,
// then two rounds of weights, since a wavefront has three of its six blocks in flight).  A
// workgroup owns 16 NT weight rows and up to 16 MT activation rows of one expert;
// its W wavefronts split K, each with D blocks of 128 in flight in registers, and their sums
// meet in LDS in wavefront order (no atomics: the same inputs give the same bits).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_fp8.h"

namespace moe_fp4 {
namespace {

// 32 bytes of a row: the 16-byte pieces g and 4 + g of a block.  (Two loads share a 128-byte
// line: the hint that drops a line after its first use made dense 6144 x 6144 of one token four
// microseconds slower, 14.7 to 10.9 then.)
__device__ __forceinline__ i32x8_t load32(rsrc_t rs, uint32_t off0, uint32_t off1, int32_t k) {
  const u32x4_t lo = __builtin_amdgcn_raw_buffer_load_b128(rs, off0, k, 0);
  const u32x4_t hi = __builtin_amdgcn_raw_buffer_load_b128(rs, off1, k, 0);
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <int NT, int MT>
struct Stage {
  i32x8_t w[NT], a[MT];
  float sa[MT];
  float sw;
};

template <int NT, int MT, int W, int D>
__global__ __launch_bounds__(W * 64) void k_gemm_fp8_stream(Fp8GemmArgs p) {
  extern __shared__ __align__(16) char smem[];
  const Fp8Item it = fp8_item<W * 64>(p, 16 * MT, 16 * NT, INT32_MAX);
  if (it.rows <= 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int32_t k = p.k, kbs = p.k_blocks, n = p.n;

  const rsrc_t w_rs = make_rsrc(p.w_q + (int64_t)it.e * n * k, (uint32_t)n * (uint32_t)k);
  const float* w_sf = p.w_sf + ((int64_t)it.e * p.n_blocks + it.n0 / kFp8Block) * kbs;
  // Without a row index the tile's rows follow each other: offsets from its first row.
  const int64_t base = p.a_row_index ? 0 : it.row0;
  const int64_t a_rows = p.a_row_index ? p.a_rows : it.rows;
  const rsrc_t a_rs = make_rsrc(p.a_q + base * k, (uint32_t)(a_rows * k));
  const rsrc_t s_rs = make_rsrc(p.a_sf + base * kbs, (uint32_t)(a_rows * kbs * 4));
  uint32_t w_off[NT], a_off[MT], s_off[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int32_t row = it.n0 + 16 * t + r;
    w_off[t] = (uint32_t)(row < n ? row : n - 1) * (uint32_t)k + 16u * g;
  }
  int32_t src[MT];  // on its way while the first weights are asked for
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int32_t row = it.row0 + min(16 * m + r, it.rows - 1);
    src[m] = p.a_row_index ? p.a_row_index[row] : row;
  }

  float4_t acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int32_t b0 = uniform(wave * kbs / W), b1 = uniform((wave + 1) * kbs / W);
  Stage<NT, MT> st[D];
  // Pieces past k (the last block's) and blocks past the share read zeros.
  auto load_w = [&](Stage<NT, MT>& s, int32_t b) {
    const bool in = b < b1;
    const bool ok0 = in && b * kFp8Block + 16 * g < k, ok1 = in && b * kFp8Block + 64 + 16 * g < k;
    const int32_t kk = uniform(b * kFp8Block);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      s.w[t] = load32(w_rs, ok0 ? w_off[t] : kOutOfRange, ok1 ? w_off[t] + 64 : kOutOfRange, kk);
  };
  auto load_a = [&](Stage<NT, MT>& s, int32_t b) {
    const bool in = b < b1;
    const bool ok0 = in && b * kFp8Block + 16 * g < k, ok1 = in && b * kFp8Block + 64 + 16 * g < k;
    const int32_t kk = uniform(b * kFp8Block);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s.a[m] = load32(a_rs, ok0 ? a_off[m] : kOutOfRange, ok1 ? a_off[m] + 64 : kOutOfRange, kk);
      s.sa[m] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(s_rs, in ? s_off[m] : kOutOfRange, uniform(b * 4), 0));
    }
    s.sw = ((sconst_f32)w_sf)[in ? b : b1 - 1];
  };
  auto multiply = [&](const Stage<NT, MT>& s) {
    float scale[MT], by[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) by[m] = scale[m] = s.sa[m] * s.sw;
    fp8_drop_far(by);
    Half32 a[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) a[m] = fp8_widen(s.a[m]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const Half32 w = fp8_widen(s.w[t]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float4_t d = fp8_block_product(w, a[m]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][m][i] = __builtin_fmaf(d[i], by[m], acc[t][m][i]);
      }
    }
    if (fp8_some_far(scale))
      fp8_add_far<NT, MT, true, false>(acc, s.a, s.sa, s.sw, scale, [&](int t) { return s.w[t]; });
  };
  if (b0 < b1) {
#pragma unroll
    for (int d = 0; d < D; ++d) load_w(st[d], b0 + d);
    __builtin_amdgcn_sched_barrier(0);
    const int32_t last = (int32_t)p.a_rows - 1;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t row = (uint32_t)(p.a_row_index ? min(max(src[m], 0), last) : src[m] - (int32_t)base);
      a_off[m] = row * (uint32_t)k + 16u * g;
      s_off[m] = row * (uint32_t)kbs * 4u;
    }
#pragma unroll
    for (int d = 0; d < D; ++d) load_a(st[d], b0 + d);
    for (int32_t b = b0; b < b1; b += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (b + d < b1) multiply(st[d]);
        load_w(st[d], b + d + D);
        load_a(st[d], b + d + D);
      }
    }
  }

  // Sums of the wavefronts, each with its tiles in LDS.
  float4_t* const sums = reinterpret_cast<float4_t*>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[((wave * NT + t) * MT + m) * 64 + lane] = acc[t][m];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * MT * 64; i += W * 64) {
    float4_t v = sums[i];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w * NT * MT * 64 + i];
    const int tile = i >> 6, t = tile / MT, m = tile % MT, l = i & 63;
    const int32_t row = 16 * m + (l & 15), col = it.n0 + 16 * t + 4 * (l >> 4);
    if (row < it.rows && col < n) fp8_store4(p, (int64_t)it.row0 + row, col, v);
  }
}

// Items of 16 x 16 a launch may have (fewer than 2^32 threads).
constexpr int64_t kFewItems = 1 << 21;

template <int NT, int MT, int W, int D>
hipError_t launch(Fp8GemmArgs p, hipStream_t stream) {
  p.n_tiles = (p.n + 16 * NT - 1) / (16 * NT);
  const unsigned grid = (unsigned)((fp8_most_items(p, 16 * MT) + 7) / 8 * 8);
  hipLaunchKernelGGL((k_gemm_fp8_stream<NT, MT, W, D>), dim3(grid), dim3(W * 64), W * NT * MT * 1024, stream, p);
  return hipGetLastError();
}

}  // namespace

// The few-row kernel for fewer than four rows an expert, and while tiles of 64 x 128 would leave
// CUs without work (its K split keeps them loading).  Both sides in us: 256 experts of 512 x 6144,
// top-8, one token 8.4 against 30 with tiles, four 20 and 30, eight 36 and 33, 32 (one row an
// expert) 80 and 77, 64 107 and 93, 96 (three rows) 120 and 112, 512 (16 rows) 199 and 141; 64 experts
// of 2048 x 4096, one row 60 and 77, three 85 and 97, four 90 and 99, 16 134 and 108; dense
// 8192 x 6144, 64 rows (128 tiles) 23.4 and 33, 128 rows (192 tiles) 31.6 and 31.5.  (Where the
// tiles are ahead below four rows, the few-row kernel's exact sums are kept.)
hipError_t launch_grouped_gemm_fp8(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t experts = p.m_total < p.experts ? p.m_total : p.experts;
  const int64_t rows = (p.m_total + p.experts - 1) / p.experts;
  const int64_t tiles = (p.m_total / 64 + experts) * ((p.n + 127) / 128);
  const bool few = p.m_total < 4 * (int64_t)p.experts || tiles < 96 || (rows <= 64 && tiles < 224);
  const int64_t items = (p.m_total / 16 + experts) * ((p.n + 15) / 16);
  if (!few || items > kFewItems) return launch_gemm_fp8_tiled(p, stream);
  // Activation rows of a workgroup: 16, 32, or 64 above that (dense 8192 x 6144, 32 rows: 17.8 with
  // room for 32, 18.7 for 16; 64 rows: 23.4 with 32, 31.6 with 64; 128 rows: 31.6 with 64, 41 with 32).
  if (rows > 64) return launch<4, 4, 4, 1>(p, stream);
  if (rows > 32) return launch<4, 2, 4, 1>(p, stream);
  if (rows > 16) return launch<2, 2, 4, 2>(p, stream);
  // Weight rows: 16 while that is about one item a CU, 32 up to twice that, else 64 (one token
  // above: 8.4, 10.9 and 16; dense 6144 x 6144, 16 rows: 17.8, 13.4 and 18.4; four tokens above:
  // 24.1, 20.3 and 19.9).
  if (items <= 320) return launch<1, 1, 8, 3>(p, stream);
  return items <= 640 ? launch<2, 1, 8, 2>(p, stream) : launch<4, 1, 4, 2>(p, stream);
}

}  // namespace moe_fp4

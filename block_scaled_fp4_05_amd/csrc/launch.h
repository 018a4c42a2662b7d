// Internal interface between the C-ABI layer (api.cpp) and the kernel
// launchers.  Arguments reaching a launcher have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe_fp4 {

// Quantiser: enqueue the kernels of moe_fp4_quantize on `stream`.
hipError_t launch_quantize(const void* x, int in_dtype, int64_t rows, int64_t k, int64_t ld_x,
                           uint8_t* q, uint8_t* sf, float* tensor_scale, int dynamic,
                           hipStream_t stream);

// Tile shapes of the grouped GEMM.  Rows per work item = 16 * m_blocks; output
// columns per wavefront = 16 * n_blocks; a workgroup holds `waves` wavefronts,
// each working on its own item; one pipeline stage covers 256 * k_sub
// elements of K.
struct GemmTile {
  int m_blocks;
  int n_blocks;
  int waves;
  int k_sub;
  int lds_scales;  // weight block scales staged through LDS (needs k % 2048 == 0)
  int tiled;       // workgroup-tiled kernel, operands shared in LDS: 1 = 128 x 128
                   // items (grouped_gemm_tiled.hip); 2 = 256 x 256 items
                   // (grouped_gemm_big.hip) for experts of kBigRows rows or more
                   // and the per-wave kernel for the rest; 3 = 256 x 256 for all;
                   // 4 = 48 x 512 items (grouped_gemm_mid.hip) for every expert;
                   // 5, 6, 7 = splits by expert size over the large tile, the
                   // 48 x 512 items and the per-wave items (launch_grouped_gemm)
  int f8 = 0;      // 256 x 256 items: split K by scale block on the FP8 MFMA
                   // instead of dequantising to FP16 (MOE_FP4_TILE "256x256f8")
};

constexpr int kKStep = 256;  // K granularity the kernels require

// Packed weight layout (moe_fp4_pack_weights): K elements per granule, and the
// bytes of one 16-row x granule block.  Rows are grouped by 64.
__host__ __device__ constexpr int32_t packed_granule(int64_t k) { return k % 512 == 0 ? 512 : 256; }
__host__ __device__ constexpr int32_t packed_block_bytes(int32_t granule) { return 8 * granule; }
constexpr int kPackRows = 64;

// Token-order combine of routed rows (combine.hip).
struct CombineArgs {
  const uint16_t* rows;  // BF16 [m_total][ld_rows]
  int64_t ld_rows;
  int64_t m_total;
  const int32_t* token_rows;     // [num_tokens][topk], row index or < 0
  const float* token_weights;    // [num_tokens][topk]
  int32_t topk;
  int64_t num_tokens;
  int64_t n;
  const float* residual;  // FP32 [num_tokens][ld_res] or NULL
  int64_t ld_res;
  void* out;              // BF16 or FP32 [num_tokens][ldo]
  int64_t ldo;
  int32_t f32_out;
};
hipError_t launch_combine(const CombineArgs& args, hipStream_t stream);

// Rearrange weight codes between the row-major and the packed layout.
hipError_t launch_repack(const uint8_t* src, uint8_t* dst, int32_t num_experts, int64_t n,
                         int64_t k, bool to_packed, hipStream_t stream);

// The tile used for a problem with these sizes; `env` (may be NULL) is the
// value of MOE_FP4_TILE ("MxN" or "MxNxK": M rows per item, N columns per
// wave, K elements per pipeline stage; a trailing 'r' keeps the weight block
// scales in registers instead of staging them through LDS).
GemmTile choose_tile(int32_t num_experts, int64_t m_total, int64_t n, int64_t k, const char* env);

// LDS bytes a workgroup of the grouped GEMM uses for `num_experts` experts.
int64_t gemm_lds_bytes(const GemmTile& t, int32_t num_experts);

// The tile `t`, or the per-wave tile of 64-row items when t is a workgroup
// tile whose output rows (128 or 256 of them, ldo BF16 values apart) would not
// fit one store resource: every kernel addresses one item's output rows with
// 32-bit buffer offsets below 2^31 - 4096 bytes.
GemmTile fit_output_range(const GemmTile& t, int64_t k, int64_t ldo);

// Rows of output one item of tile t covers.
int32_t item_rows(const GemmTile& t);

// With MOE_FP4_LOG set (to anything but "0"), print the tile an entry point
// chose to stderr, once per change of entry point, sizes or tile.
void log_tile(const char* entry, int32_t num_experts, int64_t m_total, int64_t n, int64_t k,
              int64_t ldo, const GemmTile& t);

struct GemmArgs {
  const uint8_t* a_q;
  const uint8_t* a_sf;
  const float* a_scale;
  const int32_t* a_row_index;
  const uint8_t* w_q;
  const uint8_t* w_sf;
  const float* w_scale;
  const int32_t* offsets;
  uint16_t* out;
  int64_t a_rows;
  int64_t m_total;
  int64_t n;
  int64_t k;
  int64_t ldo;
  int32_t num_experts;
  int32_t n_tiles;   // ceil(n / (16 * n_blocks))
  int32_t w_packed;  // w_q is in the packed layout
  // Experts this launch covers, by row count: rows_lo <= rows, and rows <
  // rows_hi unless rows_hi is 0 (so a zeroed GemmArgs covers every expert).
  // Launches over disjoint ranges write disjoint output rows.
  int32_t rows_lo;
  int32_t rows_hi;
  // Finalize epilogue only (moe_grouped_gemm_fp4_finalize): routed row r adds
  // row_weight[r] * its result into FP32 row out_token[r] of fin_out.
  const int32_t* out_token;
  const float* row_weight;
  float* fin_out;
  int64_t fin_ldo;
  int64_t num_tokens;
  // SwiGLU epilogue only (moe_grouped_gemm_fp4_swiglu): the NVFP4 intermediate
  // h_q [m_total][n/4], h_sf [m_total][n/32] at the static tensor scale *h_scale.
  uint8_t* h_q;
  uint8_t* h_sf;
  const float* h_scale;
};

hipError_t launch_grouped_gemm(const GemmArgs& args, const GemmTile& tile, hipStream_t stream);

// The same GEMM with the finalize epilogue (grouped_gemm_finalize.hip): per-wave
// kernels with 64-column items only.
hipError_t launch_grouped_gemm_finalize(const GemmArgs& args, const GemmTile& tile,
                                        hipStream_t stream);

// The same GEMM with the SwiGLU + NVFP4 epilogue (grouped_gemm_swiglu.hip):
// per-wave kernels, items of 32 intermediate columns (4 row blocks).
hipError_t launch_grouped_gemm_swiglu(const GemmArgs& args, const GemmTile& tile,
                                      hipStream_t stream);

// Workgroup-tiled kernel (grouped_gemm_tiled.hip): 128 x 128 items, 4 waves.
hipError_t launch_grouped_gemm_tiled(const GemmArgs& args, hipStream_t stream);
size_t tiled_lds(int32_t num_experts);

// Large-tile kernel (grouped_gemm_big.hip): 256 x 256 items, 8 waves of 128 x 64;
// f8: the split-K-by-scale-block FP8 variant.
hipError_t launch_grouped_gemm_big(const GemmArgs& args, bool f8, hipStream_t stream);
size_t big_lds(int32_t num_experts);

// Workgroup kernel for experts of a few dozen rows (grouped_gemm_mid.hip): 48 x 512
// items, 8 waves of 64 columns each, activations shared in LDS; needs k % 512 == 0.
// Sets its own n_tiles.
hipError_t launch_grouped_gemm_mid(const GemmArgs& args, hipStream_t stream);
size_t mid_lds(int32_t num_experts);

// Output types of the few-token products (the values of MOE_FP4_OUT_*).
constexpr int32_t kFewOutF32 = 1;
constexpr int32_t kFewOutF16 = 2;

// Few-token linear layer (linear.hip); sizes checked so that every byte offset
// into x and the weights is below 2^31.
struct LinearArgs {
  const void* x;  // BF16 or FP16 [m][ld_x]
  int64_t ld_x;
  const uint8_t* w_q;
  const uint8_t* w_sf;
  const float* w_scale;  // one float
  const void* residual;  // x's type [m][ld_res] or NULL
  int64_t ld_res;
  void* out;
  int64_t ldo;
  int32_t m, n, k;
  int32_t x_f16, swiglu, out_dtype;
};
hipError_t launch_linear(const LinearArgs& args, hipStream_t stream);

// Few-token Mixture-of-Experts layer (ffn.hip).
constexpr int32_t kFfnMaxTokens = 64;  // a wavefront's lanes stand for the tokens
constexpr int32_t kFfnMaxPairs = 2048;  // ids and weights of every pair in LDS
struct FfnArgs {
  const void* x;  // BF16 or FP16 [tokens][ld_x]
  int64_t ld_x;
  const int32_t* ids;    // [tokens][topk]
  const float* weights;  // [tokens][topk]
  const uint8_t* w13_q;
  const uint8_t* w13_sf;
  const float* w13_scale;
  const uint8_t* w2_q;
  const uint8_t* w2_sf;
  const float* w2_scale;
  const void* residual;  // x's type [tokens][ld_res] or NULL
  int64_t ld_res;
  void* out;
  int64_t ldo;
  int32_t tokens, topk, experts, hidden, inter;
  int32_t x_f16, out_dtype;
  // Workspace: the number of experts in use, a 16-byte record for each, and the
  // intermediate rows, 4 bytes a value.
  int32_t* ranks;
  int4* records;
  char* h;
};
hipError_t launch_ffn(const FfnArgs& args, hipStream_t stream);

// Router (route.hip).
constexpr int32_t kRouteF32 = 1, kRouteF16 = 2;  // the values of MOE_FP4_IN_*
constexpr int32_t kRouteMaxPerLane = 16;   // experts a lane holds
constexpr int32_t kRouteOneBlock = 64;     // tokens of the single-launch form
constexpr int32_t kRouteNarrow = 4096;     // tokens from which 16 lanes rank a token
constexpr int32_t kRouteMaxBlock = 512;    // tokens of a block: 16 words of marks an expert
struct RouteArgs {
  const void* logits;  // [tokens][ld] of dtype
  int64_t ld;
  const float* bias;  // [experts] or NULL
  int32_t* ids;       // [tokens][topk]
  float* weights;     // [tokens][topk]
  int32_t* offsets;   // [experts + 1]
  int32_t* row_token;   // [tokens * topk]
  int32_t* token_rows;  // [tokens][topk]
  uint16_t* counts;     // workspace: [blocks][counts_pitch]
  int32_t dtype, tokens, experts, topk, num_groups, topk_groups;
  int32_t sigmoid, renormalize;
  int32_t token_lanes;   // lanes that rank one token: 16 or 64
  int32_t group_lanes;   // lanes of one group, a power of two
  int32_t wide;          // lanes read their logits in 16-byte pieces
  int32_t per_lane;      // consecutive experts of one lane
  int32_t block_tokens;  // tokens of a block
  int32_t counts_pitch;  // experts rounded up to 8
};
hipError_t launch_route(const RouteArgs& args, hipStream_t stream);

// LDS a workgroup may use on gfx950.
constexpr size_t kLdsBytes = 160 * 1024;

// Rows from which an expert takes the 256 x 256 tile when the problem is split
// by expert size (GemmTile.tiled == 2).  Measured on the Zipf prefill shard
// (256 experts, 4096 tokens top-8): 64 -> 397 us, 96 -> 303, 128 -> 316,
// 256 -> 352, 384 -> 359.
constexpr int32_t kBigRows = 96;

// Rows from which an expert takes the 48 x 512 items when per-wave items take
// the smaller experts (GemmTile.tiled 6 and 7): one 16-row block gains nothing
// from sharing the weight conversion.
constexpr int32_t kMidRows = 17;

}  // namespace moe_fp4

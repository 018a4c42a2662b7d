// C ABI of the NVFP4 MoE grouped GEMM library (declared in include/moe_fp4.h).
//
// Every entry point validates its arguments on the host before touching the
// HIP runtime, so an argument that fails here never reaches a launch, and one
// that passes here always launches: there is no second check that could reject
// a configuration the first one accepted (the failure mode described on
// "Peering into the CUTLASS SharedStorage", section "Why This Message Was
// Written", where can_implement passed and initialize then failed).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/moe_fp4.h"
#include "api_checks.h"
#include "launch.h"

using moe_fp4::aligned;
using moe_fp4::GemmArgs;
using moe_fp4::GemmTile;
using moe_fp4::overlap;

namespace {

constexpr int kAbiVersion = 2;
// The work-list tables (8 bytes per expert) live in LDS beside each kernel's
// own buffers (at most 68 KB); 8192 experts keep every kernel within 160 KB.
constexpr int32_t kMaxExperts = 8192;

int check_gemm_shape(int32_t num_experts, int64_t m_total, int64_t n, int64_t k) {
  if (num_experts < 1 || m_total < 0 || n < 1 || k < 1) return MOE_FP4_ERR_SHAPE;
  if (num_experts > kMaxExperts) return MOE_FP4_ERR_UNSUPPORTED;
  if (n % 16 != 0 || k % moe_fp4::kKStep != 0) return MOE_FP4_ERR_UNSUPPORTED;
  // Row-index entries are addressed with 32-bit byte offsets.
  if (n > INT32_MAX / 2 || m_total > INT32_MAX / 4 - 1024) return MOE_FP4_ERR_UNSUPPORTED;
  // One expert's packed weights are addressed with 32-bit buffer offsets.
  if (k / 2 > ((int64_t)INT32_MAX - 4096) / n) return MOE_FP4_ERR_UNSUPPORTED;
  // The work-list counts items in int32: bound the largest possible count.
  const int64_t max_mtiles = m_total / 16 + (m_total < num_experts ? m_total : num_experts);
  const int64_t n_tiles = (n + 31) / 32;
  // Items and items x pipeline stages are counted in int32.
  if (max_mtiles * n_tiles * (k / moe_fp4::kKStep) >= (int64_t)INT32_MAX)
    return MOE_FP4_ERR_UNSUPPORTED;
  return MOE_FP4_OK;
}

// Byte sizes the few-token products address with 32-bit buffer offsets.
constexpr int64_t kFewLimit = (int64_t)INT32_MAX - 4096;

// Rows of a few-token linear call: 16 of them per workgroup row of the grid.
constexpr int64_t kFewMaxRows = 16 * 65535;

bool few_dtypes_ok(int x_dtype, int out_dtype) {
  return (x_dtype == MOE_FP4_IN_BF16 || x_dtype == MOE_FP4_IN_FP16) &&
         (out_dtype == MOE_FP4_OUT_BF16 || out_dtype == MOE_FP4_OUT_FP32 ||
          out_dtype == MOE_FP4_OUT_FP16);
}

int64_t out_size(int out_dtype) { return out_dtype == MOE_FP4_OUT_FP32 ? 4 : 2; }

bool few_k_ok(int64_t k) { return k % 16 == 0 && k >= 64; }

bool few_rows_aligned(const void* x, int64_t ld_x, const void* residual, const void* out,
                      int out_dtype) {
  return aligned(x, 16) && ld_x % 8 == 0 && aligned(residual, 2) && aligned(out, out_size(out_dtype));
}

// x within 32-bit offsets, and the extents of residual and out representable.
bool few_rows_fit(int64_t m, int64_t ld_x, int64_t ld_res, int64_t ldo) {
  return ld_x <= kFewLimit / 2 / m && ld_res <= INT64_MAX / 8 / m && ldo <= INT64_MAX / 8 / m;
}

// The residual and the output are the same rows (each element is read by the thread
// that writes it) or share no byte.
bool residual_ok(const void* residual, int64_t ld_res, int x_dtype, const void* out, int out_dtype,
                 int64_t ldo, int64_t m, int64_t cols) {
  if (!residual) return true;
  const bool same_type = (x_dtype == MOE_FP4_IN_BF16 && out_dtype == MOE_FP4_OUT_BF16) ||
                         (x_dtype == MOE_FP4_IN_FP16 && out_dtype == MOE_FP4_OUT_FP16);
  if (residual == out && same_type && (m == 1 || ld_res == ldo)) return true;
  return !overlap(out, ((m - 1) * ldo + cols) * out_size(out_dtype), residual,
                  ((m - 1) * ld_res + cols) * 2);
}

// End of the records in the layer's workspace: the count and one record per expert
// that `pairs` slots can name.
size_t ffn_records_end(int64_t pairs, int32_t experts) {
  return 16 + 16 * (size_t)(pairs < experts ? pairs : experts);
}

// Tokens of a router block: four, or as many more as keep the blocks, whose counts every
// block reads, at 256 or below (up to the largest block).  256 experts, top-8: 2048 tokens 11.2 us
// (128 blocks 10.9, 512 blocks 17.9), 8192 13.8 (14.8, 20.3), 16384 16.9 (22.1, 23.8).  Above 131072
// tokens, where the block no longer grows, the counts read grow with the square of the tokens.
int64_t route_block(int64_t tokens) {
  int64_t b = 4;
  while (b < moe_fp4::kRouteMaxBlock && b * 256 < tokens) b *= 2;
  return b;
}

int32_t route_pitch(int32_t experts) { return (experts + 7) / 8 * 8; }

}  // namespace

extern "C" {

int moe_fp4_abi_version(void) { return kAbiVersion; }

const char* moe_fp4_status_string(int status) {
  switch (status) {
    case MOE_FP4_OK: return "ok";
    case MOE_FP4_ERR_NULL: return "a required pointer is NULL";
    case MOE_FP4_ERR_SHAPE: return "a size is out of range or sizes are inconsistent";
    case MOE_FP4_ERR_ALIGN: return "a pointer or leading dimension is misaligned";
    case MOE_FP4_ERR_UNSUPPORTED: return "valid arguments outside what the kernels support";
    case MOE_FP4_ERR_HIP: return "the HIP runtime reported an error";
    case MOE_FP4_ERR_ARG: return "an enumerated argument has an unknown value, or buffers overlap";
    default: return "unknown status";
  }
}

int64_t moe_fp4_stage_bytes(int64_t bm, int64_t bn, int64_t bk) {
  if (bm < 1 || bn < 1 || bk < 16 || bk % 16 != 0) return -1;
  // Packed FP4 (half a byte per element) plus one E4M3 byte per 16 elements,
  // for the A tile (bm x bk) and the B tile (bn x bk).
  const int64_t a = bm * bk / 2 + bm * (bk / 16);
  const int64_t b = bn * bk / 2 + bn * (bk / 16);
  return a + b;
}

int moe_fp4_quantize(const void* x, int in_dtype, int64_t rows, int64_t k, int64_t ld_x,
                     uint8_t* q, uint8_t* sf, float* tensor_scale, int scale_mode,
                     void* stream) {
  if (in_dtype != MOE_FP4_IN_BF16 && in_dtype != MOE_FP4_IN_FP32) return MOE_FP4_ERR_ARG;
  if (scale_mode != MOE_FP4_SCALE_STATIC && scale_mode != MOE_FP4_SCALE_DYNAMIC)
    return MOE_FP4_ERR_ARG;
  if (!tensor_scale) return MOE_FP4_ERR_NULL;
  if (rows < 0 || k <= 0 || k % 16 != 0 || ld_x < k) return MOE_FP4_ERR_SHAPE;
  if (rows > 0 && (!x || !q || !sf)) return MOE_FP4_ERR_NULL;
  const int64_t esize = in_dtype == MOE_FP4_IN_BF16 ? 2 : 4;
  if (!aligned(tensor_scale, 4)) return MOE_FP4_ERR_ALIGN;
  if (rows > 0 && (!aligned(x, 16) || (ld_x * esize) % 16 != 0 || !aligned(q, 8)))
    return MOE_FP4_ERR_ALIGN;
  if (rows > 0 && (rows > INT64_MAX / k)) return MOE_FP4_ERR_SHAPE;
  // x's extent, ((rows - 1) * ld_x + k) * esize bytes, must be representable.
  if (rows > 1 && (ld_x > (INT64_MAX / esize - k) / (rows - 1))) return MOE_FP4_ERR_SHAPE;
  // The four buffers must be distinct: the dynamic mode hands the amax pass's
  // partial values to the quantise pass inside q while x is still being read,
  // and writes the tensor scale while q is being read.
  if (rows > 0) {
    const int64_t xb = ((rows - 1) * ld_x + k) * esize, qb = rows * (k / 2), sb = rows * (k / 16);
    if (overlap(x, xb, q, qb) || overlap(x, xb, sf, sb) || overlap(x, xb, tensor_scale, 4) ||
        overlap(q, qb, sf, sb) || overlap(q, qb, tensor_scale, 4) ||
        overlap(sf, sb, tensor_scale, 4))
      return MOE_FP4_ERR_ARG;
  }
  hipError_t err = moe_fp4::launch_quantize(x, in_dtype, rows, k, ld_x, q, sf, tensor_scale,
                                            scale_mode == MOE_FP4_SCALE_DYNAMIC ? 1 : 0,
                                            reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

size_t moe_grouped_gemm_fp4_workspace_size(int32_t num_experts, int64_t m_total, int64_t n,
                                           int64_t k) {
  (void)num_experts, (void)m_total, (void)n, (void)k;
  // Every kernel builds its work list in LDS from the device offsets.
  return 0;
}

int moe_grouped_gemm_fp4_plan(int32_t num_experts, int64_t m_total, int64_t n, int64_t k,
                              moe_fp4_gemm_plan* plan) {
  if (!plan) return MOE_FP4_ERR_NULL;
  const int s = check_gemm_shape(num_experts, m_total, n, k);
  if (s != MOE_FP4_OK) return s;
  const GemmTile t = moe_fp4::choose_tile(num_experts, m_total, n, k, getenv("MOE_FP4_TILE"));
  plan->tile_m = 16 * t.m_blocks;
  plan->tile_n = 16 * t.n_blocks;
  plan->k_step = (t.tiled == 4 || t.tiled == 6) ? 256 : t.tiled ? 64 : moe_fp4::kKStep * t.k_sub;
  plan->waves_per_group = t.waves;
  plan->lds_bytes = moe_fp4::gemm_lds_bytes(t, num_experts);
  return MOE_FP4_OK;
}

}  // extern "C"

namespace {

int grouped_gemm(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale, int64_t a_rows,
                 const int32_t* a_row_index, const uint8_t* w_q, const uint8_t* w_sf,
                 const float* w_scale, const int32_t* expert_offsets, int32_t num_experts,
                 int64_t m_total, int64_t n, int64_t k, uint16_t* out, int64_t ldo,
                 void* stream, bool packed) {
  if (!a_q || !a_sf || !a_scale || !w_q || !w_sf || !w_scale || !expert_offsets || !out)
    return MOE_FP4_ERR_NULL;
  if (num_experts < 1 || m_total < 0 || n < 1 || k < 1 || ldo < n || a_rows < 0)
    return MOE_FP4_ERR_SHAPE;
  if (!a_row_index && a_rows < m_total) return MOE_FP4_ERR_SHAPE;
  if (m_total > 0 && a_rows < 1) return MOE_FP4_ERR_SHAPE;
  const int s = check_gemm_shape(num_experts, m_total, n, k);
  if (s != MOE_FP4_OK) return s;
  if (!aligned(a_q, 16) || !aligned(a_sf, 16) || !aligned(w_q, 16) || !aligned(w_sf, 16) ||
      !aligned(out, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(expert_offsets, 4) || (a_row_index && !aligned(a_row_index, 4)) || ldo % 8 != 0)
    return MOE_FP4_ERR_ALIGN;
  // Activations and one item's output rows are addressed with 32-bit buffer
  // offsets as well.
  if (a_rows > ((int64_t)INT32_MAX - 4096) / (k / 2) || ldo > (1 << 23))
    return MOE_FP4_ERR_UNSUPPORTED;
  const GemmTile t = moe_fp4::fit_output_range(
      moe_fp4::choose_tile(num_experts, m_total, n, k, getenv("MOE_FP4_TILE")), k, ldo);
  // Packed weights fix the per-wavefront K step to the layout's granule.
  if (packed && !t.tiled &&
      (t.n_blocks != 4 || t.k_sub != moe_fp4::packed_granule(k) / moe_fp4::kKStep))
    return MOE_FP4_ERR_UNSUPPORTED;
  moe_fp4::log_tile(packed ? "moe_grouped_gemm_fp4_packed" : "moe_grouped_gemm_fp4", num_experts,
                    m_total, n, k, ldo, t);
  if (m_total == 0) return MOE_FP4_OK;
  GemmArgs p = {};
  p.a_q = a_q;
  p.a_sf = a_sf;
  p.a_scale = a_scale;
  p.a_row_index = a_row_index;
  p.w_q = w_q;
  p.w_sf = w_sf;
  p.w_scale = w_scale;
  p.offsets = expert_offsets;
  p.out = out;
  p.a_rows = a_rows;
  p.m_total = m_total;
  p.n = n;
  p.k = k;
  p.ldo = ldo;
  p.num_experts = num_experts;
  p.n_tiles = (int32_t)((n + 16 * t.n_blocks - 1) / (16 * t.n_blocks));
  p.w_packed = packed ? 1 : 0;
  hipError_t err = moe_fp4::launch_grouped_gemm(p, t, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

int grouped_gemm_finalize(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                          int64_t a_rows, const int32_t* a_row_index, const uint8_t* w_q,
                          const uint8_t* w_sf, const float* w_scale, int w_packed,
                          const int32_t* expert_offsets, int32_t num_experts, int64_t m_total,
                          int64_t n, int64_t k, const int32_t* out_token,
                          const float* row_weight, float* out, int64_t ldo, int64_t num_tokens,
                          void* stream) {
  if (!a_q || !a_sf || !a_scale || !w_q || !w_sf || !w_scale || !expert_offsets || !out ||
      !out_token || !row_weight)
    return MOE_FP4_ERR_NULL;
  if (w_packed != 0 && w_packed != 1) return MOE_FP4_ERR_ARG;
  if (num_experts < 1 || m_total < 0 || n < 1 || k < 1 || ldo < n || a_rows < 0 || num_tokens < 1)
    return MOE_FP4_ERR_SHAPE;
  if (!a_row_index && a_rows < m_total) return MOE_FP4_ERR_SHAPE;
  if (m_total > 0 && a_rows < 1) return MOE_FP4_ERR_SHAPE;
  const int s = check_gemm_shape(num_experts, m_total, n, k);
  if (s != MOE_FP4_OK) return s;
  if (!aligned(a_q, 16) || !aligned(a_sf, 16) || !aligned(w_q, 16) || !aligned(w_sf, 16) ||
      !aligned(out, 4) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(expert_offsets, 4) || (a_row_index && !aligned(a_row_index, 4)) ||
      !aligned(out_token, 4) || !aligned(row_weight, 4))
    return MOE_FP4_ERR_ALIGN;
  if (a_rows > ((int64_t)INT32_MAX - 4096) / (k / 2)) return MOE_FP4_ERR_UNSUPPORTED;
  // The token rows are addressed with 32-bit byte offsets.
  if (num_tokens > (int64_t)INT32_MAX / 4 || ldo > ((int64_t)INT32_MAX - 4096) / 4 / num_tokens)
    return MOE_FP4_ERR_UNSUPPORTED;
  GemmTile t = moe_fp4::choose_tile(num_experts, m_total, n, k, getenv("MOE_FP4_TILE"));
  // The finalize epilogue runs in the per-wave kernel with 64-column items;
  // experts large enough for the workgroup tile take four row blocks per item.
  if (t.tiled) t = GemmTile{4, 4, 4, k % 512 == 0 ? 2 : 1, k % 2048 == 0 ? 1 : 0, 0};
  if (t.n_blocks != 4 || t.k_sub > 2) return MOE_FP4_ERR_UNSUPPORTED;
  if (w_packed && t.k_sub != moe_fp4::packed_granule(k) / moe_fp4::kKStep)
    return MOE_FP4_ERR_UNSUPPORTED;
  moe_fp4::log_tile("moe_grouped_gemm_fp4_finalize", num_experts, m_total, n, k, ldo, t);
  if (m_total == 0) return MOE_FP4_OK;
  GemmArgs p = {};
  p.a_q = a_q;
  p.a_sf = a_sf;
  p.a_scale = a_scale;
  p.a_row_index = a_row_index;
  p.w_q = w_q;
  p.w_sf = w_sf;
  p.w_scale = w_scale;
  p.offsets = expert_offsets;
  p.out = nullptr;
  p.a_rows = a_rows;
  p.m_total = m_total;
  p.n = n;
  p.k = k;
  p.ldo = n;
  p.num_experts = num_experts;
  p.n_tiles = (int32_t)((n + 63) / 64);
  p.w_packed = w_packed;
  p.out_token = out_token;
  p.row_weight = row_weight;
  p.fin_out = out;
  p.fin_ldo = ldo;
  p.num_tokens = num_tokens;
  hipError_t err =
      moe_fp4::launch_grouped_gemm_finalize(p, t, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

int grouped_gemm_swiglu(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                        int64_t a_rows, const int32_t* a_row_index, const uint8_t* w_q,
                        const uint8_t* w_sf, const float* w_scale, int w_packed,
                        const int32_t* expert_offsets, int32_t num_experts, int64_t m_total,
                        int64_t n, int64_t k, const float* h_scale, uint8_t* h_q, uint8_t* h_sf,
                        void* stream) {
  if (!a_q || !a_sf || !a_scale || !w_q || !w_sf || !w_scale || !expert_offsets || !h_scale ||
      !h_q || !h_sf)
    return MOE_FP4_ERR_NULL;
  if (w_packed != 0 && w_packed != 1) return MOE_FP4_ERR_ARG;
  if (num_experts < 1 || m_total < 0 || n < 1 || k < 1 || a_rows < 0) return MOE_FP4_ERR_SHAPE;
  if (!a_row_index && a_rows < m_total) return MOE_FP4_ERR_SHAPE;
  if (m_total > 0 && a_rows < 1) return MOE_FP4_ERR_SHAPE;
  const int s = check_gemm_shape(num_experts, m_total, n, k);
  if (s != MOE_FP4_OK) return s;
  if (!aligned(a_q, 16) || !aligned(a_sf, 16) || !aligned(w_q, 16) || !aligned(w_sf, 16) ||
      !aligned(h_q, 16) || !aligned(h_sf, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(h_scale, 4) || !aligned(expert_offsets, 4) ||
      (a_row_index && !aligned(a_row_index, 4)))
    return MOE_FP4_ERR_ALIGN;
  if (a_rows > ((int64_t)INT32_MAX - 4096) / (k / 2)) return MOE_FP4_ERR_UNSUPPORTED;
  // The intermediate has n/2 columns in whole 16-element blocks; packed weights
  // are read in whole 64-row groups, which must not straddle the gate/up halves.
  if (n % 32 != 0 || (w_packed && (n / 2) % 64 != 0)) return MOE_FP4_ERR_UNSUPPORTED;
  // The outputs are written while the inputs are still being read.
  const int64_t hq_bytes = m_total * (n / 4), hs_bytes = m_total * (n / 32);
  if (overlap(h_q, hq_bytes, h_sf, hs_bytes) || overlap(h_q, hq_bytes, a_q, a_rows * (k / 2)) ||
      overlap(h_q, hq_bytes, a_sf, a_rows * (k / 16)) ||
      overlap(h_sf, hs_bytes, a_q, a_rows * (k / 2)) ||
      overlap(h_sf, hs_bytes, a_sf, a_rows * (k / 16)))
    return MOE_FP4_ERR_ARG;
  GemmTile t = moe_fp4::choose_tile(num_experts, m_total, n, k, getenv("MOE_FP4_TILE"));
  // Per-wave kernels with 4 row blocks (32 gate + 32 up rows) per item;
  // experts large enough for the workgroup tile take four row blocks of rows.
  if (t.tiled) t = GemmTile{4, 4, 4, k % 512 == 0 ? 2 : 1, k % 2048 == 0 ? 1 : 0, 0};
  if (t.n_blocks != 4 || t.k_sub > 2) return MOE_FP4_ERR_UNSUPPORTED;
  if (w_packed && t.k_sub != moe_fp4::packed_granule(k) / moe_fp4::kKStep)
    return MOE_FP4_ERR_UNSUPPORTED;
  moe_fp4::log_tile("moe_grouped_gemm_fp4_swiglu", num_experts, m_total, n, k, n, t);
  if (m_total == 0) return MOE_FP4_OK;
  GemmArgs p = {};
  p.a_q = a_q;
  p.a_sf = a_sf;
  p.a_scale = a_scale;
  p.a_row_index = a_row_index;
  p.w_q = w_q;
  p.w_sf = w_sf;
  p.w_scale = w_scale;
  p.offsets = expert_offsets;
  p.a_rows = a_rows;
  p.m_total = m_total;
  p.n = n;
  p.k = k;
  p.ldo = n;
  p.num_experts = num_experts;
  p.n_tiles = (int32_t)((n / 2 + 31) / 32);
  p.w_packed = w_packed;
  p.h_q = h_q;
  p.h_sf = h_sf;
  p.h_scale = h_scale;
  hipError_t err =
      moe_fp4::launch_grouped_gemm_swiglu(p, t, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

int repack(const uint8_t* src, uint8_t* dst, int32_t num_experts, int64_t n, int64_t k,
           void* stream, bool to_packed) {
  if (!src || !dst) return MOE_FP4_ERR_NULL;
  if (num_experts < 1 || n < 1 || k < 1) return MOE_FP4_ERR_SHAPE;
  if (n % 16 != 0 || k % moe_fp4::kKStep != 0) return MOE_FP4_ERR_UNSUPPORTED;
  if (n > INT32_MAX / 2 || k / 2 > ((int64_t)INT32_MAX - 4096) / n) return MOE_FP4_ERR_UNSUPPORTED;
  if (!aligned(src, 16) || !aligned(dst, 16)) return MOE_FP4_ERR_ALIGN;
  const uintptr_t bytes = (uintptr_t)num_experts * (uintptr_t)n * (uintptr_t)(k / 2);
  const uintptr_t a = reinterpret_cast<uintptr_t>(src), b = reinterpret_cast<uintptr_t>(dst);
  if (a < b + bytes && b < a + bytes) return MOE_FP4_ERR_ARG;  // overlapping buffers
  hipError_t err = moe_fp4::launch_repack(src, dst, num_experts, n, k, to_packed,
                                          reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

}  // namespace

extern "C" {

int moe_grouped_gemm_fp4(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                         int64_t a_rows, const int32_t* a_row_index,
                         const uint8_t* w_q, const uint8_t* w_sf, const float* w_scale,
                         const int32_t* expert_offsets, int32_t num_experts,
                         int64_t m_total, int64_t n, int64_t k,
                         uint16_t* out, int64_t ldo, void* stream) {
  return grouped_gemm(a_q, a_sf, a_scale, a_rows, a_row_index, w_q, w_sf, w_scale,
                      expert_offsets, num_experts, m_total, n, k, out, ldo, stream, false);
}

int moe_grouped_gemm_fp4_packed(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                                int64_t a_rows, const int32_t* a_row_index,
                                const uint8_t* w_packed, const uint8_t* w_sf,
                                const float* w_scale, const int32_t* expert_offsets,
                                int32_t num_experts, int64_t m_total, int64_t n, int64_t k,
                                uint16_t* out, int64_t ldo, void* stream) {
  return grouped_gemm(a_q, a_sf, a_scale, a_rows, a_row_index, w_packed, w_sf, w_scale,
                      expert_offsets, num_experts, m_total, n, k, out, ldo, stream, true);
}

int moe_grouped_gemm_fp4_finalize(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                                  int64_t a_rows, const int32_t* a_row_index,
                                  const uint8_t* w_q, const uint8_t* w_sf, const float* w_scale,
                                  int w_packed, const int32_t* expert_offsets,
                                  int32_t num_experts, int64_t m_total, int64_t n, int64_t k,
                                  const int32_t* out_token, const float* row_weight, float* out,
                                  int64_t ldo, int64_t num_tokens, void* stream) {
  return grouped_gemm_finalize(a_q, a_sf, a_scale, a_rows, a_row_index, w_q, w_sf, w_scale,
                               w_packed, expert_offsets, num_experts, m_total, n, k, out_token,
                               row_weight, out, ldo, num_tokens, stream);
}

int moe_grouped_gemm_fp4_swiglu(const uint8_t* a_q, const uint8_t* a_sf, const float* a_scale,
                                int64_t a_rows, const int32_t* a_row_index,
                                const uint8_t* w_q, const uint8_t* w_sf, const float* w_scale,
                                int w_packed, const int32_t* expert_offsets, int32_t num_experts,
                                int64_t m_total, int64_t n, int64_t k, const float* h_scale,
                                uint8_t* h_q, uint8_t* h_sf, void* stream) {
  return grouped_gemm_swiglu(a_q, a_sf, a_scale, a_rows, a_row_index, w_q, w_sf, w_scale,
                             w_packed, expert_offsets, num_experts, m_total, n, k, h_scale, h_q,
                             h_sf, stream);
}

int moe_fp4_combine(const uint16_t* rows, int64_t ld_rows, int64_t m_total,
                    const int32_t* token_rows, const float* token_weights, int32_t topk,
                    int64_t num_tokens, int64_t n, const float* residual, int64_t ld_res,
                    void* out, int out_dtype, int64_t ldo, void* stream) {
  if (out_dtype != MOE_FP4_OUT_BF16 && out_dtype != MOE_FP4_OUT_FP32) return MOE_FP4_ERR_ARG;
  if (!token_rows || !token_weights || !out || (m_total > 0 && !rows)) return MOE_FP4_ERR_NULL;
  if (m_total < 0 || num_tokens < 0 || topk < 1 || n < 1 || ldo < n || (m_total > 0 && ld_rows < n) ||
      (residual && ld_res < n))
    return MOE_FP4_ERR_SHAPE;
  const int64_t esize = out_dtype == MOE_FP4_OUT_FP32 ? 4 : 2;
  if ((m_total > 0 && (!aligned(rows, 16) || ld_rows % 8 != 0)) || !aligned(out, 16) ||
      (ldo * esize) % 16 != 0 || !aligned(token_rows, 4) || !aligned(token_weights, 4) ||
      (residual && (!aligned(residual, 16) || ld_res % 4 != 0)))
    return MOE_FP4_ERR_ALIGN;
  if (n % 16 != 0) return MOE_FP4_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)INT32_MAX - 4096;
  if (m_total > lim / 2 / (ld_rows > 0 ? ld_rows : 1) || num_tokens > lim / esize / ldo ||
      (residual && num_tokens > lim / 4 / ld_res) || num_tokens > lim / topk)
    return MOE_FP4_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOE_FP4_OK;
  moe_fp4::CombineArgs a;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.m_total = m_total;
  a.token_rows = token_rows;
  a.token_weights = token_weights;
  a.topk = topk;
  a.num_tokens = num_tokens;
  a.n = n;
  a.residual = residual;
  a.ld_res = ld_res;
  a.out = out;
  a.ldo = ldo;
  a.f32_out = out_dtype == MOE_FP4_OUT_FP32 ? 1 : 0;
  hipError_t err = moe_fp4::launch_combine(a, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

int moe_fp4_linear(const void* x, int x_dtype, int64_t m, int64_t ld_x, const uint8_t* w_q,
                   const uint8_t* w_sf, const float* w_scale, int64_t n, int64_t k, int swiglu,
                   const void* residual, int64_t ld_res, void* out, int out_dtype, int64_t ldo,
                   void* stream) {
  if (!few_dtypes_ok(x_dtype, out_dtype) || (swiglu != 0 && swiglu != 1)) return MOE_FP4_ERR_ARG;
  if (!w_q || !w_sf || !w_scale || (m > 0 && (!x || !out))) return MOE_FP4_ERR_NULL;
  const int64_t cols = swiglu ? n / 2 : n;
  if (m < 0 || n < 1 || k < 1 || (swiglu && (n % 2 != 0 || residual))) return MOE_FP4_ERR_SHAPE;
  if (m > 0 && (ld_x < k || ldo < cols || (residual && ld_res < n))) return MOE_FP4_ERR_SHAPE;
  if (!aligned(w_q, 16) || !aligned(w_sf, 4) || !aligned(w_scale, 4)) return MOE_FP4_ERR_ALIGN;
  if (m > 0 && !few_rows_aligned(x, ld_x, residual, out, out_dtype)) return MOE_FP4_ERR_ALIGN;
  if (!few_k_ok(k) || k / 2 > kFewLimit / n || m > kFewMaxRows) return MOE_FP4_ERR_UNSUPPORTED;
  if (m == 0) return MOE_FP4_OK;
  if (!few_rows_fit(m, ld_x, residual ? ld_res : 0, ldo)) return MOE_FP4_ERR_UNSUPPORTED;
  const int64_t ob = ((m - 1) * ldo + cols) * out_size(out_dtype);
  if (overlap(out, ob, x, ((m - 1) * ld_x + k) * 2) || overlap(out, ob, w_q, n * (k / 2)) ||
      overlap(out, ob, w_sf, n * (k / 16)) || overlap(out, ob, w_scale, 4) ||
      !residual_ok(residual, ld_res, x_dtype, out, out_dtype, ldo, m, cols))
    return MOE_FP4_ERR_ARG;
  moe_fp4::LinearArgs a;
  a.x = x;
  a.ld_x = ld_x;
  a.w_q = w_q;
  a.w_sf = w_sf;
  a.w_scale = w_scale;
  a.residual = residual;
  a.ld_res = ld_res;
  a.out = out;
  a.ldo = ldo;
  a.m = (int32_t)m;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.x_f16 = x_dtype == MOE_FP4_IN_FP16 ? 1 : 0;
  a.swiglu = swiglu;
  a.out_dtype = out_dtype;
  hipError_t err = moe_fp4::launch_linear(a, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

size_t moe_fp4_ffn_workspace_size(int64_t tokens, int32_t topk, int32_t num_experts, int64_t inter) {
  if (tokens < 1 || topk < 1 || num_experts < 1 || inter < 1) return 0;
  if (tokens > moe_fp4::kFfnMaxTokens || topk > moe_fp4::kFfnMaxPairs / tokens ||
      inter > kFewLimit / 4 / (tokens * topk))
    return 0;
  return ffn_records_end(tokens * topk, num_experts) + (size_t)(tokens * topk * inter * 4);
}

int moe_fp4_ffn(const void* x, int x_dtype, int64_t tokens, int64_t ld_x, const int32_t* ids,
                const float* weights, int32_t topk, const uint8_t* w13_q, const uint8_t* w13_sf,
                const float* w13_scale, const uint8_t* w2_q, const uint8_t* w2_sf,
                const float* w2_scale, int32_t num_experts, int64_t hidden, int64_t inter,
                const void* residual, int64_t ld_res, void* out, int out_dtype, int64_t ldo,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!few_dtypes_ok(x_dtype, out_dtype)) return MOE_FP4_ERR_ARG;
  if (!w13_q || !w13_sf || !w13_scale || !w2_q || !w2_sf || !w2_scale) return MOE_FP4_ERR_NULL;
  if (tokens > 0 && (!x || !ids || !weights || !out)) return MOE_FP4_ERR_NULL;
  if (tokens < 0 || topk < 1 || num_experts < 1 || hidden < 1 || inter < 1) return MOE_FP4_ERR_SHAPE;
  if (tokens > 0 && (ld_x < hidden || ldo < hidden || (residual && ld_res < hidden)))
    return MOE_FP4_ERR_SHAPE;
  if (!aligned(w13_q, 16) || !aligned(w13_sf, 4) || !aligned(w13_scale, 4) || !aligned(w2_q, 16) ||
      !aligned(w2_sf, 4) || !aligned(w2_scale, 4))
    return MOE_FP4_ERR_ALIGN;
  if (tokens > 0 && (!few_rows_aligned(x, ld_x, residual, out, out_dtype) || !aligned(ids, 4) ||
                     !aligned(weights, 4) || !aligned(workspace, 16)))
    return MOE_FP4_ERR_ALIGN;
  if (!few_k_ok(hidden) || !few_k_ok(inter) || num_experts > kMaxExperts ||
      inter > kFewLimit / hidden)
    return MOE_FP4_ERR_UNSUPPORTED;
  // Code bytes of one expert, multiples of 128: every expert's codes are aligned.
  const int64_t w13_b = hidden * inter, w2_b = hidden * inter / 2;
  if (tokens == 0) return MOE_FP4_OK;
  if (!few_rows_fit(tokens, ld_x, residual ? ld_res : 0, ldo)) return MOE_FP4_ERR_UNSUPPORTED;
  const size_t need = moe_fp4_ffn_workspace_size(tokens, topk, num_experts, inter);
  if (need == 0) return MOE_FP4_ERR_UNSUPPORTED;
  if (!workspace) return MOE_FP4_ERR_NULL;
  if (workspace_bytes < need) return MOE_FP4_ERR_SHAPE;
  const int64_t ob = ((tokens - 1) * ldo + hidden) * out_size(out_dtype);
  const int64_t pb = tokens * topk * 4, xb = ((tokens - 1) * ld_x + hidden) * 2;
  struct {
    const void* p;
    int64_t bytes;
  } const in[] = {{x, xb},
                  {ids, pb},
                  {weights, pb},
                  {w13_q, num_experts * w13_b},
                  {w13_sf, num_experts * (w13_b / 8)},
                  {w13_scale, num_experts * (int64_t)4},
                  {w2_q, num_experts * w2_b},
                  {w2_sf, num_experts * (w2_b / 8)},
                  {w2_scale, num_experts * (int64_t)4}};
  for (const auto& b : in)
    if (overlap(workspace, (int64_t)need, b.p, b.bytes) || overlap(out, ob, b.p, b.bytes))
      return MOE_FP4_ERR_ARG;
  if (overlap(workspace, (int64_t)need, out, ob) ||
      (residual && overlap(workspace, (int64_t)need, residual, ((tokens - 1) * ld_res + hidden) * 2)) ||
      !residual_ok(residual, ld_res, x_dtype, out, out_dtype, ldo, tokens, hidden))
    return MOE_FP4_ERR_ARG;
  moe_fp4::FfnArgs a;
  a.x = x;
  a.ld_x = ld_x;
  a.ids = ids;
  a.weights = weights;
  a.w13_q = w13_q;
  a.w13_sf = w13_sf;
  a.w13_scale = w13_scale;
  a.w2_q = w2_q;
  a.w2_sf = w2_sf;
  a.w2_scale = w2_scale;
  a.residual = residual;
  a.ld_res = ld_res;
  a.out = out;
  a.ldo = ldo;
  a.tokens = (int32_t)tokens;
  a.topk = topk;
  a.experts = num_experts;
  a.hidden = (int32_t)hidden;
  a.inter = (int32_t)inter;
  a.x_f16 = x_dtype == MOE_FP4_IN_FP16 ? 1 : 0;
  a.out_dtype = out_dtype;
  char* ws = static_cast<char*>(workspace);
  a.ranks = reinterpret_cast<int32_t*>(ws);
  a.records = reinterpret_cast<int4*>(ws + 16);
  a.h = ws + ffn_records_end(tokens * topk, num_experts);
  hipError_t err = moe_fp4::launch_ffn(a, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

size_t moe_fp4_route_workspace_size(int64_t tokens, int32_t num_experts) {
  if (tokens <= moe_fp4::kRouteOneBlock || num_experts < 1 || num_experts > 1024 ||
      tokens > kFewLimit)
    return 0;
  const int64_t block = route_block(tokens);
  return (size_t)((tokens + block - 1) / block) * route_pitch(num_experts) * 2;
}

int moe_fp4_route(const void* logits, int dtype, int64_t tokens, int32_t num_experts, int64_t ld,
                  int score, const float* bias, int renormalize, int32_t topk, int32_t num_groups,
                  int32_t topk_groups, int32_t* ids, float* weights, int32_t* offsets,
                  int32_t* row_token, int32_t* token_rows, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (dtype != MOE_FP4_IN_BF16 && dtype != MOE_FP4_IN_FP32 && dtype != MOE_FP4_IN_FP16)
    return MOE_FP4_ERR_ARG;
  if ((score != MOE_FP4_SCORE_SOFTMAX && score != MOE_FP4_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1) || (bias && score != MOE_FP4_SCORE_SIGMOID))
    return MOE_FP4_ERR_ARG;
  if (!offsets || (tokens > 0 && (!logits || !ids || !weights || !row_token || !token_rows)))
    return MOE_FP4_ERR_NULL;
  if (tokens < 0 || num_experts < 1 || num_groups < 1 || num_experts % num_groups != 0 ||
      topk_groups < 1 || topk_groups > num_groups || topk < 1 ||
      topk > (int64_t)(num_experts / num_groups) * topk_groups || (tokens > 0 && ld < num_experts))
    return MOE_FP4_ERR_SHAPE;
  const int64_t esize = dtype == MOE_FP4_IN_FP32 ? 4 : 2;
  if (!aligned(logits, esize) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(token_rows, 4) ||
      !aligned(workspace, 16))
    return MOE_FP4_ERR_ALIGN;
  if (num_experts > 1024 || topk > 32 || num_groups > 64) return MOE_FP4_ERR_UNSUPPORTED;
  const int32_t group_size = num_experts / num_groups;
  int32_t token_lanes = tokens >= moe_fp4::kRouteNarrow ? 16 : 64, group_lanes = 0, per_lane = 0;
  for (; token_lanes <= 64; token_lanes *= 4) {
    group_lanes = token_lanes;
    while (group_lanes * num_groups > token_lanes) group_lanes /= 2;
    per_lane = group_lanes ? (group_size + group_lanes - 1) / group_lanes : 0;
    if (group_lanes > 0 && per_lane <= moe_fp4::kRouteMaxPerLane && topk <= token_lanes) break;
  }
  if (token_lanes > 64) return MOE_FP4_ERR_UNSUPPORTED;
  if (tokens > 0 && (tokens > kFewLimit / topk || ld > kFewLimit / tokens))
    return MOE_FP4_ERR_UNSUPPORTED;
  const size_t need = moe_fp4_route_workspace_size(tokens, num_experts);
  if (need > 0 && !workspace) return MOE_FP4_ERR_NULL;
  if (workspace_bytes < need) return MOE_FP4_ERR_SHAPE;
  const int64_t pb = tokens * topk * 4;
  struct {
    const void* p;
    int64_t bytes;
  } const bufs[] = {{logits, tokens > 0 ? ((tokens - 1) * ld + num_experts) * esize : 0},
                    {bias, bias ? num_experts * (int64_t)4 : 0},
                    {ids, pb},
                    {weights, pb},
                    {row_token, pb},
                    {token_rows, pb},
                    {offsets, (num_experts + 1) * (int64_t)4},
                    {workspace, (int64_t)need}};
  for (int i = 2; i < 8; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes)) return MOE_FP4_ERR_ARG;
  moe_fp4::RouteArgs a;
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.row_token = row_token;
  a.token_rows = token_rows;
  a.counts = static_cast<uint16_t*>(workspace);
  a.dtype = dtype;
  a.tokens = (int32_t)tokens;
  a.experts = num_experts;
  a.topk = topk;
  a.num_groups = num_groups;
  a.topk_groups = topk_groups;
  a.sigmoid = score == MOE_FP4_SCORE_SIGMOID ? 1 : 0;
  a.renormalize = renormalize;
  a.token_lanes = token_lanes;
  a.group_lanes = group_lanes;
  // Every lane holds none or per_lane experts, a power of two, at 16-byte addresses.
  a.wide = aligned(logits, 16) && ld * esize % 16 == 0 && (per_lane & (per_lane - 1)) == 0 &&
           per_lane * esize % 16 == 0 && group_size % per_lane == 0;
  a.per_lane = per_lane;
  a.block_tokens = (int32_t)route_block(tokens);
  a.counts_pitch = route_pitch(num_experts);
  hipError_t err = moe_fp4::launch_route(a, reinterpret_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP;
}

int moe_fp4_pack_weights(const uint8_t* w_q, uint8_t* w_packed, int32_t num_experts,
                         int64_t n, int64_t k, void* stream) {
  return repack(w_q, w_packed, num_experts, n, k, stream, true);
}

int moe_fp4_unpack_weights(const uint8_t* w_packed, uint8_t* w_q, int32_t num_experts,
                           int64_t n, int64_t k, void* stream) {
  return repack(w_packed, w_q, num_experts, n, k, stream, false);
}

}  // extern "C"

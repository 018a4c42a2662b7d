// C ABI of the FP8 block-scaled operators and of the rows' and router's gradients (declared in
// include/moe_fp4.h).  As in api.cpp, every argument is checked on the host before the HIP
// runtime is touched, and what passes always launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_fp4.h"
#include "api_checks.h"
#include "launch.h"

using moe_fp4::aligned;
using moe_fp4::overlap;

namespace {

// Byte sizes that are addressed with 32-bit buffer offsets.
constexpr int64_t kLimit = (int64_t)INT32_MAX - 4096;
constexpr int32_t kMaxExperts = 8192;

bool in_dtype_ok(int t) { return t == MOE_FP4_IN_BF16 || t == MOE_FP4_IN_FP32 || t == MOE_FP4_IN_FP16; }
int64_t in_size(int t) { return t == MOE_FP4_IN_FP32 ? 4 : t == MOE_FP4_IN_FP8 ? 1 : 2; }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Bytes that `rows` rows of `cols` elements at a pitch take; a negative number where that is
// not representable.
int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  if (rows == 0) return 0;
  if (ld > INT64_MAX / 16 / rows) return -1;
  return ((rows - 1) * ld + cols) * size;
}

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether one of the last `written` ranges shares a byte with any range before it.
template <int N>
bool clash(const Range (&r)[N], int written) {
  for (int i = N - written; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes)) return true;
  return false;
}

int status_of(hipError_t err) { return err == hipSuccess ? MOE_FP4_OK : MOE_FP4_ERR_HIP; }

}  // namespace

extern "C" {

int moe_fp8_quantize(const void* x, int in_dtype, int64_t rows, int64_t k, int64_t ld_x, int swiglu,
                     const void* grad, int64_t ld_grad, int power_of_two, uint8_t* q, float* sf,
                     void* stream) {
  if (!in_dtype_ok(in_dtype) || (swiglu != 0 && swiglu != 1) || (grad && !swiglu) ||
      (power_of_two != 0 && power_of_two != 1))
    return MOE_FP4_ERR_ARG;
  if (rows > 0 && (!x || !q || !sf)) return MOE_FP4_ERR_NULL;
  if (rows < 0 || k < 1 || k % 16 != 0) return MOE_FP4_ERR_SHAPE;
  if (k > kLimit / 4) return MOE_FP4_ERR_UNSUPPORTED;
  const int64_t in_cols = swiglu ? 2 * k : k, cols = grad ? 2 * k : k;
  if (rows > 0 && (ld_x < in_cols || (grad && ld_grad < k))) return MOE_FP4_ERR_SHAPE;
  const int64_t es = in_size(in_dtype);
  if (!aligned(x, 16) || !aligned(grad, 16) || !aligned(q, 16) || !aligned(sf, 4)) return MOE_FP4_ERR_ALIGN;
  if (rows > 0 && ((ld_x % 16 * es) % 16 != 0 || (grad && (ld_grad % 16 * es) % 16 != 0))) return MOE_FP4_ERR_ALIGN;
  if (rows == 0) return MOE_FP4_OK;
  const int64_t xb = extent(rows, in_cols, ld_x, es), gb = grad ? extent(rows, k, ld_grad, es) : 0;
  if (xb < 0 || gb < 0) return MOE_FP4_ERR_SHAPE;
  // Eight threads or fewer a block, fewer than 2^32 in a launch.
  if (rows > ((1 << 29) - (1 << 17)) / blocks(cols)) return MOE_FP4_ERR_UNSUPPORTED;
  const Range r[] = {{x, xb}, {grad, gb}, {q, rows * cols}, {sf, rows * blocks(cols) * 4}};
  if (clash(r, 2)) return MOE_FP4_ERR_ARG;
  moe_fp4::Fp8QuantArgs a;
  a.x = x;
  a.ld_x = ld_x;
  a.grad = grad;
  a.ld_grad = ld_grad;
  a.q = q;
  a.sf = sf;
  a.per_row = moe_fp4::FastDiv::of((uint32_t)blocks(cols));
  a.blocks = (uint32_t)(rows * blocks(cols));
  a.rows = rows;
  a.k = (int32_t)cols;
  a.dtype = in_dtype;
  a.swiglu = swiglu;
  a.pow2 = power_of_two;
  return status_of(moe_fp4::launch_quantize_fp8(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_fp8_quantize_weights(const void* w, int in_dtype, int32_t num_experts, int64_t n, int64_t k,
                             int power_of_two, uint8_t* q, float* sf, uint8_t* qt, float* sft,
                             void* stream) {
  if (!in_dtype_ok(in_dtype) || (power_of_two != 0 && power_of_two != 1)) return MOE_FP4_ERR_ARG;
  if (!w || !q || !sf || (!qt != !sft)) return MOE_FP4_ERR_NULL;
  if (num_experts < 1 || n < 1 || k < 1 || k % 16 != 0 || (qt && n % 16 != 0)) return MOE_FP4_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(sf, 4) || !aligned(qt, 16) || !aligned(sft, 4))
    return MOE_FP4_ERR_ALIGN;
  if (num_experts > kMaxExperts || n > kLimit / k || blocks(n) > 65535) return MOE_FP4_ERR_UNSUPPORTED;
  const int64_t qb = num_experts * n * k, sb = num_experts * blocks(n) * blocks(k) * 4;
  const Range r[] = {{w, qb * in_size(in_dtype)}, {q, qb}, {sf, sb}, {qt, qt ? qb : 0}, {sft, sft ? sb : 0}};
  if (clash(r, 4)) return MOE_FP4_ERR_ARG;
  moe_fp4::Fp8WeightArgs a;
  a.w = w;
  a.q = q;
  a.sf = sf;
  a.qt = qt;
  a.sft = sft;
  a.experts = num_experts;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.dtype = in_dtype;
  a.pow2 = power_of_two;
  return status_of(moe_fp4::launch_quantize_fp8_weights(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_grouped_gemm_fp8(const uint8_t* a_q, const float* a_sf, int64_t a_rows,
                         const int32_t* a_row_index, const uint8_t* w_q, const float* w_sf,
                         const int32_t* expert_offsets, int32_t num_experts, int64_t m_total, int64_t n,
                         int64_t k, void* out, int out_dtype, int64_t ldo, void* stream) {
  if (out_dtype != MOE_FP4_OUT_BF16 && out_dtype != MOE_FP4_OUT_FP32 && out_dtype != MOE_FP4_OUT_FP16)
    return MOE_FP4_ERR_ARG;
  if (!w_q || !w_sf || (num_experts > 1 && !expert_offsets) || (m_total > 0 && (!a_q || !a_sf || !out)))
    return MOE_FP4_ERR_NULL;
  if (num_experts < 1 || m_total < 0 || n < 1 || k < 1) return MOE_FP4_ERR_SHAPE;
  if (m_total > 0 && (ldo < n || a_rows < (a_row_index ? 1 : m_total))) return MOE_FP4_ERR_SHAPE;
  const int64_t es = out_dtype == MOE_FP4_OUT_FP32 ? 4 : 2;
  if (!aligned(a_q, 16) || !aligned(a_sf, 4) || !aligned(w_q, 16) || !aligned(w_sf, 4) ||
      !aligned(a_row_index, 4) || !aligned(expert_offsets, 4) || !aligned(out, es))
    return MOE_FP4_ERR_ALIGN;
  if (k % 16 != 0 || k > (1 << 22) || num_experts > kMaxExperts || n > kLimit / k || m_total > kLimit / 4 ||
      a_rows > kLimit || (a_row_index && a_rows > kLimit / k))
    return MOE_FP4_ERR_UNSUPPORTED;
  if (m_total == 0) return MOE_FP4_OK;
  if (ldo > (1 << 20)) return MOE_FP4_ERR_UNSUPPORTED;  // 256 rows of FP32 within 32-bit offsets
  // Items are counted in 32 bits.
  const int64_t m_tiles = m_total / 16 + (m_total < num_experts ? m_total : num_experts) + 1;
  if (m_tiles > kLimit / ((n + 15) / 16)) return MOE_FP4_ERR_UNSUPPORTED;
  const int64_t ob = extent(m_total, n, ldo, es), nb = blocks(n), kb = blocks(k);
  const Range r[] = {{a_q, a_rows * k},
                     {a_sf, a_rows * kb * 4},
                     {a_row_index, a_row_index ? m_total * 4 : 0},
                     {w_q, num_experts * n * k},
                     {w_sf, num_experts * nb * kb * 4},
                     {expert_offsets, expert_offsets ? (num_experts + 1) * (int64_t)4 : 0},
                     {out, ob}};
  if (clash(r, 1)) return MOE_FP4_ERR_ARG;
  moe_fp4::Fp8GemmArgs a;
  a.a_q = a_q;
  a.a_sf = a_sf;
  a.a_rows = a_rows;
  a.a_row_index = a_row_index;
  a.w_q = w_q;
  a.w_sf = w_sf;
  a.offsets = expert_offsets;
  a.m_total = m_total;
  a.experts = num_experts;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.n_blocks = (int32_t)nb;
  a.k_blocks = (int32_t)kb;
  a.out = out;
  a.ldo = ldo;
  a.out_dtype = out_dtype;
  a.vec4 = ldo % 4 == 0 && aligned(out, 4 * es);
  return status_of(moe_fp4::launch_grouped_gemm_fp8(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_fp4_dispatch(const void* x, int dtype, int64_t tokens, int64_t n, int64_t ld_x,
                     const int32_t* row_token, int64_t m_total, void* out, int64_t ldo, void* stream) {
  if (!in_dtype_ok(dtype) && dtype != MOE_FP4_IN_FP8) return MOE_FP4_ERR_ARG;
  if (m_total > 0 && (!row_token || !out || (tokens > 0 && !x))) return MOE_FP4_ERR_NULL;
  if (tokens < 0 || m_total < 0 || n < 1) return MOE_FP4_ERR_SHAPE;
  if (m_total > 0 && (ldo < n || (tokens > 0 && ld_x < n))) return MOE_FP4_ERR_SHAPE;
  const int64_t es = in_size(dtype);
  if (!aligned(x, es) || !aligned(out, es) || !aligned(row_token, 4)) return MOE_FP4_ERR_ALIGN;
  if (tokens > INT32_MAX || m_total > INT32_MAX) return MOE_FP4_ERR_UNSUPPORTED;
  if (m_total == 0) return MOE_FP4_OK;
  const int64_t xb = extent(tokens, n, ld_x, es), ob = extent(m_total, n, ldo, es);
  if (xb < 0 || ob < 0) return MOE_FP4_ERR_SHAPE;
  const Range r[] = {{x, xb}, {row_token, m_total * 4}, {out, ob}};
  if (clash(r, 1)) return MOE_FP4_ERR_ARG;
  moe_fp4::RowsArgs a;
  a.x = x;
  a.ld_x = tokens > 0 ? ld_x * es : 0;
  a.source_rows = tokens;
  a.map = row_token;
  a.topk = 1;
  a.out = out;
  a.ld_out = ldo * es;
  a.rows = m_total;
  a.cols = n;
  a.row_bytes = n * es;
  a.esize = (int32_t)es;
  a.dtype = dtype;
  return status_of(moe_fp4::launch_dispatch(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_fp4_dispatch_backward(const void* dy, int dtype, int64_t m_total, int64_t n, int64_t ld_dy,
                              const int32_t* token_rows, int32_t topk, int64_t tokens, void* dx,
                              int64_t ld_dx, void* stream) {
  if (!in_dtype_ok(dtype)) return MOE_FP4_ERR_ARG;
  if (tokens > 0 && (!token_rows || !dx || (m_total > 0 && !dy))) return MOE_FP4_ERR_NULL;
  if (tokens < 0 || m_total < 0 || n < 1 || topk < 1) return MOE_FP4_ERR_SHAPE;
  if (tokens > 0 && (ld_dx < n || (m_total > 0 && ld_dy < n))) return MOE_FP4_ERR_SHAPE;
  const int64_t es = in_size(dtype);
  if (!aligned(dy, es) || !aligned(dx, es) || !aligned(token_rows, 4)) return MOE_FP4_ERR_ALIGN;
  if (tokens > INT32_MAX || m_total > INT32_MAX || topk > 1024) return MOE_FP4_ERR_UNSUPPORTED;
  if (tokens == 0) return MOE_FP4_OK;
  const int64_t yb = extent(m_total, n, ld_dy, es), xb = extent(tokens, n, ld_dx, es);
  if (yb < 0 || xb < 0) return MOE_FP4_ERR_SHAPE;
  const Range r[] = {{dy, yb}, {token_rows, tokens * topk * 4}, {dx, xb}};
  if (clash(r, 1)) return MOE_FP4_ERR_ARG;
  moe_fp4::RowsArgs a;
  a.x = dy;
  a.ld_x = m_total > 0 ? ld_dy * es : 0;
  a.source_rows = m_total;
  a.map = token_rows;
  a.topk = topk;
  a.out = dx;
  a.ld_out = ld_dx * es;
  a.rows = tokens;
  a.cols = n;
  a.row_bytes = n * es;
  a.esize = (int32_t)es;
  a.dtype = dtype;
  return status_of(moe_fp4::launch_dispatch_backward(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_fp4_combine_backward(const void* dout, int dout_dtype, int64_t num_tokens, int64_t n, int64_t ld_dout,
                             const uint16_t* rows, int64_t ld_rows, int64_t m_total,
                             const int32_t* token_rows, const float* token_weights, int32_t topk,
                             const int32_t* row_token, uint16_t* drows, int64_t ld_drows, float* dweights,
                             void* stream) {
  if (dout_dtype != MOE_FP4_OUT_BF16 && dout_dtype != MOE_FP4_OUT_FP32) return MOE_FP4_ERR_ARG;
  if (num_tokens > 0 && (!dout || !token_rows || !token_weights || !dweights)) return MOE_FP4_ERR_NULL;
  if (m_total > 0 && num_tokens > 0 && !rows) return MOE_FP4_ERR_NULL;
  if (m_total > 0 && (num_tokens > 0 || row_token) && !drows) return MOE_FP4_ERR_NULL;
  if (num_tokens < 0 || m_total < 0 || topk < 1 || n < 1) return MOE_FP4_ERR_SHAPE;
  if ((num_tokens > 0 && ld_dout < n) || (m_total > 0 && ((num_tokens > 0 && ld_rows < n) || ld_drows < n)))
    return MOE_FP4_ERR_SHAPE;
  const int64_t es = dout_dtype == MOE_FP4_OUT_FP32 ? 4 : 2;
  if (!aligned(dout, 16) || (num_tokens > 0 && (ld_dout % 16 * es) % 16 != 0) || !aligned(token_rows, 4) ||
      !aligned(token_weights, 4) || !aligned(dweights, 4) || !aligned(row_token, 4))
    return MOE_FP4_ERR_ALIGN;
  if (m_total > 0 && (!aligned(rows, 16) || !aligned(drows, 16) || (num_tokens > 0 && ld_rows % 8 != 0) ||
                      ld_drows % 8 != 0))
    return MOE_FP4_ERR_ALIGN;
  // One workgroup a token.
  if (n % 16 != 0 || num_tokens > (1 << 23) || m_total > kLimit / 16 || topk > 1024) return MOE_FP4_ERR_UNSUPPORTED;
  if (num_tokens == 0 && (m_total == 0 || !row_token)) return MOE_FP4_OK;
  const int64_t gb = extent(num_tokens, n, ld_dout, es), pb = num_tokens * topk * 4;
  const int64_t rb = num_tokens > 0 ? extent(m_total, n, ld_rows, 2) : 0, db = extent(m_total, n, ld_drows, 2);
  if (gb < 0 || rb < 0 || db < 0) return MOE_FP4_ERR_SHAPE;
  const Range r[] = {{dout, gb}, {rows, rb}, {token_rows, pb}, {token_weights, pb},
                     {row_token, row_token ? m_total * 4 : 0}, {drows, db}, {dweights, pb}};
  if (clash(r, 2)) return MOE_FP4_ERR_ARG;
  moe_fp4::CombineBackwardArgs a;
  a.dout = dout;
  a.ld_dout = ld_dout;
  a.f32_dout = dout_dtype == MOE_FP4_OUT_FP32 ? 1 : 0;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.m_total = m_total;
  a.token_rows = token_rows;
  a.token_weights = token_weights;
  a.row_token = row_token;
  a.topk = topk;
  a.num_tokens = num_tokens;
  a.n = n;
  a.drows = drows;
  a.ld_drows = ld_drows;
  a.dweights = dweights;
  return status_of(moe_fp4::launch_combine_backward(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_fp4_route_backward(const void* logits, int dtype, int64_t tokens, int32_t num_experts, int64_t ld,
                           const int32_t* ids, const float* dweights, int32_t topk, int score,
                           int renormalize, void* dlogits, int64_t ld_out, void* stream) {
  if (!in_dtype_ok(dtype) || (score != MOE_FP4_SCORE_SOFTMAX && score != MOE_FP4_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1))
    return MOE_FP4_ERR_ARG;
  if (tokens > 0 && (!logits || !ids || !dweights || !dlogits)) return MOE_FP4_ERR_NULL;
  if (tokens < 0 || num_experts < 1 || topk < 1) return MOE_FP4_ERR_SHAPE;
  if (tokens > 0 && (ld < num_experts || ld_out < num_experts)) return MOE_FP4_ERR_SHAPE;
  const int64_t es = in_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(ids, 4) || !aligned(dweights, 4))
    return MOE_FP4_ERR_ALIGN;
  if (num_experts > 1024 || topk > 32 || tokens > (1 << 24)) return MOE_FP4_ERR_UNSUPPORTED;
  if (tokens == 0) return MOE_FP4_OK;
  const int64_t xb = extent(tokens, num_experts, ld, es), ob = extent(tokens, num_experts, ld_out, es);
  if (xb < 0 || ob < 0) return MOE_FP4_ERR_SHAPE;
  const Range r[] = {{logits, xb}, {ids, tokens * topk * 4}, {dweights, tokens * topk * 4}, {dlogits, ob}};
  if (clash(r, 1)) return MOE_FP4_ERR_ARG;
  moe_fp4::RouteBackwardArgs a;
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.ld_out = ld_out;
  a.tokens = tokens;
  a.experts = num_experts;
  a.topk = topk;
  a.dtype = dtype;
  a.sigmoid = score == MOE_FP4_SCORE_SIGMOID ? 1 : 0;
  a.renormalize = renormalize;
  return status_of(moe_fp4::launch_route_backward(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

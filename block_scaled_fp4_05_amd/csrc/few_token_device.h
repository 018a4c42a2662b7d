// Device pieces of the few-token products (linear.hip, ffn.hip): 16-bit rows times
// NVFP4 weights, on the 16 x 16 x 32 matrix instruction.
//
// The weights are the A operand (16 weight rows), the tokens the B operand (up to
// 16 columns), so lane l holds weight row l % 16 and token l % 16, both at the K
// slice of lane group g = l / 16, and the result's four values are four
// consecutive weight rows of one token.  The order of K inside a product is free
// as long as both operands agree: a wavefront takes 256 elements of K per step
// and lane group g the 64 consecutive ones at 64 g, so that a lane's codes are two
// 16-byte loads and its four block scales one dword.
//
// What reaches a lane through LDS, private to its wavefront (no barriers; lds_handover):
//   - activations: loaded in whole 512-byte pieces of a token's row and read back as
//     operands.  Loading operands straight from memory costs eight instructions a step
//     whatever the token count, each touching 64 places.
//   - block scales: one load covers four steps (64 bytes of each row); a dword a
//     step and lane touches as many lines as the codes do for an eighth of the bytes.
//   - codes, in the variants that stream much for few tokens: see Pieces below.
// No load takes the non-temporal hint: two loads share each line of codes (65536 x 6144,
// codes alone: 57 us with it against 48).
//
// Any K that is a multiple of 16 and at least 64 runs: a lane whose 64 elements pass
// the end of the row reads the row's last 64 and moves them down; scales and
// activations past the end are zeros.
#pragma once

#include "fp4_device.h"
#include "gemm_common.h"

namespace moe_fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kFewStep = 256;  // elements of K per wavefront step

// Between a wavefront's writes to its own LDS and other lanes' reads of them, and between
// those reads and the next writes.  The hardware keeps a wavefront's LDS operations in order;
// this keeps the compiler from moving them past each other.  No instruction.
__device__ __forceinline__ void lds_handover() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Eight codes (one dword) times one block scale as eight exact 16-bit values: the
// product has at most 6 significant bits and lies in [2^-10, 2688], inside both
// types' normal range.  A NaN scale stays NaN.  FP16: packed multiply.  BF16 has
// no packed multiply on gfx950, so the product is taken in FP32 and its upper half
// kept (exact, the lower half being zero).
template <bool F16>
__device__ __forceinline__ u32x4_t dequant8_16bit(uint32_t codes, float scale) {
  if (F16) {
    const _Float16 h = (_Float16)scale;
    const half2_t s2 = {h, h};
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s2;
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s2;
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s2;
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s2;
    return u32x4_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                   __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
  }
  auto pair = [&](auto v) {
    const float lo = v[0] * scale, hi = v[1] * scale;
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo),
                                 0x07060302u);
  };
  return u32x4_t{pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2)),
                 pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3))};
}

template <bool F16>
__device__ __forceinline__ float4_t mfma16(u32x4_t a, u32x4_t b, float4_t c) {
  if (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Blocks (0..4) of a row that lie in a lane's 64 elements from k0.
__device__ __forceinline__ int32_t blocks_left(int32_t k0, int32_t k) {
  const int32_t b = (k - k0) >> 4;
  return b < 0 ? 0 : b < 4 ? b : 4;
}

// The codes of a step for NT x 16 weight rows.
template <int NT>
struct Codes {
  u32x4_t q[NT][2];
};

// Byte offset, in a row of codes, of a lane's 32 bytes of a step: the row's last 32
// where they would pass its end.
__device__ __forceinline__ uint32_t code_offset(int32_t step, int32_t g, int32_t k) {
  const uint32_t o = (uint32_t)(step * (kFewStep / 2) + 32 * g), last = (uint32_t)(k / 2 - 32);
  return o < last ? o : last;
}

template <int NT>
__device__ __forceinline__ void load_codes(Codes<NT>& c, rsrc_t q_rs, const uint32_t (&row_off)[NT],
                                           uint32_t off) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    c.q[t][0] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, row_off[t] + off, 0, 0);
    c.q[t][1] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, row_off[t] + off + 16u, 0, 0);
  }
}

// Move the last `left` (1..3) blocks of a lane's window down to its start; 0 and 4 stay.
template <int NT>
__device__ __forceinline__ void move_codes(Codes<NT>& c, int32_t left) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t w[8] = {c.q[t][0][0], c.q[t][0][1], c.q[t][0][2], c.q[t][0][3],
                           c.q[t][1][0], c.q[t][1][1], c.q[t][1][2], c.q[t][1][3]};
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v = w[i];
      if (left == 3) v = i + 2 < 8 ? w[i + 2 < 8 ? i + 2 : 0] : 0u;
      if (left == 2) v = i + 4 < 8 ? w[i + 4 < 8 ? i + 4 : 0] : 0u;
      if (left == 1) v = i + 6 < 8 ? w[i + 6 < 8 ? i + 6 : 0] : 0u;
      m[i] = v;
    }
    c.q[t][0] = u32x4_t{m[0], m[1], m[2], m[3]};
    c.q[t][1] = u32x4_t{m[4], m[5], m[6], m[7]};
  }
}

// Pieces: the codes of a step on their way, as four neighbouring lanes read them from 64
// consecutive bytes of a row: lane l holds pieces of row l / 4 of each tile, which the
// wavefront turns into Codes through its own LDS.  Read as the products want them,
// neighbouring lanes read different rows, and the L1 cache takes one line at a time.
// 65536 x 6144, four tokens: 47.8 us against 52.0 with Codes read directly; eight
// tokens 59 against 63.  Variants of one tile a wavefront (few rows: latency) or of more
// tokens (LDS, registers) read directly: 6144 x 6144, one token 8.8 us against 9.3 turned; up
// projections of 64 experts, 32 tokens 60.5 against 61.6.  So does the layer's down projection,
// which has a step or a few an expert: 256 experts, eight tokens 16.7 us against 21.4 (with its
// activations in two parts).
constexpr int kPieceBytes = 2048;  // LDS in which one tile's codes are turned

// Which of the four 16-byte pieces of a 64-byte half lane l reads of row l / 4: staggered,
// so that sixteen rows' equal pieces lie in different banks.
__device__ __forceinline__ int32_t piece_of(int32_t lane) { return (lane ^ (lane >> 4)) & 3; }

// row_off: start of row lane / 4 of each tile.  A piece that passes the row's end, k / 2, is
// read 8 bytes earlier or, past the end, from its last 16 bytes: its scales are 0.
template <int NT>
__device__ __forceinline__ void load_pieces(Codes<NT>& c, rsrc_t q_rs, const uint32_t (&row_off)[NT],
                                            int32_t step, int32_t end, int32_t lane, int32_t k) {
  uint32_t off0 = (uint32_t)(step * (kFewStep / 2) + 16 * piece_of(lane)), off1 = off0 + 64u;
  if ((step + 1) * kFewStep > k) {  // uniform
    const uint32_t last = (uint32_t)(k / 2 - 16);
    off0 = off0 < last ? off0 : last;
    off1 = off1 < last ? off1 : last;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t row = step < end ? row_off[t] : kOutOfRange;
    c.q[t][0] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, row + off0, 0, 0);
    c.q[t][1] = __builtin_amdgcn_raw_buffer_load_b128(q_rs, row + off1, 0, 0);
  }
}

// Pieces to Codes, through NT * kPieceBytes of the wavefront's LDS; hands over whatever else
// has been written to it.
template <int NT>
__device__ __forceinline__ void turn_pieces(Codes<NT>& c, char* lds, int32_t step, int32_t lane, int32_t k) {
  if ((step + 1) * kFewStep > k) {  // uniform: a piece may have been read 8 bytes early
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool early = step * (kFewStep / 2) + 64 * h + 16 * piece_of(lane) == k / 2 - 8;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (early) c.q[t][h] = u32x4_t{c.q[t][h][2], c.q[t][h][3], 0u, 0u};
    }
  }
  const int32_t r = lane & 15, g = lane >> 4;
  const char* from = lds + (g >> 1) * 1024 + 64 * r;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<u32x4_t*>(lds + t * kPieceBytes + h * 1024 + 16 * lane) = c.q[t][h];
  }
  lds_handover();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      c.q[t][h] = *reinterpret_cast<const u32x4_t*>(from + t * kPieceBytes + 16 * ((2 * (g & 1) + h) ^ (r >> 2)));
  }
}

// The eight matrix products of a step: operand J covers elements 8J .. 8J+7 of each
// lane's 64.  x(J): the token operands; f(J, t, a, x): multiply tile t.
template <bool F16, int NT, int J, typename X, typename F>
__device__ __forceinline__ void for_operands(const Codes<NT>& c, const uint32_t (&s)[NT], X&& x, F&& f) {
  if constexpr (J < 8) {
    const auto xv = x(J);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t codes = c.q[t][J / 4][J % 4];
      f(J, t, dequant8_16bit<F16>(codes, __builtin_amdgcn_cvt_f32_fp8((int)s[t], J / 2)), xv);
    }
    for_operands<F16, NT, J + 1>(c, s, x, f);
  }
}

__device__ __forceinline__ float bf16_value(uint16_t b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// A 16-bit input element as FP32.
template <bool F16>
__device__ __forceinline__ float value16(uint16_t b) {
  return F16 ? (float)__builtin_bit_cast(_Float16, b) : bf16_value(b);
}

// Store one result in the output's type (rounded to nearest even).
__device__ __forceinline__ void store_as(void* out, int64_t i, float v, int32_t dtype) {
  if (dtype == kFewOutF32)
    static_cast<float*>(out)[i] = v;
  else if (dtype == kFewOutF16)
    static_cast<_Float16*>(out)[i] = (_Float16)v;
  else
    static_cast<__bf16*>(out)[i] = (__bf16)v;
}

// x / (1 + e^-x): exactly 0 or the identity where e^-x overflows or vanishes.  expf, since the
// fast exponential's relative error grows with |x|; a thread takes four, in the epilogues.
__device__ __forceinline__ float silu(float x) { return x / (1.0f + expf(-x)); }

// The sums of NT x 16 weight rows times up to 16 tokens over a wavefront's steps
// [s0, s1).  XR = loads of two tokens each that a step takes at most (8), PF of
// them kept in flight, the rest (where there are as many tokens) loaded when needed.
// Two steps are in flight; a load that has nothing to fetch is sent out of range
// instead of being branched around, so that the compiler's counts of outstanding
// loads stay exact.  TURN: codes are read as Pieces.
template <bool F16, int NT, int XR, int PF, bool TURN>
struct FewLoop {
  struct Stage {
    Codes<NT> c;
    u32x4_t x[PF];
  };
  static constexpr int kChunk = 8;  // steps whose scales are in LDS at once
  static constexpr int kXBytes = XR * 1024, kSBytes = NT * 2048;
  // Of a wavefront; its sums take the place of all.
  static constexpr int kLdsBytes = kXBytes + kSBytes + (TURN ? NT * kPieceBytes : 0);

  // The weight row (0..15 of a tile) whose codes and scales a lane loads, and which quarter of
  // what is read of that row.
  static __device__ __forceinline__ int row_of(int lane) { return TURN ? lane >> 2 : lane & 15; }
  static __device__ __forceinline__ int quarter_of(int lane) { return TURN ? lane & 3 : lane >> 4; }

  rsrc_t q_rs, s_rs, x_rs;
  uint32_t q_off[NT], s_off[NT];  // starts of row row_of(lane) of each tile, bytes
  uint32_t x_off[XR];             // start of this lane's 16 bytes of token 2i + lane / 32
  char* lds;                      // kLdsBytes of this wavefront
  int32_t k, tokens, lane;

  // Steps from `end` on are not fetched (in all that follows).
  __device__ __forceinline__ uint32_t x_offset(int i, int32_t step, int32_t end) const {
    return step * kFewStep + 8 * (lane & 31) < k && step < end
               ? x_off[i] + (uint32_t)(2 * kFewStep * step) : kOutOfRange;
  }

  __device__ __forceinline__ void load(Stage& r, int32_t step, int32_t end) const {
    if (TURN)
      load_pieces<NT>(r.c, q_rs, q_off, step, end, lane, k);
    else
      load_codes<NT>(r.c, q_rs, q_off, step < end ? code_offset(step, lane >> 4, k) : kOutOfRange);
#pragma unroll
    for (int i = 0; i < PF; ++i)
      r.x[i] = __builtin_amdgcn_raw_buffer_load_b128(x_rs, x_offset(i, step, end), 0, 0);
  }

  // Scales of steps base .. base + 3: a row's quarter i is the 16 bytes of step base + i.
  __device__ __forceinline__ void load_scales(u32x4_t (&s)[NT], int32_t base, int32_t end) const {
    const int32_t step = base + quarter_of(lane);
    const int32_t last = base + 4 < end ? base + 4 : end;
    if (last * kFewStep <= k) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        s[t] = __builtin_amdgcn_raw_buffer_load_b128(
            s_rs, step < end ? s_off[t] + (uint32_t)(16 * step) : kOutOfRange, 0, 0);
    } else {  // a row ends inside: a dword reads the row's last four where it would pass the end
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t left = blocks_left(step * kFewStep + 64 * i, k);
          const uint32_t d = __builtin_amdgcn_raw_buffer_load_b32(
              s_rs, step < end && left > 0 ? s_off[t] + (uint32_t)(16 * step + 4 * i - (4 - left))
                                          : kOutOfRange, 0, 0);
          s[t][i] = left > 0 ? d >> (8 * (4 - left)) : 0u;
        }
    }
  }

  __device__ __forceinline__ void put_scales(const u32x4_t (&s)[NT], int h) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<u32x4_t*>(lds + kXBytes + (t * 2 + h) * 1024 + (quarter_of(lane) * 16 + row_of(lane)) * 16) = s[t];
  }

  // 16-byte piece c (0..31) of token t is kept at piece c ^ t: sixteen tokens'
  // equal pieces lie in different banks.
  __device__ __forceinline__ void put_x(int i, u32x4_t v) const {
    const int32_t t = 2 * i + (lane >> 5);
    *reinterpret_cast<u32x4_t*>(lds + t * 512 + (((lane & 31) ^ t) << 4)) = v;
  }

  // Step `step`, the i-th of those whose scales are in LDS.
  __device__ __forceinline__ void compute(Stage& r, float4_t (&acc)[NT], int32_t step, int i) const {
    lds_handover();  // the previous step's operands have been read
#pragma unroll
    for (int j = 0; j < PF; ++j) put_x(j, r.x[j]);
#pragma unroll
    for (int j = PF; j < XR; ++j)
      if (2 * j < tokens)
        put_x(j, __builtin_amdgcn_raw_buffer_load_b128(x_rs, x_offset(j, step, step + 1), 0, 0));
    const int32_t g = lane >> 4, col = lane & 15;
    if (TURN)
      turn_pieces<NT>(r.c, lds + kXBytes + kSBytes, step, lane, k);
    else
      lds_handover();
    if (!TURN && (step + 1) * kFewStep > k) move_codes<NT>(r.c, blocks_left(step * kFewStep + 64 * g, k));
    uint32_t s[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
      s[t] = *reinterpret_cast<const uint32_t*>(lds + kXBytes + t * 2048 + (col + 16 * i) * 16 + 4 * g);
    const int32_t tok = col < tokens ? col : tokens - 1;
    const uint32_t at = (uint32_t)(tok * 512 + (((8 * g) ^ tok) << 4));
    for_operands<F16, NT, 0>(
        r.c, s,
        [&](int j) { return *reinterpret_cast<const u32x4_t*>(lds + (at ^ (uint32_t)(j << 4))); },
        [&](int, int t, u32x4_t a, u32x4_t x) { acc[t] = mfma16<F16>(a, x, acc[t]); });
  }

  // kChunk steps at a time: their scales first, then two steps in flight.
  __device__ __forceinline__ void run(float4_t (&acc)[NT], int32_t s0, int32_t s1) const {
    for (int32_t c0 = s0; c0 < s1; c0 += kChunk) {
      const int32_t c1 = c0 + kChunk < s1 ? c0 + kChunk : s1;
      u32x4_t sc[2][NT];
      Stage a, b;
      load_scales(sc[0], c0, c1);
      load(a, c0, c1);
      load_scales(sc[1], c0 + 4, c1);
      load(b, c0 + 1, c1);
      lds_handover();  // the previous scales have been read
      put_scales(sc[0], 0);
      put_scales(sc[1], 1);
      int32_t s = c0;
      for (; s + 2 < c1; s += 2) {
        compute(a, acc, s, s - c0);
        load(a, s + 2, c1);
        compute(b, acc, s + 1, s + 1 - c0);
        load(b, s + 3, c1);
      }
      compute(a, acc, s, s - c0);
      if (s + 1 < c1) compute(b, acc, s + 1, s + 1 - c0);
    }
  }
};

// Leave a wavefront's sums in its own LDS: [tile][lane], four values each.
template <int NT>
__device__ __forceinline__ void put_sums(char* lds, const float4_t (&acc)[NT], int lane) {
  lds_handover();  // the last operands have been read
#pragma unroll
  for (int t = 0; t < NT; ++t) reinterpret_cast<float4_t*>(lds)[t * 64 + lane] = acc[t];
}

// The sum over the wavefronts, in wavefront order, of one lane's values of a tile.
__device__ __forceinline__ float4_t take_sum(const char* lds, int pitch, int tile, int lane, int waves) {
  const int at = (tile * 64 + lane) * 16;
  float4_t v = *reinterpret_cast<const float4_t*>(lds + at);
  for (int w = 1; w < waves; ++w) v += *reinterpret_cast<const float4_t*>(lds + w * pitch + at);
  return v;
}

}  // namespace moe_fp4

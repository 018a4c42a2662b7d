// A whole Mixture-of-Experts feed-forward layer for a few tokens (moe_fp4_ffn), two
// kernels:
//
//   k_ffn_up    h[t, e] = silu(g) * u,  (g, u) = w13_scale[e] * W13[e] x[t]
//   k_ffn_down  out[t]  = residual[t] + sum_e W2[e] (c[t, e] h[t, e]),
//               c[t, e] = w2_scale[e] * (sum of t's routing weights for e)
//
// Experts no token is routed to are not read.  A routed expert's down projection is read once,
// its gate and up projections once for every 2 XR of its tokens (launch_typed: the room goes by
// the experts' average, so a much fuller expert takes several passes).
// k_ffn_up is bound by its weight stream (2/3 of the layer's bytes), k_ffn_down by what follows
// its loads (below); with one token both by the chain launch - ids - weights - sum.
//
// Measured, kernel times: 64 experts of 4096 x 1024, 32 FP16 tokens, top-6: up 60 us (4.8 TB/s;
// a large copy reaches 5.05), down 65.5 us (2.2 TB/s: half of its wavefronts' time waits for
// loads and LDS, and every column tile reads all rows of h and takes them apart again).
// 256 experts of 6144 x 256, top-8: eight tokens 22.1 and 18.2 us, one token 9.5 and 6.0 us.
//
// Experts in use are found on the device: every workgroup marks the ids in an LDS
// bitmap and takes the r-th marked expert (ascending), so the grid needs only
// min(experts, pairs) ranks and no host knowledge of the routing.  k_ffn_up leaves one record
// per rank (expert, its first row of h, its tokens as a 64-bit mask) for k_ffn_down.
//
// h is kept in FP32, already times c.  k_ffn_down takes each value apart into three BF16 values
// of 8 significant bits each, whose sum is the value exactly (24 bits; BF16 has FP32's range), and
// multiplies all three on the matrix cores: nothing of h is rounded away.  (Two parts, rounded to
// 2^-17, were 1.5 us faster for the eight tokens and 15 for the 32; an FP32 output showed it.)
//
// The sum over a token's experts: every wavefront of k_ffn_down adds its experts'
// results, in ascending order, into a token array of its own in LDS, and the
// wavefronts' arrays are added in wavefront order: no atomics, and the same inputs give the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "launch.h"
#include "few_token_device.h"

namespace moe_fp4 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kDownWaves = 8;

// What k_ffn_up tells k_ffn_down about one rank.
struct __align__(16) RankRecord {
  int32_t expert;
  int32_t row0;  // first row of h of this expert
  uint32_t tokens_lo, tokens_hi;
};

// Dynamic LDS of k_ffn_up before the sums: ids and weights of every pair, the
// bitmap, and the expert's token list and coefficients.
__host__ __device__ constexpr size_t up_table_bytes(int pairs, int experts) {
  return ((size_t)pairs * 8 + (size_t)((experts + 31) / 32) * 4 + 64 * 8 + 15) / 16 * 16;
}

// A step's first two loads of x (four tokens) are kept in flight, the rest of a larger
// expert's are loaded when needed.
template <bool F16, int NT, int XR>
using FfnLoop = FewLoop<F16, NT, XR, (XR < 2 ? XR : 2), (NT > 1 && XR <= 2)>;

template <bool F16, int NT, int XR>
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
  char* work = smem + up_table_bytes(pairs, a.experts);

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
  typedef FfnLoop<F16, NT, XR> Loop;
  Loop loop;
  const int64_t wrow = (int64_t)expert * 2 * inter;
  loop.q_rs = make_rsrc(a.w13_q + wrow * (k / 2), (uint32_t)(2 * inter) * (uint32_t)(k / 2));
  loop.s_rs = make_rsrc(a.w13_sf + wrow * (k / 16), (uint32_t)(2 * inter) * (uint32_t)(k / 16));
  loop.x_rs = make_rsrc(a.x, (uint32_t)(((a.tokens - 1) * a.ld_x + k) * 2));
  loop.lds = work + wave * Loop::kLdsBytes;
  loop.k = k;
  loop.lane = lane;
  const int r = lane & 15;
#pragma unroll
  for (int t = 0; t < NT; ++t) {  // rows 0-7 of a tile: gate; 8-15: the same columns of up
    const int lr = Loop::row_of(lane);
    const int32_t col = c0 + 8 * t + (lr & 7);
    const uint32_t row = (uint32_t)((lr >> 3) * inter + (col < inter ? col : inter - 1));
    loop.q_off[t] = row * (uint32_t)(k / 2);
    loop.s_off[t] = row * (uint32_t)(k / 16);
  }
  const int32_t steps = (k + kFewStep - 1) / kFewStep;
  const int32_t s0 = uniform(wave * steps / waves), s1 = uniform((wave + 1) * steps / waves);
  const int tile = tid >> 6;
  // An expert of more than 2 XR tokens takes several passes over its weights.
  for (int32_t first = 0; first < rows; first += 2 * XR) {
    loop.tokens = rows - first < 2 * XR ? rows - first : 2 * XR;
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const int32_t j = 2 * i + (lane >> 5);
      loop.x_off[i] = j < loop.tokens ? (uint32_t)(list[first + j] * a.ld_x * 2 + 16 * (lane & 31)) : kOutOfRange;
    }
    float4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (first > 0) __syncthreads();  // the previous sums have been taken
    loop.run(acc, s0, s1);
    put_sums<NT>(loop.lds, acc, lane);
    __syncthreads();
    const int32_t j = first + r;
    const int32_t col = c0 + tile * 8 + 4 * ((lane >> 4) & 1);
    if (tile < NT && lane < 32 && r < loop.tokens && col < inter) {
      const float4_t gate = take_sum(work, Loop::kLdsBytes, tile, lane, waves);
      const float4_t up = take_sum(work, Loop::kLdsBytes, tile, lane + 32, waves);
      const float cf = coef[j];
      float4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu(gate[i] * scale) * (up[i] * scale) * cf;
      *reinterpret_cast<float4_t*>(a.h + ((int64_t)(row0 + j) * inter + col) * 4) = v;
    }
  }
}

// One wavefront's unit, 256 elements of K of one expert, on its way: codes, scales and
// the first PF rows of h.
template <int NT, int PF>
struct DownStage {
  RankRecord rec;
  Codes<NT> c;
  uint32_t s[NT];
  u32x4_t h[PF];
};

constexpr int kDepth = 2;     // units in flight
constexpr int kParts = 3;     // BF16 values that hold an FP32 one
constexpr int kRowGroup = 5;  // rows of h in one product: part p of row j in column 3 j + p
constexpr int kRowBytes = kParts * 512;  // a row's parts of a unit, in LDS

// Groups of rows that a dequantised weight is multiplied with at once: two where experts
// have several tokens (PF), which take more LDS.
__host__ __device__ constexpr int row_groups(int pf) { return pf > kRowGroup ? 2 : 1; }

// Four FP32 values as three BF16 parts each, by taking off the upper half twice: the three
// hold the leading, next and last 8 bits exactly.
__device__ __forceinline__ void split_h(u32x4_t v, u32x2_t (&parts)[kParts]) {
  float rest[4], last[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = v[i];
    rest[i] = __builtin_bit_cast(float, b) - __builtin_bit_cast(float, b & 0xFFFF0000u);
    const uint32_t m = __builtin_bit_cast(uint32_t, rest[i]) & 0xFFFF0000u;
    last[i] = rest[i] - __builtin_bit_cast(float, m);
  }
  const float sum = (last[0] + last[1]) + (last[2] + last[3]);
  if (__ballot(sum != sum)) {  // uniform: some value is not finite, and has no rest
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (last[i] != last[i]) rest[i] = last[i] = 0.0f;
  }
  auto upper = [](uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); };
  auto bits = [](float f) { return __builtin_bit_cast(uint32_t, f); };
  parts[0] = u32x2_t{upper(v[0], v[1]), upper(v[2], v[3])};
  parts[1] = u32x2_t{upper(bits(rest[0]), bits(rest[1])), upper(bits(rest[2]), bits(rest[3]))};
  parts[2] = u32x2_t{upper(bits(last[0]), bits(last[1])), upper(bits(last[2]), bits(last[3]))};
}

template <bool F16, int NT, int PF>
__global__ __launch_bounds__(kMaxThreads, PF > 4 ? 2 : 4) void k_ffn_down(FfnArgs a) {
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  constexpr int kCols = 16 * NT;
  constexpr int GR = row_groups(PF), kRows = GR * kRowGroup;  // rows multiplied at once
  const int hrows = a.tokens < kRows ? a.tokens : kRows;
  char* hs = smem + wave * hrows * kRowBytes;
  float* sums = reinterpret_cast<float*>(smem + waves * hrows * kRowBytes);  // [wave][token][kCols]
  int32_t* list = reinterpret_cast<int32_t*>(sums + (size_t)waves * a.tokens * kCols) + wave * 64;
  float* mysum = sums + (size_t)wave * a.tokens * kCols;
  const int32_t k = a.inter;
  const int32_t n0 = blockIdx.x * kCols;
  for (int i = lane; i < a.tokens * kCols; i += 64) mysum[i] = 0.0f;
  lds_handover();

  uint32_t q_off[NT], s_off[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int32_t c = n0 + 16 * t + r;
    const uint32_t row = (uint32_t)(c < a.hidden ? c : a.hidden - 1);
    q_off[t] = row * (uint32_t)(k / 2);
    s_off[t] = row * (uint32_t)(k / 16);
  }
  const rsrc_t h_rs = make_rsrc(a.h, (uint32_t)(a.tokens * a.topk) * (uint32_t)k * 4u);
  const int32_t steps = (k + kFewStep - 1) / kFewStep;
  const int32_t units = ((sconst_i32)a.ranks)[0] * steps;
  const int32_t u0 = uniform((int32_t)((int64_t)wave * units / waves));
  const int32_t u1 = uniform((int32_t)((int64_t)(wave + 1) * units / waves));

  auto tokens_of = [](const RankRecord& rec) { return (uint64_t)rec.tokens_hi << 32 | rec.tokens_lo; };
  // Byte offset of this lane's 16 bytes of row j of an expert's h.
  auto h_offset = [&](const RankRecord& rec, int32_t rows, int32_t step, int32_t j) {
    return j < rows && step * kFewStep + 4 * lane < k
               ? ((uint32_t)(rec.row0 + j) * (uint32_t)k + (uint32_t)(step * kFewStep)) * 4u + 16u * lane
               : kOutOfRange;
  };
  // 16-byte piece i (0..31, eight values) of column c is kept at piece i ^ c: sixteen columns' equal
  // pieces lie in different banks.
  auto put_h = [&](int j, u32x4_t v) {
    u32x2_t parts[kParts];
    split_h(v, parts);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int c = kParts * j + p;
      *reinterpret_cast<u32x2_t*>(hs + c * 512 + (((lane >> 1) ^ c) << 4) + 8 * (lane & 1)) = parts[p];
    }
  };
  // Where loading and computing stand: units in order are (rank, step).
  struct Cursor {
    int32_t rank, step;
  };
  auto advance = [&](Cursor& c) {
    if (++c.step == steps) c.step = 0, ++c.rank;
  };
  auto load = [&](DownStage<NT, PF>& d, const Cursor& c, bool on) {
    const sconst_i32 p = (sconst_i32)(const void*)(a.records + (on ? c.rank : 0));
    d.rec.expert = p[0], d.rec.row0 = p[1], d.rec.tokens_lo = (uint32_t)p[2], d.rec.tokens_hi = (uint32_t)p[3];
    const int64_t wrow = (int64_t)d.rec.expert * a.hidden;
    const rsrc_t q_rs = make_rsrc(a.w2_q + wrow * (k / 2), (uint32_t)a.hidden * (uint32_t)(k / 2));
    const rsrc_t s_rs = make_rsrc(a.w2_sf + wrow * (k / 16), (uint32_t)a.hidden * (uint32_t)(k / 16));
    load_codes<NT>(d.c, q_rs, q_off, on ? code_offset(c.step, g, k) : kOutOfRange);
    const uint32_t so = (uint32_t)(c.step * 16 + 4 * g), last = (uint32_t)(k / 16 - 4);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      d.s[t] = __builtin_amdgcn_raw_buffer_load_b32(
          s_rs, on ? s_off[t] + (so < last ? so : last) : kOutOfRange, 0, 0);
    const int32_t rows = on ? __popcll(tokens_of(d.rec)) : 0;
#pragma unroll
    for (int j = 0; j < PF; ++j)
      if (j < 2 || j < rows) d.h[j] = __builtin_amdgcn_raw_buffer_load_b128(h_rs, h_offset(d.rec, rows, c.step, j), 0, 0);
  };

  // The sums of a lane for the groups of rows.
  struct Sums {
    float4_t v[GR][NT][2];
  };
  auto clear = [&](Sums& s) {
#pragma unroll
    for (int q = 0; q < GR; ++q)
#pragma unroll
      for (int t = 0; t < NT; ++t) s.v[q][t][0] = s.v[q][t][1] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // The row of a group whose sum this lane carries, none for the columns of second and third parts.
  const int32_t my_row = r % kParts == 0 && r < kParts * kRowGroup ? r / kParts : INT32_MAX / 2;
  // Where the sums of that row of group q of rows first .. are in mysum, negative for none.
  auto place = [&](int32_t first, int q, int32_t rows) {
    const int32_t j = first + q * kRowGroup + my_row;
    return j < rows ? list[j] * kCols + 4 * g : -1;
  };
  // Add what a group of rows has summed to its tokens' sums, a row's three columns first.
  auto flush = [&](const float4_t (&s)[NT][2], int32_t to) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float4_t v = s[t][0] + s[t][1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = __builtin_bit_cast(int, (float)v[i]);  // the columns one and two to the right
        const float second = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x101, 0xf, 0xf, true));
        const float third = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x102, 0xf, 0xf, true));
        v[i] += second + third;
      }
      if (to >= 0) *reinterpret_cast<float4_t*>(mysum + to + 16 * t) += v;
    }
  };
  // Multiply the first G groups of the `here` rows in LDS.
  auto multiply = [&](DownStage<NT, PF> d, int32_t here, Sums& s, auto groups) {
    // Each product dequantises for itself: carried from one to the next, the weights' values
    // would take more registers than there are.
#pragma unroll
    for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(d.c.q[t][0]), "+v"(d.c.q[t][1]));
    constexpr int G = decltype(groups)::value;
    struct Operands {
      u32x4_t v[G];
    };
    uint32_t at[G];
#pragma unroll
    for (int q = 0; q < G; ++q) {
      const int32_t left = here - q * kRowGroup, last = kParts * (left < kRowGroup ? left : kRowGroup) - 1;
      const int32_t c = q * kParts * kRowGroup + (r < last ? r : last);
      at[q] = (uint32_t)(c * 512 + (((8 * g) ^ c) << 4));
    }
    for_operands<false, NT, 0>(
        d.c, d.s,
        [&](int j) {
          Operands x;
#pragma unroll
          for (int q = 0; q < G; ++q) x.v[q] = *reinterpret_cast<const u32x4_t*>(hs + (at[q] ^ (uint32_t)(j << 4)));
          return x;
        },
        [&](int j, int t, u32x4_t w, const Operands& x) {
#pragma unroll
          for (int q = 0; q < G; ++q) s.v[q][t][j & 1] = mfma16<false>(w, x.v[q], s.v[q][t][j & 1]);
        });
  };
  auto multiply_rows = [&](const DownStage<NT, PF>& d, int32_t here, Sums& s) {
    lds_handover();  // the rows have been written
    if (GR == 1 || here <= kRowGroup)
      multiply(d, here, s, std::integral_constant<int, 1>());
    else
      multiply(d, here, s, std::integral_constant<int, GR>());
    lds_handover();  // and read
  };
  // The expert being summed: its first rows' sums stay in registers until the expert ends.
  Sums acc;
  int32_t dest[GR];
  clear(acc);
  auto compute = [&](DownStage<NT, PF>& d, const Cursor& c, bool begins, bool ends) {
    const uint64_t tokens = tokens_of(d.rec);
    const int32_t rows = __popcll(tokens);
    if ((c.step + 1) * kFewStep > k) {
      const int32_t left = blocks_left(c.step * kFewStep + 64 * g, k);
      move_codes<NT>(d.c, left);
#pragma unroll
      for (int t = 0; t < NT; ++t) d.s[t] = left > 0 ? d.s[t] >> (8 * (4 - left)) : 0u;
    }
    if (begins) {
      lds_handover();  // the previous expert's tokens have been read
      if (tokens >> lane & 1) list[__popcll(tokens & ((1ull << lane) - 1))] = lane;
      lds_handover();
#pragma unroll
      for (int q = 0; q < GR; ++q) dest[q] = place(0, q, rows);
    }
#pragma unroll
    for (int j = 0; j < PF; ++j)
      if (j < rows) put_h(j, d.h[j]);
    for (int32_t j = PF; j < rows && j < kRows; ++j)
      put_h(j, __builtin_amdgcn_raw_buffer_load_b128(h_rs, h_offset(d.rec, rows, c.step, j), 0, 0));
    multiply_rows(d, rows < kRows ? rows : kRows, acc);
    for (int32_t first = kRows; first < rows; first += kRows) {  // an expert of many tokens
      const int32_t here = rows - first < kRows ? rows - first : kRows;
      for (int32_t j = 0; j < here; ++j)
        put_h(j, __builtin_amdgcn_raw_buffer_load_b128(h_rs, h_offset(d.rec, rows, c.step, first + j), 0, 0));
      Sums more;
      clear(more);
      multiply_rows(d, here, more);
#pragma unroll
      for (int q = 0; q < GR; ++q)
        if (q * kRowGroup < here) flush(more.v[q], place(first, q, rows));
    }
    if (ends) {
#pragma unroll
      for (int q = 0; q < GR; ++q)
        if (q * kRowGroup < rows) flush(acc.v[q], dest[q]);
      clear(acc);
    }
  };
  if (u0 < u1) {
    DownStage<NT, PF> st[kDepth];
    Cursor in{u0 / steps, u0 % steps}, at = in;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      load(st[d], in, u0 + d < u1);
      advance(in);
    }
    for (int32_t u = u0; u < u1; u += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (u + d < u1)
          compute(st[d], at, u + d == u0 || at.step == 0, u + d + 1 == u1 || at.step + 1 == steps);
        advance(at);
        load(st[d], in, u + d + kDepth < u1);
        advance(in);
      }
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

template <bool F16, int NT, int XR>
hipError_t launch_up(const FfnArgs& a, int waves, hipStream_t stream) {
  const int pairs = a.tokens * a.topk;
  const dim3 grid((a.inter + 8 * NT - 1) / (8 * NT), pairs < a.experts ? pairs : a.experts);
  const size_t lds = up_table_bytes(pairs, a.experts) + (size_t)waves * FfnLoop<F16, NT, XR>::kLdsBytes;
  hipLaunchKernelGGL((k_ffn_up<F16, NT, XR>), grid, dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
}

template <bool F16, int NT, int PF>
hipError_t launch_down(const FfnArgs& a, hipStream_t stream) {
  constexpr int kRows = row_groups(PF) * kRowGroup;
  const int hrows = a.tokens < kRows ? a.tokens : kRows;
  const size_t lds = (size_t)kDownWaves * (hrows * kRowBytes + (a.tokens * 16 * NT + 64) * 4);
  const dim3 grid((a.hidden + 16 * NT - 1) / (16 * NT));
  hipLaunchKernelGGL((k_ffn_down<F16, NT, PF>), grid, dim3(kDownWaves * 64), lds, stream, a);
  return hipGetLastError();
}

// k_ffn_up: two tiles an item and four wavefronts (64 experts, 32 tokens top-6, 4096 x
// 1024: the layer takes 122 us against 134 with one tile and 170 with one tile and eight
// wavefronts); where that leaves CUs without an item, one tile and eight wavefronts
// (one token, eight experts of 6144 x 256: 15.0 us against 15.2 with four and 17.9 with two tiles).
// Room for 2, 4, 8 or 16 tokens of an expert at once, by how many it has on average; the
// wavefronts that fit on a CU depend on it (the first layer above: 122 us with 8, 125
// with 16, 128 with 4; eight tokens of 256 experts 43 with 4, 44 with 8 and 16).
// k_ffn_down: eight wavefronts (121 us for the first layer, 43 for eight tokens of 256 experts,
// 15.0 for one; four: 153, 44 and 15.3; sixteen: 118, 47 and 18.5) and one tile (two were slower by
// a third).  Eight of the ten rows of h that are multiplied at once are kept in flight where experts
// have two tokens or more on average (121 against 135 us), else four of five (eight of ten: 50 us
// against 43 for the eight tokens, with one workgroup a CU instead of two).
template <bool F16>
hipError_t launch_typed(const FfnArgs& a, hipStream_t stream) {
  const int64_t pairs = (int64_t)a.tokens * a.topk;
  const int64_t tiles = (a.inter + 7) / 8 * (pairs < a.experts ? pairs : a.experts);
  const bool pair = tiles >= 512;
  hipError_t err;
  if (a.tokens <= 2)
    err = pair ? launch_up<F16, 2, 1>(a, 4, stream) : launch_up<F16, 1, 1>(a, 8, stream);
  else if (pairs <= a.experts)
    err = pair ? launch_up<F16, 2, 2>(a, 4, stream) : launch_up<F16, 1, 2>(a, 8, stream);
  else if (pairs <= 4 * (int64_t)a.experts)
    err = pair ? launch_up<F16, 2, 4>(a, 4, stream) : launch_up<F16, 1, 4>(a, 8, stream);
  else
    err = pair ? launch_up<F16, 2, 8>(a, 4, stream) : launch_up<F16, 1, 8>(a, 8, stream);
  if (err != hipSuccess) return err;
  if (a.tokens == 1) return launch_down<F16, 1, 1>(a, stream);
  return pairs >= 2 * (int64_t)a.experts ? launch_down<F16, 1, 8>(a, stream) : launch_down<F16, 1, 4>(a, stream);
}

}  // namespace

hipError_t launch_ffn(const FfnArgs& a, hipStream_t stream) {
  return a.x_f16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace moe_fp4

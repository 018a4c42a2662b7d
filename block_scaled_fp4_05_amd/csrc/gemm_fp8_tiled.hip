// FP8 block-scaled grouped product for experts of many rows and the dense case
// (moe_grouped_gemm_fp8), tiles of BM activation rows x BN weight rows a workgroup.
//
// Bound: the matrix cores for large dense products (8192^3: 480-512 us, 2.2 PFLOP/s), the weight stream
// for experts of some 16 rows (512 tokens of 256 experts of 512 x 6144: 140 us, 5.8 TB/s), the copies
// between them (4096 tokens of the same 253 us; 60 experts of 273 rows, 1444 x 1552: 99 us), with an
// FP32 result the conversions (4096 tokens 316 us, 4096^3 135).  A stage is one block of 128
// of every row of the tile, copied from memory straight into LDS (no registers) while the stage before
// it is multiplied.
// Each wavefront owns 128 weight rows x 16 MT activation rows, so a stage takes one weight scale
// (uniform) and MT activation scales (one a lane).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_fp8.h"

namespace moe_fp4 {
namespace {

// Weight row that is row i of a wavefront's 16-row tile t (of its 128): tiles 2p and 2p + 1
// interleave in fours, so that a lane's results of the two are eight consecutive columns, one
// 16-byte store of 16-bit values.
__device__ __forceinline__ int tile_row(int t, int i) { return 32 * (t >> 1) + 4 * (t & 1) + 8 * (i >> 2) + (i & 3); }

// Row r of a stage is 8 pieces of 16 bytes; piece c is stored at position c ^ swz(r).  A 16-byte
// LDS read serves 16 lanes a clock, lanes 0-3, 12-15 and 20-27 of a wavefront together, then
// 4-11, 16-19 and 28-31, and the same of the upper half: with pieces g and g + 1 of tile rows i as
// lanes (i, g) read them, every 16 touch 16 different 16-byte places of a 256-byte line (two
// rows) if swz is i / 2.  A swizzle that served 16 consecutive lanes alone made every read
// take twice as long.  Activation tiles are 16 consecutive rows, weight tiles tile_row's.
__device__ __forceinline__ int swz_a(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_w(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }


// R: stages in LDS.
template <int WN, int WM, int MT, int R>
struct Tile {
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int BN = 128 * WN, BM = 16 * MT * WM;
  static constexpr int kRows = BN + BM;         // weight rows, then activation rows
  static constexpr int kStage = kRows * 128;    // bytes
  static constexpr int kRound = kThreads / 8;   // rows that all threads copy at once
  static constexpr int kWRounds = BN / kRound, kARounds = BM / kRound, kCopies = kWRounds + kARounds;
  // Weight tiles, and stages of activation tiles, in registers: reads run WD - 1 tiles ahead, which
  // with few products a tile has to be more.
  static constexpr int WD = MT >= 3 ? 2 : 4, AD = MT >= 3 ? 1 : 2;
  static constexpr int kScales = BM > 64 * kWaves ? BM : 64 * kWaves;
  static_assert(BN % kRound == 0 && BM % kRound == 0 && kCopies % 2 == 0, "whole rounds, an even number");
};

// 16 (or 4) bytes a lane from memory to LDS: lane l's to `to` + 16 l (4 l), `to` uniform; ONCE:
// with the hint that they are not read again.  In
// assembly, because the compiler, which cannot tell the stages apart in a loop, otherwise waits
// for copies of later stages before it reads an earlier one; all waits for copies are
// stage_barrier's.  (The compiler sets M0 itself wherever it uses it.)  Five wait states: M0 before
// its use, and a scalar register that a vector instruction may just have written.
template <bool ONCE = false>
__device__ __forceinline__ void copy16(const u32x4_t& rs, uint8_t* to, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass has no such registers)
  typedef uint8_t __attribute__((address_space(3))) lds_byte;
  const uint32_t at = (uint32_t)(uintptr_t)(lds_byte*)to;
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(at), "v"(off), "s"(rs) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rs) : "memory");
#endif
}
__device__ __forceinline__ void copy4(const u32x4_t& rs, float* to, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef float __attribute__((address_space(3))) lds_float;
  const uint32_t at = (uint32_t)(uintptr_t)(lds_float*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rs) : "memory");
#endif
}

// A raw buffer resource as four words (make_rsrc's), in scalar registers whatever the compiler
// makes of the arguments.
__device__ __forceinline__ u32x4_t rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t at = (uint64_t)reinterpret_cast<uintptr_t>(base);
  return u32x4_t{(uint32_t)uniform((int32_t)at), (uint32_t)uniform((int32_t)(at >> 32)) & 0xFFFFu, (uint32_t)uniform((int32_t)bytes),
                 (uint32_t)kRawBufferWord3};
}

// Everything this wavefront has read from LDS is in registers and what it copied there is complete,
// but for its last LEFT copies; then all wavefronts meet.
template <int LEFT>
__device__ __forceinline__ void stage_barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
#endif
}

// Order of a tile's instructions: a product, then the additions of an earlier one.
template <int MT>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instruction
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // vector instructions
  }
}

// acc += d * s, here and not later: left alone, the compiler collects all of a stage's additions
// behind its last product, and with them all products.
__device__ __forceinline__ void add_scaled(float4_t& acc, const float4_t& d, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d[i], s, acc[i]);
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(acc));
#endif
}

template <int I>
struct Index {
  static constexpr int value = I;
};

// A wavefront's 16 MT x 128 results into `out`, from row row0 (rows of which there are) and column
// col0 on.  Where there is no row or column a store is sent out of range.
template <int MT, bool EXACT>
__device__ __forceinline__ void store_tile(const Fp8GemmArgs& p, const float4_t (&acc)[8][MT], int32_t row0, int32_t rows,
                                           int32_t first, int32_t col0, int r, int g) {
  const int32_t n = p.n;
  constexpr int es = EXACT ? 4 : 2;
  const rsrc_t o = make_rsrc(static_cast<char*>(p.out) + (int64_t)row0 * p.ldo * es, (uint32_t)rows * (uint32_t)p.ldo * es);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int32_t row = first + 16 * m + r;
    const uint32_t row_at = (uint32_t)row * (uint32_t)p.ldo;
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
      const int32_t col = col0 + tile_row(t, 4 * g);
      const uint32_t to = row < rows && col < n ? (row_at + (uint32_t)col) * es : kOutOfRange;
      const u32x4_t v = fp8_round8(acc[t][m], acc[t + 1][m], p.out_dtype);
      if (p.store_cols == 8) {
        if constexpr (EXACT) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[t][m]), o, to, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[t + 1][m]), o, to, 16, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(v, o, to, 0, 0);
        }
      } else if (p.store_cols == 4) {
        const uint32_t to_hi = col + 4 < n ? to + 4 * es : kOutOfRange;
        if constexpr (EXACT) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[t][m]), o, to, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[t + 1][m]), o, to_hi, 0, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{v[0], v[1]}, o, to, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{v[2], v[3]}, o, to_hi, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t to_i = col + i < n ? to + i * es : kOutOfRange;
          if constexpr (EXACT) {
            const float f = i < 4 ? acc[t][m][i & 3] : acc[t + 1][m][i & 3];
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, f), o, to_i, 0, 0);
          } else {
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[i >> 1] >> (16 * (i & 1))), o, to_i, 0, 0);
          }
        }
      }
    }
  }
}

template <int WN, int WM, int MT, bool EXACT, int R>
__global__ __launch_bounds__(64 * WN * WM) __attribute__((amdgpu_waves_per_eu(2, MT >= 3 ? 2 : 4)))
void k_gemm_fp8_tiled(Fp8GemmArgs p) {
  typedef Tile<WN, WM, MT, R> T;
  static_assert(R == 2 || (R == 3 && MT == 1), "with three stages the copies of one are counted");
  constexpr int WD = T::WD, AD = T::AD;
  __shared__ __align__(1024) uint8_t stages[R][T::kStage];
  __shared__ __align__(1024) float scales[R][T::kScales];  // of the stages' activation rows
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const int r = lane & 15, g = lane >> 4;
  const int32_t k = p.k, kbs = p.k_blocks, n = p.n;

  const Fp8Item it = fp8_item<T::kThreads>(p, T::BM, T::BN, 4);
  if (it.rows <= 0) return;

  // ---- copies: this thread moves piece lane % 8 of rows tid / 8 + kRound * j, swizzled, and
  // wavefront w the scales of activation rows 64 w ...
  // (swz_a has a period of 16 rows, swz_w of 32: every round's rows have the same pieces.)
  static_assert(T::kRound % 32 == 0, "rows of a round");
  const int piece_a = (lane & 7) ^ swz_a(tid >> 3), piece_w = (lane & 7) ^ swz_w(tid >> 3);
  const uint8_t* const w_base = p.w_q + (int64_t)it.e * n * k;
  // Without a row index the tile's rows follow each other: offsets from its first row.
  const int64_t base = p.a_row_index ? 0 : it.row0, a_rows = p.a_row_index ? p.a_rows : (int64_t)it.rows;
  uint32_t off[T::kCopies], scale_off;
#pragma unroll
  for (int j = 0; j < T::kWRounds; ++j) {
    const int32_t row = it.n0 + (tid >> 3) + T::kRound * j;
    off[j] = (uint32_t)(row < n ? row : n - 1) * (uint32_t)k + 16u * piece_w;
  }
  {
    int32_t row[T::kARounds + 1];
#pragma unroll
    for (int j = 0; j < T::kARounds; ++j) row[j] = min((tid >> 3) + T::kRound * j, it.rows - 1);
    row[T::kARounds] = min(tid, it.rows - 1);
    if (p.a_row_index) {
      const int32_t last = (int32_t)p.a_rows - 1;
#pragma unroll
      for (int j = 0; j <= T::kARounds; ++j) row[j] = p.a_row_index[it.row0 + row[j]];
#pragma unroll
      for (int j = 0; j <= T::kARounds; ++j) row[j] = min(max(row[j], 0), last);
    }
#pragma unroll
    for (int j = 0; j < T::kARounds; ++j) off[T::kWRounds + j] = (uint32_t)row[j] * (uint32_t)k + 16u * piece_a;
    scale_off = (uint32_t)row[T::kARounds] * (uint32_t)kbs * 4u;
  }
  // A piece past k (only the last block has any) is copied from the row's start instead: its
  // products are made zero below, and a NaN there is in the result already.  Behind the last
  // block nothing is fetched (a resource of no bytes, without a branch).
  const u32x4_t w_rs = rsrc_words(w_base, (uint32_t)n * (uint32_t)k);
  const u32x4_t a_rs = rsrc_words(p.a_q + base * k, (uint32_t)(a_rows * k));
  const u32x4_t s_rs = rsrc_words(p.a_sf + base * kbs, (uint32_t)(a_rows * kbs * 4));
  const uint32_t last_at = (uint32_t)(kbs - 1) * 128u;
  const uint32_t last_w = last_at + 16u * piece_w >= (uint32_t)k ? 0u - 16u * piece_w : last_at;
  const uint32_t last_a = last_at + 16u * piece_a >= (uint32_t)k ? 0u - 16u * piece_a : last_at;
  auto within = [&](const u32x4_t& rs, int32_t b) { return u32x4_t{rs[0], rs[1], b < kbs ? rs[2] : 0u, rs[3]}; };
  auto copy = [&](uint8_t* to, int32_t b, int from, int end) {
    const u32x4_t w_now = within(w_rs, b), a_now = within(a_rs, b);
    const uint32_t here = (uint32_t)b * 128u;
    const uint32_t at_w = b == kbs - 1 ? last_w : here, at_a = b == kbs - 1 ? last_a : here;
    const int w_end = end < T::kWRounds ? end : T::kWRounds;
    // Weights that no other workgroup reads do not stay in the caches (512 tokens of 256 experts 139
    // us instead of 154; experts of 64 rows, where a second tile often reads them too, 155 instead
    // of 133 with the hint for all, 133 so.  Not in taller tiles: ragged experts 104 instead of 101.)
    if (MT == 1 && it.once) {
#pragma unroll
      for (int j = from; j < w_end; ++j) copy16<true>(w_now, to + (T::kRound * j + 8 * wave) * 128, off[j] + at_w);
    } else {
#pragma unroll
      for (int j = from; j < w_end; ++j) copy16(w_now, to + (T::kRound * j + 8 * wave) * 128, off[j] + at_w);
    }
#pragma unroll
    for (int j = from < T::kWRounds ? T::kWRounds : from; j < end; ++j) {
      // Eight activation rows that are not there stay what they were: they reach only results that
      // are not stored.  (Ragged experts of 273 rows on average 105 -> 101 us; but tiles of 64
      // rows copy their last row again, 512 tokens of 256 experts 165 us, left out 172.)
      if (MT >= 2 && T::kRound * (j - T::kWRounds) + 8 * wave >= it.rows) continue;
      copy16(a_now, to + (T::kRound * j + 8 * wave) * 128, off[j] + at_a);
    }
  };
  auto copy_scales = [&](float* to, int32_t b) { copy4(within(s_rs, b), to + 64 * wave, scale_off + (uint32_t)b * 4u); };

  // ---- products
  const float* const w_sf = p.w_sf + ((int64_t)it.e * p.n_blocks + min(it.n0 / kFp8Block + wn, p.n_blocks - 1)) * kbs;
  float4_t acc[8][MT];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // Pieces g and 4 + g of this lane's row of a 16-row tile.
  const int at_w = tile_row(0, r) * 128 + 16 * (g ^ (r >> 1)), at_a = r * 128 + 16 * (g ^ (r >> 1));
  auto fragment = [&](const uint8_t* from, int row0, int at) {
    const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(from + row0 * 128 + at);
    const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(from + row0 * 128 + (at ^ 64));
    return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  typedef typename Operand<EXACT>::type operand_t;
  i32x8_t a[AD][MT], w[WD];
  float4_t d[MT];
  float next_w = ((sconst_f32)w_sf)[0];
  auto read_w = [&](const uint8_t* from, int t) { w[t % WD] = fragment(from, 128 * wn + tile_row(t, 0), at_w); };
  auto read_a = [&](const uint8_t* from, i32x8_t (&to)[MT], int m) { to[m] = fragment(from, T::BN + 16 * (MT * wm + m), at_a); };

  // One stage, tile by tile: a tile's products are issued while tiles ahead are read and the tile
  // before it is scaled and added.  The last two tiles wait in registers for the barrier, behind
  // which the stage's place is filled anew, two stages ahead, and the next stage's first operands
  // are read while those tiles are multiplied.  The fences keep the compiler from reading all
  // tiles first, which spills.
  // A stage's copies are issued in four parts.  256 x 256: behind the barrier (tiles 6 and 7) and in
  // the next stage's tiles 0 and 1, so that a wavefront's products do not queue behind eight of
  // them (8192^3: 5% less than with all behind the barrier); smaller tiles behind the barrier, since
  // what they wait for is the copies (4096 tokens of 256 experts: 259 us, spread 277).
  constexpr int kPart = MT >= 3 ? T::kCopies / 4 : T::kCopies / 2;
  constexpr int kLeft = (R - 2) * (T::kCopies + 1);  // copies that may still be on their way
  int i = 0;  // the stage's place
  auto after = [](int x) { return x + 1 == R ? 0 : x + 1; };
  auto step = [&](auto which, int32_t b) {
    constexpr int S = decltype(which)::value;
    if (R == 2) i = S;
    uint8_t *const cur = stages[i], *const nxt = stages[after(i)];
    i32x8_t(&now_a)[MT] = a[S % AD];
    i32x8_t(&next_a)[MT] = a[(S + 1) % AD];
    if (b == kbs - 1 && k % kFp8Block != 0) {
      const bool z0 = b * 128 + 16 * g >= k, z1 = b * 128 + 64 + 16 * g >= k;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (z0) now_a[m][i] = 0;
          if (z1) now_a[m][4 + i] = 0;
        }
    }
    float scale[MT], sa[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sa[m] = scales[i][16 * (MT * wm + m) + r];
      scale[m] = sa[m] * next_w;
    }
    if (fp8_some_far(scale)) {
      fp8_add_far<8, MT, EXACT, true>(acc, now_a, sa, next_w, scale,
                                      [&](int t) { return fragment(cur, 128 * wn + tile_row(t, 0), at_w); });
      fp8_drop_far(scale);
    }
    next_w = ((sconst_f32)w_sf)[b + 1 < kbs ? b + 1 : b];
    operand_t ao[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ao[m] = Operand<EXACT>::of(now_a[m]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      if (t == 6) {
        stage_barrier<kLeft>();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (AD == 2) {
#pragma unroll
          for (int m = 0; m < MT; ++m) read_a(nxt, next_a, m);
        }
      }
      const operand_t wo = Operand<EXACT>::of(w[t % WD]);
      if (t + WD - 1 < (WD == 2 ? 7 : 8)) read_w(cur, t + WD - 1);  // (two buffers: tile 7 below)
      if (t == 6) {
#pragma unroll
        for (int j = 0; j < WD - 2; ++j) read_w(nxt, j);
      }
      if (t == 7) read_w(nxt, WD - 2);
      if (t == 6) copy(cur, b + R, 0, kPart);
      if (t == 7) {
        copy(cur, b + R, kPart, 2 * kPart);
        copy_scales(scales[i], b + R);
      }
      if (t == 0) copy(nxt, b + 1, 2 * kPart, min(3 * kPart, T::kCopies));
      if (t == 1) copy(nxt, b + 1, 3 * kPart, T::kCopies);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float4_t now = fp8_block_product(wo, ao[m]);
        if (t > 0) add_scaled(acc[t - 1][m], d[m], scale[m]);
        d[m] = now;
        if (AD == 1 && t == 7) {
          __builtin_amdgcn_sched_barrier(0);
          read_a(nxt, next_a, m);
        }
      }
      if (WD == 2 && t == 5) {  // where tile 5's registers are free
        __builtin_amdgcn_sched_barrier(0);
        read_w(cur, 7);
      }
      interleave<MT>();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m) add_scaled(acc[7][m], d[m], scale[m]);
    i = after(i);
  };

  copy(stages[0], 0, 0, T::kCopies);
  copy_scales(scales[0], 0);
  if constexpr (R == 3) {  // every stage's copies are kCopies and one: none is left out
    copy(stages[1], 1, 0, T::kCopies);
    copy_scales(scales[1], 1);
    stage_barrier<T::kCopies + 1>();
    copy(stages[2], 2, 0, T::kCopies);
    copy_scales(scales[2], 2);
  } else {
    stage_barrier<0>();
    copy(stages[1], 1, 0, 2 * kPart);
    copy_scales(scales[1], 1);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) read_a(stages[0], a[0], m);
#pragma unroll
  for (int t = 0; t < WD - 1; ++t) read_w(stages[0], t);
  if (16 * MT * wm < it.rows) {
    for (int32_t b = 0; b < kbs; b += 2) {
      step(Index<0>{}, b);
      if (b + 1 < kbs) step(Index<1>{}, b + 1);
    }
  } else {  // no rows here: its copies, and the matrix core is another workgroup's (4096 tokens of 256 experts 260 -> 255 us)
    for (int32_t b = 0; b < kbs; ++b) {
      copy(stages[after(i)], b + 1, 2 * kPart, T::kCopies);
      stage_barrier<kLeft>();
      copy(stages[i], b + R, 0, 2 * kPart);
      copy_scales(scales[i], b + R);
      i = after(i);
    }
  }
  // Nothing is on its way into LDS when the workgroup ends.
  stage_barrier<0>();

  store_tile<MT, EXACT>(p, acc, it.row0, it.rows, 16 * MT * wm, it.n0 + 128 * wn, r, g);
}

// Products of KB blocks, up to four: a workgroup keeps its 64 MT activation rows in registers and
// runs along `span` tiles of 128 weight rows, a stage in LDS being one block of a tile.
// Rows are found, read and scaled once and the copies never stop, where the kernel above spends
// most of a short item on its start and its end.  Bound: the weights and results (6144 x 256,
// 256 experts: 512 tokens 82 us, 5.5 TB/s; 4096 tokens 172 us, 4.7 TB/s).
constexpr int kShortRing = 3;

template <int KB, int MT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(KB * MT <= 4 ? 3 : 2, 3)))
void k_gemm_fp8_short(Fp8GemmArgs p) {
  constexpr int R = kShortRing, kCopies = 4, WD = 4;
  __shared__ __align__(1024) uint8_t stages[R][128 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int32_t k = p.k, n = p.n;

  const Fp8Item it = fp8_item<256>(p, 64 * MT, 128 * p.span, 4);
  if (it.rows <= 0) return;
  const int32_t tiles = min(p.span, (n - it.n0 + 127) / 128), all = tiles * KB;

  // ---- copies of weights, as in the kernel above
  const int piece = (lane & 7) ^ swz_w(tid >> 3);
  const u32x4_t w_rs = rsrc_words(p.w_q + (int64_t)it.e * n * k, (uint32_t)n * (uint32_t)k);
  // Block b's (static) piece; one past k is copied from the row's start (its products are zero).
  auto copy = [&](uint8_t* to, int b, int32_t tile) {
    const u32x4_t now = u32x4_t{w_rs[0], w_rs[1], tile < tiles ? w_rs[2] : 0u, w_rs[3]};
    const int32_t at = b * 128 + 16 * piece;
    const uint32_t in_row = at < k ? (uint32_t)at : 0u;
    uint32_t from[kCopies];
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      from[j] = (uint32_t)min(it.n0 + 128 * tile + (tid >> 3) + 32 * j, n - 1) * (uint32_t)k + in_row;
    if (it.once) {  // (6144 x 256: 85 us instead of 94; K = 512: 150 instead of 170)
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy16<true>(now, to + (32 * j + 8 * wave) * 128, from[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy16(now, to + (32 * j + 8 * wave) * 128, from[j]);
    }
  };
#pragma unroll
  for (int s = 0; s < R; ++s) copy(stages[s], s % KB, s / KB);

  // ---- this wavefront's rows; the pieces past k are zeros
  const bool live = 16 * MT * wave < it.rows;
  i32x8_t a[KB][MT];
  float sa[KB][MT];
  if (live) {
    const int64_t base = p.a_row_index ? 0 : it.row0, a_rows = p.a_row_index ? p.a_rows : (int64_t)it.rows;
    const rsrc_t a_rs = make_rsrc(p.a_q + base * k, (uint32_t)(a_rows * k));
    const rsrc_t s_rs = make_rsrc(p.a_sf + base * KB, (uint32_t)(a_rows * KB * 4));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      int32_t row = min(16 * (MT * wave + m) + r, it.rows - 1);
      if (p.a_row_index) row = min(max(p.a_row_index[it.row0 + row], 0), (int32_t)p.a_rows - 1);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const int32_t at = 128 * b + 16 * g;
        const uint32_t from = (uint32_t)row * (uint32_t)k + (uint32_t)at;
        const u32x4_t lo = __builtin_amdgcn_raw_buffer_load_b128(a_rs, at < k ? from : kOutOfRange, 0, 0);
        const u32x4_t hi = __builtin_amdgcn_raw_buffer_load_b128(a_rs, at + 64 < k ? from + 64 : kOutOfRange, 0, 0);
        a[b][m] = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
        sa[b][m] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(s_rs, (uint32_t)(row * KB + b) * 4u, 0, 0));
      }
    }
  }

  // ---- products
  const float* const w_sf = p.w_sf + ((int64_t)it.e * p.n_blocks + it.n0 / kFp8Block) * KB;  // of stage s at s
  const int at_w = tile_row(0, r) * 128 + 16 * (g ^ (r >> 1));
  i32x8_t w[WD];
  auto fragment = [&](const uint8_t* from, int t) {
    const uint8_t* const row = from + tile_row(t, 0) * 128;
    const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(row + at_w);
    const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(row + (at_w ^ 64));
    return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto read_w = [&](const uint8_t* from, int t) { w[t % WD] = fragment(from, t); };
  auto after = [](int x) { return x + 1 == R ? 0 : x + 1; };
  float4_t acc[8][MT], d[MT];
  float next_w = ((sconst_f32)w_sf)[0];
  int i = 0;  // the stage's place
  // (What a wavefront has loaded for itself is older than the copies that may still be on their way.)
  auto step = [&](auto which, int32_t tile) {
    constexpr int b = decltype(which)::value;
    uint8_t *const cur = stages[i], *const nxt = stages[after(i)];
    const int32_t s = tile * KB + b;
    float scale[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) scale[m] = sa[b][m] * next_w;
    if (fp8_some_far(scale)) {
      fp8_add_far<8, MT, false, true>(acc, a[b], sa[b], next_w, scale, [&](int t) { return fragment(cur, t); });
      fp8_drop_far(scale);
    }
    next_w = ((sconst_f32)w_sf)[s + 1 < all ? s + 1 : s];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      if (t == 6) {
        stage_barrier<(R - 2) * kCopies>();
        __builtin_amdgcn_sched_barrier(0);
      }
      const i32x8_t wo = w[t % WD];
      if (t + WD - 1 < 8) read_w(cur, t + WD - 1);
      if (t == 6) {
#pragma unroll
        for (int j = 0; j < WD - 2; ++j) read_w(nxt, j);
        copy(cur, (b + R) % KB, tile + (b + R) / KB);
      }
      if (t == 7) read_w(nxt, WD - 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float4_t now = fp8_block_product(wo, a[b][m]);
        if (t > 0) add_scaled(acc[t - 1][m], d[m], scale[m]);
        d[m] = now;
      }
      interleave<MT>();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m) add_scaled(acc[7][m], d[m], scale[m]);
    i = after(i);
  };
  stage_barrier<0>();
  if (live) {
#pragma unroll
    for (int t = 0; t < WD - 1; ++t) read_w(stages[0], t);
    for (int32_t tile = 0; tile < tiles; ++tile) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      step(Index<0>{}, tile);
      if constexpr (KB > 1) step(Index<1>{}, tile);
      if constexpr (KB > 2) step(Index<2>{}, tile);
      if constexpr (KB > 3) step(Index<3>{}, tile);
      store_tile<MT, false>(p, acc, it.row0, it.rows, 16 * MT * wave, it.n0 + 128 * tile, r, g);
    }
  } else {
    for (int32_t tile = 0; tile < tiles; ++tile)
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        stage_barrier<(R - 2) * kCopies>();
        copy(stages[i], (b + R) % KB, tile + (b + R) / KB);
        i = after(i);
      }
  }
  // Nothing is on its way into LDS when the workgroup ends.
  stage_barrier<0>();
}

// Sets how results are stored; workgroups for every tile of bm rows.
dim3 fp8_grid(Fp8GemmArgs& p, int bm, uint64_t es) {
  // Columns that can be stored together everywhere: 8 (16-bit results) or 4 of them in one piece.
  const uint64_t where = reinterpret_cast<uintptr_t>(p.out) | (uint64_t)p.ldo * es;
  p.store_cols = where % 16 == 0 && p.n % 8 == 0 ? 8 : where % (4 * es) == 0 && p.n % 4 == 0 ? 4 : 1;
  const int64_t items = (fp8_most_items(p, bm) + 7) / 8 * 8, row = 1 << 16;
  return items <= row ? dim3((unsigned)items) : dim3((unsigned)row, (unsigned)((items + row - 1) / row));
}

template <int WN, int WM, int MT, bool EXACT, int R>
hipError_t launch(Fp8GemmArgs p, hipStream_t stream) {
  typedef Tile<WN, WM, MT, R> T;
  p.n_tiles = (p.n + T::BN - 1) / T::BN;
  const dim3 grid = fp8_grid(p, T::BM, EXACT ? 4 : 2);
  hipLaunchKernelGGL((k_gemm_fp8_tiled<WN, WM, MT, EXACT, R>), grid, dim3(T::kThreads), 0, stream, p);
  return hipGetLastError();
}

template <int KB, int MT>
hipError_t launch_short(Fp8GemmArgs p, hipStream_t stream) {
  p.n_tiles = (p.n + 128 * p.span - 1) / (128 * p.span);
  const dim3 grid = fp8_grid(p, 64 * MT, 2);
  hipLaunchKernelGGL((k_gemm_fp8_short<KB, MT>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_short_sized(const Fp8GemmArgs& p, hipStream_t stream) {
  switch (p.k_blocks) {
    case 1: return launch_short<1, MT>(p, stream);
    case 2: return launch_short<2, MT>(p, stream);
    case 3: return launch_short<3, MT>(p, stream);
    default: return launch_short<4, MT>(p, stream);
  }
}

// The tile by the average rows of an expert; both sides in us:
//   64 x 128 below 96 rows (6144 x 256, 32 rows: 123 against 153 with 128 x 128), and while 128 x
//     128 would leave CUs without two workgroups (dense 8192 x 6144, 256 rows: 34 against 38); with
//     three stages in LDS, two workgroups a CU instead of three, from
//     32 blocks (512 tokens of 256 experts, 512 x 6144: 141 against 151 with two stages; 512 x 4096:
//     114 and 131; 512 x 1024: 31 and 33; 6144 x 512: 187 and 173; FP32 results the same);
//   256 x 256 from 384 rows (8 experts of 8192 x 4096, 512 rows: 147 against 200 with 128 x 128;
//     1024 rows: 275 against 378; 64 experts of 2048 x 4096, 256 rows: 225 against 233, in another
//     session 260 against 253) where they
//     fill most of a round of 256 CUs (dense 8192^2, 2048 rows: 122 against 161; 8192 x 4096, 2500
//     rows, 320 tiles: 110 against 101);
//   128 x 128 else (4096 tokens of 256 experts, 512 x 6144: 253 against 266 with 64 x 128).
//   Up to four blocks the workgroups that run along the weights' tiles, of 64 or 128 rows as above,
//     four tiles each or, so that there are 512 at least, two or three (512 tokens of 256 experts,
//     6144 x 256: 82 against 112, 4096 tokens 172 against 268; 6144 x 512: 153 against 173 and 252 against 347;
//     dense 8192 x 8192 x 256 34 against 48; with eight tiles 84, 178, 156, 254 and 32); below 1024
//     tiles those above (dense 4096 x 256, 512 rows: 7.1 both).
template <bool EXACT>
hipError_t launch_sized(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t experts = p.m_total < p.experts ? p.m_total : p.experts, avg = p.m_total / p.experts;
  const int64_t middle = (p.m_total / 128 + experts) * ((p.n + 127) / 128);
  const bool low = avg < 96 || middle < 512;
  if (!EXACT && p.k_blocks <= 4) {
    const int64_t tiles = (p.m_total / (low ? 64 : 128) + experts) * ((p.n + 127) / 128);
    if (tiles >= 1024) {
      Fp8GemmArgs a = p;
      a.span = tiles < 2048 ? (int32_t)(tiles / 512) : 4;
      return low ? launch_short_sized<1>(a, stream) : launch_short_sized<2>(a, stream);
    }
  }
  if (low)
    return !EXACT && p.k_blocks >= 32 ? launch<1, 4, 1, false, 3>(p, stream) : launch<1, 4, 1, EXACT, 2>(p, stream);
  const int64_t big = (p.m_total + 255) / 256 * ((p.n + 255) / 256), rest = big % 256;
  if (!EXACT && avg >= 384 && big >= 224 && (rest == 0 || rest >= 160 || big >= 1024))
    return launch<2, 4, 4, false, 2>(p, stream);
  return launch<1, 4, 2, EXACT, 2>(p, stream);
}

}  // namespace

hipError_t launch_gemm_fp8_tiled(const Fp8GemmArgs& p, hipStream_t stream) {
  return p.out_dtype == kFewOutF32 ? launch_sized<true>(p, stream) : launch_sized<false>(p, stream);
}

}  // namespace moe_fp4

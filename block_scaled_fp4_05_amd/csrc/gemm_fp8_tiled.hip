// FP8 block-scaled grouped product for experts of many rows and the dense case
// (moe_grouped_gemm_fp8), tiles of BM activation rows x BN weight rows a workgroup.
//
// Bound: the matrix cores.  A stage is one block of 128 of every row of the tile, copied from
// memory straight into LDS (no registers) while the stage before it is multiplied.
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

template <int WN, int WM, int MT, bool EXACT>
struct Tile {
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int BN = 128 * WN, BM = 16 * MT * WM;
  static constexpr int kRows = BN + BM;         // weight rows, then activation rows
  static constexpr int kStage = kRows * 128;    // bytes
  static constexpr int kRound = kThreads / 8;   // rows that all threads copy at once
  static constexpr int kWRounds = BN / kRound, kARounds = BM / kRound;
  static_assert(BN % kRound == 0 && BM % kRound == 0, "whole rounds");
};

// 16 bytes a lane from memory to LDS: lane l's to `to` + 16 l (uniform).
__device__ __forceinline__ void copy16(rsrc_t rs, uint8_t* to, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass knows neither this width nor the registers below)
  typedef uint8_t __attribute__((address_space(3))) lds_byte;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_byte*)to, 16, off, 0, 0, 0);
#endif
}

// What the matrix cores are given.
template <bool EXACT>
struct Operand {
  typedef i32x8_t type;
  static __device__ __forceinline__ const i32x8_t& of(const i32x8_t& x) { return x; }
};
template <>
struct Operand<true> {
  typedef Half32 type;
  static __device__ __forceinline__ Half32 of(const i32x8_t& x) { return fp8_widen(x); }
};

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

template <int WN, int WM, int MT, bool EXACT>
__global__ __launch_bounds__(64 * WN * WM) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_gemm_fp8_tiled(Fp8GemmArgs p) {
  typedef Tile<WN, WM, MT, EXACT> T;
  __shared__ __align__(1024) uint8_t stage0[T::kStage], stage1[T::kStage];
  const Fp8Item it = fp8_locate<T::kThreads>(p, T::BM, T::BN, 4);
  if (it.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const int r = lane & 15, g = lane >> 4;
  const int32_t k = p.k, kbs = p.k_blocks, n = p.n;

  // What this thread copies: piece (lane % 8) of rows tid / 8 + kRound * j, swizzled.
  const uint8_t* const w_base = p.w_q + (int64_t)it.e * n * k;
  const uint32_t w_bytes = (uint32_t)n * (uint32_t)k;
  const int64_t base = p.a_row_index ? 0 : it.row0;
  const int64_t a_rows = p.a_row_index ? p.a_rows : it.rows;
  const uint8_t* const a_base = p.a_q + base * k;
  const uint32_t a_bytes = (uint32_t)(a_rows * k);
  const int piece_w = (lane & 7) ^ swz_w(tid >> 3), piece_a = (lane & 7) ^ swz_a(tid >> 3);
  uint32_t off[T::kWRounds + T::kARounds];
#pragma unroll
  for (int j = 0; j < T::kWRounds; ++j) {
    const int32_t row = it.n0 + (tid >> 3) + T::kRound * j;
    off[j] = (uint32_t)(row < n ? row : n - 1) * (uint32_t)k + 16u * piece_w;
  }
#pragma unroll
  for (int j = 0; j < T::kARounds; ++j) {
    const int32_t row = (tid >> 3) + T::kRound * j;
    const int32_t src = fp8_source_row(p, it.row0 + (row < it.rows ? row : it.rows - 1)) - (int32_t)base;
    off[T::kWRounds + j] = (uint32_t)src * (uint32_t)k + 16u * piece_a;
  }
  // A piece past k (only the last block has any) is copied from the row's start instead: its
  // products are made zero below, and a NaN there is in the result already.
  // Behind the last block nothing is fetched (a resource of no bytes, without a branch).
  auto copy = [&](uint8_t* stage, int32_t b, int j) {
    const uint32_t kk = (uint32_t)b * 128;
    const int piece = j < T::kWRounds ? piece_w : piece_a;
    const uint32_t at = b * 128 + 16 * piece >= k ? 0u - 16u * piece : kk;
    const bool in = b < kbs;
    const rsrc_t rs = j < T::kWRounds ? make_rsrc(w_base, in ? w_bytes : 0u) : make_rsrc(a_base, in ? a_bytes : 0u);
    copy16(rs, stage + (T::kRound * j + 8 * wave) * 128, off[j] + at);
  };

  // Scales: one weight scale a block, one activation scale a lane and 16 rows.
  const int32_t nb = min(it.n0 / kFp8Block + wn, p.n_blocks - 1);
  const float* w_sf = p.w_sf + ((int64_t)it.e * p.n_blocks + nb) * kbs;
  const float* a_sf[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int32_t row = 16 * (MT * wm + m) + r;
    a_sf[m] = p.a_sf + (int64_t)fp8_source_row(p, it.row0 + (row < it.rows ? row : it.rows - 1)) * kbs;
  }

  float4_t acc[8][MT];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Pieces g and 4 + g of this lane's row of a 16-row tile.
  const int at_w = tile_row(0, r) * 128 + 16 * (g ^ (r >> 1)), at_a = r * 128 + 16 * (g ^ (r >> 1));
  auto fragment = [&](const uint8_t* stage, int row0, int at) {
    const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(stage + row0 * 128 + at);
    const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(stage + row0 * 128 + (at ^ 64));
    return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  typedef typename Operand<EXACT>::type operand_t;
  i32x8_t a[MT], w[2];
  float scale[MT], next[MT], next_w = ((sconst_f32)w_sf)[0];
  float4_t d[MT];
  auto read_w = [&](const uint8_t* stage, int t) { w[t & 1] = fragment(stage, 128 * wn + tile_row(t, 0), at_w); };
  auto read_a = [&](const uint8_t* stage, int m) { a[m] = fragment(stage, T::BN + 16 * (MT * wm + m), at_a); };

  // One stage, tile by tile: tile t's products are issued while tile t + 1 is read and tile t - 1
  // is scaled and added; the copies of the next stage are spread over the first tiles.  The
  // last two tiles wait in registers for the barrier: their products run while the next
  // stage's first operands are read.  The fences keep the compiler from reading all tiles
  // first, which spills.
  constexpr int kCopies = T::kWRounds + T::kARounds, kPerTile = (kCopies + 1) / 2;
  auto step = [&](uint8_t* cur, uint8_t* nxt, int32_t b) {
    const bool more = b + 1 < kbs;
    if (b == kbs - 1 && k % kFp8Block != 0) {
      const bool z0 = b * 128 + 16 * g >= k, z1 = b * 128 + 64 + 16 * g >= k;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (z0) a[m][i] = 0;
          if (z1) a[m][4 + i] = 0;
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) scale[m] = next[m] * next_w;
    const int32_t ahead = more ? b + 1 : b;
    next_w = ((sconst_f32)w_sf)[ahead];
#pragma unroll
    for (int m = 0; m < MT; ++m) next[m] = a_sf[m][ahead];
    operand_t ao[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ao[m] = Operand<EXACT>::of(a[m]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      if (t == 6) {
        __syncthreads();  // the next stage is there, and this one is in registers
        __builtin_amdgcn_sched_barrier(0);
      }
      const operand_t wo = Operand<EXACT>::of(w[t & 1]);
      if (t < 6) read_w(cur, t + 1);  // (tile 7 below, where tile 5's registers are free)
      if (t == 7) read_w(nxt, 0);
      if (t >= 6) {
#pragma unroll
        for (int j = (t - 6) * kPerTile; j < (t - 5) * kPerTile && j < kCopies; ++j) copy(cur, b + 2, j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float4_t now = fp8_block_product(wo, ao[m]);
        if (t > 0) add_scaled(acc[t - 1][m], d[m], scale[m]);
        d[m] = now;
        if (t == 7) {
          __builtin_amdgcn_sched_barrier(0);
          read_a(nxt, m);
        }
      }
      if (t == 5) {
        __builtin_amdgcn_sched_barrier(0);
        read_w(cur, 7);
      }
      interleave<MT>();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m) add_scaled(acc[7][m], d[m], scale[m]);
  };

#pragma unroll
  for (int m = 0; m < MT; ++m) next[m] = a_sf[m][0];
#pragma unroll
  for (int j = 0; j < kCopies; ++j) copy(stage0, 0, j);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kCopies; ++j) copy(stage1, 1, j);
  read_w(stage0, 0);
#pragma unroll
  for (int m = 0; m < MT; ++m) read_a(stage0, m);
  for (int32_t b = 0; b < kbs; b += 2) {
    step(stage0, stage1, b);
    if (b + 1 < kbs) step(stage1, stage0, b + 1);
  }

  // Nothing is on its way into LDS when the workgroup ends.
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int32_t row = 16 * (MT * wm + m) + r;
    if (row >= it.rows) continue;
#pragma unroll
    for (int t = 0; t < 8; t += 2)
      fp8_store8(p, (int64_t)it.row0 + row, it.n0 + 128 * wn + tile_row(t, 4 * g), acc[t][m], acc[t + 1][m]);
  }
}

template <int WN, int WM, int MT, bool EXACT>
hipError_t launch(Fp8GemmArgs p, hipStream_t stream) {
  typedef Tile<WN, WM, MT, EXACT> T;
  p.n_tiles = (p.n + T::BN - 1) / T::BN;
  hipLaunchKernelGGL((k_gemm_fp8_tiled<WN, WM, MT, EXACT>), fp8_grid(p, T::BM), dim3(T::kThreads), 0, stream, p);
  return hipGetLastError();
}

template <bool EXACT>
hipError_t launch_sized(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t tiles = p.m_total * p.n / (256 * 256), avg = p.m_total / p.experts;
  if (tiles >= 192 && avg >= 192) return launch<2, 4, EXACT ? 2 : 4, EXACT>(p, stream);
  return launch<1, 4, 2, EXACT>(p, stream);
}

}  // namespace

hipError_t launch_gemm_fp8_tiled(const Fp8GemmArgs& p, hipStream_t stream) {
  return p.out_dtype == kFewOutF32 ? launch_sized<true>(p, stream) : launch_sized<false>(p, stream);
}

}  // namespace moe_fp4

// The Mixture-of-Experts router (moe_fp4_route): each token's best topk experts and
// their weights, and the routed rows grouped by expert as the grouped GEMM and the
// token-order combine take them (offsets, row -> token, token -> rows).
//
//   scores    softmax:  p = e^x / sum e^x, ranked by the logit x itself
//             sigmoid:  p = 1 / (1 + e^-x), ranked by p + bias
//   groups    with num_groups > 1 only the best topk_groups runs of experts stay
//             open; a group's score is its best rank value (softmax) or the sum of its
//             two best (sigmoid)
//   ties      go to the lower index, in groups and experts
//
// A token is ranked by 64 lanes, or from kRouteNarrow tokens on by 16 where they can
// hold its experts (16 each).  Four tokens a wavefront share every instruction: 16384
// tokens of 256 BF16 logits, top-8, rank in 12.4 us against 21.5 (10.7 with the
// expert in the key); but each lane then works through four times the experts, which
// shows while there is a wavefront or two for a SIMD: 2048 tokens with sigmoid scores in
// groups take 17.8 us against 16.0, one token 6.7 against 5.3.  A lane holds
// consecutive experts of one group, so the order of (lane, place) is the order of
// experts and the first holder of the maximum wins a tie.  Sigmoid values are ranked in
// FP64: neighbouring scores of a few hundred experts come closer than an FP32 step
// often enough to swap experts.
//
// Bound: instructions (each slot is two reductions over a token's lanes) and, up to a
// few thousand tokens, the launches; the bytes (16384 tokens: 10.5 MB) would take 2 us.
//
// Grouping is a counting sort by expert, stable in token order and without a
// scatter order that could vary: a block of tokens marks each expert's tokens in an
// LDS bitmap, so the row of (token, expert) is the expert's offset, plus its rows in
// earlier blocks, plus the marks before the token.  Up to kRouteOneBlock tokens take one
// launch; more take two, the second reading the first's per-block counts.
//
// Measured, kernel times: one token of 256 experts, top-8: 4.7 us; 512 tokens with sigmoid scores
// in groups: 6.9 us to rank, 5.7 to place; 16384 tokens: 10.7 and 7.7 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4_device.h"
#include "gemm_common.h"
#include "launch.h"

namespace moe_fp4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kFewPairs = 32;
// Ranking values below every score: a NaN (below -inf), and an expert that is taken,
// closed or no expert at all.
constexpr double kKeyMinusInf = -1.0e308, kKeyNaN = -1.5e308;

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}

// Ranking keys: FP32 logits as integers of the same order; 16-bit logits so too, with
// the expert's complement below them, which makes every key different and carries the
// expert along; FP64 scores as they are.
struct Key32 {
  typedef uint32_t T;
  static constexpr bool kUnique = false;
  static __device__ __forceinline__ T none() { return 0u; }
  static __device__ __forceinline__ T of(float x) {
    if (x != x) return 1u;
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 ranks as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  static __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
  static __device__ __forceinline__ T smaller(T a, T b) { return a < b ? a : b; }
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ T moved(T v) {
    return dpp<CTRL, ROWS>(0u, v);
  }
  static __device__ __forceinline__ T lane(T v, int l) {
    return (T)__builtin_amdgcn_readlane((int)v, l);
  }
};

struct Key16 : Key32 {
  static constexpr bool kUnique = true;
  static __device__ __forceinline__ T of(float x, bool f16, int32_t expert) {
    x += 0.0f;  // -0 ranks as +0
    const uint32_t b = f16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint32_t, x) >> 16;
    const uint32_t order = x != x ? 1u : (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
    return order << 16 | (0xFFFFu - (uint32_t)expert);
  }
};

struct Key64 {
  typedef double T;
  static constexpr bool kUnique = false;
  static __device__ __forceinline__ T none() { return -__builtin_inf(); }
  static __device__ __forceinline__ T of(double s) {
    return s != s ? kKeyNaN : s < kKeyMinusInf ? kKeyMinusInf : s + 0.0;
  }
  static __device__ __forceinline__ T larger(T a, T b) { return __builtin_fmax(a, b); }
  static __device__ __forceinline__ T smaller(T a, T b) { return __builtin_fmin(a, b); }
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ T moved(T v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL, ROWS>(0u, (uint32_t)b);
    const uint32_t hi = dpp<CTRL, ROWS>(0xFFF00000u, (uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
  static __device__ __forceinline__ T lane(T v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
};

// The largest key of a token's lanes (LT = 16, a row of the wavefront, or 64), in each
// of them.
template <typename K, int LT>
__device__ __forceinline__ typename K::T token_max(typename K::T v) {
  v = K::larger(v, K::template moved<0x128, 0xf>(v));  // row rotations by 8, 4, 2, 1
  v = K::larger(v, K::template moved<0x124, 0xf>(v));
  v = K::larger(v, K::template moved<0x122, 0xf>(v));
  v = K::larger(v, K::template moved<0x121, 0xf>(v));
  if (LT == 16) return v;
  v = K::larger(v, K::template moved<0x142, 0xa>(v));  // row ends into the next rows
  v = K::larger(v, K::template moved<0x143, 0xc>(v));
  return K::lane(v, 63);
}

struct Word {  // an unsigned number as a key
  typedef uint32_t T;
  static __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ T moved(T v) {
    return dpp<CTRL, ROWS>(0u, v);
  }
  static __device__ __forceinline__ T lane(T v, int l) {
    return (T)__builtin_amdgcn_readlane((int)v, l);
  }
};

// The lanes of the wavefront that hold its largest key.
template <typename K>
__device__ __forceinline__ uint64_t wave_holders(typename K::T v) {
  if constexpr (sizeof(typename K::T) == 4) {
    return __ballot(v == token_max<K, 64>(v));
  } else {
    // By the upper halves, as integers of the same order; by the lower ones only where
    // several lanes share the upper one.
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = (int64_t)b < 0 ? ~b : b | 0x8000000000000000ull;
    const uint32_t hi = (uint32_t)(o >> 32);
    const bool top = hi == token_max<Word, 64>(hi);
    const uint64_t tops = __ballot(top);
    if (__popcll(tops) == 1) return tops;
    const uint32_t lo = top ? (uint32_t)o : 0u;
    const uint32_t most = token_max<Word, 64>(lo);
    return __ballot(top && lo == most);
  }
}

template <int LT, typename T>
__device__ __forceinline__ T token_sum(T v) {
#pragma unroll
  for (int d = 1; d < LT; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <int LT>
__device__ __forceinline__ float token_max_f(float v) {
#pragma unroll
  for (int d = 1; d < LT; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.dtype == kRouteF32) return static_cast<const float*>(a.logits)[i];
  const uint16_t b = static_cast<const uint16_t*>(a.logits)[i];
  return a.dtype == kRouteF16 ? (float)__builtin_bit_cast(_Float16, b)
                              : __builtin_bit_cast(float, (uint32_t)b << 16);
}

// A lane's logits x[0 .. per_lane) from element i on; valid ones are j < count.
template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t i, int32_t count, float (&x)[VPL]) {
  if (a.dtype == kRouteF32) {
    const float* p = static_cast<const float*>(a.logits) + i;
    if (VPL % 4 == 0 && a.wide) {
      const float4_t* w = reinterpret_cast<const float4_t*>(p);
#pragma unroll
      for (int c = 0; c < VPL / 4; ++c) {
        const float4_t v = count > 0 ? w[c] : float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * c + e] = v[e];
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = j < count ? p[j] : 0.0f;
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(a.logits) + i;
  uint16_t raw[VPL];
  if (VPL % 8 == 0 && a.wide) {
    const u32x4_t* w = reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int c = 0; c < VPL / 8; ++c) {
      const u32x4_t v = count > 0 ? w[c] : u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) raw[8 * c + e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) raw[j] = j < count ? p[j] : 0;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    x[j] = a.dtype == kRouteF16 ? (float)__builtin_bit_cast(_Float16, raw[j])
                                : __builtin_bit_cast(float, (uint32_t)raw[j] << 16);
}

// kind of ranking: by FP32 logits, by 16-bit logits, by sigmoid scores
enum { kByLogit = 0, kByShortLogit = 1, kByScore = 2 };
template <int KIND>
using KeyOf = std::conditional_t<KIND == kByScore, Key64, std::conditional_t<KIND == kByShortLogit, Key16, Key32>>;

// Rank token t with LT lanes; `on`: there is such a token (lanes of a wavefront may hold
// several).  Lane s < topk of the token's returns the expert and weight of slot s.
template <int KIND, int LT, int VPL>
__device__ __forceinline__ void rank_token(const RouteArgs& a, int32_t t, bool on, int lane, int32_t* id,
                                           float* weight) {
  typedef KeyOf<KIND> K;
  typedef typename K::T KeyT;
  constexpr bool SIGMOID = KIND == kByScore;
  const int32_t own = lane % LT;                  // among the token's lanes
  const int32_t size = a.experts / a.num_groups;  // experts of a group
  const int32_t group = own / a.group_lanes;
  const int32_t first = own % a.group_lanes * a.per_lane;
  const int32_t expert0 = group * size + first;
  int32_t count = on && group < a.num_groups ? size - first : 0;  // experts of this lane
  count = count < a.per_lane ? count : a.per_lane;
  KeyT key[VPL];
  float val[VPL];
  load_logits<VPL>(a, (int64_t)t * a.ld + expert0, count, val);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const bool ok = j < count;
    if constexpr (SIGMOID) {
      const double p = 1.0 / (1.0 + exp(-(double)val[j]));
      key[j] = ok ? K::of(a.bias ? p + (double)a.bias[ok ? expert0 + j : 0] : p) : K::none();
    } else if constexpr (K::kUnique) {
      key[j] = ok ? K::of(val[j], a.dtype == kRouteF16, expert0 + j) : K::none();
    } else {
      key[j] = ok ? K::of(val[j]) : K::none();
    }
  }
  float top = 0.0f, sum = 0.0f;
  if (!SIGMOID && !a.renormalize) {
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < VPL; ++j) m = j < count ? fmaxf(m, val[j]) : m;
    top = token_max_f<LT>(m);
    // Terms far below the largest weigh little, so the fast exponential's error, which
    // grows with the distance, does not show in the sum.
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += j < count ? __expf(val[j] - top) : 0.0f;
    sum = token_sum<LT>(sum);
  }
  if (a.topk_groups < a.num_groups) {
    KeyT best = K::none(), second = K::none();
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const KeyT low = K::smaller(best, key[j]);
      best = K::larger(best, key[j]);
      second = K::larger(second, low);
    }
    // Over the group's lanes: neighbours, pairs, halves and rows of a row by lane moves.
    auto join = [&](KeyT b, KeyT s) {
      const KeyT low = K::smaller(best, b);
      best = K::larger(best, b);
      second = K::larger(low, K::larger(second, s));
    };
    const int32_t gl = a.group_lanes;
    if (gl > 1) join(K::template moved<0xB1, 0xf>(best), K::template moved<0xB1, 0xf>(second));
    if (gl > 2) join(K::template moved<0x4E, 0xf>(best), K::template moved<0x4E, 0xf>(second));
    if (gl > 4) join(K::template moved<0x141, 0xf>(best), K::template moved<0x141, 0xf>(second));
    if (gl > 8) join(K::template moved<0x140, 0xf>(best), K::template moved<0x140, 0xf>(second));
    for (int d = 16; d < gl; d <<= 1) join(__shfl_xor(best, d, 64), __shfl_xor(second, d, 64));
    const KeyT score = SIGMOID && size > 1 ? best + second : best;
    int32_t ahead = 0;
    for (int32_t o = 0; o < a.num_groups; ++o) {
      const KeyT other = LT == 64 ? K::lane(score, o * a.group_lanes)
                                  : __shfl(score, lane - own + o * a.group_lanes, 64);
      ahead += other > score || (other == score && o < group) ? 1 : 0;
    }
    if (ahead >= a.topk_groups) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = K::none();
    }
  }
  int32_t my_id = 0;
  for (int32_t s = 0; s < a.topk; ++s) {
    KeyT best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = K::larger(best, key[j]);
    int32_t chosen;
    if constexpr (K::kUnique) {
      chosen = (int32_t)(0xFFFFu - (token_max<K, LT>(best) & 0xFFFFu));
    } else if constexpr (LT == 64) {
      const int holder = __ffsll((unsigned long long)wave_holders<K>(best)) - 1;
      int32_t at = 0;
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j) at = key[j] == best ? j : at;
      chosen = __builtin_amdgcn_readlane(expert0 + at, holder);
    } else {
      // The lowest expert that holds it, as the largest complement.
      const KeyT m = token_max<K, LT>(best);
      uint32_t not_expert = 0;
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j) not_expert = key[j] == m ? ~(uint32_t)(expert0 + j) : not_expert;
      chosen = (int32_t)~token_max<Word, LT>(not_expert);
    }
    if (own == s) my_id = chosen;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (expert0 + j == chosen) key[j] = K::none();
  }
  // The chosen logits are read again (they are in the caches) rather than carried.
  const bool mine = on && own < a.topk;
  const float my_val = mine ? load_logit(a, (int64_t)t * a.ld + my_id) : 0.0f;
  float w;
  if (SIGMOID) {
    // In FP64 up to the quotient: scores below 2^-126 lose their proportions in FP32.
    const double p = 1.0 / (1.0 + exp(-(double)my_val));
    w = (float)(a.renormalize ? p / token_sum<LT>(mine ? p : 0.0) : p);
  } else if (a.renormalize) {
    // The full softmax's denominator cancels: only the chosen experts' terms are needed.
    const float m = token_max_f<LT>(mine ? my_val : -__builtin_inff());
    const float e = expf(my_val - m);
    w = e / token_sum<LT>(mine ? e : 0.0f);
  } else {
    w = expf(my_val - top) / sum;
  }
  *id = my_id;
  *weight = w;
}

// Exclusive scan of total[0 .. experts) in LDS into base, plus `before` (rows of
// earlier blocks); block 0 also writes the offsets.  All threads; barriers inside.
__device__ __forceinline__ void scan_offsets(const RouteArgs& a, const int32_t* total,
                                             int32_t* before, int32_t* wave_sums, bool write) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  int32_t carry = 0;
  for (int32_t e0 = 0; e0 < a.experts; e0 += blockDim.x) {
    const int32_t e = e0 + tid;
    const int32_t c = e < a.experts ? total[e] : 0;
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sums[wave] = incl;
    __syncthreads();
    int32_t base = carry;
    for (int w = 0; w < waves; ++w) {
      const int32_t v = wave_sums[w];
      if (w < wave) base += v;
      carry += v;
    }
    if (e < a.experts) {
      const int32_t off = base + incl - c;
      if (write) a.offsets[e] = off;
      before[e] += off;
    }
    __syncthreads();
  }
  if (write && tid == 0) a.offsets[a.experts] = carry;
}

// Rows of a block's pairs: the marks before each token in its expert's bitmap.
__device__ __forceinline__ void place_rows(const RouteArgs& a, const int32_t* ids,
                                           const uint32_t* marks, const int32_t* base, int32_t t0,
                                           int32_t count, int words) {
  for (int32_t p = threadIdx.x; p < count * a.topk; p += blockDim.x) {
    const int32_t e = ids[p], tl = p / a.topk;
    const uint32_t* m = marks + e * words;
    int32_t r = base[e];
    for (int w = 0; w < tl >> 5; ++w) r += __popc(m[w]);
    r += __popc(m[tl >> 5] & ((1u << (tl & 31)) - 1));
    a.token_rows[(int64_t)t0 * a.topk + p] = r;
    a.row_token[r] = t0 + tl;
  }
}

__device__ __forceinline__ void mark(uint32_t* marks, int32_t e, int32_t tl, int words) {
  atomicOr(&marks[e * words + (tl >> 5)], 1u << (tl & 31));
}

// Ranks a block of tokens; leaves the block's rows per expert (16-bit) in counts.
template <int KIND, int LT, int VPL>
__global__ __launch_bounds__(kThreads) void k_rank(RouteArgs a) {
  extern __shared__ __align__(16) int32_t count[];  // [counts_pitch]
  const int tid = threadIdx.x, lane = tid & 63, own = lane % LT;
  const int32_t t0 = blockIdx.x * a.block_tokens;
  const int32_t here = a.tokens - t0 < a.block_tokens ? a.tokens - t0 : a.block_tokens;
  for (int i = tid; i < a.counts_pitch; i += blockDim.x) count[i] = 0;
  __syncthreads();
  for (int32_t first = 0; first < here; first += blockDim.x / LT) {
    const int32_t tl = first + tid / LT;
    const bool on = tl < here;
    int32_t id;
    float w;
    rank_token<KIND, LT, VPL>(a, t0 + (on ? tl : 0), on, lane, &id, &w);
    if (on && own < a.topk) {
      const int64_t o = (int64_t)(t0 + tl) * a.topk + own;
      a.ids[o] = id;
      a.weights[o] = w;
      atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  uint16_t* out = a.counts + (int64_t)blockIdx.x * a.counts_pitch;
  for (int i = tid; i < a.counts_pitch; i += blockDim.x) out[i] = (uint16_t)count[i];
}

// Places a block's rows: offsets from every block's counts, then the marks.
__global__ __launch_bounds__(kThreads) void k_place(RouteArgs a) {
  extern __shared__ __align__(16) int32_t lds[];
  const int words = a.block_tokens / 32 > 1 ? a.block_tokens / 32 : 1;
  int32_t* total = lds;
  int32_t* before = total + a.counts_pitch;
  int32_t* wave_sums = before + a.counts_pitch;
  uint32_t* marks = reinterpret_cast<uint32_t*>(wave_sums + kWaves);
  const int tid = threadIdx.x;
  const int32_t t0 = blockIdx.x * a.block_tokens;
  const int32_t here = a.tokens - t0 < a.block_tokens ? a.tokens - t0 : a.block_tokens;
  const int32_t* ids = a.ids + (int64_t)t0 * a.topk;
  for (int i = tid; i < 2 * a.counts_pitch; i += kThreads) total[i] = 0;
  for (int i = tid; i < a.experts * words; i += kThreads) marks[i] = 0;
  __syncthreads();
  for (int32_t p = tid; p < here * a.topk; p += kThreads) mark(marks, ids[p], p / a.topk, words);
  // A thread sums four experts (8 bytes of counts) over every `stride`-th block.
  const int cols = a.counts_pitch / 4, stride = kThreads / cols;
  const int col = tid % cols, row = tid / cols;
  if (row < stride) {
    int32_t all[4] = {}, low[4] = {};
#pragma unroll 8
    for (int32_t b = row; b < (int32_t)gridDim.x; b += stride) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(a.counts + (int64_t)b * a.counts_pitch + 4 * col);
      const bool earlier = b < (int32_t)blockIdx.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t c = (int32_t)((uint32_t)v[i / 2] >> (16 * (i % 2)) & 0xFFFFu);
        all[i] += c;
        low[i] += earlier ? c : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (all[i]) atomicAdd(&total[4 * col + i], all[i]);
      if (low[i]) atomicAdd(&before[4 * col + i], low[i]);
    }
  }
  __syncthreads();
  scan_offsets(a, total, before, wave_sums, blockIdx.x == 0);
  place_rows(a, ids, marks, before, t0, here, words);
}

// Both steps of at most kRouteOneBlock tokens in one workgroup.
template <int KIND, int LT, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_small(RouteArgs a) {
  extern __shared__ __align__(16) int32_t lds[];
  const int words = a.tokens > 32 ? 2 : 1;
  int32_t* total = lds;
  int32_t* before = total + a.experts;
  int32_t* wave_sums = before + a.experts;
  uint32_t* marks = reinterpret_cast<uint32_t*>(wave_sums + kWaves);
  int32_t* ids = reinterpret_cast<int32_t*>(marks + a.experts * words);
  const int tid = threadIdx.x, lane = tid & 63, own = lane % LT;
  for (int i = tid; i < a.experts * words; i += blockDim.x) marks[i] = 0;
  for (int i = tid; i < a.experts; i += blockDim.x) before[i] = 0;
  __syncthreads();
  for (int32_t first = 0; first < a.tokens; first += blockDim.x / LT) {
    const int32_t t = first + tid / LT;
    const bool on = t < a.tokens;
    int32_t id;
    float w;
    rank_token<KIND, LT, VPL>(a, on ? t : 0, on, lane, &id, &w);
    if (on && own < a.topk) {
      a.ids[t * a.topk + own] = id;
      a.weights[t * a.topk + own] = w;
      ids[t * a.topk + own] = id;
      mark(marks, id, t, words);
    }
  }
  __syncthreads();
  const int32_t pairs = a.tokens * a.topk;
  if (pairs <= kFewPairs) {
    // Few enough to compare each with all: no scan.
    for (int e = tid; e <= a.experts; e += blockDim.x) {
      int32_t lower = 0;
      for (int q = 0; q < pairs; ++q) lower += ids[q] < e ? 1 : 0;
      a.offsets[e] = lower;
    }
    if (tid < pairs) {
      const int32_t id = ids[tid];
      int32_t row = 0;
      for (int q = 0; q < pairs; ++q) row += ids[q] < id || (ids[q] == id && q < tid) ? 1 : 0;
      a.token_rows[tid] = row;
      a.row_token[row] = tid / a.topk;
    }
    return;
  }
  for (int i = tid; i < a.experts; i += blockDim.x) {
    int32_t c = 0;
    for (int w = 0; w < words; ++w) c += __popc(marks[i * words + w]);
    total[i] = c;
  }
  __syncthreads();
  scan_offsets(a, total, before, wave_sums, true);
  place_rows(a, ids, marks, before, 0, a.tokens, words);
}

// Threads that rank `tokens` at once, LT lanes each: whole wavefronts, up to kThreads.
int rank_threads(int64_t tokens, int lt) {
  const int64_t t = (tokens * lt + 63) / 64 * 64;
  return t < 64 ? 64 : t < kThreads ? (int)t : kThreads;
}

template <int KIND, int LT, int VPL>
hipError_t launch(const RouteArgs& a, hipStream_t stream) {
  if (a.tokens <= kRouteOneBlock) {
    // At least four wavefronts: they share the scan over the experts.
    const int threads = rank_threads(a.tokens, LT);
    const size_t lds = (size_t)((2 + (a.tokens > 32 ? 2 : 1)) * a.experts + kWaves + a.tokens * a.topk) * 4;
    hipLaunchKernelGGL((k_route_small<KIND, LT, VPL>), dim3(1), dim3(threads < 256 ? 256 : threads), lds,
                       stream, a);
    return hipGetLastError();
  }
  const int blocks = (int)((a.tokens + a.block_tokens - 1) / a.block_tokens);
  hipLaunchKernelGGL((k_rank<KIND, LT, VPL>), dim3(blocks), dim3(rank_threads(a.block_tokens, LT)),
                     (size_t)a.counts_pitch * 4, stream, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int words = a.block_tokens / 32 > 1 ? a.block_tokens / 32 : 1;
  const size_t lds = (size_t)(2 * a.counts_pitch + kWaves + a.experts * words) * 4;
  hipLaunchKernelGGL(k_place, dim3(blocks), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

template <int KIND, int LT>
hipError_t launch_sized(const RouteArgs& a, hipStream_t stream) {
  if (a.per_lane <= 1) return launch<KIND, LT, 1>(a, stream);
  if (a.per_lane <= 2) return launch<KIND, LT, 2>(a, stream);
  if (a.per_lane <= 4) return launch<KIND, LT, 4>(a, stream);
  if (a.per_lane <= 8) return launch<KIND, LT, 8>(a, stream);
  return launch<KIND, LT, 16>(a, stream);
}

template <int KIND>
hipError_t launch_lanes(const RouteArgs& a, hipStream_t stream) {
  return a.token_lanes == 16 ? launch_sized<KIND, 16>(a, stream) : launch_sized<KIND, 64>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.sigmoid) return launch_lanes<kByScore>(a, stream);
  return a.dtype == kRouteF32 ? launch_lanes<kByLogit>(a, stream) : launch_lanes<kByShortLogit>(a, stream);
}

}  // namespace moe_fp4

// Host-side checks that the C-ABI files share.
#pragma once

#include <stdint.h>

namespace moe_fp4 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether the byte ranges [p, p + pb) and [q, q + qb) share a byte.
inline bool overlap(const void* p, int64_t pb, const void* q, int64_t qb) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return pb > 0 && qb > 0 && a < b + (uintptr_t)qb && b < a + (uintptr_t)pb;
}

}  // namespace moe_fp4

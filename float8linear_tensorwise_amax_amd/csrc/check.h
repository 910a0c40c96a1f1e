// Argument checks shared by the C-ABI layers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/f8lin.h"

namespace f8lin {

constexpr int64_t kMaxDim = (int64_t)1 << 22;        // per matrix dimension (32-bit tile offsets)
constexpr int64_t kMaxElems = (int64_t)1 << 40;      // per tensor

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// A data pointer may be NULL only when its tensor is empty.
inline bool missing(const void *p, int64_t elems) { return p == nullptr && elems > 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

struct Range {
  const void *p;
  int64_t bytes;
};

inline bool overlaps(const Range &a, const Range &b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, a1 = a0 + (uintptr_t)a.bytes;
  const uintptr_t b0 = (uintptr_t)b.p, b1 = b0 + (uintptr_t)b.bytes;
  return a0 < b1 && b0 < a1;
}

// Every output range must be disjoint from every other range.
inline bool any_overlap(const Range *outs, int nout, const Range *ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(outs[i], outs[j])) return true;
    for (int j = 0; j < nin; ++j)
      if (overlaps(outs[i], ins[j])) return true;
  }
  return false;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? F8LIN_OK : F8LIN_EHIP; }

}  // namespace f8lin

#define F8_TRY(expr)                 \
  do {                               \
    const int st_ = (expr);          \
    if (st_ != F8LIN_OK) return st_; \
  } while (0)

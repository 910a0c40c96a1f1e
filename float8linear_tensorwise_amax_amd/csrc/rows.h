// Loads of a few consecutive elements of a row, whatever its length and
// alignment, without a branch for each.
#pragma once

#include "mx_common.h"

namespace f8lin {

// V consecutive elements (1, 2, 4 or 8 of a 16-bit type, 1, 2 or 4 of
// binary32) as words: a word holds two 16-bit elements, or a lone one in its
// low half.
template <int DT, int V>
struct Few {
  static constexpr int kWords = DT == F8LIN_FP32 ? V : (V + 1) / 2;
  uint32_t w[kWords];
};

// V elements at p, all there.  PAST: past the caches (16 bytes only).
template <int DT, int V, bool PAST = false>
__device__ __forceinline__ Few<DT, V> load_whole(const typename MxElem<DT>::type *p) {
  Few<DT, V> f;
  constexpr int kW = Few<DT, V>::kWords;
  if constexpr (DT != F8LIN_FP32 && V == 1) {
    f.w[0] = *p;
  } else if constexpr (kW == 1) {
    typedef uint32_t u32_u __attribute__((aligned(2)));
    f.w[0] = *reinterpret_cast<const u32_u *>(p);
  } else if constexpr (kW == 2) {
    const u32x2 v = *reinterpret_cast<const u32x2_u *>(p);
    f.w[0] = v.x, f.w[1] = v.y;
  } else {
    const u32x4_u *const q = reinterpret_cast<const u32x4_u *>(p);
    const u32x4 v = PAST ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.w[i] = v[i];
  }
  return f;
}

// Elements d .. V - 1 moved to the front, zeros behind them (d >= V: zeros).
template <int DT, int V>
__device__ __forceinline__ Few<DT, V> moved(Few<DT, V> f, int d) {
  constexpr int kW = Few<DT, V>::kWords;
  const int words = DT == F8LIN_FP32 ? d : d >> 1;
#pragma unroll
  for (int s = 1; s < kW; s *= 2) {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const uint32_t from = i + s < kW ? f.w[(i + s) % kW] : 0u;
      f.w[i] = words & s ? from : f.w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kW; ++i) f.w[i] = words >= kW ? 0u : f.w[i];
  if constexpr (DT != F8LIN_FP32) {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const uint32_t next = i + 1 < kW ? f.w[(i + 1) % kW] : 0u;
      f.w[i] = d & 1 ? f.w[i] >> 16 | next << 16 : f.w[i];
    }
  }
  return f;
}

// V elements from place `at` of a row of n >= V, zeros past its end: read from
// where V are there, and moved.
template <int DT, int V>
__device__ __forceinline__ Few<DT, V> load_to_end(const typename MxElem<DT>::type *row, int at, int n) {
  const int from = min(at, n - V);
  return moved<DT, V>(load_whole<DT, V>(row + from), min(at - from, V));
}

// The same of a row of any length n >= 1, an element at a time.
template <int DT, int V>
__device__ __forceinline__ Few<DT, V> load_each(const typename MxElem<DT>::type *row, int64_t at, int64_t n) {
  uint32_t e[V];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = (uint32_t)row[at + i < n ? at + i : n - 1];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = at + i < n ? e[i] : 0u;
  Few<DT, V> f;
#pragma unroll
  for (int i = 0; i < Few<DT, V>::kWords; ++i) {
    if constexpr (DT == F8LIN_FP32) f.w[i] = e[i];
    else f.w[i] = e[(2 * i) % V] | (2 * i + 1 < V ? e[(2 * i + 1) % V] << 16 : 0u);
  }
  return f;
}

// The first d elements as zeros.
template <int DT, int V>
__device__ __forceinline__ void clear_first(Few<DT, V> &f, int d) {
#pragma unroll
  for (int i = 0; i < Few<DT, V>::kWords; ++i) {
    if constexpr (DT == F8LIN_FP32) f.w[i] = i < d ? 0u : f.w[i];
    else f.w[i] = 2 * i + 1 < d ? 0u : 2 * i < d ? f.w[i] & 0xFFFF0000u : f.w[i];
  }
}
template <int DT, int V>
__device__ __forceinline__ void clear(Few<DT, V> &f) {
#pragma unroll
  for (int i = 0; i < Few<DT, V>::kWords; ++i) f.w[i] = 0u;
}

}  // namespace f8lin

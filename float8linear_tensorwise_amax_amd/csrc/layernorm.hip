// Layer norm of the rows of a matrix, forward and backward:
//   mean = sum(x) / n,  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps),  xhat = (x - mean) * rstd
//   y  = xhat * w + b
//   dx = rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n),  g = dy * w
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// HBM-bound: the forward reads x and writes y once, the backward reads x and
// dy and writes dx once (65536 x 4096 bf16, in a loop over two inputs and
// outputs: 235 us, 4.6 TB/s, and 297 us, 5.4 TB/s; with one output, as a program
// calls it again, forward 200; 12288 x 1600: 19 and 32 us).  A row stays in the registers of the wave
// (or of the workgroup) that normalises it, so that the mean, the centred
// squares and the output are three passes over registers, not memory; only
// rows of more than 16384 values are read again.  Everything is computed in
// binary32 from the values as read, and rounded once.  The backward's
// workgroups keep dw and db of their rows in registers too and leave one
// partial sum each, which a second launch adds in a fixed order (no atomics:
// the same bits on every run).
//
// A wave a row up to 2048 values in the forward (12288 x 1600: 19 us, a
// workgroup a row 22), a workgroup a row above (8192 x 4096: 25 us, a wave a row
// 32; 1021 x 2055 fp32 6.9 and 8.9; but 65536 x 4096 235 and 218) and from 512 in the backward, whose sums need the registers (12288 x
// 1600: 32 us, a wave a row 46).  From 8193 to 16384 values the backward keeps
// more than its registers hold (17 spilled in the 16-bit types, 345 in binary32:
// 4096 x 16384 110 us, 3.7 TB/s, and 370 us, 2.2 TB/s).  Longer rows are read
// three times forward and back (4096 x 20000 bf16: 99 and 211 us; 1024 x 70000:
// 101 and 250).
#include <algorithm>

#include "rows.h"

namespace f8lin {
namespace {

// What is read and written goes past the caches where it is more than they
// hold (65536 x 4096 bf16: forward 235 us, through them 248; backward 297 and
// 321; 8192 x 4096: forward 32 past and 25 through them; the backward of 4096 x
// 16384 in binary32, which spills, the other way: 370 and 361).
constexpr int64_t kPastBytes = (int64_t)256 << 20;

// Sum over the G threads of a row (G = 64: a wave; else the workgroup), the
// same in all of them.  Consecutive sums take different `red`: a wave may still
// read the last one's.
template <int G, int S>
__device__ __forceinline__ void row_sum(float (&v)[S], float (*red)[S]) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
#pragma unroll
    for (int s = 0; s < S; ++s) v[s] += __shfl_xor(v[s], off, 64);
  }
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int s = 0; s < S; ++s) red[threadIdx.x >> 6][s] = v[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) t += red[w][s];
      v[s] = t;
    }
  }
}

// Eight values of a row of n, from place `at` of it on, as binary32.  A load
// that would pass the row's end ends there instead, and its values move to
// their places: columns past the end are zero.  (Rows of fewer than eight:
// TINY, an element at a time.)
template <int DT, bool TINY, bool PAST = false>
struct Load8 {
  static constexpr int kHalf = DT == F8LIN_FP32 ? 4 : 8, kCount = 8 / kHalf;
  Few<DT, kHalf> f[kCount];
  int d;
  __device__ __forceinline__ void from(const void *p, int at, int n) {
    typedef typename MxElem<DT>::type elem;
    const elem *const row = reinterpret_cast<const elem *>(p);
    if constexpr (TINY) {
#pragma unroll
      for (int h = 0; h < kCount; ++h) f[h] = load_each<DT, kHalf>(row, at + kHalf * h, n);
    } else {
      const int start = min(at, n - 8);
      d = at - start;
#pragma unroll
      for (int h = 0; h < kCount; ++h) f[h] = load_whole<DT, kHalf, PAST>(row + start + kHalf * h);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (DT == F8LIN_FP32) v[e] = __uint_as_float(f[e / 4].w[e % 4]);
      else v[e] = elem_f32<DT>((f[0].w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    }
    if (!TINY && d > 0) {
#pragma unroll
      for (int s = 1; s < 8; s *= 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = e + s < 8 ? v[(e + s) % 8] : 0.0f;
          v[e] = d & s ? u : v[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = d >= 8 ? 0.0f : v[e];
    }
  }
};

// Eight parameters from column c of n, as binary32.
template <bool TINY>
__device__ __forceinline__ void load_param8(const void *p, int dt, int c, int n, float (&v)[8]) {
  if (dt == F8LIN_FP32) {
    Load8<F8LIN_FP32, TINY> l;
    l.from(p, c, n), l.values(v);
  } else if (dt == F8LIN_BF16) {
    Load8<F8LIN_BF16, TINY> l;
    l.from(p, c, n), l.values(v);
  } else {
    Load8<F8LIN_FP16, TINY> l;
    l.from(p, c, n), l.values(v);
  }
}

// Two values rounded to the 16-bit type DT, as a packed pair.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  if constexpr (DT == F8LIN_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// Stores the first n of eight values, rounded to DT; returns the largest
// magnitude stored, as binary32 bits (NaN above all).  PAST: past the caches.
template <int DT, bool PAST = false>
__device__ __forceinline__ uint32_t store8(void *p, int64_t at, int n, const float (&v)[8], bool mag) {
  typedef typename MxElem<DT>::type elem;
  constexpr bool F32 = DT == F8LIN_FP32;
  elem *const y = reinterpret_cast<elem *>(p) + at;
  uint32_t o[F32 ? 8 : 4];
#pragma unroll
  for (int e = 0; e < (F32 ? 8 : 4); ++e) o[e] = F32 ? __float_as_uint(v[e]) : pack2<DT>(v[(2 * e) % 8], v[(2 * e + 1) % 8]);
  auto bits = [&](int e) { return F32 ? o[e] : (o[e >> 1] >> (16 * (e & 1))) & 0xFFFFu; };
  uint32_t m = 0;
  if (mag) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) m = max(m, __float_as_uint(elem_f32<DT>(bits(e))) & 0x7FFFFFFFu);
  }
  if (n >= 8) {
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
      const u32x4 w = {o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]};
      u32x4_u *const to = reinterpret_cast<u32x4_u *>(y + 4 * h);
      if constexpr (PAST) __builtin_nontemporal_store(w, to);
      else *to = w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) y[e] = (elem)bits(e);
  }
  return m;
}

// Eight values from column col of the row that starts at element `at`.
template <int DT>
__device__ __forceinline__ void load_row8(const void *p, int64_t at, int64_t col, int64_t cols, float (&v)[8]) {
  Load8<DT, false> l;
  l.from(reinterpret_cast<const typename MxElem<DT>::type *>(p) + at, (int)col, (int)cols);
  l.values(v);
}

// Folds this wave's largest magnitude into the amax word (the order of the
// bits is the order of the values).
__device__ __forceinline__ void fold_amax(float *amax, uint32_t m) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  uint32_t *const word = reinterpret_cast<uint32_t *>(amax);
  if ((threadIdx.x & 63) == 0 && m > __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
    __hip_atomic_fetch_max(word, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ void ln_clear_kernel(float *word) { *word = 0.0f; }

// Rows of up to 8 * C * G values: G threads a row, C chunks of 8 a thread.
template <int XT, int YT, int G, int C, bool TINY, bool PAST>
__global__ __launch_bounds__(G > 256 ? G : 256) void ln_forward_kernel(const LayerNormFwd a) {
  __shared__ float red[2][16][1];
  constexpr int kRows = G == 64 ? 4 : 1;  // rows of a workgroup
  const int lane = G == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = a.first + (int64_t)blockIdx.x * kRows + (G == 64 ? threadIdx.x >> 6 : 0);
  if (G == 64 && row >= a.rows) return;  // (no barrier below for G = 64)
  const int cols = (int)a.cols;
  Load8<XT, TINY, PAST> raw[C];
#pragma unroll
  for (int c = 0; c < C; ++c)
    raw[c].from(reinterpret_cast<const typename MxElem<XT>::type *>(a.x) + row * a.ldx, 8 * (c * G + lane), cols);
  float v[C][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    raw[c].values(v[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += v[c][e];
  }
  row_sum<G, 1>(s, red[0]);
  const float mean = s[0] / (float)cols;
  float q[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = cols - 8 * (c * G + lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[c][e] = e < n ? v[c][e] - mean : 0.0f;
      q[0] = fmaf(v[c][e], v[c][e], q[0]);
    }
  }
  row_sum<G, 1>(q, red[1]);
  const float rstd = 1.0f / sqrtf(q[0] / (float)cols + a.eps);
  if (a.stats && lane == 0) {
    a.stats[row] = mean;
    a.stats[a.rows + row] = rstd;
  }
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (c * G + lane), n = cols - col;
    if (n <= 0) break;
    float w[8], b[8];
    if (a.weight) load_param8<TINY>(a.weight, a.weight_dtype, col, cols, w);
    if (a.bias) load_param8<TINY>(a.bias, a.bias_dtype, col, cols, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[c][e] *= rstd;
      if (a.weight) v[c][e] *= w[e];
      if (a.bias) v[c][e] += b[e];
    }
    m = max(m, store8<YT, PAST>(a.y, row * a.cols + col, n, v[c], a.amax != nullptr));
  }
  if (a.amax) fold_amax(a.amax, m);
}

// Rows of any length: the row is read three times (from the L2, where it fits).
template <int XT, int YT>
__global__ __launch_bounds__(1024) void ln_forward_wide_kernel(const LayerNormFwd a) {
  __shared__ float red[2][16][1];
  const int64_t row = a.first + blockIdx.x, at = row * a.ldx, cols = a.cols;
  float v[8];
  float s[1] = {0.0f}, q[1] = {0.0f};
  for (int64_t col = 8 * (int64_t)threadIdx.x; col < cols; col += 8 * 1024) {
    load_row8<XT>(a.x, at, col, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += v[e];
  }
  row_sum<1024, 1>(s, red[0]);
  const float mean = s[0] / (float)cols;
  for (int64_t col = 8 * (int64_t)threadIdx.x; col < cols; col += 8 * 1024) {
    const int n = (int)min((int64_t)8, cols - col);
    load_row8<XT>(a.x, at, col, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) q[0] = fmaf(v[e] - mean, v[e] - mean, q[0]);
  }
  row_sum<1024, 1>(q, red[1]);
  const float rstd = 1.0f / sqrtf(q[0] / (float)cols + a.eps);
  if (a.stats && threadIdx.x == 0) {
    a.stats[row] = mean;
    a.stats[a.rows + row] = rstd;
  }
  uint32_t m = 0;
  for (int64_t col = 8 * (int64_t)threadIdx.x; col < cols; col += 8 * 1024) {
    const int n = (int)min((int64_t)8, cols - col);
    float w[8], b[8];
    load_row8<XT>(a.x, at, col, cols, v);
    if (a.weight) load_param8<false>(a.weight, a.weight_dtype, (int)col, (int)cols, w);
    if (a.bias) load_param8<false>(a.bias, a.bias_dtype, (int)col, (int)cols, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = (v[e] - mean) * rstd;
      if (a.weight) v[e] *= w[e];
      if (a.bias) v[e] += b[e];
    }
    m = max(m, store8<YT>(a.y, row * cols + col, n, v, a.amax != nullptr));
  }
  if (a.amax) fold_amax(a.amax, m);
}

// dx of a workgroup's rows, and their dw and db, which stay in registers; the
// next row is on its way while one is reduced.
template <int XT, int YT, int G, int C, bool TINY, bool PAST>
__global__ __launch_bounds__(G > 256 ? G : 256) void ln_backward_kernel(const LayerNormBwd a, int64_t rows_each) {
  constexpr int kRows = G == 64 ? 4 : 1;
  __shared__ float red[2][16][2];
  __shared__ float join[G == 64 ? 2 * 8 * 64 * C : 1];
  const int wave = threadIdx.x >> 6;
  const int lane = G == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const bool params = a.part != nullptr;
  float w[C][8], dw[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = 1.0f, dw[c][e] = 0.0f, db[c][e] = 0.0f;
    if (a.weight) load_param8<TINY>(a.weight, a.weight_dtype, 8 * (c * G + lane), cols, w[c]);
  }
  const int64_t first = (int64_t)blockIdx.x * rows_each, last = min(a.rows, first + rows_each);
  Load8<XT, TINY, PAST> rx[C];
  Load8<YT, TINY, PAST> rd[C];
  float mean_next = 0.0f, rstd_next = 0.0f;
  auto load = [&](int64_t row) {
    mean_next = a.stats[row], rstd_next = a.stats[a.rows + row];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (c * G + lane);
      rx[c].from(reinterpret_cast<const typename MxElem<XT>::type *>(a.x) + row * a.ldx, col, cols);
      rd[c].from(reinterpret_cast<const typename MxElem<YT>::type *>(a.dy) + row * a.lddy, col, cols);
    }
  };
  int parity = 0;
  int64_t row = first + (G == 64 ? wave : 0);
  if (row < last) load(row);
  for (; row < last; row += kRows) {
    const float mean = mean_next, rstd = rstd_next;
    float x[C][8], d[C][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) rx[c].values(x[c]), rd[c].values(d[c]);
    if (row + kRows < last) load(row + kRows);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int n = cols - 8 * (c * G + lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // (a column past the end: nothing of the row's mean gets in)
        const float xh = e < n ? (x[c][e] - mean) * rstd : 0.0f, g = d[c][e] * w[c][e];
        x[c][e] = xh;
        s[0] += g;
        s[1] = fmaf(g, xh, s[1]);
        dw[c][e] = fmaf(d[c][e], xh, dw[c][e]);
        db[c][e] += d[c][e];
        d[c][e] = g;
      }
    }
    if (!a.dx) continue;
    row_sum<G, 2>(s, red[parity]);
    parity ^= 1;  // (the other buffer: a wave may still read this one)
    const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (c * G + lane), n = cols - col;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (d[c][e] - m0 - x[c][e] * m1);
      if (n > 0) store8<XT, PAST>(a.dx, row * a.cols + col, n, o, false);
    }
  }
  if (!params) return;
  float *const part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (G == 64) {
    // the four waves' sums, in their order
    for (int t = 0; t < 4; ++t) {
      if (wave == t) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float *const j0 = join + (c * 8 + e) * 64 + lane, *const j1 = j0 + 8 * 64 * C;
            if (t > 0) dw[c][e] += *j0, db[c][e] += *j1;
            *j0 = dw[c][e], *j1 = db[c][e];
          }
      }
      __syncthreads();
    }
    if (wave != 3) return;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (c * G + lane), n = cols - col;
    if (n > 0) {
      store8<F8LIN_FP32>(part, col, n, dw[c], false);
      store8<F8LIN_FP32>(part + a.cols, col, n, db[c], false);
    }
  }
}

// Rows of any length, dx alone.
template <int XT, int YT>
__global__ __launch_bounds__(1024) void ln_backward_wide_kernel(const LayerNormBwd a) {
  __shared__ float red[16][2];
  const int64_t row = a.first + blockIdx.x, cols = a.cols;
  const float mean = a.stats[row], rstd = a.stats[a.rows + row], inv = 1.0f / (float)cols;
  float s[2] = {0.0f, 0.0f}, x[8], d[8], w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  for (int64_t col = 8 * (int64_t)threadIdx.x; col < cols; col += 8 * 1024) {
    const int n = (int)min((int64_t)8, cols - col);
    load_row8<XT>(a.x, row * a.ldx, col, cols, x);
    load_row8<YT>(a.dy, row * a.lddy, col, cols, d);
    if (a.weight) load_param8<false>(a.weight, a.weight_dtype, (int)col, (int)cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e >= n) continue;
      const float g = d[e] * w[e];
      s[0] += g;
      s[1] = fmaf(g, (x[e] - mean) * rstd, s[1]);
    }
  }
  row_sum<1024, 2>(s, red);
  const float m0 = s[0] * inv, m1 = s[1] * inv;
  for (int64_t col = 8 * (int64_t)threadIdx.x; col < cols; col += 8 * 1024) {
    const int n = (int)min((int64_t)8, cols - col);
    load_row8<XT>(a.x, row * a.ldx, col, cols, x);
    load_row8<YT>(a.dy, row * a.lddy, col, cols, d);
    if (a.weight) load_param8<false>(a.weight, a.weight_dtype, (int)col, (int)cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = rstd * (d[e] * w[e] - m0 - (x[e] - mean) * rstd * m1);
    store8<XT>(a.dx, row * cols + col, n, x, false);
  }
}

// Rows of any length, dw and db of rows_each rows for 2048 columns a workgroup.
template <int XT, int YT>
__global__ __launch_bounds__(256) void ln_param_kernel(const LayerNormBwd a, int64_t rows_each, int col_blocks) {
  const int64_t block = blockIdx.x / col_blocks;
  const int64_t col = 8 * ((int64_t)(blockIdx.x % col_blocks) * 256 + threadIdx.x);
  if (col >= a.cols) return;
  const int n = (int)min((int64_t)8, a.cols - col);
  float dw[8], db[8], x[8], d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
  const int64_t first = block * rows_each, last = min(a.rows, first + rows_each);
  for (int64_t row = first; row < last; ++row) {
    const float mean = a.stats[row], rstd = a.stats[a.rows + row];
    load_row8<XT>(a.x, row * a.ldx, col, a.cols, x);
    load_row8<YT>(a.dy, row * a.lddy, col, a.cols, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] = fmaf(d[e], (x[e] - mean) * rstd, dw[e]);
      db[e] += d[e];
    }
  }
  float *const part = a.part + block * 2 * a.cols;
  store8<F8LIN_FP32>(part, col, n, dw, false);
  store8<F8LIN_FP32>(part + a.cols, col, n, db, false);
}

// dw[c], db[c] = the sums of `parts` partial sums, in a fixed order: 32 columns
// a workgroup, 32 groups of threads over the partial sums.
__global__ __launch_bounds__(1024) void ln_join_kernel(const float *part, int parts, int64_t cols, void *dw, int dw_dtype,
                                                       void *db, int db_dtype) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int64_t blocks = (cols + 31) / 32;
  const bool bias = blockIdx.x >= blocks;
  const int64_t col = (int64_t)(blockIdx.x - (bias ? blocks : 0)) * 32 + lane;
  void *const out = bias ? db : dw;
  if (!out) return;
  const int dt = bias ? db_dtype : dw_dtype;
  const int64_t ld = 2 * cols;
  float s = 0.0f;
  if (col < cols) {
    const float *p = part + (bias ? cols : 0) + col;
    int i = group;
    for (; i + 7 * 32 < parts; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(i + 32 * k) * ld];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
#pragma unroll 4
    for (; i < parts; i += 32) s += p[i * ld];
  }
  red[group][lane] = s;
  __syncthreads();
  if (group != 0 || col >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += red[i][lane];
  const uint32_t o = f32_to_elem(s, dt);
  if (dt == F8LIN_FP32) reinterpret_cast<uint32_t *>(out)[col] = o;
  else reinterpret_cast<uint16_t *>(out)[col] = (uint16_t)o;
}

// Rows of a launch: a grid has fewer than 2^32 threads.
constexpr int64_t kMaxRows = (int64_t)1 << 21;

template <int XT, int YT, bool PAST>
void forward_sized(const LayerNormFwd &a, hipStream_t s) {
  const unsigned rows = (unsigned)std::min(a.rows - a.first, kMaxRows), quads = (rows + 3) / 4;
  if (a.cols <= 512) ln_forward_kernel<XT, YT, 64, 1, false, PAST><<<quads, 256, 0, s>>>(a);
  else if (a.cols <= 1024) ln_forward_kernel<XT, YT, 64, 2, false, PAST><<<quads, 256, 0, s>>>(a);
  else if (a.cols <= 2048) ln_forward_kernel<XT, YT, 64, 4, false, PAST><<<quads, 256, 0, s>>>(a);
  else if (a.cols <= 4096) ln_forward_kernel<XT, YT, 256, 2, false, PAST><<<rows, 256, 0, s>>>(a);
  else if (a.cols <= 8192) ln_forward_kernel<XT, YT, 256, 4, false, PAST><<<rows, 256, 0, s>>>(a);
  else if (a.cols <= 16384) ln_forward_kernel<XT, YT, 1024, 2, false, PAST><<<rows, 1024, 0, s>>>(a);
  else ln_forward_wide_kernel<XT, YT><<<rows, 1024, 0, s>>>(a);
}
template <int XT, int YT>
void forward_typed(const LayerNormFwd &a, hipStream_t s) {
  if (a.cols < 8)
    ln_forward_kernel<XT, YT, 64, 1, true, false><<<(unsigned)((std::min(a.rows - a.first, kMaxRows) + 3) / 4), 256, 0, s>>>(a);
  else if (a.rows * a.cols * (elem_bytes(XT) + elem_bytes(YT)) > kPastBytes) forward_sized<XT, YT, true>(a, s);
  else forward_sized<XT, YT, false>(a, s);
}

template <int XT, int YT, bool PAST>
void backward_sized(const LayerNormBwd &a, int parts, int64_t each, hipStream_t s) {
  if (a.cols <= 512) ln_backward_kernel<XT, YT, 64, 1, false, PAST><<<parts, 256, 0, s>>>(a, each);
  else if (a.cols <= 2048) ln_backward_kernel<XT, YT, 256, 1, false, PAST><<<parts, 256, 0, s>>>(a, each);
  else if (a.cols <= 4096) ln_backward_kernel<XT, YT, 256, 2, false, PAST><<<parts, 256, 0, s>>>(a, each);
  else if (a.cols <= 8192) ln_backward_kernel<XT, YT, 512, 2, false, PAST><<<parts, 512, 0, s>>>(a, each);
  else if (a.cols <= 16384) ln_backward_kernel<XT, YT, 512, 4, false, PAST><<<parts, 512, 0, s>>>(a, each);
  else {
    LayerNormBwd b = a;
    for (; a.dx && b.first < a.rows; b.first += kMaxRows)
      ln_backward_wide_kernel<XT, YT><<<(unsigned)std::min(a.rows - b.first, kMaxRows), 1024, 0, s>>>(b);
    const int blocks = (int)((a.cols + 2047) / 2048);
    if (a.part) ln_param_kernel<XT, YT><<<(unsigned)parts * blocks, 256, 0, s>>>(a, each, blocks);
  }
}
template <int XT, int YT>
void backward_typed(const LayerNormBwd &a, hipStream_t s) {
  const int parts = ln_parts(a.rows, a.cols);
  const int64_t each = (a.rows + parts - 1) / parts;
  if (a.cols < 8) ln_backward_kernel<XT, YT, 64, 1, true, false><<<parts, 256, 0, s>>>(a, each);
  else if (a.rows * a.cols * (2 * elem_bytes(XT) + elem_bytes(YT)) > kPastBytes) backward_sized<XT, YT, true>(a, parts, each, s);
  else backward_sized<XT, YT, false>(a, parts, each, s);
}

template <int XT>
void forward_by_y(const LayerNormFwd &a, int y_dtype, hipStream_t s) {
  if constexpr (XT == F8LIN_FP32) {
    if (y_dtype == F8LIN_BF16) return forward_typed<XT, F8LIN_BF16>(a, s);
    if (y_dtype == F8LIN_FP16) return forward_typed<XT, F8LIN_FP16>(a, s);
  }
  forward_typed<XT, XT>(a, s);
}
template <int XT>
void backward_by_y(const LayerNormBwd &a, int dy_dtype, hipStream_t s) {
  if constexpr (XT == F8LIN_FP32) {
    if (dy_dtype == F8LIN_BF16) return backward_typed<XT, F8LIN_BF16>(a, s);
    if (dy_dtype == F8LIN_FP16) return backward_typed<XT, F8LIN_FP16>(a, s);
  }
  backward_typed<XT, XT>(a, s);
}

}  // namespace

// Partial sums of dw and db, one a workgroup: enough workgroups to fill the
// chip, but at least two rows each up to 256 of them and eight beyond, since a
// partial sum is written and read again (1021 x 2055 fp32 into 511: 16.2 us,
// into 256: 14.8; 12288 x 1600 bf16 into 512: 39 us, into 1024: 32).
int ln_parts(int64_t rows, int64_t cols) {
  const int64_t most = std::max(std::min<int64_t>((rows + 1) / 2, 256), rows / 8);
  const int64_t fill = cols <= 2048 ? 1024 : cols <= 4096 ? 512 : 256;
  return (int)std::max<int64_t>(1, std::min(most, fill));
}

hipError_t launch_layer_norm_forward(const LayerNormFwd &a, int x_dtype, int y_dtype, hipStream_t stream) {
  if (!a.amax && (a.rows == 0 || a.cols == 0)) return hipSuccess;
  if (a.amax) ln_clear_kernel<<<1, 1, 0, stream>>>(a.amax);
  LayerNormFwd k = a;
  for (; a.cols > 0 && k.first < a.rows; k.first += kMaxRows) {
    if (x_dtype == F8LIN_BF16) forward_by_y<F8LIN_BF16>(k, y_dtype, stream);
    else if (x_dtype == F8LIN_FP16) forward_by_y<F8LIN_FP16>(k, y_dtype, stream);
    else forward_by_y<F8LIN_FP32>(k, y_dtype, stream);
  }
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const LayerNormBwd &a, int x_dtype, int dy_dtype, void *dw, int dw_dtype, void *db,
                                      int db_dtype, hipStream_t stream) {
  if (a.cols == 0 || (a.rows == 0 && !dw && !db)) return hipSuccess;
  // (no rows: the parameters' gradients are zero)
  const int parts = a.rows > 0 ? ln_parts(a.rows, a.cols) : 0;
  if (parts) {
    if (x_dtype == F8LIN_BF16) backward_by_y<F8LIN_BF16>(a, dy_dtype, stream);
    else if (x_dtype == F8LIN_FP16) backward_by_y<F8LIN_FP16>(a, dy_dtype, stream);
    else backward_by_y<F8LIN_FP32>(a, dy_dtype, stream);
  }
  if (dw || db)
    ln_join_kernel<<<2 * (unsigned)((a.cols + 31) / 32), 1024, 0, stream>>>(a.part, parts, a.cols, dw, dw_dtype, db,
                                                                            db_dtype);
  return hipGetLastError();
}

}  // namespace f8lin

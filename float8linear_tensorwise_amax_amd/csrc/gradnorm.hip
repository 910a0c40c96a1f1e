// Global norm of a list of tensors, and scaling them to a largest norm: the
// step between the layers' backward passes and the optimiser.
//   n = sqrt(sum g^2), sum |g| or max |g| over every element of every tensor;
//   c = min(1, max_norm / (n + 1e-6)) in binary32;  out = c * g, rounded once.
// A NaN anywhere makes n and c NaN; an Inf makes n Inf and c 0 (so that Inf
// elements become NaN and the others 0), unless max_norm is Inf too: then c is 1.
//
// HBM-bound: the norm reads every element once, the scaling reads it again
// and writes it (872M bf16 elements into fp32: 254 us, 6.9 TB/s, and 970 us,
// 5.4 TB/s).  Sums are taken in binary64: the square of a 16-bit float is
// exact in it, cannot overflow or vanish, and the order of a fixed grid is
// the same on every run (no atomics).
// Tables of up to kGradBatch tensors go to the kernel as an argument, so a
// call copies nothing to the device; the tensors are cut into pieces of
// kPiece elements, dealt to the workgroups round robin.  Longer lists take one
// launch per table, each adding to the partial results of the one before.
// The scaling kernel's workgroups each reduce the partial results (at most 8
// KB, from the L2) themselves, so that norm and clipping are two launches: a
// launch of its own for it took 4 us, more than the rest of a small list.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 16384;
constexpr int kNormGrid = kGradPartials;
constexpr int kScaleGrid = 2048;
// 16-byte loads a thread has in flight, in both passes (the norm of 872M bf16
// elements through the caches: 289 us, with one load 349 us)
constexpr int kAhead = 4;

struct GradTable {
  const void *g[kGradBatch];
  void *out[kGradBatch];
  int64_t n[kGradBatch];
  int first[kGradBatch];  // first piece of each tensor
  uint8_t in_dtype[kGradBatch], out_dtype[kGradBatch];
  int count, pieces;
};

// Tensor of piece p: the last one whose first piece is at or before p.
__device__ __forceinline__ int tensor_of(const GradTable &t, int p) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int P>
__device__ __forceinline__ void fold(double &s, float v) {
  if constexpr (P == F8LIN_NORM_2) s = fma((double)v, (double)v, s);
  if constexpr (P == F8LIN_NORM_1) s += (double)fabsf(v);
  if constexpr (P == F8LIN_NORM_INF) s = (v != v) ? (double)v : fmax(s, (double)fabsf(v));  // (a NaN in s: below)
}
template <int P>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (P != F8LIN_NORM_INF) return a + b;
  return (a != a) ? a : (b != b) ? b : fmax(a, b);
}

template <int P>
__device__ __forceinline__ double block_join(double s) {
  __shared__ double red[kThreads / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s = join<P>(s, __shfl_xor(s, off, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return join<P>(join<P>(red[0], red[1]), join<P>(red[2], red[3]));
}

template <int P, int DT, bool PAST>
__device__ __forceinline__ double piece_norm(const void *g, int64_t begin, int64_t n) {
  typedef typename MxElem<DT>::type elem;
  const elem *x = reinterpret_cast<const elem *>(g) + begin;
  const int len = (int)min((int64_t)kPiece, n - begin);
  double s = 0.0;
  bool nan = false;
  auto add = [&](const Raw8<DT> &r) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = raw_value<DT>(r, k);
      if (P == F8LIN_NORM_INF) nan = nan || v != v;
      fold<P>(s, v);
    }
  };
  constexpr int kStep = 8 * kThreads;
  int at = 0;
  for (; at + kAhead * kStep <= len; at += kAhead * kStep) {  // kAhead loads in flight
    Raw8<DT> r[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) r[a] = load_raw8<DT, PAST>(x + at + a * kStep + 8 * (int)threadIdx.x, 8);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) add(r[a]);
  }
  for (int i = at + 8 * (int)threadIdx.x; i < len; i += kStep) add(load_raw8<DT>(x + i, len - i));
  return nan ? __builtin_nan("") : s;
}

template <int P, bool PAST>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const GradTable tab, double *partials, int add) {
  double s = 0.0;
  for (int p = blockIdx.x; p < tab.pieces; p += gridDim.x) {
    const int t = tensor_of(tab, p);
    const int64_t begin = (int64_t)(p - tab.first[t]) * kPiece;
    double v;
    if (tab.in_dtype[t] == F8LIN_BF16) v = piece_norm<P, F8LIN_BF16, PAST>(tab.g[t], begin, tab.n[t]);
    else if (tab.in_dtype[t] == F8LIN_FP16) v = piece_norm<P, F8LIN_FP16, PAST>(tab.g[t], begin, tab.n[t]);
    else v = piece_norm<P, F8LIN_FP32, PAST>(tab.g[t], begin, tab.n[t]);
    s = join<P>(s, v);
  }
  s = block_join<P>(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = add ? join<P>(partials[blockIdx.x], s) : s;
}

// The norm from the first `count` partial results, in every thread.
template <int P>
__device__ __forceinline__ float norm_of(const double *partials, int count) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s = join<P>(s, partials[i]);
  s = block_join<P>(s);
  return (float)(P == F8LIN_NORM_2 ? sqrt(s) : s);
}

template <int P>
__global__ __launch_bounds__(kThreads) void grad_norm_final_kernel(const double *partials, int count, float *norm) {
  const float n = norm_of<P>(partials, count);
  if (threadIdx.x == 0) norm[0] = n;
}

// E consecutive elements per thread and step, so that a step's stores are 16
// bytes a lane and contiguous whatever the types (16-bit gradients into
// 32-bit outputs with eight elements a lane: 1142 us for 872M elements, with
// four 995 us); kAhead steps' loads in flight.
template <int DI, int DO, bool PAST>
__device__ __forceinline__ void piece_scale(const void *g, void *out, int64_t begin, int64_t n, float c) {
  typedef typename MxElem<DI>::type ielem;
  typedef typename MxElem<DO>::type oelem;
  constexpr int E = DO == F8LIN_FP32 ? 4 : 8;
  constexpr int kInWords = E * (int)sizeof(ielem) / 4, kOutWords = 4;
  const ielem *x = reinterpret_cast<const ielem *>(g) + begin;
  oelem *y = reinterpret_cast<oelem *>(out) + begin;
  const int len = (int)min((int64_t)kPiece, n - begin);
  const int whole = len / E;  // whole groups of E
  auto value = [&](const uint32_t(&w)[kInWords], int k) {
    if constexpr (DI == F8LIN_FP32) return __uint_as_float(w[k]);
    else return elem_f32<DI>((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
  };
  for (int i0 = threadIdx.x; i0 < whole; i0 += kAhead * kThreads) {
    uint32_t w[kAhead][kInWords];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kThreads;
      if (i >= whole) continue;
      if constexpr (kInWords == 2) {
        const u32x2_u *src = reinterpret_cast<const u32x2_u *>(x + E * i);
        const u32x2 v = PAST ? __builtin_nontemporal_load(src) : *src;
        w[a][0] = v.x, w[a][1] = v.y;
      } else {
#pragma unroll
        for (int q = 0; q < kInWords; q += 4) {
          const u32x4_u *src = reinterpret_cast<const u32x4_u *>(x + E * i + q * 4 / (int)sizeof(ielem));
          const u32x4 v = PAST ? __builtin_nontemporal_load(src) : *src;
          w[a][q] = v.x, w[a][q + 1] = v.y, w[a][q + 2] = v.z, w[a][q + 3] = v.w;
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kThreads;
      uint32_t o[kOutWords];
#pragma unroll
      for (int k = 0; k < kOutWords; ++k) {
        if constexpr (DO == F8LIN_FP32)
          o[k] = __float_as_uint(value(w[a], k) * c);
        else
          o[k] = f32_to_elem(value(w[a], 2 * k) * c, DO) | f32_to_elem(value(w[a], 2 * k + 1) * c, DO) << 16;
      }
      if (i >= whole) continue;
      const u32x4 v = {o[0], o[1], o[2], o[3]};
      u32x4_u *const dst = reinterpret_cast<u32x4_u *>(y + E * i);
      if constexpr (PAST) __builtin_nontemporal_store(v, dst);
      else *dst = v;
    }
  }
  const int at = whole * E + (int)threadIdx.x;  // fewer than E elements left
  if (at < len) y[at] = (oelem)f32_to_elem(elem_f32<DI>((uint32_t)x[at]) * c, DO);
}

template <int DI, bool PAST>
__device__ __forceinline__ void piece_scale_to(const void *g, void *out, int out_dtype, int64_t begin, int64_t n, float c) {
  if (out_dtype == F8LIN_BF16) piece_scale<DI, F8LIN_BF16, PAST>(g, out, begin, n, c);
  else if (out_dtype == F8LIN_FP16) piece_scale<DI, F8LIN_FP16, PAST>(g, out, begin, n, c);
  else piece_scale<DI, F8LIN_FP32, PAST>(g, out, begin, n, c);
}

// P < 0: norm[0] holds the norm; otherwise it comes from the partial results,
// and the first workgroup writes it there.
template <int P, bool PAST>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradTable tab, const double *partials, int count,
                                                              float *norm, float max_norm) {
  float n;
  if constexpr (P < 0) {
    n = norm[0];
  } else {
    n = norm_of<P>(partials, count);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = n;
  }
  float c = max_norm / (n + 1e-6f);
  c = c > 1.0f ? 1.0f : c;  // (a NaN stays one)
  if (max_norm == __builtin_inff() && n == max_norm) c = 1.0f;  // (no limit: Inf / Inf above)
  // from the end: what the norm's pass read last is still in the caches
  for (int p = tab.pieces - 1 - (int)blockIdx.x; p >= 0; p -= (int)gridDim.x) {
    const int t = tensor_of(tab, p);
    // a factor of one leaves a tensor scaled in place as it is
    if (c == 1.0f && tab.g[t] == tab.out[t]) continue;
    const int64_t begin = (int64_t)(p - tab.first[t]) * kPiece;
    if (tab.in_dtype[t] == F8LIN_BF16)
      piece_scale_to<F8LIN_BF16, PAST>(tab.g[t], tab.out[t], tab.out_dtype[t], begin, tab.n[t], c);
    else if (tab.in_dtype[t] == F8LIN_FP16)
      piece_scale_to<F8LIN_FP16, PAST>(tab.g[t], tab.out[t], tab.out_dtype[t], begin, tab.n[t], c);
    else
      piece_scale_to<F8LIN_FP32, PAST>(tab.g[t], tab.out[t], tab.out_dtype[t], begin, tab.n[t], c);
  }
}

// Fills the table with the next tensors of the list (empty ones left out);
// returns the index after the last one taken.
int fill(GradTable &tab, const f8lin_grad *list, int at, int count, bool outs) {
  int64_t pieces = 0;
  tab.count = 0;
  for (; at < count && tab.count < kGradBatch; ++at) {
    const f8lin_grad &g = list[at];
    if (g.n == 0) continue;
    const int64_t np = (g.n + kPiece - 1) / kPiece;
    if (pieces + np > 0x7FFFFFFF) break;  // (one tensor of 2^40 elements has 2^26 pieces)
    tab.g[tab.count] = g.g;
    tab.out[tab.count] = outs ? g.out : nullptr;
    tab.n[tab.count] = g.n;
    tab.first[tab.count] = (int)pieces;
    tab.in_dtype[tab.count] = (uint8_t)g.dtype;
    tab.out_dtype[tab.count] = (uint8_t)g.out_dtype;
    ++tab.count;
    pieces += np;
  }
  tab.pieces = (int)pieces;
  return at;
}

// Whether gradients and outputs go past the caches (PAST): where they are more
// than the 256 MB last-level cache keeps between the two passes.  Clipping
// bf16 into bf16, past and through them: 256 MB in all 70 and 67 us, 384 MB
// 103 and 107 us, 1.6 GB 404 and 452 us; into fp32: 192 MB 51 and 46 us, 384
// MB 96 and 95 us, 576 MB 142 and 153 us.
constexpr int64_t kCached = (int64_t)320 << 20;
bool past_caches(const f8lin_grad *list, int count, bool outs) {
  auto size = [](int64_t n, int dt) { return n * (dt == F8LIN_FP32 ? 4 : 2); };
  int64_t bytes = 0;
  for (int i = 0; i < count; ++i) {
    bytes += size(list[i].n, list[i].dtype);
    if (outs && list[i].out != list[i].g) bytes += size(list[i].n, list[i].out_dtype);
  }
  return bytes > kCached;
}

// The norm's partial results; returns how many there are.
template <int P, bool PAST>
int launch_partials(const f8lin_grad *list, int count, double *partials, hipStream_t stream) {
  int at = 0, grid = kNormGrid;
  bool add = false;
  do {
    GradTable tab = {};
    at = fill(tab, list, at, count, false);
    // (a list of one table needs no more workgroups than it has pieces)
    if (!add && at >= count) grid = std::max(1, std::min(tab.pieces, kNormGrid));
    grad_norm_kernel<P, PAST><<<grid, kThreads, 0, stream>>>(tab, partials, add ? 1 : 0);
    add = true;
  } while (at < count);
  return grid;
}

template <int P, bool PAST>
void launch_scale(const f8lin_grad *list, int count, const double *partials, int nparts, float *norm, float max_norm,
                  hipStream_t stream) {
  int at = 0;
  do {
    GradTable tab = {};
    at = fill(tab, list, at, count, true);
    const unsigned grid = (unsigned)std::max(1, std::min(tab.pieces, kScaleGrid));
    grad_scale_kernel<P, PAST><<<grid, kThreads, 0, stream>>>(tab, partials, nparts, norm, max_norm);
  } while (at < count);
}

template <int P, bool PAST>
void launch_norm(const f8lin_grad *list, int count, double *partials, float *norm, bool clip, float max_norm,
                 hipStream_t stream) {
  const int nparts = launch_partials<P, PAST>(list, count, partials, stream);
  if (clip)
    launch_scale<P, PAST>(list, count, partials, nparts, norm, max_norm, stream);
  else
    grad_norm_final_kernel<P><<<1, kThreads, 0, stream>>>(partials, nparts, norm);
}

template <int P>
void launch_type(const f8lin_grad *list, int count, double *partials, float *norm, bool clip, float max_norm,
                 hipStream_t stream) {
  if (past_caches(list, count, clip))
    launch_norm<P, true>(list, count, partials, norm, clip, max_norm, stream);
  else
    launch_norm<P, false>(list, count, partials, norm, clip, max_norm, stream);
}

}  // namespace

hipError_t launch_grad_norm(const f8lin_grad *list, int count, int norm_type, double *partials, float *norm, bool clip,
                            float max_norm, hipStream_t stream) {
  if (norm_type == F8LIN_NORM_2) launch_type<F8LIN_NORM_2>(list, count, partials, norm, clip, max_norm, stream);
  else if (norm_type == F8LIN_NORM_1) launch_type<F8LIN_NORM_1>(list, count, partials, norm, clip, max_norm, stream);
  else launch_type<F8LIN_NORM_INF>(list, count, partials, norm, clip, max_norm, stream);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const f8lin_grad *list, int count, float *norm, float max_norm, hipStream_t stream) {
  if (count == 0) return hipSuccess;
  if (past_caches(list, count, true))
    launch_scale<-1, true>(list, count, nullptr, 0, norm, max_norm, stream);
  else
    launch_scale<-1, false>(list, count, nullptr, 0, norm, max_norm, stream);
  return hipGetLastError();
}

}  // namespace f8lin

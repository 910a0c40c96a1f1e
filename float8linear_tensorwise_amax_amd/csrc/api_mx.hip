// C ABI of the MXFP4 operators and of gradient clipping (declared in
// include/f8lin.h): argument validation, then the launches on the caller's
// stream.  Nothing here synchronises, reads device memory, or allocates on
// the device.
#include <math.h>

#include <algorithm>
#include <vector>

#include "check.h"
#include "internal.h"

namespace f8lin {
namespace {

constexpr int64_t kMxMaxLd = kMaxDim;

bool bad_size(int64_t d) { return d < 0 || d > kMaxDim; }
bool bad_matrix(int64_t r, int64_t c) { return bad_size(r) || bad_size(c) || r * c > kMaxElems; }
int es_of(int dt) { return dt == F8LIN_FP32 ? 4 : 2; }
int check_dtype(int dt) { return dt >= F8LIN_BF16 && dt <= F8LIN_FP32 ? F8LIN_OK : F8LIN_EINVAL; }
int check_rule(int r) { return r == F8LIN_MX_FLOOR || r == F8LIN_MX_CEIL ? F8LIN_OK : F8LIN_EINVAL; }
bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Bytes a (rows, cols) tensor with row stride ld elements spans.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int es) {
  return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

// A (rows, cols) MXFP4 tensor: pointers, alignment, strides.
int check_mx(const f8lin_mxfp4 &q, int64_t rows, int64_t cols) {
  if (rows * cols == 0) return F8LIN_OK;
  if (!q.codes || !q.scales) return F8LIN_EINVAL;
  if (!aligned16(q.codes) || !aligned16(q.scales)) return F8LIN_EALIGN;
  const int64_t nb = (cols + 31) / 32;
  if (q.ld % 16 || q.scale_ld % 16 || q.ld < 16 * nb || q.scale_ld < (nb + 15) / 16 * 16 || q.ld > kMxMaxLd ||
      q.scale_ld > kMxMaxLd)
    return F8LIN_ESHAPE;
  return F8LIN_OK;
}
Range mx_codes(const f8lin_mxfp4 &q, int64_t rows, int64_t cols) {
  return Range{q.codes, rows * cols > 0 ? (rows - 1) * q.ld + 16 * ((cols + 31) / 32) : 0};
}
Range mx_scales(const f8lin_mxfp4 &q, int64_t rows, int64_t cols) {
  return Range{q.scales, rows * cols > 0 ? rows * q.scale_ld : 0};
}

struct Ranges {
  Range r[16];
  int n = 0;
  void add(const void *p, int64_t bytes) { r[n++] = Range{p, bytes}; }
  void add(const f8lin_mxfp4 &q, int64_t rows, int64_t cols) {
    r[n++] = mx_codes(q, rows, cols);
    r[n++] = mx_scales(q, rows, cols);
  }
};

// A dense (rows, cols) input or output of type dt.
int check_dense(const void *p, int dt, int64_t rows, int64_t cols, int64_t ld, int align) {
  F8_TRY(check_dtype(dt));
  if (missing(p, rows * cols)) return F8LIN_EINVAL;
  if (rows * cols > 0 && (ld < cols || ld > kMaxElems)) return F8LIN_ESHAPE;
  if (rows * cols > 0 && !aligned_to(p, align)) return F8LIN_EALIGN;
  return F8LIN_OK;
}

int64_t dbias_tiles(int64_t M) { return M > 0 ? (M + kMxTile - 1) / kMxTile : 0; }

}  // namespace
}  // namespace f8lin

using namespace f8lin;

extern "C" {

int64_t f8lin_mxfp4_ld(int64_t cols) { return cols < 0 ? 0 : mx_ld(cols); }

int64_t f8lin_mxfp4_scale_ld(int64_t cols) { return cols < 0 ? 0 : (cols + 511) / 512 * 16; }

int f8lin_mxfp4_quantize(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const f8lin_mxfp4 *q,
                         const f8lin_mxfp4 *qt, int rule, void *stream) {
  F8_TRY(check_dtype(dtype));
  F8_TRY(check_rule(rule));
  if (bad_matrix(rows, cols)) return F8LIN_ESHAPE;
  if (ldx == 0) ldx = cols;
  const int es = es_of(dtype);
  F8_TRY(check_dense(x, dtype, rows, cols, ldx, es));
  const bool has_q = q && q->codes, has_t = qt && qt->codes;
  if (!has_q && !has_t) return rows * cols > 0 ? F8LIN_EINVAL : F8LIN_OK;
  Ranges outs;
  MxQuant t = {x, dtype, rows, cols, ldx, {}, {}, nullptr};
  if (has_q) {
    F8_TRY(check_mx(*q, rows, cols));
    t.q = *q;
    outs.add(*q, rows, cols);
  }
  if (has_t) {
    F8_TRY(check_mx(*qt, cols, rows));
    t.qt = *qt;
    outs.add(*qt, cols, rows);
  }
  const Range in = {x, span(rows, cols, ldx, es)};
  if (any_overlap(outs.r, outs.n, &in, 1)) return F8LIN_EINVAL;
  return status_of(launch_mx_quantize(&t, 1, rule, (hipStream_t)stream));
}

int f8lin_mxfp4_dequantize(const f8lin_mxfp4 *q, int64_t rows, int64_t cols, int dtype, void *out, void *stream) {
  if (!q) return F8LIN_EINVAL;
  if (bad_matrix(rows, cols)) return F8LIN_ESHAPE;
  F8_TRY(check_dense(out, dtype, rows, cols, cols, es_of(dtype)));
  F8_TRY(check_mx(*q, rows, cols));
  Ranges ins;
  ins.add(*q, rows, cols);
  const Range o = {out, rows * cols * es_of(dtype)};
  if (any_overlap(&o, 1, ins.r, ins.n)) return F8LIN_EINVAL;
  return status_of(launch_mx_dequantize(*q, rows, cols, dtype, out, (hipStream_t)stream));
}

int f8lin_mxfp4_gemm(const f8lin_mxfp4_gemm_desc *d, int count, void *stream) {
  static_assert(F8LIN_MXFP4_MAX_BATCH == kMxMaxGemms, "batch limit");
  if (!d || count < 1 || count > kMxMaxGemms) return F8LIN_EINVAL;
  Ranges outs, ins;
  MxGemm g[kMxMaxGemms];
  for (int i = 0; i < count; ++i) {
    const f8lin_mxfp4_gemm_desc &e = d[i];
    if (bad_matrix(e.M, e.N) || bad_matrix(e.M, e.K) || bad_matrix(e.N, e.K)) return F8LIN_ESHAPE;
    F8_TRY(check_dense(e.c, e.c_dtype, e.M, e.N, e.N, es_of(e.c_dtype)));
    F8_TRY(check_mx(e.a, e.M, e.K));
    F8_TRY(check_mx(e.b, e.N, e.K));
    if (e.bias) F8_TRY(check_dense(e.bias, e.bias_dtype, 1, e.N, e.N, es_of(e.bias_dtype)));
    outs.add(e.c, e.M * e.N * es_of(e.c_dtype));
    ins.add(e.a, e.M, e.K);
    ins.add(e.b, e.N, e.K);
    ins.add(e.bias, e.bias ? e.N * es_of(e.bias_dtype) : 0);
    g[i] = MxGemm{e.a, e.b, e.c, e.bias, e.M, e.N, e.K, e.c_dtype, e.bias_dtype};
  }
  if (any_overlap(outs.r, outs.n, ins.r, ins.n)) return F8LIN_EINVAL;
  return status_of(launch_mx_gemms(g, count, (hipStream_t)stream));
}

int f8lin_mxfp4_forward(const f8lin_mxfp4_fwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_mxfp4_fwd_args &a = *p;
  F8_TRY(check_rule(a.rule));
  const int64_t M = a.M, N = a.N, K = a.K, ldx = a.ldx ? a.ldx : K;
  if (bad_matrix(M, N) || bad_matrix(M, K) || bad_matrix(N, K)) return F8LIN_ESHAPE;
  F8_TRY(check_dense(a.x, a.x_dtype, M, K, ldx, es_of(a.x_dtype)));
  F8_TRY(check_dense(a.y, a.y_dtype, M, N, N, es_of(a.y_dtype)));
  if (a.bias) F8_TRY(check_dense(a.bias, a.bias_dtype, 1, N, N, es_of(a.bias_dtype)));
  const bool xt = a.x4t.codes != nullptr, quant_w = a.w != nullptr, wt = quant_w && a.w4t.codes != nullptr;
  const bool fused = !a.x4.codes && !xt && !quant_w && mx_linear_fused(M, N, K);
  if (!fused) F8_TRY(check_mx(a.x4, M, K));
  if (xt) F8_TRY(check_mx(a.x4t, K, M));
  F8_TRY(check_mx(a.w4, N, K));
  if (quant_w) F8_TRY(check_dense(a.w, a.w_dtype, N, K, K, es_of(a.w_dtype)));
  if (wt) F8_TRY(check_mx(a.w4t, K, N));
  Ranges outs, ins;
  outs.add(a.y, M * N * es_of(a.y_dtype));
  if (!fused) outs.add(a.x4, M, K);
  if (xt) outs.add(a.x4t, K, M);
  (quant_w ? outs : ins).add(a.w4, N, K);
  if (wt) outs.add(a.w4t, K, N);
  ins.add(a.x, span(M, K, ldx, es_of(a.x_dtype)));
  ins.add(a.w, quant_w ? N * K * es_of(a.w_dtype) : 0);
  ins.add(a.bias, a.bias ? N * es_of(a.bias_dtype) : 0);
  if (any_overlap(outs.r, outs.n, ins.r, ins.n)) return F8LIN_EINVAL;

  hipStream_t s = (hipStream_t)stream;
  if (fused) {
    const MxLinear l = {a.x, a.x_dtype, ldx, a.w4, a.y, a.y_dtype, a.bias, a.bias_dtype, M, N, K, a.rule};
    return status_of(launch_mx_linear(l, s));
  }
  MxQuant q[2] = {{a.x, a.x_dtype, M, K, ldx, a.x4, xt ? a.x4t : f8lin_mxfp4{}, nullptr},
                  {a.w, a.w_dtype, N, K, K, a.w4, wt ? a.w4t : f8lin_mxfp4{}, nullptr}};
  // one launch for both where they agree in type and layouts
  const bool both = quant_w && a.w_dtype == a.x_dtype && xt == wt;
  F8_TRY(status_of(launch_mx_quantize(q, both ? 2 : 1, a.rule, s)));
  if (quant_w && !both) F8_TRY(status_of(launch_mx_quantize(q + 1, 1, a.rule, s)));
  const MxGemm g = {a.x4, a.w4, a.y, a.bias, M, N, K, a.y_dtype, a.bias_dtype};
  return status_of(launch_mx_gemms(&g, 1, s));
}

int f8lin_mxfp4_forward_fused(int64_t M, int64_t N, int64_t K) { return mx_linear_fused(M, N, K) ? 1 : 0; }

size_t f8lin_mxfp4_dbias_workspace_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0) return 0;
  return (size_t)dbias_tiles(M) * (size_t)N * sizeof(float);
}

int f8lin_mxfp4_backward(const f8lin_mxfp4_bwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_mxfp4_bwd_args &a = *p;
  F8_TRY(check_rule(a.rule));
  const int64_t M = a.M, N = a.N, K = a.K, lddy = a.lddy ? a.lddy : N;
  if (bad_matrix(M, N) || bad_matrix(M, K) || bad_matrix(N, K)) return F8LIN_ESHAPE;
  F8_TRY(check_dense(a.dy, a.dy_dtype, M, N, lddy, es_of(a.dy_dtype)));
  if (!a.dx && !a.dw && !a.dbias) return F8LIN_OK;
  Ranges outs, ins;
  ins.add(a.dy, span(M, N, lddy, es_of(a.dy_dtype)));
  if (a.dx) {
    F8_TRY(check_dense(a.dx, a.dx_dtype, M, K, K, es_of(a.dx_dtype)));
    F8_TRY(check_mx(a.dy4, M, N));
    F8_TRY(check_mx(a.w4t, K, N));
    outs.add(a.dx, M * K * es_of(a.dx_dtype));
    outs.add(a.dy4, M, N);
    ins.add(a.w4t, K, N);
  }
  // (the column sums ride on the pass that quantises along the columns)
  const bool cols = a.dw || a.dbias;
  if (cols) {
    F8_TRY(check_mx(a.dy4t, N, M));
    outs.add(a.dy4t, N, M);
  }
  if (a.dw) {
    F8_TRY(check_dense(a.dw, a.dw_dtype, N, K, K, es_of(a.dw_dtype)));
    F8_TRY(check_mx(a.x4t, K, M));
    outs.add(a.dw, N * K * es_of(a.dw_dtype));
    ins.add(a.x4t, K, M);
  }
  const int64_t db_ws = a.dbias ? (int64_t)f8lin_mxfp4_dbias_workspace_bytes(M, N) : 0;
  if (a.dbias) {
    F8_TRY(check_dense(a.dbias, a.dbias_dtype, 1, N, N, es_of(a.dbias_dtype)));
    if (db_ws > 0 && (!a.dbias_ws || a.dbias_ws_bytes < (size_t)db_ws)) return F8LIN_EWORKSPACE;
    if (!aligned16(a.dbias_ws)) return F8LIN_EALIGN;
    outs.add(a.dbias, N * es_of(a.dbias_dtype));
    outs.add(a.dbias_ws, db_ws);
  }
  if (any_overlap(outs.r, outs.n, ins.r, ins.n)) return F8LIN_EINVAL;

  hipStream_t s = (hipStream_t)stream;
  const MxQuant q = {a.dy, a.dy_dtype, M, N, lddy, a.dx ? a.dy4 : f8lin_mxfp4{}, cols ? a.dy4t : f8lin_mxfp4{},
                     a.dbias ? a.dbias_ws : nullptr};
  F8_TRY(status_of(launch_mx_quantize(&q, 1, a.rule, s)));
  if (a.dbias) F8_TRY(status_of(launch_mx_dbias(a.dbias_ws, dbias_tiles(M), N, a.dbias, a.dbias_dtype, s)));
  MxGemm g[2];
  int n = 0;
  if (a.dx) g[n++] = MxGemm{a.dy4, a.w4t, a.dx, nullptr, M, K, N, a.dx_dtype, 0};
  if (a.dw) g[n++] = MxGemm{a.dy4t, a.x4t, a.dw, nullptr, N, K, M, a.dw_dtype, 0};
  return n ? status_of(launch_mx_gemms(g, n, s)) : F8LIN_OK;
}

size_t f8lin_grad_workspace_bytes(void) { return kGradPartials * sizeof(double); }

}  // extern "C"

namespace f8lin {
namespace {

int check_grads(const f8lin_grad *list, int count, int norm_type, bool outs) {
  if (count < 0 || (count > 0 && !list)) return F8LIN_EINVAL;
  if (norm_type != F8LIN_NORM_2 && norm_type != F8LIN_NORM_1 && norm_type != F8LIN_NORM_INF) return F8LIN_EINVAL;
  for (int i = 0; i < count; ++i) {
    const f8lin_grad &g = list[i];
    F8_TRY(check_dtype(g.dtype));
    if (g.n < 0 || g.n > kMaxElems) return F8LIN_ESHAPE;
    if (missing(g.g, g.n)) return F8LIN_EINVAL;
    if (!aligned_to(g.g, es_of(g.dtype))) return F8LIN_EALIGN;
    if (outs) {
      F8_TRY(check_dtype(g.out_dtype));
      if (missing(g.out, g.n)) return F8LIN_EINVAL;
      if (!aligned_to(g.out, es_of(g.out_dtype))) return F8LIN_EALIGN;
      if (g.n > 0 && g.out == g.g && g.out_dtype != g.dtype) return F8LIN_EINVAL;
    }
  }
  return F8LIN_OK;
}

// Whether a written range overlaps any other range (ranges in any order).
struct Span {
  uintptr_t begin, end;
  bool written;
};
bool spans_clash(std::vector<Span> &v) {
  std::sort(v.begin(), v.end(), [](const Span &a, const Span &b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;
  for (const Span &s : v) {
    if (s.begin < (s.written ? any : written)) return true;
    any = std::max(any, s.end);
    if (s.written) written = std::max(written, s.end);
  }
  return false;
}
void add_span(std::vector<Span> &v, const void *p, int64_t bytes, bool written) {
  if (bytes > 0) v.push_back(Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
}

int check_grad_ws(const void *ws, size_t bytes) {
  return !ws || bytes < f8lin_grad_workspace_bytes() || !aligned16(ws) ? F8LIN_EWORKSPACE : F8LIN_OK;
}

int grad_impl(const f8lin_grad *list, int count, int norm_type, bool clip, float max_norm, float *norm, bool given,
              void *ws, size_t ws_bytes, void *stream) {
  F8_TRY(check_grads(list, count, norm_type, clip));
  if (!norm) return F8LIN_EINVAL;
  if (!aligned4(norm)) return F8LIN_EALIGN;
  if (clip && !(max_norm >= 0.0f)) return F8LIN_EINVAL;
  if (!given) F8_TRY(check_grad_ws(ws, ws_bytes));
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)count + 2);
  for (int i = 0; i < count; ++i) {
    const f8lin_grad &g = list[i];
    const bool same = clip && g.out == g.g;
    add_span(spans, g.g, g.n * es_of(g.dtype), same);
    if (clip && !same) add_span(spans, g.out, g.n * es_of(g.out_dtype), true);
  }
  add_span(spans, norm, 4, !given);
  if (!given) add_span(spans, ws, (int64_t)f8lin_grad_workspace_bytes(), true);
  if (spans_clash(spans)) return F8LIN_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  if (given) return status_of(launch_grad_scale(list, count, norm, max_norm, s));
  return status_of(launch_grad_norm(list, count, norm_type, (double *)ws, norm, clip, max_norm, s));
}

}  // namespace
}  // namespace f8lin

extern "C" {

// (the overlap check sorts the ranges on the host: no exception leaves a C entry)
int f8lin_grad_norm(const f8lin_grad *list, int count, int norm_type, float *norm_out, void *ws, size_t ws_bytes,
                    void *stream) {
  try {
    return grad_impl(list, count, norm_type, false, 0.0f, norm_out, false, ws, ws_bytes, stream);
  } catch (...) {
    return F8LIN_EHIP;
  }
}

int f8lin_grad_clip(const f8lin_grad *list, int count, int norm_type, float max_norm, float *norm, int norm_given,
                    void *ws, size_t ws_bytes, void *stream) {
  try {
    return grad_impl(list, count, norm_type, true, max_norm, norm, norm_given != 0, ws, ws_bytes, stream);
  } catch (...) {
    return F8LIN_EHIP;
  }
}

}  // extern "C"

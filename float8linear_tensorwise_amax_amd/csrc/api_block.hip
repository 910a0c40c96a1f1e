// C ABI of the operators around a block's linears, layer norm and low-rank
// adapters (declared in include/f8lin.h): argument validation, then the
// launches on the caller's stream.  Nothing here synchronises, reads device
// memory, or allocates.
#include "check.h"
#include "internal.h"
#include "lora.h"

namespace f8lin {
namespace {

bool bad_size(int64_t d) { return d < 0 || d > kMaxDim; }
bool bad_matrix(int64_t r, int64_t c) { return bad_size(r) || bad_size(c) || r * c > kMaxElems; }
// Of a layer norm: its rows are only counted.
bool bad_rows(int64_t r, int64_t c) { return r < 0 || r > kMaxElems || bad_size(c) || (c > 0 && r > kMaxElems / c); }
int es_of(int dt) { return dt == F8LIN_FP32 ? 4 : 2; }
int check_dtype(int dt) { return dt >= F8LIN_BF16 && dt <= F8LIN_FP32 ? F8LIN_OK : F8LIN_EINVAL; }
bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// A (rows, cols) input or output of type dt whose rows are ld elements apart.
int check_dense(const void *p, int dt, int64_t rows, int64_t cols, int64_t ld) {
  F8_TRY(check_dtype(dt));
  if (rows * cols == 0) return F8LIN_OK;
  if (!p) return F8LIN_EINVAL;
  if (ld < cols || ld > kMaxElems || ld > kMaxBytes / rows) return F8LIN_ESHAPE;
  return aligned_to(p, es_of(dt)) ? F8LIN_OK : F8LIN_EALIGN;
}
Range span(const void *p, int dt, int64_t rows, int64_t cols, int64_t ld) {
  return Range{p, p && rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es_of(dt) : 0};
}
int check_f32(const float *p, int64_t n) {
  if (n == 0) return F8LIN_OK;
  if (!p) return F8LIN_EINVAL;
  return aligned4(p) ? F8LIN_OK : F8LIN_EALIGN;
}

// y's type: x's, or with binary32 x any.
bool types_pair(int x, int y) { return x == y || x == F8LIN_FP32; }

}  // namespace
}  // namespace f8lin

using namespace f8lin;

extern "C" {

// ------------------------------------------------------------- layer norm

int f8lin_layer_norm_forward(const f8lin_layer_norm_fwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_layer_norm_fwd_args &a = *p;
  if (bad_rows(a.rows, a.cols)) return F8LIN_ESHAPE;
  const int64_t R = a.rows, C = a.cols, ldx = a.ldx ? a.ldx : C;
  F8_TRY(check_dense(a.x, a.x_dtype, R, C, ldx));
  F8_TRY(check_dense(a.y, a.y_dtype, R, C, C));
  if (!types_pair(a.x_dtype, a.y_dtype)) return F8LIN_EINVAL;
  if (a.weight) F8_TRY(check_dense(a.weight, a.weight_dtype, 1, C, C));
  if (a.bias) F8_TRY(check_dense(a.bias, a.bias_dtype, 1, C, C));
  if (!(a.eps >= 0.0f)) return F8LIN_EINVAL;
  if (a.stats) F8_TRY(check_f32(a.stats, R));
  if (a.y_amax && !aligned4(a.y_amax)) return F8LIN_EALIGN;
  const Range outs[] = {span(a.y, a.y_dtype, R, C, C), {a.stats, a.stats ? 8 * R : 0}, {a.y_amax, a.y_amax ? 4 : 0}};
  const Range ins[] = {span(a.x, a.x_dtype, R, C, ldx), span(a.weight, a.weight_dtype, 1, C, C),
                       span(a.bias, a.bias_dtype, 1, C, C)};
  if (any_overlap(outs, 3, ins, 3)) return F8LIN_EINVAL;
  const LayerNormFwd k = {a.x, R, C, ldx, a.weight, a.bias, a.weight_dtype, a.bias_dtype, a.eps, a.y, a.stats, a.y_amax};
  return status_of(launch_layer_norm_forward(k, a.x_dtype, a.y_dtype, (hipStream_t)stream));
}

size_t f8lin_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
  if (bad_rows(rows, cols) || rows == 0) return 0;
  return (size_t)ln_parts(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

int f8lin_layer_norm_backward(const f8lin_layer_norm_bwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_layer_norm_bwd_args &a = *p;
  if (bad_rows(a.rows, a.cols)) return F8LIN_ESHAPE;
  const int64_t R = a.rows, C = a.cols, ldx = a.ldx ? a.ldx : C, lddy = a.lddy ? a.lddy : C;
  F8_TRY(check_dense(a.dy, a.dy_dtype, R, C, lddy));
  F8_TRY(check_dense(a.x, a.x_dtype, R, C, ldx));
  if (!types_pair(a.x_dtype, a.dy_dtype)) return F8LIN_EINVAL;
  if (a.weight) F8_TRY(check_dense(a.weight, a.weight_dtype, 1, C, C));
  F8_TRY(check_f32(a.stats, C > 0 ? R : 0));
  if (a.dx) F8_TRY(check_dense(a.dx, a.x_dtype, R, C, C));
  if (a.dweight) F8_TRY(check_dense(a.dweight, a.dweight_dtype, 1, C, C));
  if (a.dbias) F8_TRY(check_dense(a.dbias, a.dbias_dtype, 1, C, C));
  const bool params = a.dweight || a.dbias;
  if (!a.dx && !params) return F8LIN_OK;
  const size_t need = params ? f8lin_layer_norm_workspace_bytes(R, C) : 0;
  if (need > 0) {
    if (!a.ws || a.ws_bytes < need) return F8LIN_EWORKSPACE;
    if (!aligned16(a.ws)) return F8LIN_EALIGN;
  }
  const Range outs[] = {span(a.dx, a.x_dtype, R, C, C), span(a.dweight, a.dweight_dtype, 1, C, C),
                        span(a.dbias, a.dbias_dtype, 1, C, C), {a.ws, (int64_t)need}};
  const Range ins[] = {span(a.dy, a.dy_dtype, R, C, lddy), span(a.x, a.x_dtype, R, C, ldx),
                       span(a.weight, a.weight_dtype, 1, C, C), {a.stats, 8 * R}};
  if (any_overlap(outs, 4, ins, 4)) return F8LIN_EINVAL;
  const LayerNormBwd k = {a.dy, a.x, R, C, lddy, ldx, a.weight, a.weight_dtype, a.stats, a.dx,
                          need > 0 ? a.ws : nullptr};
  return status_of(launch_layer_norm_backward(k, a.x_dtype, a.dy_dtype, a.dweight, a.dweight_dtype, a.dbias,
                                              a.dbias_dtype, (hipStream_t)stream));
}

// ------------------------------------------------------ low-rank adapters

size_t f8lin_lora_plan_bytes(int64_t tokens, int adapters) {
  if (bad_size(tokens) || adapters < 1 || adapters > kLoraMaxAdapters) return 0;
  return (size_t)lora_plan_words(tokens, adapters) * sizeof(int);
}

int f8lin_lora_plan(const void *index, int index_bytes, int64_t tokens, int adapters, void *plan, size_t plan_bytes,
                    void *stream) {
  if (index_bytes != 4 && index_bytes != 8) return F8LIN_EINVAL;
  if (bad_size(tokens) || adapters < 1 || adapters > kLoraMaxAdapters) return F8LIN_ESHAPE;
  if (missing(index, tokens)) return F8LIN_EINVAL;
  const size_t need = f8lin_lora_plan_bytes(tokens, adapters);
  if (!plan || plan_bytes < need) return F8LIN_EWORKSPACE;
  if (!aligned16(plan) || (tokens > 0 && !aligned_to(index, index_bytes))) return F8LIN_EALIGN;
  const Range o = {plan, (int64_t)need}, in = {index, tokens * index_bytes};
  if (any_overlap(&o, 1, &in, 1)) return F8LIN_EINVAL;
  return status_of(launch_lora_plan(index, index_bytes == 8, (int)tokens, adapters, (int *)plan, (hipStream_t)stream));
}

}  // extern "C"

namespace f8lin {
namespace {

int check_lora(int64_t T, int64_t K, int64_t N, int rank, int adapters, int dtype) {
  F8_TRY(check_dtype(dtype));
  if (bad_matrix(T, K) || bad_matrix(T, N) || rank < 1 || rank > kLoraMaxRank || adapters < 1 ||
      adapters > kLoraMaxAdapters)
    return F8LIN_ESHAPE;
  return (int64_t)adapters * rank * K > kMaxElems || (int64_t)adapters * rank * N > kMaxElems ? F8LIN_ESHAPE : F8LIN_OK;
}
int check_plan(const void *plan) {
  if (!plan) return F8LIN_EINVAL;
  return aligned16(plan) ? F8LIN_OK : F8LIN_EALIGN;
}
int check_ws(const void *ws, size_t bytes, int64_t need) {
  if (need == 0) return F8LIN_OK;
  if (!ws || (int64_t)bytes < need) return F8LIN_EWORKSPACE;
  return aligned16(ws) ? F8LIN_OK : F8LIN_EALIGN;
}

// What the calls keep in their workspace, in bytes from its start: H's parts,
// or H in fragments and then its exponents; in the backward G's, G by rank, and
// the partial sums of dA and dB.
struct LoraWs {
  bool split;
  int parts;
  int64_t h_bytes, exps_at, ht_at, part_a_at, part_b_at, bytes;
  int chunk, chunks;
};
int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }
int64_t h_bytes_of(int64_t T, int rank) { return T * lora_rank_pad(rank) * 4; }
LoraWs lora_forward_ws(int64_t T, int64_t cols, int rank, int adapters) {
  LoraWs w = {};
  w.split = lora_split(T);
  w.parts = lora_parts(T, adapters, cols, rank);
  w.h_bytes = h_bytes_of(T, rank);
  w.exps_at = w.split ? w.parts * w.h_bytes
                      : lora_max_tiles(T, adapters) * lora_tile(T) * (int64_t)lora_rank_pad(rank) * 4;
  w.bytes = w.exps_at + (w.split ? 0 : up16((rank + 63) / 64 * T * 4));
  return w;
}
LoraWs lora_backward_ws(int64_t T, int64_t K, int64_t N, int rank, int adapters) {
  LoraWs w = lora_forward_ws(T, N, rank, adapters);
  w.ht_at = w.bytes;
  w.chunk = lora_chunk(T, K, N, rank);
  w.chunks = (int)((T + w.chunk - 1) / w.chunk);
  w.part_a_at = w.ht_at + w.h_bytes;
  // (one chunk: nothing reaches over several)
  const int64_t slots = w.chunks > 1 ? 2 * (int64_t)w.chunks : 0;
  w.part_b_at = w.part_a_at + up16(slots * rank * K * 4);
  w.bytes = w.part_b_at + up16(slots * rank * N * 4);
  return w;
}

}  // namespace
}  // namespace f8lin

extern "C" {

size_t f8lin_lora_forward_workspace_bytes(int64_t T, int64_t K, int64_t N, int rank, int adapters) {
  if (check_lora(T, K, N, rank, adapters, F8LIN_FP32) != F8LIN_OK) return 0;
  return (size_t)lora_forward_ws(T, K, rank, adapters).bytes;
}

size_t f8lin_lora_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, int rank, int adapters) {
  if (check_lora(T, K, N, rank, adapters, F8LIN_FP32) != F8LIN_OK) return 0;
  return (size_t)lora_backward_ws(T, K, N, rank, adapters).bytes;
}

int f8lin_lora_forward(const f8lin_lora_fwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_lora_fwd_args &a = *p;
  const int64_t T = a.tokens, K = a.K, N = a.N, ldx = a.ldx ? a.ldx : K, ldb = a.ldbase ? a.ldbase : N;
  F8_TRY(check_lora(T, K, N, a.rank, a.adapters, a.dtype));
  const int64_t per = (int64_t)a.adapters * a.rank;
  F8_TRY(check_dense(a.x, a.dtype, T, K, ldx));
  F8_TRY(check_dense(a.a, a.dtype, per, K, K));
  F8_TRY(check_dense(a.b, a.dtype, per, N, N));
  if (a.base) F8_TRY(check_dense(a.base, a.dtype, T, N, ldb));
  F8_TRY(check_dense(a.y, a.dtype, T, N, N));
  if (a.scales && !aligned4(a.scales)) return F8LIN_EALIGN;
  F8_TRY(check_plan(a.plan));
  const LoraWs w = lora_forward_ws(T, K, a.rank, a.adapters);
  F8_TRY(check_ws(a.ws, a.ws_bytes, w.bytes));
  if (!aligned16(a.h)) return F8LIN_EALIGN;
  const Range y = span(a.y, a.dtype, T, N, N), base = span(a.base, a.dtype, T, N, ldb);
  // (y may be base itself)
  const bool same = a.base == a.y && ldb == N;
  const Range outs[] = {y, {a.h, a.h ? w.h_bytes : 0}, {a.ws, w.bytes}};
  const Range ins[] = {span(a.x, a.dtype, T, K, ldx), span(a.a, a.dtype, per, K, K), span(a.b, a.dtype, per, N, N),
                       {a.scales, a.scales ? 4 * (int64_t)a.adapters : 0},
                       {a.plan, (int64_t)f8lin_lora_plan_bytes(T, a.adapters)}, same ? Range{nullptr, 0} : base};
  if (any_overlap(outs, 3, ins, 6)) return F8LIN_EINVAL;
  if (T == 0 || N == 0) return F8LIN_OK;
  hipStream_t s = (hipStream_t)stream;
  const bool split = w.split;
  const int tiles = (int)lora_max_tiles(T, a.adapters);
  int *const exps = (int *)((uint8_t *)a.ws + w.exps_at);
  const LoraDown d = {(const int *)a.plan, (int)T, a.adapters, a.rank, tiles, a.x, ldx, K, a.a, a.scales,
                      split ? nullptr : (uint32_t *)a.ws, a.h, exps, split ? (float *)a.ws : nullptr, w.parts};
  F8_TRY(status_of(launch_lora_down(d, a.dtype, false, s)));
  const LoraUp u = {(const int *)a.plan, (int)T, a.adapters, a.rank, tiles, split ? nullptr : (const uint32_t *)a.ws, exps,
                    split ? (const float *)a.ws : nullptr, w.parts, a.b, a.base, ldb, N, a.y, N};
  return status_of(launch_lora_up(u, a.dtype, false, s));
}

int f8lin_lora_backward(const f8lin_lora_bwd_args *p, void *stream) {
  if (!p) return F8LIN_EINVAL;
  const f8lin_lora_bwd_args &a = *p;
  const int64_t T = a.tokens, K = a.K, N = a.N, ldx = a.ldx ? a.ldx : K, lddy = a.lddy ? a.lddy : N;
  F8_TRY(check_lora(T, K, N, a.rank, a.adapters, a.dtype));
  if (!a.dx && !a.da && !a.db) return F8LIN_OK;
  const int64_t per = (int64_t)a.adapters * a.rank;
  const bool g = a.dx || a.da;
  F8_TRY(check_dense(a.dy, a.dtype, T, N, lddy));
  if (a.dx) F8_TRY(check_dense(a.a, a.dtype, per, K, K));
  if (g) F8_TRY(check_dense(a.b, a.dtype, per, N, N));
  if (a.da) F8_TRY(check_dense(a.x, a.dtype, T, K, ldx));
  if (a.dx) F8_TRY(check_dense(a.dx, a.dtype, T, K, K));
  if (a.da) F8_TRY(check_dense(a.da, a.dtype, per, K, K));
  if (a.db) {
    F8_TRY(check_dense(a.db, a.dtype, per, N, N));
    if (missing(a.h, T)) return F8LIN_EINVAL;
    if (!aligned16(a.h)) return F8LIN_EALIGN;
  }
  if (a.scales && !aligned4(a.scales)) return F8LIN_EALIGN;
  F8_TRY(check_plan(a.plan));
  const LoraWs w = lora_backward_ws(T, K, N, a.rank, a.adapters);
  F8_TRY(check_ws(a.ws, a.ws_bytes, w.bytes));
  const Range outs[] = {span(a.dx, a.dtype, T, K, K), span(a.da, a.dtype, per, K, K), span(a.db, a.dtype, per, N, N),
                        {a.ws, w.bytes}};
  const Range none = {nullptr, 0};
  const Range ins[] = {span(a.dy, a.dtype, T, N, lddy), a.da ? span(a.x, a.dtype, T, K, ldx) : none,
                       a.dx ? span(a.a, a.dtype, per, K, K) : none, g ? span(a.b, a.dtype, per, N, N) : none,
                       {a.scales, a.scales ? 4 * (int64_t)a.adapters : 0}, {a.h, a.db ? w.h_bytes : 0},
                       {a.plan, (int64_t)f8lin_lora_plan_bytes(T, a.adapters)}};
  if (any_overlap(outs, 4, ins, 7)) return F8LIN_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *const ws = (uint8_t *)a.ws;
  const bool split = w.split;
  const int tiles = (int)lora_max_tiles(T, a.adapters);
  int *const exps = (int *)(ws + w.exps_at);
  float *const gt = (float *)(ws + w.ht_at);
  if (g) {
    const LoraDown d = {(const int *)a.plan, (int)T, a.adapters, a.rank, tiles, a.dy, lddy, N, a.b, a.scales,
                        split ? nullptr : (uint32_t *)ws, a.da ? gt : nullptr, exps, split ? (float *)ws : nullptr, w.parts};
    F8_TRY(status_of(launch_lora_down(d, a.dtype, true, s)));
    const LoraUp u = {(const int *)a.plan, (int)T, a.adapters, a.rank, tiles, split ? nullptr : (const uint32_t *)ws, exps,
                      split ? (const float *)ws : nullptr, w.parts, a.a, nullptr, K, K, a.dx, K};
    if (a.dx) F8_TRY(status_of(launch_lora_up(u, a.dtype, true, s)));
  }
  if (!a.da && !a.db) return F8LIN_OK;
  LoraOuter o = {(const int *)a.plan, (int)T, a.adapters, a.rank, w.chunk, w.chunks, {}, 0};
  o.side[0] = LoraOuterSide{a.x, ldx, K, gt, a.da, 0, (float *)(ws + w.part_a_at), 0, 0};
  o.side[1] = LoraOuterSide{a.dy, lddy, N, a.h, a.db, 1, (float *)(ws + w.part_b_at), 0, 0};
  return status_of(launch_lora_outer(o, a.dtype, s));
}

}  // extern "C"

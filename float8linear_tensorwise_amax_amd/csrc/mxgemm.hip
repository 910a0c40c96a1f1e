// MXFP4 product  C (M, N) = A (M, K) . B (N, K)^T (+ bias), operands as e2m1
// codes with an e8m0 scale per 32 elements of K, fp32 accumulation.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes four K blocks of 32: lane l feeds
// the 16 code bytes and the one scale byte of block l / 16 of row l % 16, so
// a block's scale is applied by the matrix core and costs no instruction.
// The instruction runs on C^T (B as its first operand): lane l then holds
// columns 4 (l / 16) .. + 3 of row l % 16.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

struct MxProblem {
  const uint8_t *a, *as, *b, *bs;
  void *c;
  const void *bias;
  int M, N, K;
  int64_t lda, lsa, ldb, lsb;
  int c_dtype, bias_dtype;
  int tiles_m, tiles_n, first;
};
struct MxBatch {
  MxProblem p[kMxMaxGemms];
  int count;
};

__device__ __forceinline__ v4f mfma_fp4(const u32x4 &a, int sa, const u32x4 &b, int sb, const v4f &c) {
  const v8i x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

__device__ __forceinline__ float load_elem(const void *p, int64_t i, int dt) {
  if (dt == F8LIN_BF16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
  if (dt == F8LIN_FP16) return f16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
  return reinterpret_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v, int dt) {
  if (dt == F8LIN_FP32)
    reinterpret_cast<float *>(p)[i] = v;
  else
    reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_elem(v, dt);
}

// One workgroup of four waves per 64 x 64 tile, a wave 32 x 32, operands
// straight from global memory.
__global__ __launch_bounds__(256) void mx_gemm_kernel(const MxBatch batch) {
  int pi = 0;
#pragma unroll
  for (int i = 1; i < kMxMaxGemms; ++i)
    if (i < batch.count && (int)blockIdx.x >= batch.p[i].first) pi = i;
  const MxProblem P = batch.p[pi];
  const int t = (int)blockIdx.x - P.first;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int m0 = t / P.tiles_n * 64 + (wave >> 1) * 32, n0 = t % P.tiles_n * 64 + (wave & 1) * 32;
  const int nb = (P.K + kMxBlock - 1) / kMxBlock;
  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b0 = 0; b0 < nb; b0 += 4) {
    const int blk = b0 + g;
    u32x4 fa[2], fb[2];
    int sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = fb[i] = u32x4{0, 0, 0, 0};
      sa[i] = sb[i] = 0;
      const int64_t ra = m0 + 16 * i + r, rb = n0 + 16 * i + r;
      if (blk < nb && ra < P.M) {
        fa[i] = *reinterpret_cast<const u32x4 *>(P.a + ra * P.lda + 16 * blk);
        sa[i] = P.as[ra * P.lsa + blk];
      }
      if (blk < nb && rb < P.N) {
        fb[i] = *reinterpret_cast<const u32x4 *>(P.b + rb * P.ldb + 16 * blk);
        sb[i] = P.bs[rb * P.lsb + blk];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_fp4(fb[j], sb[j], fa[i], sa[i], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = m0 + 16 * i + r, col = n0 + 16 * j + 4 * g + v;
        if (row < P.M && col < P.N) {
          const float b = P.bias ? load_elem(P.bias, col, P.bias_dtype) : 0.0f;
          store_elem(P.c, (int64_t)row * P.N + col, acc[i][j][v] + b, P.c_dtype);
        }
      }
}

}  // namespace

size_t mx_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
bool mx_linear_fused(int64_t, int64_t, int64_t) { return false; }
hipError_t launch_mx_linear(const MxLinear &, hipStream_t) { return hipErrorInvalidValue; }

hipError_t launch_mx_gemms(const MxGemm *d, int count, void *, size_t, hipStream_t stream) {
  MxBatch b = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (d[i].M == 0 || d[i].N == 0) continue;
    MxProblem &p = b.p[b.count++];
    p = MxProblem{d[i].a.codes,    d[i].a.scales, d[i].b.codes,  d[i].b.scales,  d[i].c,          d[i].bias,
                  (int)d[i].M,     (int)d[i].N,   (int)d[i].K,   d[i].a.ld,      d[i].a.scale_ld, d[i].b.ld,
                  d[i].b.scale_ld, d[i].c_dtype,  d[i].bias_dtype, (int)((d[i].M + 63) / 64), (int)((d[i].N + 63) / 64),
                  (int)total};
    total += (int64_t)p.tiles_m * p.tiles_n;
  }
  if (b.count == 0) return hipSuccess;
  mx_gemm_kernel<<<(unsigned)total, 256, 0, stream>>>(b);
  return hipGetLastError();
}

}  // namespace f8lin

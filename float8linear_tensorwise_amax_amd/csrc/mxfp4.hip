// Quantisation of a (rows, cols) tensor to MXFP4 along its rows, along its
// columns (the transposed copy a backward product contracts over), or both in
// one pass over the data; the way back; and the column sums a bias gradient
// needs.  The block arithmetic is in mx_common.h.
//
// HBM-bound: es bytes read and 17/32 byte written per element and layout.
// Work decomposition: one workgroup of 256 threads per 128 x 128 tile.
//   load : thread t reads 8 consecutive elements of rows t/16 + 16 p: sixteen
//          lanes cover 128 columns of a row.
//   rows : a block is four lanes; its maximum meets by two DPP quad
//          permutations, each lane converts its eight values to one 32-bit
//          word, and sixteen lanes store 64 contiguous bytes.
//   cols : the tile goes to LDS as it is; thread t then owns the 32-row block
//          t % 4 of column pair t / 4: it reads 32 words down the tile, has
//          both columns' maxima in its own registers, and stores 16 bytes
//          for each column, four lanes covering 64 contiguous bytes of a
//          transposed row.  Words are XOR-ed with 16 * (row / 32), so that the
//          four row blocks that one read touches fall in different banks.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;

struct QuantJob {
  const void *x;
  int64_t rows, cols, ldx;
  f8lin_mxfp4 q, qt;
  float *colsum;
  int tiles_x, first;
};
struct QuantJobs {
  QuantJob j[kMxMaxQuant];
  int count;
};

template <int DT, int RULE, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const QuantJobs jobs) {
  typedef typename MxElem<DT>::type elem;
  constexpr int kWords = DT == F8LIN_FP32 ? 2 : 1;  // 32-bit words of a column pair
  __shared__ __attribute__((aligned(16))) uint32_t tile[COLS ? kTile * kTile / 2 * kWords : 4];
  const int job = jobs.count > 1 && (int)blockIdx.x >= jobs.j[1].first ? 1 : 0;
  const QuantJob &jb = jobs.j[job];
  const int64_t rows = jb.rows, cols = jb.cols;
  const int local = (int)blockIdx.x - jb.first;
  const int64_t row0 = (int64_t)(local / jb.tiles_x) * kTile, col0 = (int64_t)(local % jb.tiles_x) * kTile;
  const int t = threadIdx.x, c8 = t & 15;
  const elem *x = reinterpret_cast<const elem *>(jb.x);
  const int64_t gcol = col0 + 8 * c8;
  const int have = (int)min((int64_t)8, max((int64_t)0, cols - gcol));

#pragma unroll 4
  for (int p = 0; p < 8; ++p) {
    const int r = (t >> 4) + 16 * p;
    const int64_t grow = row0 + r;
    float v[8];
    load8<DT>(x + grow * jb.ldx + gcol, grow < rows ? have : 0, v);
    if constexpr (ROWS) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      const int e = mx_scale_byte<RULE>(quad_max(m));
      const uint32_t code = e == kMxNan ? 0u : mx_cvt8(v, mx_scale_f32(e));
      // the four blocks' scale bytes of the row meet in one word
      int sw = e << (8 * (c8 >> 2));
      sw |= __builtin_amdgcn_mov_dpp(sw, 0x124, 0xF, 0xF, true);  // row_ror 4
      sw |= __builtin_amdgcn_mov_dpp(sw, 0x128, 0xF, 0xF, true);  // row_ror 8
      if (grow < rows) {
        // (a block that starts inside the row is stored whole: its codes past cols are +0)
        if (col0 + 32 * (c8 >> 2) < cols)
          *reinterpret_cast<uint32_t *>(jb.q.codes + grow * jb.q.ld + col0 / 2 + 4 * c8) = code;
        if (c8 == 0) *reinterpret_cast<int *>(jb.q.scales + grow * jb.q.scale_ld + col0 / 32) = sw;
      }
    }
    if constexpr (COLS) {
      const int rb = r >> 5;
      if constexpr (DT == F8LIN_FP32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int w = (8 * c8 + 4 * h) ^ (32 * rb);
          *reinterpret_cast<u32x4 *>(&tile[r * 128 + w]) =
              u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                    __float_as_uint(v[4 * h + 3])};
        }
      } else {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = f32_to_elem(v[2 * i], DT) | f32_to_elem(v[2 * i + 1], DT) << 16;
        *reinterpret_cast<u32x4 *>(&tile[r * 64 + ((4 * c8) ^ (16 * rb))]) = w;
      }
    }
  }

  if constexpr (COLS) {
    __syncthreads();
    const int rb = t & 3, cp = t >> 2;
    const bool block_ok = row0 + 32 * rb < rows;
    float v[2][32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int r = 32 * rb + i;
      if constexpr (DT == F8LIN_FP32) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(&tile[r * 128 + ((2 * cp) ^ (32 * rb))]);
        v[0][i] = __uint_as_float(w.x), v[1][i] = __uint_as_float(w.y);
      } else {
        const uint32_t w = tile[r * 64 + (cp ^ (16 * rb))];
        v[0][i] = elem_f32<DT>(w & 0xFFFFu), v[1][i] = elem_f32<DT>(w >> 16);
      }
    }
    float cs[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t col = col0 + 2 * cp + h;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[h][i]) & 0x7FFFFFFFu);
      const int e = mx_scale_byte<RULE>(m);
      u32x4 out;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = v[h][8 * d + i];
        out[d] = e == kMxNan ? 0u : mx_cvt8(g, mx_scale_f32(e));
      }
      int sw = e << (8 * rb);
      sw |= __builtin_amdgcn_mov_dpp(sw, 0xB1, 0xF, 0xF, true);
      sw |= __builtin_amdgcn_mov_dpp(sw, 0x4E, 0xF, 0xF, true);
      if (col < cols) {
        if (block_ok) *reinterpret_cast<u32x4 *>(jb.qt.codes + col * jb.qt.ld + row0 / 2 + 16 * rb) = out;
        if (rb == 0) *reinterpret_cast<int *>(jb.qt.scales + col * jb.qt.scale_ld + row0 / 32) = sw;
      }
      if (jb.colsum) {
#pragma unroll
        for (int i = 0; i < 32; ++i) cs[h] += v[h][i];
        // the four row blocks in a fixed order: (0 + 1) + (2 + 3)
        cs[h] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(cs[h]), 0xB1, 0xF, 0xF, true));
        cs[h] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(cs[h]), 0x4E, 0xF, 0xF, true));
        if (rb == 0 && col < cols) jb.colsum[(row0 / kTile) * cols + col] = cs[h];
      }
    }
  }
}

// Eight codes (one 32-bit word) per thread back to values of type dt.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(f8lin_mxfp4 q, int64_t rows, int64_t cols,
                                                                 typename MxElem<DT>::type *out) {
  const int64_t words = (cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows * words; i += (int64_t)gridDim.x * kThreads) {
    const int64_t r = i / words, w = i % words;
    const uint32_t c = *reinterpret_cast<const uint32_t *>(q.codes + r * q.ld + 4 * w);
    const int e = q.scales[r * q.scale_ld + w / 4];
    const float s = mx_scale_f32(e);
    float v[8];
    f32x2_t p;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), v[0] = p.x, v[1] = p.y;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1), v[2] = p.x, v[3] = p.y;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), v[4] = p.x, v[5] = p.y;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3), v[6] = p.x, v[7] = p.y;
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = f32_to_elem(e == kMxNan ? __builtin_nanf("") : v[k], DT);
    typename MxElem<DT>::type *dst = out + r * cols + 8 * w;
    if (8 * w + 8 <= cols) {
      if constexpr (DT == F8LIN_FP32) {
        reinterpret_cast<u32x4_u *>(dst)[0] = u32x4{o[0], o[1], o[2], o[3]};
        reinterpret_cast<u32x4_u *>(dst)[1] = u32x4{o[4], o[5], o[6], o[7]};
      } else {
        *reinterpret_cast<u32x4_u *>(dst) =
            u32x4{o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16};
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (8 * w + k < cols) dst[k] = (typename MxElem<DT>::type)o[k];
    }
  }
}

// Bias gradient from the 128-row column sums, in order of the tiles.
__global__ __launch_bounds__(kThreads) void mx_dbias_kernel(const float *__restrict__ colsum, int64_t tiles, int64_t n,
                                                            void *db, int dt) {
  const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (col >= n) return;
  float s = 0.0f;
  for (int64_t i = 0; i < tiles; ++i) s += colsum[i * n + col];
  const uint32_t o = f32_to_elem(s, dt);
  if (dt == F8LIN_FP32)
    reinterpret_cast<uint32_t *>(db)[col] = o;
  else
    reinterpret_cast<uint16_t *>(db)[col] = (uint16_t)o;
}

template <int DT, int RULE>
void launch_quant(const QuantJobs &jobs, unsigned grid, bool rows, bool cols, hipStream_t stream) {
  if (rows && cols)
    mx_quantize_kernel<DT, RULE, true, true><<<grid, kThreads, 0, stream>>>(jobs);
  else if (rows)
    mx_quantize_kernel<DT, RULE, true, false><<<grid, kThreads, 0, stream>>>(jobs);
  else
    mx_quantize_kernel<DT, RULE, false, true><<<grid, kThreads, 0, stream>>>(jobs);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuant *ts, int count, int rule, hipStream_t stream) {
  QuantJobs jobs = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const MxQuant &t = ts[i];
    if (t.rows == 0 || t.cols == 0) continue;
    const int64_t gx = (t.cols + kTile - 1) / kTile, gy = (t.rows + kTile - 1) / kTile;
    jobs.j[jobs.count++] =
        QuantJob{t.x, t.rows, t.cols, t.ldx, t.q, t.qt, t.colsum, (int)gx, (int)total};
    total += gx * gy;
  }
  if (jobs.count == 0) return hipSuccess;
  const bool rows = ts[0].q.codes != nullptr, cols = ts[0].qt.codes != nullptr;
  const unsigned grid = (unsigned)total;
#define F8_MX_Q(DT)                                                             \
  if (rule == F8LIN_MX_CEIL)                                                    \
    launch_quant<DT, F8LIN_MX_CEIL>(jobs, grid, rows, cols, stream);            \
  else                                                                          \
    launch_quant<DT, F8LIN_MX_FLOOR>(jobs, grid, rows, cols, stream)
  if (ts[0].dtype == F8LIN_BF16) {
    F8_MX_Q(F8LIN_BF16);
  } else if (ts[0].dtype == F8LIN_FP16) {
    F8_MX_Q(F8LIN_FP16);
  } else {
    F8_MX_Q(F8LIN_FP32);
  }
#undef F8_MX_Q
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const f8lin_mxfp4 &q, int64_t rows, int64_t cols, int dtype, void *out,
                                hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const int64_t work = rows * ((cols + 7) / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((work + kThreads - 1) / kThreads, 65536);
  if (dtype == F8LIN_BF16)
    mx_dequantize_kernel<F8LIN_BF16><<<grid, kThreads, 0, stream>>>(q, rows, cols, (uint16_t *)out);
  else if (dtype == F8LIN_FP16)
    mx_dequantize_kernel<F8LIN_FP16><<<grid, kThreads, 0, stream>>>(q, rows, cols, (uint16_t *)out);
  else
    mx_dequantize_kernel<F8LIN_FP32><<<grid, kThreads, 0, stream>>>(q, rows, cols, (uint32_t *)out);
  return hipGetLastError();
}

hipError_t launch_mx_dbias(const float *colsum, int64_t tiles, int64_t n, void *db, int dtype, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  mx_dbias_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(colsum, tiles, n, db, dtype);
  return hipGetLastError();
}

}  // namespace f8lin

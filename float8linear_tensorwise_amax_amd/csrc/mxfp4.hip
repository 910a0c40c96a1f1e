// Quantisation of a (rows, cols) tensor to MXFP4 along its rows, along its
// columns (the transposed copy a backward product contracts over), or both in
// one pass over the data; the way back; and the column sums a bias gradient
// needs.  The block arithmetic is in mx_common.h.
//
// HBM-bound: es bytes read and 17/32 byte written per element and layout.
// 65536 x 4096 bf16: rows 109 us (6.2 TB/s), columns 133 us (5.1), both 157 us
// (5.2), the way back 103 us (6.6); a plain copy moves 5.0-5.3 TB/s on this
// card and a read alone 6.3, both through the caches.
// Rows alone (mx_rows_kernel): a thread takes eight consecutive elements of
// four rows, all four loads in flight; a block is four lanes, whose maxima
// meet by two DPP quad permutations.
// Columns, or both (mx_quantize_kernel): one workgroup per tile of 256 (or 128)
// rows x 128 columns, a wave per 32 rows, all of its loads in flight at once.
//   rows : sixteen lanes cover 128 columns of a row and store 64 contiguous
//          bytes of codes and one word of scales.
//   cols : the tile goes to LDS as it is; thread t then owns the 32-row block
//          t % 8 of column pair t / 8: it reads 32 words down the tile, has
//          both columns' maxima in its own registers, and stores 16 bytes
//          for each column, eight lanes covering a 128-byte line of a
//          transposed row.  Words are XOR-ed with 8 * (row / 32), so that the
//          eight row blocks that one read touches fall in different banks.
//   An XCD takes a contiguous run of tiles (workgroup b runs on XCD b % 8),
//   so that the halves of a 128-byte line of codes meet in one L2.
// 16-bit elements stay packed pairs throughout: maxima by packed 16-bit max,
// codes by v_cvt_scalef32_pk_fp4_{bf16,f16}.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

constexpr int kThreads = 256;
constexpr int kTileCols = 128;
constexpr int64_t kFewTiles = 256;  // tiles of 256 x 128 elements: fewer leave CUs idle
constexpr int64_t kManyTiles = 1280;  // 80 MB of 16-bit elements

struct QuantJob {
  const void *x;
  int64_t rows, cols, ldx;
  f8lin_mxfp4 q, qt;
  float *colsum;
  int tiles_x, first, log_tx;
};
struct QuantJobs {
  QuantJob j[kMxMaxQuant];
  int count;
};

// The scale bytes of the four blocks that sixteen lanes hold (block q in lanes
// 4 q .. 4 q + 3), as one word in all of them.
__device__ __forceinline__ int scales_of_16(int e, int q) {
  int sw = e << (8 * q);
  sw |= __builtin_amdgcn_mov_dpp(sw, 0x124, 0xF, 0xF, true);         // row_ror 4
  return sw | __builtin_amdgcn_mov_dpp(sw, 0x128, 0xF, 0xF, true);  // row_ror 8
}

// Rows alone; in large calls 16-bit X is read past the L2 (65536 x 4096 bf16
// 109 us, through it 126 us; 3001 x 2504 fp16 8.4 us, through it 7.4 us).  A
// workgroup covers tx = 2^log_tx chunks of eight elements by
// kRowsPer * 256 / tx rows: four rows a thread, or one where that leaves few
// workgroups.
template <int DT, int RULE, int kRowsPer>
__global__ __launch_bounds__(kThreads) void mx_rows_kernel(const QuantJobs jobs) {
  typedef typename MxElem<DT>::type elem;
  const int job = jobs.count > 1 && (int)blockIdx.x >= jobs.j[1].first ? 1 : 0;
  const QuantJob &jb = jobs.j[job];
  const int local = (int)blockIdx.x - jb.first;
  const int tx = (int)threadIdx.x & ((1 << jb.log_tx) - 1), ty = (int)threadIdx.x >> jb.log_tx;
  const int64_t col = ((int64_t)(local % jb.tiles_x) << (jb.log_tx + 3)) + 8 * tx;
  const int64_t row0 = (int64_t)(local / jb.tiles_x) * (kRowsPer * (kThreads >> jb.log_tx)) + ty;
  const int have = (int)min((int64_t)8, max((int64_t)0, jb.cols - col));
  const elem *x = reinterpret_cast<const elem *>(jb.x);
  Raw8<DT> v[kRowsPer];
#pragma unroll
  for (int p = 0; p < kRowsPer; ++p) {
    const int64_t row = row0 + (int64_t)p * (kThreads >> jb.log_tx);
    v[p] = load_raw8<DT, DT != F8LIN_FP32 && kRowsPer == 4>(x + row * jb.ldx + col, row < jb.rows ? have : 0);
  }
#pragma unroll
  for (int p = 0; p < kRowsPer; ++p) {
    const int64_t row = row0 + (int64_t)p * (kThreads >> jb.log_tx);
    const int e = mx_scale_byte<RULE>(mag_f32_bits<DT>(quad_max(raw_mag<DT>(v[p]))));
    const uint32_t code = e == kMxNan ? 0u : raw_codes<DT>(v[p], mx_scale_f32(e));
    const int sw = scales_of_16(e, (tx >> 2) & 3);
    if (row < jb.rows) {
      // (a block that starts inside the row is stored whole: its codes past cols are +0)
      if ((col & ~31) < jb.cols) *reinterpret_cast<uint32_t *>(jb.q.codes + row * jb.q.ld + col / 2) = code;
      if ((tx & 15) == 0 && col < jb.cols) *reinterpret_cast<int *>(jb.q.scales + row * jb.q.scale_ld + col / 32) = sw;
    }
  }
}

// ONCE: X is read, and the transposed codes (which a backward reads much later)
// are written, past the L2, so that the lines that tiles fill together stay
// there (65536 x 4096 bf16, both layouts: 157 us, otherwise 185 us).
template <int DT, int RULE, bool ROWS, int kRowBlocks, bool ONCE>
__global__ __launch_bounds__(64 * kRowBlocks) void mx_quantize_kernel(const QuantJobs jobs) {
  typedef typename MxElem<DT>::type elem;
  constexpr int kTileRows = 32 * kRowBlocks;  // a wave per 32 rows
  constexpr int kWords = DT == F8LIN_FP32 ? 2 : 1;  // 32-bit words of a column pair
  constexpr int kPitch = kTileCols / 2 * kWords;
  constexpr int kSkew = 64 / kRowBlocks;  // words that a row block is set apart by
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTileRows * kPitch];
  const int per = (int)gridDim.x / 8, rem = (int)gridDim.x % 8, xcd = (int)blockIdx.x % 8;
  const int wg = xcd * per + min(xcd, rem) + (int)blockIdx.x / 8;
  const int job = jobs.count > 1 && wg >= jobs.j[1].first ? 1 : 0;
  const QuantJob &jb = jobs.j[job];
  const int64_t rows = jb.rows, cols = jb.cols;
  const int local = wg - jb.first;
  // 32-bit elements: pairs of 128-row tiles one after the other, for the
  // halves of a 128-byte line of transposed codes (65536 x 4096, both layouts:
  // 269 us, tile-row by tile-row 287 us; 1021 x 2055: 7.9 and 7.7 us)
  constexpr int kGroup = DT == F8LIN_FP32 ? 2 : 1;
  const int tiles_y = (int)((rows + kTileRows - 1) / kTileRows);
  const int group = local / (kGroup * jb.tiles_x), in_group = local - group * kGroup * jb.tiles_x;
  const int group_rows = min(kGroup, tiles_y - group * kGroup);
  const int64_t row0 = (int64_t)(group * kGroup + in_group % group_rows) * kTileRows;
  const int64_t col0 = (int64_t)(in_group / group_rows) * kTileCols;
  const int t = threadIdx.x, c8 = t & 15;
  const elem *x = reinterpret_cast<const elem *>(jb.x);
  const int64_t gcol = col0 + 8 * c8;
  const int have = (int)min((int64_t)8, max((int64_t)0, cols - gcol));
  Raw8<DT> in[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t grow = row0 + (t >> 4) + 4 * kRowBlocks * p;
    in[p] = load_raw8<DT, ONCE>(x + grow * jb.ldx + gcol, grow < rows ? have : 0);
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = (t >> 4) + 4 * kRowBlocks * p, rb = r >> 5;
    const int64_t grow = row0 + r;
    if constexpr (DT == F8LIN_FP32) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4 *>(&tile[r * kPitch + ((8 * c8 + 4 * h) ^ (2 * kSkew * rb))]) = in[p].w[h];
    } else {
      *reinterpret_cast<u32x4 *>(&tile[r * kPitch + ((4 * c8) ^ (kSkew * rb))]) = in[p].w[0];
    }
    if constexpr (ROWS) {
      const int e = mx_scale_byte<RULE>(mag_f32_bits<DT>(quad_max(raw_mag<DT>(in[p]))));
      const uint32_t code = e == kMxNan ? 0u : raw_codes<DT>(in[p], mx_scale_f32(e));
      const int sw = scales_of_16(e, c8 >> 2);
      if (grow < rows) {
        if (col0 + 32 * (c8 >> 2) < cols)
          *reinterpret_cast<uint32_t *>(jb.q.codes + grow * jb.q.ld + col0 / 2 + 4 * c8) = code;
        if (c8 == 0) *reinterpret_cast<int *>(jb.q.scales + grow * jb.q.scale_ld + col0 / 32) = sw;
      }
    }
  }
  __syncthreads();
  const int rb = t % kRowBlocks, cp = t / kRowBlocks;
  const bool block_ok = row0 + 32 * rb < rows;
  // the column pair's 32 rows, and its two maxima
  uint32_t v[kWords][32], m[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int r = 32 * rb + i;
    if constexpr (DT == F8LIN_FP32) {
      const u32x2 w = *reinterpret_cast<const u32x2 *>(&tile[r * kPitch + ((2 * cp) ^ (2 * kSkew * rb))]);
      v[0][i] = w.x, v[1][i] = w.y;
      m[0] = max(m[0], w.x & 0x7FFFFFFFu);
      m[1] = max(m[1], w.y & 0x7FFFFFFFu);
    } else {
      v[0][i] = tile[r * kPitch + (cp ^ (kSkew * rb))];
      m[0] = pair_mag_max(m[0], v[0][i]);
    }
  }
  if constexpr (DT != F8LIN_FP32) m[1] = m[0] >> 16, m[0] &= 0xFFFFu;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = col0 + 2 * cp + h;
    const int e = mx_scale_byte<RULE>(mag_f32_bits<DT>(m[h]));
    const float s = mx_scale_f32(e);
    u32x4 out;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (DT == F8LIN_FP32) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = __uint_as_float(v[h][8 * d + i]);
        out[d] = mx_cvt8(g, s);
      } else {
        // the column's elements of two rows side by side
        constexpr uint32_t kSel[2] = {0x05040100u, 0x07060302u};
        uint32_t g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = __builtin_amdgcn_perm(v[0][8 * d + 2 * i + 1], v[0][8 * d + 2 * i], kSel[h]);
        out[d] = cvt_pairs<DT>(g[0], g[1], g[2], g[3], s);
      }
      if (e == kMxNan) out[d] = 0;
    }
    int sw = e << (8 * (rb & 3));
    sw |= __builtin_amdgcn_mov_dpp(sw, 0xB1, 0xF, 0xF, true);
    sw |= __builtin_amdgcn_mov_dpp(sw, 0x4E, 0xF, 0xF, true);
    if (col < cols) {
      u32x4 *const dst = reinterpret_cast<u32x4 *>(jb.qt.codes + col * jb.qt.ld + row0 / 2 + 16 * rb);
      if (block_ok) {
        if constexpr (ROWS && ONCE) __builtin_nontemporal_store(out, dst);
        else *dst = out;
      }
      if ((rb & 3) == 0 && block_ok)
        *reinterpret_cast<int *>(jb.qt.scales + col * jb.qt.scale_ld + row0 / 32 + rb) = sw;
    }
    if (jb.colsum) {
      float cs = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if constexpr (DT == F8LIN_FP32) cs += __uint_as_float(v[h][i]);
        else cs += elem_f32<DT>((v[0][i] >> (16 * h)) & 0xFFFFu);
      }
      // four row blocks (kMxTile rows) in a fixed order: (0 + 1) + (2 + 3)
      cs += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(cs), 0xB1, 0xF, 0xF, true));
      cs += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(cs), 0x4E, 0xF, 0xF, true));
      if ((rb & 3) == 0 && col < cols && block_ok) jb.colsum[(row0 / kMxTile + rb / 4) * cols + col] = cs;
    }
  }
}

// The way back.  E codes per thread, so that its values are one 16-byte store,
// of kRowsPer rows; a workgroup covers 2^log_tx such groups by kRowsPer * 256 /
// 2^log_tx rows.
template <int DT, int kRowsPer, bool PAST>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(f8lin_mxfp4 q, int64_t rows, int64_t cols,
                                                                 typename MxElem<DT>::type *out, int tiles_x, int log_tx) {
  constexpr int E = DT == F8LIN_FP32 ? 4 : 8;
  const int tx = (int)threadIdx.x & ((1 << log_tx) - 1), ty = (int)threadIdx.x >> log_tx;
  const int64_t col = ((int64_t)((int)blockIdx.x % tiles_x) * E << log_tx) + E * tx;
  const int64_t row0 = (int64_t)((int)blockIdx.x / tiles_x) * (kRowsPer * (kThreads >> log_tx)) + ty;
  if (col >= cols) return;
  uint32_t code[kRowsPer];
  int exps[kRowsPer];
#pragma unroll
  for (int p = 0; p < kRowsPer; ++p) {
    const int64_t row = row0 + (int64_t)p * (kThreads >> log_tx);
    code[p] = 0, exps[p] = 0;
    if (row >= rows) continue;
    const uint8_t *c = q.codes + row * q.ld + col / 2;
    code[p] = E == 8 ? *reinterpret_cast<const uint32_t *>(c) : *reinterpret_cast<const uint16_t *>(c);
    exps[p] = q.scales[row * q.scale_ld + col / 32];
  }
#pragma unroll
  for (int p = 0; p < kRowsPer; ++p) {
    const int64_t row = row0 + (int64_t)p * (kThreads >> log_tx);
    if (row >= rows) continue;
    const uint32_t c = code[p];
    const int e = exps[p];
    const float s = mx_scale_f32(e);
    f32x2_t v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    uint32_t o[E];
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = f32_to_elem(e == kMxNan ? __builtin_nanf("") : v[k >> 1][k & 1], DT);
    typename MxElem<DT>::type *dst = out + row * cols + col;
    if (col + E <= cols) {
      u32x4 v;
      if constexpr (DT == F8LIN_FP32) v = u32x4{o[0], o[1], o[2], o[3]};
      else v = u32x4{o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16};
      if constexpr (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_u *>(dst));
      else *reinterpret_cast<u32x4_u *>(dst) = v;
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k)
        if (col + k < cols) dst[k] = (typename MxElem<DT>::type)o[k];
    }
  }
}

// Bias gradient from the 128-row column sums.  A workgroup owns 32 columns (a
// 128-byte line of a tile's sums); 32 groups of threads take every 32nd tile,
// eight loads in flight each, and meet in LDS in the groups' order.  (65536 x
// 4096: 4.1 us, with a thread a column 164 us: the loads of 512 tiles one after
// the other on 16 CUs.)
constexpr int kDbCols = 32, kDbGroups = 32;
__global__ __launch_bounds__(kDbCols * kDbGroups) void mx_dbias_kernel(const float *__restrict__ colsum, int64_t tiles,
                                                                       int64_t n, void *db, int dt) {
  constexpr int kAhead = 8;
  __shared__ float part[kDbGroups][kDbCols];
  const int c = (int)threadIdx.x % kDbCols, grp = (int)threadIdx.x / kDbCols;
  const int64_t col = (int64_t)blockIdx.x * kDbCols + c;
  float s = 0.0f;
  if (col < n) {
    for (int64_t i0 = grp; i0 < tiles; i0 += kAhead * kDbGroups) {
      float v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int64_t i = i0 + a * kDbGroups;
        v[a] = i < tiles ? colsum[i * n + col] : 0.0f;
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) s += v[a];
    }
  }
  part[grp][c] = s;
  __syncthreads();
  if (grp != 0 || col >= n) return;
#pragma unroll
  for (int g = 1; g < kDbGroups; ++g) s += part[g][c];
  const uint32_t o = f32_to_elem(s, dt);
  if (dt == F8LIN_FP32)
    reinterpret_cast<uint32_t *>(db)[col] = o;
  else
    reinterpret_cast<uint16_t *>(db)[col] = (uint16_t)o;
}

template <int DT, int RULE, int RB, bool ONCE>
void launch_cols(const QuantJobs &jobs, unsigned grid, bool rows, hipStream_t stream) {
  if (rows)
    mx_quantize_kernel<DT, RULE, true, RB, ONCE><<<grid, 64 * RB, 0, stream>>>(jobs);
  else
    mx_quantize_kernel<DT, RULE, false, RB, ONCE><<<grid, 64 * RB, 0, stream>>>(jobs);
}

template <int DT, int RULE>
void launch_quant(const QuantJobs &jobs, unsigned grid, bool rows, int row_blocks, bool once, hipStream_t stream) {
  if constexpr (DT != F8LIN_FP32) {
    if (row_blocks == 8 && once) return launch_cols<DT, RULE, 8, true>(jobs, grid, rows, stream);
    if (row_blocks == 8) return launch_cols<DT, RULE, 8, false>(jobs, grid, rows, stream);
  }
  if (row_blocks == 4)
    launch_cols<DT, RULE, 4, false>(jobs, grid, rows, stream);
  else
    row_blocks == 0 ? mx_rows_kernel<DT, RULE, 4><<<grid, kThreads, 0, stream>>>(jobs)
                    : mx_rows_kernel<DT, RULE, 1><<<grid, kThreads, 0, stream>>>(jobs);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuant *ts, int count, int rule, hipStream_t stream) {
  const bool rows = ts[0].q.codes != nullptr, cols = ts[0].qt.codes != nullptr;
  // 256-row tiles fill whole 128-byte lines of the transposed codes (65536 x
  // 4096 bf16, both layouts: 157 us, with 128-row tiles 214 us); 128-row
  // tiles for 32-bit elements, whose tile would take 128 KB of LDS (270 us,
  // with 256 rows 342 us), and where there are few tiles (256 x 4096 bf16:
  // 5.6 us, with 256 rows 6.3 us).
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i)
    tiles += ((ts[i].rows + 255) / 256) * ((ts[i].cols + kTileCols - 1) / kTileCols);
  // (rows alone: 0, or 1 for one row a thread)
  const int row_blocks = !cols ? (tiles < kFewTiles ? 1 : 0) : (ts[0].dtype != F8LIN_FP32 && tiles >= kFewTiles) ? 8 : 4;
  QuantJobs jobs = {};
  int64_t total = 0;
  // X past the L2: where its rows are whole 128-byte lines, that no two tiles
  // share (65535 x 4095 bf16, both layouts: 218 us so, 214 us otherwise), and
  // there is more of it than the caches may hold from whoever wrote it (an
  // element-wise launch, the forward and another one: 8192 x 4096 x 4096, 96
  // MB in X and W, 159 us, otherwise 166 us; 4096 x 4096 x 4096, 64 MB, 92 and
  // 90 us).
  bool once = tiles >= kManyTiles;
  for (int i = 0; i < count; ++i) {
    const MxQuant &t = ts[i];
    if (t.rows == 0 || t.cols == 0) continue;
    once = once && ((uintptr_t)t.x | (uintptr_t)t.ldx * 2) % 128 == 0;
    int64_t gx, gy;
    int log_tx = 0;
    if (cols) {
      gx = (t.cols + kTileCols - 1) / kTileCols, gy = (t.rows + 32 * row_blocks - 1) / (32 * row_blocks);
    } else {
      // as many threads along a row as it has chunks, 16 to 256
      log_tx = 4;
      while (log_tx < 8 && (8 << log_tx) < t.cols) ++log_tx;
      const int64_t per = (row_blocks ? 1 : 4) * (kThreads >> log_tx);
      gx = (t.cols + (8 << log_tx) - 1) / (8 << log_tx), gy = (t.rows + per - 1) / per;
    }
    jobs.j[jobs.count++] =
        QuantJob{t.x, t.rows, t.cols, t.ldx, t.q, t.qt, t.colsum, (int)gx, (int)total, log_tx};
    total += gx * gy;
  }
  if (jobs.count == 0) return hipSuccess;
  const unsigned grid = (unsigned)total;
#define F8_MX_Q(DT)                                                             \
  if (rule == F8LIN_MX_CEIL)                                                    \
    launch_quant<DT, F8LIN_MX_CEIL>(jobs, grid, rows, row_blocks, once, stream);      \
  else                                                                          \
    launch_quant<DT, F8LIN_MX_FLOOR>(jobs, grid, rows, row_blocks, once, stream)
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
  const int64_t per = dtype == F8LIN_FP32 ? 4 : 8;
  int log_tx = 2;
  while (log_tx < 8 && (per << log_tx) < cols) ++log_tx;
  const int64_t gx = (cols + (per << log_tx) - 1) / (per << log_tx), few = rows * cols < kFewTiles * 256 * kTileCols,
                rows_per = (few ? 1 : 4) * (kThreads >> log_tx);
  const unsigned grid = (unsigned)(gx * ((rows + rows_per - 1) / rows_per));
  // an output that the caches cannot hold for its reader goes past them (65536
  // x 4096 bf16 103 us, through them 122 us)
  const bool past = rows * cols * (dtype == F8LIN_FP32 ? 4 : 2) > (int64_t)320 << 20;
#define F8_MX_D(DT, T)                                                                                             \
  past  ? mx_dequantize_kernel<DT, 4, true><<<grid, kThreads, 0, stream>>>(q, rows, cols, (T *)out, (int)gx, log_tx) \
  : few ? mx_dequantize_kernel<DT, 1, false><<<grid, kThreads, 0, stream>>>(q, rows, cols, (T *)out, (int)gx, log_tx) \
        : mx_dequantize_kernel<DT, 4, false><<<grid, kThreads, 0, stream>>>(q, rows, cols, (T *)out, (int)gx, log_tx)
  if (dtype == F8LIN_BF16)
    F8_MX_D(F8LIN_BF16, uint16_t);
  else if (dtype == F8LIN_FP16)
    F8_MX_D(F8LIN_FP16, uint16_t);
  else
    F8_MX_D(F8LIN_FP32, uint32_t);
#undef F8_MX_D
  return hipGetLastError();
}

hipError_t launch_mx_dbias(const float *colsum, int64_t tiles, int64_t n, void *db, int dtype, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  mx_dbias_kernel<<<(unsigned)((n + kDbCols - 1) / kDbCols), kDbCols * kDbGroups, 0, stream>>>(colsum, tiles, n, db,
                                                                                              dtype);
  return hipGetLastError();
}

}  // namespace f8lin

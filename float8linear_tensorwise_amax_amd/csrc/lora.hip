// Low-rank adapters of many requests beside a shared projection.  Token t of
// adapter i (A_i (R, K), B_i (N, R), scale s_i):
//   H[t] = s_i * x[t] . A_i^T                          "down"
//   y[t] = base[t] + H[t] . B_i^T                      "up"
//   G[t] = s_i * dy[t] . B_i,  dx[t] = G[t] . A_i      the same two kernels, the other operand layouts
//   dA_i = sum of G[t]^T x[t],  dB_i = sum of dy[t]^T H[t]   over the adapter's tokens: "outer"
// and a token without an adapter has y = base, dx = 0.
//
// A plan, made once per batch on the device, sorts the tokens by adapter
// (stably: every sum has a fixed order) and cuts them into tiles of up to 64
// rows of one adapter, so that the products run on the matrix cores whatever
// the mix: a tile reads its adapter once, and a batch of single tokens reads
// each adapter it uses once.  Rows are gathered through the plan; nothing is
// copied into sorted order.
//
// All of it is bound by memory up to ranks of about 64 (R flops a byte of x):
// down reads x, up reads base and writes y, outer reads x and dy once more.
// Operands go from memory to registers in the matrix instructions' own layout,
// with no LDS between: the contraction's order is free, so that a lane's 16
// bytes are whatever 8 (4 in binary32) values are contiguous, and where the
// contraction runs across rows a lane takes 8 rows of a block of columns and
// transposes them in registers.
//
// H and G are (T, R) in binary32.  They enter the second product as a sum of
// two bf16 values (16 bits of mantissa; an fp16 operand beside them as such a
// sum too), so that the rounding of the intermediate, 2^-17, stays below the
// output's; binary32 data use the binary32 matrix instruction throughout.
#include <algorithm>

#include "lora.h"
#include "mx_common.h"

namespace f8lin {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = kLoraTile;

// ---------------------------------------------------------------- plan

// The buffer's words: {magic, tokens, adapters, tiles}, starts[adapters + 2]
// (first sorted position of each adapter; then of the tokens without one, and
// the end), tiles {adapter, position, rows, 0}, order[tokens] (token of each
// sorted position), owner[tokens] (its adapter).
__device__ __forceinline__ const int *plan_starts(const int *p) { return p + 4; }
__device__ __forceinline__ const i32x4 *plan_tiles(const int *p, int adapters) {
  return reinterpret_cast<const i32x4 *>(p + lora_tiles_at(adapters));
}
__device__ __forceinline__ const int *plan_order(const int *p, int tokens, int adapters) {
  return p + lora_order_at(tokens, adapters);
}
__device__ __forceinline__ const int *plan_owner(const int *p, int tokens, int adapters) {
  return p + lora_order_at(tokens, adapters) + tokens;
}
// Tiles of the plan, or -1 where the buffer is no plan of this batch size.
__device__ __forceinline__ int plan_tile_count(const int *p, int tokens, int adapters) {
  const i32x4 h = *reinterpret_cast<const i32x4 *>(p);
  return h.x == kLoraMagic && h.y == tokens && h.z == adapters ? h.w : -1;
}

// A stable counting sort in one workgroup: each wave owns a contiguous part of
// the tokens and, 64 at a time, finds the lanes that share an adapter; counts
// and cursors are a wave's own, so that no two waves meet at one.
template <int WAVES, int MAXA>
__global__ __launch_bounds__(64 * WAVES) void lora_plan_kernel(const void *index, int wide, int tokens, int adapters,
                                                               int *plan) {
  constexpr int kThreads = 64 * WAVES;
  __shared__ int count[WAVES][MAXA + 1];
  __shared__ int starts[MAXA + 2], tile_first[MAXA + 2];
  __shared__ int sums[2][WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int groups = adapters + 1;  // the last: no adapter
  for (int i = tid; i < WAVES * (MAXA + 1); i += kThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  const int each = ((tokens + WAVES - 1) / WAVES + 63) / 64 * 64;
  const int begin = min(tokens, wave * each), end = min(tokens, begin + each);
  auto adapter_of = [&](int t) {
    if (t >= end) return -1;
    const int64_t v = wide ? reinterpret_cast<const int64_t *>(index)[t] : (int64_t) reinterpret_cast<const int *>(index)[t];
    return v >= 0 && v < adapters ? (int)v : adapters;
  };
  // f(adapter, lanes that have it) for each adapter among 64 tokens
  auto each_adapter = [&](int a, auto f) {
    uint64_t left = __ballot(a >= 0);
    while (left) {
      const int av = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
      const uint64_t same = __ballot(a == av);
      f(av, same);
      left &= ~same;
    }
  };
  int next = adapter_of(begin + lane);
  for (int t = begin; t < end; t += 64) {
    const int a = next;
    next = adapter_of(t + 64 + lane);
    each_adapter(a, [&](int av, uint64_t same) {
      if (lane == 0) count[wave][av] += __builtin_popcountll(same);
    });
  }
  __syncthreads();
  // exclusive prefix sums over the adapters, of tokens and of tiles
  int tokens_before = 0, tiles_before = 0;
  for (int a0 = 0; a0 < groups; a0 += kThreads) {
    const int a = a0 + tid;
    int n = 0;
    if (a < groups) {
#pragma unroll
      for (int w = 0; w < WAVES; ++w) n += count[w][a];
    }
    const int nt = (n + kTile - 1) / kTile;
    int s = n, st = nt;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(s, off, 64), ut = __shfl_up(st, off, 64);
      if (lane >= off) s += u, st += ut;
    }
    __syncthreads();
    if (lane == 63) sums[0][wave] = s, sums[1][wave] = st;
    __syncthreads();
    int total = 0, total_tiles = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) s += sums[0][w], st += sums[1][w];
      total += sums[0][w], total_tiles += sums[1][w];
    }
    if (a < groups) {
      int at = tokens_before + s - n;
      starts[a] = at;
      tile_first[a] = tiles_before + st - nt;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {  // counts become cursors
        const int c = count[w][a];
        count[w][a] = at;
        at += c;
      }
    }
    tokens_before += total;
    tiles_before += total_tiles;
  }
  if (tid == 0) starts[groups] = tokens, tile_first[groups] = tiles_before;
  __syncthreads();
  int *const order = plan + lora_order_at(tokens, adapters), *const owner = order + tokens;
  next = adapter_of(begin + lane);
  for (int t = begin; t < end; t += 64) {
    const int a = next;
    next = adapter_of(t + 64 + lane);
    each_adapter(a, [&](int av, uint64_t same) {
      const int at = count[wave][av];
      if (a == av) {
        const int p = at + __builtin_popcountll(same & ((1ull << lane) - 1));
        order[p] = t + lane;
        owner[p] = av;
      }
      if (lane == 0) count[wave][av] = at + __builtin_popcountll(same);
    });
  }
  for (int a = tid; a <= groups; a += kThreads) plan[4 + a] = starts[a];
  i32x4 *const tiles = reinterpret_cast<i32x4 *>(plan + lora_tiles_at(adapters));
  for (int i = tid; i < tiles_before; i += kThreads) {
    int lo = 0, hi = groups - 1;  // the last adapter whose first tile is at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int p = starts[lo] + (i - tile_first[lo]) * kTile;
    tiles[i] = i32x4{lo, p, min(kTile, starts[lo + 1] - p), 0};
  }
  if (tid == 0) *reinterpret_cast<i32x4 *>(plan) = i32x4{kLoraMagic, tokens, adapters, tiles_before};
}

// ---------------------------------------------------------------- fragments

// 16 bytes of an operand a lane: 8 values of a 16-bit type along a contraction
// of 32, or 4 binary32 ones along a contraction of 16 (lane l: row or column
// l & 15, values (l >> 4) * kE ..).
template <int DT>
constexpr int kE = DT == F8LIN_FP32 ? 4 : 8;

template <int DT>
__device__ __forceinline__ v4f mma(u32x4 a, u32x4 b, v4f c) {
  if constexpr (DT == F8LIN_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else if constexpr (DT == F8LIN_FP16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
}

// kE values at p, of which n exist (the others are 0).
template <int DT>
__device__ __forceinline__ u32x4 load_frag(const typename MxElem<DT>::type *p, int64_t n) {
  if (n >= kE<DT>) return *reinterpret_cast<const u32x4_u *>(p);
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < kE<DT>; ++i) e[i] = i < n ? (uint32_t)p[i] : 0u;
  if constexpr (DT == F8LIN_FP32) return u32x4{e[0], e[1], e[2], e[3]};
  else return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

// V consecutive elements (V = 1, 2, 4, 8 16-bit ones or 1, 2, 4 binary32 ones)
// as words; a word holds two 16-bit elements, or a lone one in its low half.
template <int DT, int V>
struct Few {
  static constexpr int kWords = DT == F8LIN_FP32 ? V : (V + 1) / 2;
  uint32_t w[kWords];
};
template <int DT, int V>
__device__ __forceinline__ Few<DT, V> load_few(const typename MxElem<DT>::type *p, int n) {
  Few<DT, V> f;
  constexpr int kW = Few<DT, V>::kWords;
  if (n >= V) {
    if constexpr (DT != F8LIN_FP32 && V == 1) {
      f.w[0] = *p;
    } else if constexpr (kW == 1) {
      typedef uint32_t u32_u __attribute__((aligned(2)));
      f.w[0] = *reinterpret_cast<const u32_u *>(p);
    } else if constexpr (kW == 2) {
      const u32x2 v = *reinterpret_cast<const u32x2_u *>(p);
      f.w[0] = v.x, f.w[1] = v.y;
    } else {
      const u32x4 v = *reinterpret_cast<const u32x4_u *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.w[i] = v[i];
    }
  } else {
    uint32_t e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = i < n ? (uint32_t)p[i] : 0u;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      if constexpr (DT == F8LIN_FP32) f.w[i] = e[i];
      else f.w[i] = e[2 * i] | (2 * i + 1 < V ? e[(2 * i + 1) % V] << 16 : 0u);
    }
  }
  return f;
}
// Element j of each of kE rows, packed as a fragment.
template <int DT, int V>
__device__ __forceinline__ u32x4 pick(const Few<DT, V> (&rows)[kE<DT>], int j) {
  u32x4 f;
  if constexpr (DT == F8LIN_FP32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = rows[e].w[j];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = rows[2 * e].w[j >> 1], hi = rows[2 * e + 1].w[j >> 1];
      f[e] = __builtin_amdgcn_perm(hi, lo, (j & 1) ? 0x07060302u : 0x05040100u);
    }
  }
  return f;
}

// Two binary32 values rounded to a packed pair of bf16.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
// What rounding a to the bf16 in `bits` (its low or high half) left over; an
// infinity leaves nothing.
__device__ __forceinline__ float left_over(float a, float rounded) {
  return (__float_as_uint(rounded) & 0x7F800000u) == 0x7F800000u ? 0.0f : a - rounded;
}
// Eight values as bf16 plus bf16.
__device__ __forceinline__ void split8(const float (&v)[8], u32x4 &hi, u32x4 &lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    lo[e] = pack_bf16(left_over(v[2 * e], bf16_lo(hi[e])), left_over(v[2 * e + 1], bf16_hi(hi[e])));
  }
}
// Pairs of bf16 with infinities and NaN as zeros.
__device__ __forceinline__ u32x4 no_inf(u32x4 f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((f[e] & 0x7F80u) == 0x7F80u) f[e] &= 0xFFFF0000u;
    if ((f[e] & 0x7F800000u) == 0x7F800000u) f[e] &= 0x0000FFFFu;
  }
  return f;
}
__device__ __forceinline__ void split_f16(u32x4 f, u32x4 &hi, u32x4 &lo) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = f16_bits_to_f32(f[e] & 0xFFFFu);
    v[2 * e + 1] = f16_bits_to_f32(f[e] >> 16);
  }
  split8(v, hi, lo);
}

// ---------------------------------------------------------------- down

// H[part][position][r] = scale * sum over part's columns of X[t][c] * W(r, c),
// W (R, C) as rows, or (C, R) where W_T.  A workgroup takes 64 rows, 16 * NT
// ranks and one part of the columns, 64 (32 in binary32: 128 bytes a row) at a
// time, dealt to its four waves.
template <int DT, int NT, bool W_T>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraDown a) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>, kBlock = 8 * E, RB = 16 * NT;
  __shared__ float red[3][kTile][RB + 1];
  const int tiles = plan_tile_count(a.plan, a.tokens, a.adapters);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int rblocks = (a.rank + RB - 1) / RB, per_tile = rblocks * a.parts;
  const int64_t total = (int64_t)tiles * per_tile;
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int64_t C = a.cols;
  const int blocks = (int)((C + kBlock - 1) / kBlock), part_blocks = (blocks + a.parts - 1) / a.parts;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const i32x4 tile = plan_tiles(a.plan, a.adapters)[id / per_tile];
    const int sub = (int)(id % per_tile), part = sub % a.parts, r0 = sub / a.parts * RB;
    if (tile.x >= a.adapters) break;  // (tokens without an adapter come last)
    const elem *const w = reinterpret_cast<const elem *>(a.w) + (int64_t)tile.x * a.rank * C;
    const elem *x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      x[m] = reinterpret_cast<const elem *>(a.x) + (int64_t)order[tile.y + min(16 * m + i, tile.z - 1)] * a.ldx;
    const int groups = (tile.z + 15) >> 4;
    v4f acc[4][NT];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[m][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int b1 = min(blocks, (part + 1) * part_blocks);
    for (int b = part * part_blocks + wave; b < b1; b += 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = (int64_t)b * kBlock + (2 * g + h) * E;
        const int64_t left = C - c;  // (may be 0 or less)
        u32x4 wf[NT];
        if constexpr (!W_T) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int r = r0 + 16 * j + i;
            wf[j] = load_frag<DT>(w + (int64_t)min(r, a.rank - 1) * C + c, r < a.rank ? left : 0);
          }
        } else {
          Few<DT, NT> rows[E];
          const int r = r0 + i * NT;
#pragma unroll
          for (int e = 0; e < E; ++e) rows[e] = load_few<DT, NT>(w + (c + e) * a.rank + r, e < left ? a.rank - r : 0);
#pragma unroll
          for (int j = 0; j < NT; ++j) wf[j] = pick<DT, NT>(rows, j);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= groups) break;
          const u32x4 xf = load_frag<DT>(x[m] + c, left);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[m][j] = mma<DT>(wf[j], xf, acc[m][j]);
        }
      }
    }
    // the four waves' sums, in their order
    auto rank_of = [&](int j, int q) { return W_T ? (4 * g + q) * NT + j : 16 * j + 4 * g + q; };
    __syncthreads();  // (of the last tile's reads)
    if (wave > 0) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) red[wave - 1][16 * m + i][rank_of(j, q)] = acc[m][j][q];
    }
    __syncthreads();
    if (wave == 0) {
      const float s = a.scales ? a.scales[tile.x] : 1.0f;
      const int rp = lora_rank_pad(a.rank);
      float *const out = a.h + (int64_t)part * a.tokens * rp;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (16 * m + i >= tile.z) continue;
        float *const row = out + (int64_t)(tile.y + 16 * m + i) * rp + r0;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = rank_of(j, q);
            float v = acc[m][j][q];
#pragma unroll
            for (int t = 0; t < 3; ++t) v += red[t][16 * m + i][r];
            // (past the rank: zero, also where x is not finite)
            if (r0 + r < rp) row[r] = r0 + r < a.rank ? s * v : 0.0f;
          }
      }
    }
  }
}

// ---------------------------------------------------------------- up

// Y[t][c] = base[t][c] + sum over r of H[position][r] * W(c, r), W (C, R) as
// rows, or (R, C) where W_T; base may be missing.  A wave takes 64 columns of
// up to 64 rows; lane (i, g) ends with 16 consecutive columns of rows i, i +
// 16, ...: row 4 * p + q of operand tile j stands for column 4 * (4 * p + q) + j.
template <int DT, bool W_T>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraUp a) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>;
  const int tiles = plan_tile_count(a.plan, a.tokens, a.adapters);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t C = a.cols;
  const int cblocks = (int)((C + 255) / 256);
  const int64_t total = (int64_t)tiles * cblocks;
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int rp = lora_rank_pad(a.rank);
  const int64_t part_ld = (int64_t)a.tokens * rp;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const i32x4 tile = plan_tiles(a.plan, a.adapters)[id / cblocks];
    const int64_t c0 = (id % cblocks) * 256 + 64 * wave;
    const int groups = (tile.z + 15) >> 4;
    v4f acc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (tile.x < a.adapters) {
      const elem *const w = reinterpret_cast<const elem *>(a.w) + (int64_t)tile.x * a.rank * C;
      const bool keep = a.sum && id % cblocks == 0 && wave == 0;
      for (int r0 = 0; r0 < rp; r0 += 16) {
        // this lane's ranks: E of 16 (in the 16-bit types lanes of g and g + 2 hold the same, for H's two halves)
        const int rg = r0 + (DT == F8LIN_FP32 ? g : (g & 1)) * E;
        u32x4 wf[4];
        if constexpr (!W_T) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + 4 * i + j;
            wf[j] = load_frag<DT>(w + min(c, C - 1) * a.rank + rg, c < C ? a.rank - rg : 0);
          }
        } else {
          Few<DT, 4> rows[E];
          const int64_t c = c0 + 4 * i;
#pragma unroll
          for (int e = 0; e < E; ++e)
            rows[e] = load_few<DT, 4>(w + (int64_t)(rg + e) * C + c, rg + e < a.rank ? (int)min((int64_t)4, C - c) : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) wf[j] = pick<DT, 4>(rows, j);
        }
        u32x4 wl[4];
        if constexpr (DT == F8LIN_FP16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) split_f16(wf[j], wf[j], wl[j]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= groups) break;
          const int p = tile.y + min(16 * m + i, tile.z - 1);
          const float *const h = a.h + (int64_t)p * rp + rg;
          float v[E];
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            v4f s = *reinterpret_cast<const v4f *>(h + e);
            for (int k = 1; k < a.parts; ++k) s += *reinterpret_cast<const v4f *>(h + k * part_ld + e);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[e + k] = s[k];
            if (keep && (DT == F8LIN_FP32 || g < 2) && 16 * m + i < tile.z)
              *reinterpret_cast<v4f *>(a.sum + (int64_t)p * rp + rg + e) = s;
          }
          if constexpr (DT == F8LIN_FP32) {
            const u32x4 hf = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][j] = mma<DT>(wf[j], hf, acc[m][j]);
          } else {
            u32x4 hi, lo;
            split8(v, hi, lo);
            const u32x4 hf = g < 2 ? hi : lo;
            // (an infinite H meets the operand's main half only: the other is often zero)
            const u32x4 finite = DT == F8LIN_FP16 ? no_inf(hf) : hf;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[m][j] = mma<F8LIN_BF16>(wf[j], hf, acc[m][j]);
              if constexpr (DT == F8LIN_FP16) acc[m][j] = mma<F8LIN_BF16>(wl[j], finite, acc[m][j]);
            }
          }
        }
      }
    }
    const int64_t c = c0 + 16 * g;
    const int n = (int)max((int64_t)0, min((int64_t)16, C - c));
    if (n == 0) continue;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (16 * m + i >= tile.z) break;
      const int64_t t = order[tile.y + 16 * m + i];
      elem *const y = reinterpret_cast<elem *>(a.y) + t * a.ldy + c;
      const elem *const base = a.base ? reinterpret_cast<const elem *>(a.base) + t * a.ldbase + c : nullptr;
#pragma unroll
      for (int h = 0; h < 16; h += E) {
        if (h >= n) break;
        const u32x4 raw = base ? load_frag<DT>(base + h, n - h) : u32x4{0, 0, 0, 0};
        uint32_t o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t bits = DT == F8LIN_FP32 ? raw[e & 3] : (raw[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
          const float v = acc[m][(h + e) & 3][(h + e) >> 2];
          // (a token without an adapter keeps base's bits)
          o[e] = tile.x < a.adapters ? f32_to_elem(base ? elem_f32<DT>(bits) + v : v, DT) : bits;
        }
        if (n - h >= E) {
          if constexpr (DT == F8LIN_FP32) *reinterpret_cast<u32x4_u *>(y + h) = u32x4{o[0], o[1], o[2], o[3]};
          else
            *reinterpret_cast<u32x4_u *>(y + h) =
                u32x4{o[0] | o[1] << 16, o[2] | o[3] << 16, o[4 % E] | o[5 % E] << 16, o[6 % E] | o[7 % E] << 16};
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (h + e < n) y[h + e] = (elem)o[e];
        }
      }
    }
  }
}

// The sum of H's parts, in their order.
__global__ __launch_bounds__(256) void lora_sum_kernel(const float *h, int parts, int64_t n, float *sum) {
  const int64_t at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);  // (n is a multiple of 16)
  if (at >= n) return;
  v4f s = *reinterpret_cast<const v4f *>(h + at);
  for (int k = 1; k < parts; ++k) s += *reinterpret_cast<const v4f *>(h + k * n + at);
  *reinterpret_cast<v4f *>(sum + at) = s;
}

// ---------------------------------------------------------------- outer

// D_i(c, r) = sum over adapter i's positions p of X[order[p]][c] * H[p][r], as
// (R, C), or (C, R) where d_t.  A wave takes 16 * E columns (lane i the
// contiguous block of E at E * i, which become E operand tiles), 16 * NT ranks
// and `chunk` sorted positions, which may hold several adapters.  An adapter
// that lies within one chunk is written as it is; one that reaches over
// several leaves a binary32 partial sum for each (slot 2 * chunk, or 2 * chunk
// + 1 in the chunk where it begins), which lora_outer_join_kernel adds up.
template <int DT, int NT>
__global__ __launch_bounds__(256) void lora_outer_kernel(const LoraOuter a) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>, kCols = 16 * E, kStep = 4 * E;
  if (plan_tile_count(a.plan, a.tokens, a.adapters) < 0) return;
  const int *const starts = plan_starts(a.plan);
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int *const owner = plan_owner(a.plan, a.tokens, a.adapters);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int rp = lora_rank_pad(a.rank);
  const int adapted = starts[a.adapters];
  int id = blockIdx.x;
  const LoraOuterSide &side = id < a.side[0].blocks * a.units ? a.side[0] : a.side[1];
  if (id >= a.side[0].blocks * a.units) id -= a.side[0].blocks * a.units;
  // columns fastest: the workgroups of a chunk read the same H
  const int64_t c0 = (int64_t)(id % side.blocks) * 4 * kCols + wave * kCols + E * i;
  const int unit = id / side.blocks, chunk = unit % a.chunks, r0 = unit / a.chunks * 16 * NT;
  const int64_t C = side.cols;
  const int64_t first = (int64_t)chunk * a.chunk;
  const int end = (int)min((int64_t)adapted, first + a.chunk);
  const int cn = (int)max((int64_t)0, min((int64_t)E, C - c0));
  for (int p0 = (int)min((int64_t)adapted, first); p0 < end;) {
    const int ad = owner[p0], p1 = min(end, starts[ad + 1]);
    v4f acc[E][NT];
#pragma unroll
    for (int c = 0; c < E; ++c)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[c][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = p0; p < p1; p += kStep) {
      Few<DT, E> rows[E];
      float h[NT][E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = p + g * E + e;
        const bool in = at < p1;  // (nothing behind the adapter's tokens gets in, whatever it holds)
        const int64_t t = in ? order[at] : 0;
        rows[e] = load_few<DT, E>(reinterpret_cast<const elem *>(side.x) + t * side.ldx + c0, in ? cn : 0);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = r0 + 16 * j + i;
          h[j][e] = in && r < rp ? side.h[(int64_t)at * rp + r] : 0.0f;
        }
      }
      u32x4 hi[NT], lo[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (DT == F8LIN_FP32)
          hi[j] = u32x4{__float_as_uint(h[j][0]), __float_as_uint(h[j][1]), __float_as_uint(h[j][2]), __float_as_uint(h[j][3])};
        else split8(h[j], hi[j], lo[j]);
      }
#pragma unroll
      for (int c = 0; c < E; ++c) {
        u32x4 xf = pick<DT, E>(rows, c);
        if constexpr (DT == F8LIN_FP32) {
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[c][j] = mma<DT>(xf, hi[j], acc[c][j]);
        } else {
          u32x4 xl;
          if constexpr (DT == F8LIN_FP16) split_f16(xf, xf, xl);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[c][j] = mma<F8LIN_BF16>(xf, hi[j], acc[c][j]);
            acc[c][j] = mma<F8LIN_BF16>(xf, lo[j], acc[c][j]);
            if constexpr (DT == F8LIN_FP16) acc[c][j] = mma<F8LIN_BF16>(xl, hi[j], acc[c][j]);
          }
        }
      }
    }
    // lane (i, g) holds rank r0 + 16 j + i of columns E * (4 g + q) + c of the wave's
    const bool whole = starts[ad] >= first && starts[ad + 1] <= first + a.chunk;
    const int slot = 2 * chunk + (starts[ad] >= first ? 1 : 0);
    const int64_t elems = (int64_t)a.rank * C;
    auto put = [&](int64_t at, float v) {
      if (!whole) side.part[(int64_t)slot * elems + at] = v;
      else if constexpr (DT == F8LIN_FP32) reinterpret_cast<float *>(side.d)[(int64_t)ad * elems + at] = v;
      else reinterpret_cast<uint16_t *>(side.d)[(int64_t)ad * elems + at] = (uint16_t)f32_to_elem(v, DT);
    };
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = r0 + 16 * j + i;
      if (r >= a.rank) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < E; ++c) {
          const int64_t col = c0 - E * i + E * (4 * g + q) + c;
          if (col < C) put(side.d_t ? col * a.rank + r : (int64_t)r * C + col, acc[c][j][q]);
        }
    }
    p0 = p1;
  }
}

// Adds the partial sums of the adapters that reach over several chunks, and
// clears the gradients of those without a token.
template <int DT>
__global__ __launch_bounds__(256) void lora_outer_join_kernel(const LoraOuter a) {
  if (plan_tile_count(a.plan, a.tokens, a.adapters) < 0) return;
  const int *const starts = plan_starts(a.plan);
  const int64_t per0 = a.side[0].join_blocks, per1 = a.side[1].join_blocks, per = per0 + per1;
  for (int64_t id = blockIdx.x; id < per * a.adapters; id += gridDim.x) {
    const int ad = (int)(id / per);
    const bool second = id % per >= per0;
    const LoraOuterSide &side = second ? a.side[1] : a.side[0];
    const int s = starts[ad], e = starts[ad + 1];
    const int j0 = s / a.chunk, j1 = e > s ? (e - 1) / a.chunk : j0;
    if (e > s && j0 == j1) continue;
    const int64_t elems = (int64_t)a.rank * side.cols;
    const int64_t at = (id % per - (second ? per0 : 0)) * 1024 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t o = at + 256 * k;
      if (o >= elems) break;
      float v = 0.0f;
      if (e > s) {
        v = side.part[(int64_t)(2 * j0 + 1) * elems + o];
        for (int j = j0 + 1; j <= j1; ++j) v += side.part[(int64_t)(2 * j) * elems + o];
      }
      if constexpr (DT == F8LIN_FP32) reinterpret_cast<float *>(side.d)[(int64_t)ad * elems + o] = v;
      else reinterpret_cast<uint16_t *>(side.d)[(int64_t)ad * elems + o] = (uint16_t)f32_to_elem(v, DT);
    }
  }
}

// ---------------------------------------------------------------- launches

constexpr int64_t kMaxGrid1 = (int64_t)1 << 22;  // workgroups; the kernels stride over the rest
unsigned grid_of(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min(n, kMaxGrid1)); }

// Ranks of 16 a workgroup takes: one, two or four.
int rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }

template <int DT, bool W_T>
void down_typed(const LoraDown &a, hipStream_t s) {
  const int nt = rank_tiles(a.rank), rblocks = (a.rank + 16 * nt - 1) / (16 * nt);
  const unsigned grid = grid_of(lora_max_tiles(a.tokens, a.adapters) * rblocks * a.parts);
  if (nt == 1) lora_down_kernel<DT, 1, W_T><<<grid, 256, 0, s>>>(a);
  else if (nt == 2) lora_down_kernel<DT, 2, W_T><<<grid, 256, 0, s>>>(a);
  else lora_down_kernel<DT, 4, W_T><<<grid, 256, 0, s>>>(a);
}
template <int DT>
void down_by_layout(const LoraDown &a, bool w_t, hipStream_t s) {
  if (w_t) down_typed<DT, true>(a, s);
  else down_typed<DT, false>(a, s);
}
template <int DT>
void up_by_layout(const LoraUp &a, bool w_t, hipStream_t s) {
  const unsigned grid = grid_of(lora_max_tiles(a.tokens, a.adapters) * ((a.cols + 255) / 256));
  if (w_t) lora_up_kernel<DT, true><<<grid, 256, 0, s>>>(a);
  else lora_up_kernel<DT, false><<<grid, 256, 0, s>>>(a);
}
template <int DT>
void outer_typed(LoraOuter a, hipStream_t s) {
  const int nt = rank_tiles(a.rank), rblocks = (a.rank + 16 * nt - 1) / (16 * nt);
  const int64_t cols = 4 * 16 * kE<DT>;
  a.units = a.chunks * rblocks;
  for (int i = 0; i < 2; ++i) {
    a.side[i].blocks = a.side[i].d ? (int)((a.side[i].cols + cols - 1) / cols) : 0;
    a.side[i].join_blocks = a.side[i].d ? (a.rank * a.side[i].cols + 1023) / 1024 : 0;
  }
  const int64_t grid = (int64_t)(a.side[0].blocks + a.side[1].blocks) * a.units;
  if (grid > 0) {
    if (nt == 1) lora_outer_kernel<DT, 1><<<(unsigned)grid, 256, 0, s>>>(a);
    else if (nt == 2) lora_outer_kernel<DT, 2><<<(unsigned)grid, 256, 0, s>>>(a);
    else lora_outer_kernel<DT, 4><<<(unsigned)grid, 256, 0, s>>>(a);
  }
  const int64_t joins = (a.side[0].join_blocks + a.side[1].join_blocks) * a.adapters;
  if (joins > 0) lora_outer_join_kernel<DT><<<grid_of(joins), 256, 0, s>>>(a);
}

}  // namespace

int lora_parts(int64_t tokens, int adapters, int64_t cols, int rank) {
  // enough workgroups for the chip, each with two 64-column blocks a wave at least
  const int64_t groups = std::max<int64_t>(1, lora_max_tiles(tokens, adapters)) * ((rank + 63) / 64);
  const int64_t want = (1024 + groups - 1) / groups, most = (cols + 511) / 512;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), 16));
}

int lora_chunk(int64_t tokens, int64_t K, int64_t N, int rank) {
  const int64_t per_chunk = ((K + 511) / 512 + (N + 511) / 512) * ((rank + 63) / 64);
  const int64_t chunks = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, per_chunk));
  const int64_t each = ((tokens + chunks - 1) / chunks + 31) / 32 * 32;
  return (int)std::min<int64_t>(4096, std::max<int64_t>(128, each));
}

hipError_t launch_lora_plan(const void *index, bool wide, int tokens, int adapters, int *plan, hipStream_t stream) {
  if (adapters <= 255) lora_plan_kernel<16, 255><<<1, 1024, 0, stream>>>(index, wide, tokens, adapters, plan);
  else lora_plan_kernel<16, kLoraMaxAdapters><<<1, 1024, 0, stream>>>(index, wide, tokens, adapters, plan);
  return hipGetLastError();
}

hipError_t launch_lora_down(const LoraDown &a, int dtype, bool w_t, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  if (dtype == F8LIN_BF16) down_by_layout<F8LIN_BF16>(a, w_t, stream);
  else if (dtype == F8LIN_FP16) down_by_layout<F8LIN_FP16>(a, w_t, stream);
  else down_by_layout<F8LIN_FP32>(a, w_t, stream);
  return hipGetLastError();
}

hipError_t launch_lora_up(const LoraUp &a, int dtype, bool w_t, hipStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return hipSuccess;
  if (dtype == F8LIN_BF16) up_by_layout<F8LIN_BF16>(a, w_t, stream);
  else if (dtype == F8LIN_FP16) up_by_layout<F8LIN_FP16>(a, w_t, stream);
  else up_by_layout<F8LIN_FP32>(a, w_t, stream);
  return hipGetLastError();
}

hipError_t launch_lora_sum(const LoraUp &a, hipStream_t stream) {
  const int64_t n = (int64_t)a.tokens * lora_rank_pad(a.rank);
  if (n > 0) lora_sum_kernel<<<(unsigned)((n + 1023) / 1024), 256, 0, stream>>>(a.h, a.parts, n, a.sum);
  return hipGetLastError();
}

hipError_t launch_lora_outer(const LoraOuter &a, int dtype, hipStream_t stream) {
  if (dtype == F8LIN_BF16) outer_typed<F8LIN_BF16>(a, stream);
  else if (dtype == F8LIN_FP16) outer_typed<F8LIN_FP16>(a, stream);
  else outer_typed<F8LIN_FP32>(a, stream);
  return hipGetLastError();
}

}  // namespace f8lin

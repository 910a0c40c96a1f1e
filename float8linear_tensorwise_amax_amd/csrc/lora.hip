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
// 65535 bf16 tokens, 4096 x 4096, rank 16, in a training step: down 93 us (5.8
// TB/s), up 210 (5.1), down from dy 122, dx 138 (3.9, all of it written), outer
// 228 (4.7).  8192 tokens from 4096 to 14336 at rank 64: 29 and 127 us (3.7
// TB/s: the adapter's rows, read by every tile, are half of what passes the L2).
// 64 single tokens of as many adapters, rank 16: 6 and 14.5 us for 37 MB, two
// chains of dependent cold reads.
// Rows and weights go from memory to registers in the matrix instructions' own
// layout, with no LDS between (a tile's H passes through it, once for the four
// waves): the contraction's order is free, so that a lane's 16 bytes are
// whatever 8 (4 in binary32) values are contiguous, and where the contraction
// runs across rows a lane takes 8 rows of a block of columns and transposes
// them in registers.  Loads stand in straight lines, whole blocks ahead of
// their use: with a bounds check at each load down took 186 us and outer 379
// where they took 92 and 200 without.
//
// H and G are (T, R), summed and handed on in binary32.  Beside 16-bit operands
// each value becomes a sum of three 16-bit ones, all of its 24 bits, where it
// meets the matrix instruction: three bf16 (an fp16 operand beside them becomes
// two, exactly, and all six products are taken), or in the tiled products over
// ranks in fp16 three fp16 values scaled by a power of two a token.  Two of them
// (2^-17) showed in the outputs wherever a sum cancels.  Binary32 data use the
// binary32 matrix instruction throughout.
//
// An infinity times a value's parts is NaN where one of them is zero, although
// the product is infinite.  Sums that come out as NaN are therefore taken once
// more, an infinite value with the other side's main part alone (which is zero
// only where the value is, or in bf16 below 2^-133); products of ordinary data
// pay a comparison.
#include <algorithm>
#include <type_traits>

#include "lora.h"
#include "rows.h"

namespace f8lin {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- plan

// The buffer's words: {magic, tokens, adapters, tiles}, starts[adapters + 2]
// (first sorted position of each adapter; then of the tokens without one, and
// the end), tiles {adapter, position, rows, first token}, order[tokens] (token
// of each sorted position), owner[tokens] (its adapter).
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
// Tiles of the plan, or -1 where the buffer is no plan of this batch size; it may
// then be shorter than such a plan, and nothing more of it is read.
__device__ __forceinline__ int plan_tile_count(const int *p, int tokens, int adapters) {
  const i32x4 h = *reinterpret_cast<const i32x4 *>(p);
  return h.x == kLoraMagic && h.y == tokens && h.z == adapters ? h.w : -1;
}

// A stable counting sort in one workgroup: each wave owns a contiguous part of
// the tokens and, 64 at a time, finds for each the others of its adapter, one
// ballot a bit of the adapters' numbers; counts and cursors are a wave's own,
// so that no two waves meet at one.  Bound by the latency of its passes over
// the index, and past a few thousand tokens by what one workgroup computes (64
// tokens 5.5 us, 65536 of 4 adapters 41 in runs and 66 mixed, of 1000 mixed 125;
// one adapter after the other among 64 tokens 12.9, 108 mixed, 946), once a
// batch.
template <int WAVES, int MAXA>
__global__ __launch_bounds__(64 * WAVES) void lora_plan_kernel(const void *index, int wide, int tokens, int adapters,
                                                               int *plan) {
  constexpr int kThreads = 64 * WAVES;
  __shared__ int count[WAVES][MAXA + 1];
  __shared__ int starts[MAXA + 2], tile_first[MAXA + 2];
  __shared__ int sums[2][WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile_rows = lora_tile(tokens);
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
  // f(token, its adapter, the lanes that have the same) for 64 tokens at a time, lanes past the wave's last with none
  const int bits = 32 - __builtin_clz(adapters);
  constexpr int kAhead = 4;  // loads on their way
  auto each_group = [&](auto f) {
    int next[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) next[k] = adapter_of(begin + 64 * k + lane);
    for (int t0 = begin; t0 < end; t0 += 64 * kAhead) {
      int now[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) now[k] = next[k], next[k] = adapter_of(t0 + 64 * (kAhead + k) + lane);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int a = now[k];
        uint64_t same = __ballot(a >= 0);
        if (same == 0) break;
        // (often all 64 are one adapter's; lane 0 is there)
        if (__ballot(a == __builtin_amdgcn_readfirstlane(a)) != same) {
          uint32_t lo = (uint32_t)same, hi = (uint32_t)(same >> 32);
          for (int b = 0; b < bits; ++b) {
            const uint32_t bit = (uint32_t)(a << (31 - b) >> 31);  // of this lane, 32 times
            const uint64_t with = __ballot(bit != 0);
            lo &= ~((uint32_t)with ^ bit), hi &= ~((uint32_t)(with >> 32) ^ bit);
          }
          same = (uint64_t)hi << 32 | lo;
        }
        if (a >= 0) f(t0 + 64 * k + lane, a, same);
        // (the next group reads what other lanes have written)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
  };
  const uint64_t before = (1ull << lane) - 1;
  // (the first lane of an adapter's counts for all)
  each_group([&](int, int a, uint64_t same) {
    if ((same & before) == 0) atomicAdd(&count[wave][a], __builtin_popcountll(same));
  });
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
    const int nt = (n + tile_rows - 1) / tile_rows;
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
  each_group([&](int t, int a, uint64_t same) {
    const int p = count[wave][a] + __builtin_popcountll(same & before);
    order[p] = t;
    owner[p] = a;
    if ((same & before) == 0) atomicAdd(&count[wave][a], __builtin_popcountll(same));
  });
  __syncthreads();  // (order, by other waves)
  for (int a = tid; a <= groups; a += kThreads) plan[4 + a] = starts[a];
  i32x4 *const tiles = reinterpret_cast<i32x4 *>(plan + lora_tiles_at(adapters));
  for (int i = tid; i < tiles_before; i += kThreads) {
    int lo = 0, hi = groups - 1;  // the last adapter whose first tile is at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int p = starts[lo] + (i - tile_first[lo]) * tile_rows;
    tiles[i] = i32x4{lo, p, min(tile_rows, starts[lo + 1] - p), order[p]};
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

// The same with 8 bytes of a 16-bit type along a contraction of 16.
template <int DT>
__device__ __forceinline__ v4f mma16(u32x2 a, u32x2 b, v4f c) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  if constexpr (DT == F8LIN_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ u32x4 frag_of(const Few<DT, kE<DT>> &f) {
  return u32x4{f.w[0], f.w[1], f.w[2], f.w[3]};
}

// Element j of each of four rows, packed.
template <int V>
__device__ __forceinline__ u32x2 pick4(const Few<F8LIN_BF16, V> &a, const Few<F8LIN_BF16, V> &b, const Few<F8LIN_BF16, V> &c,
                                       const Few<F8LIN_BF16, V> &d, int j) {
  const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
  return u32x2{__builtin_amdgcn_perm(b.w[j >> 1], a.w[j >> 1], sel), __builtin_amdgcn_perm(d.w[j >> 1], c.w[j >> 1], sel)};
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
// The same of the type DT.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  if constexpr (DT == F8LIN_BF16) return pack_bf16(a, b);
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
// What rounding a leaves over; an infinity leaves nothing.
__device__ __forceinline__ float left_over(float a, float rounded) {
  return (__float_as_uint(rounded) & 0x7F800000u) == 0x7F800000u ? 0.0f : a - rounded;
}
// A pair of DT with infinities and NaN as zeros.
template <int DT>
__device__ __forceinline__ uint32_t finite_of(uint32_t f) {
  constexpr uint32_t top = DT == F8LIN_BF16 ? 0x7F80u : 0x7C00u;
  if ((f & top) == top) f &= 0xFFFF0000u;
  if ((f & (top << 16)) == top << 16) f &= 0x0000FFFFu;
  return f;
}
// Whether there is a NaN among n sums.
template <int N>
__device__ __forceinline__ bool has_nan(const v4f (&v)[N]) {
  bool nan = false;
#pragma unroll
  for (int k = 0; k < N; ++k) nan |= __builtin_isunordered(v[k].x, v[k].y) || __builtin_isunordered(v[k].z, v[k].w);
  return nan;
}
// A pair of fp16 as pairs of bf16: rounded, and what that left over.
__device__ __forceinline__ void split_f16(uint32_t f, uint32_t &hi, uint32_t &lo) {
  const float a = f16_bits_to_f32(f & 0xFFFFu), b = f16_bits_to_f32(f >> 16);
  hi = pack_bf16(a, b);
  lo = pack_bf16(left_over(a, bf16_lo(hi)), left_over(b, bf16_hi(hi)));
}

// ---------------------------------------------------------------- intermediates

// Beside 16-bit operands a value of H is a sum of three values of DT.  bf16: cut
// off after 8 bits each, which leaves nothing.
constexpr int kParts = 3;
// Two values' parts, as packed pairs.
template <int DT>
__device__ __forceinline__ void h_parts(float a, float b, uint32_t (&p)[kParts]) {
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    if constexpr (DT == F8LIN_BF16) {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      p[k] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
      if (k + 1 == kParts) break;
      a = left_over(a, __uint_as_float(ua & 0xFFFF0000u)), b = left_over(b, __uint_as_float(ub & 0xFFFF0000u));
    } else {
      p[k] = pack2<DT>(a, b);
      if (k == 0) {  // (the main part of a value that is not zero is not: 2^-24, which the others make up for)
        if ((p[0] & 0x7FFFu) == 0 && a != 0.0f) p[0] |= 1u;
        if ((p[0] & 0x7FFF0000u) == 0 && b != 0.0f) p[0] |= 0x10000u;
      }
      if (k + 1 == kParts) break;
      a = left_over(a, f16_bits_to_f32(p[k] & 0xFFFFu)), b = left_over(b, f16_bits_to_f32(p[k] >> 16));
    }
  }
}
// The same of n consecutive values: part k of them in words k * n / 2 ...
template <int DT, int N>
__device__ __forceinline__ void h_parts_of(const float (&v)[N], uint32_t *w) {
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    uint32_t p[kParts];
    h_parts<DT>(v[2 * e], v[2 * e + 1], p);
#pragma unroll
    for (int k = 0; k < kParts; ++k) w[k * (N / 2) + e] = p[k];
  }
}
// With fp16 operands the products over ranks take v * 2^-e, e by the largest
// finite value of a token's block of 64 ranks, which becomes one of 2^13 to 2^14: three
// fp16 values then hold every bit of what is at least 2^-15 of it, and 2^-39 of
// it is the most that is lost of the rest.
__device__ __forceinline__ int up_exponent(uint32_t mag) {
  const int field = (int)(mag >> 23);
  return field == 0 ? 0 : field - 127 - 13;
}
// ---------------------------------------------------------------- down

// H[position][r] = scale * sum over columns of X[t][c] * W(r, c), W (R, C) as
// rows, or (C, R) where W_T.  A workgroup takes a tile of up to 16 * M rows,
// 16 * NT ranks and one part of the columns, 64 (32 in binary32: 128 bytes a
// row) at a time, dealt to its waves, whose sums meet in the LDS.  With one
// part H is written as the later products take it, by position (h) and by rank
// (ht); else each part's sum in binary32, by position.
//
// Each step's loads are on their way while the step before is multiplied.  The
// last block of columns ends with the row, what it shares with the one before
// taken as zero (SMALL, fewer columns than a block: an element at a time).
template <int DT, int NT, bool W_T, int M>
struct DownStep {
  Few<DT, kE<DT>> x[2][M];
  Few<DT, kE<DT>> w[2][W_T ? 1 : NT];  // !W_T
  Few<DT, NT> rows[2][kE<DT>];         // W_T
};
template <int DT, int NT, bool W_T, int M, int WAVES, bool SMALL>
__global__ __launch_bounds__(64 * WAVES) void lora_down_kernel(const LoraDown a) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>, kBlock = 8 * E, RB = 16 * NT, kRows = 16 * M, kThreads = 64 * WAVES;
  __shared__ float red[WAVES][kRows][RB + 1];
  const int tiles = plan_tile_count(a.plan, a.tokens, a.adapters);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  // (a tile's rows are dealt to as many workgroups as M leaves)
  const int part = blockIdx.x % a.parts, first_row = blockIdx.x / a.parts * kRows, r0 = blockIdx.z * RB;
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int64_t C = a.cols;
  const int blocks = (int)((C + kBlock - 1) / kBlock), part_blocks = (blocks + a.parts - 1) / a.parts;
  const int rp = lora_rank_pad(a.rank), tile_rows = lora_tile(a.tokens);
  const bool whole_ranks = !W_T || a.rank % NT == 0;
  for (int at = blockIdx.y; at < tiles; at += gridDim.y) {
    i32x4 tile = plan_tiles(a.plan, a.adapters)[at];
    if (tile.x >= a.adapters) break;  // (tokens without an adapter come last)
    tile.y += first_row, tile.z -= first_row;
    if (tile.z <= 0) continue;
    const elem *const w = reinterpret_cast<const elem *>(a.w) + (int64_t)tile.x * a.rank * C;
    const elem *x[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
      x[m] = reinterpret_cast<const elem *>(a.x) + (int64_t)order[tile.y + min(16 * m + i, tile.z - 1)] * a.ldx;
    v4f acc[M][NT];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[m][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // Ranks past the end read a row (or a place in one) that is there: their sums are dropped below.
    auto load = [&](int b, DownStep<DT, NT, W_T, M> &s) {
      const bool last = !SMALL && (int64_t)(b + 1) * kBlock > C;
      const int64_t at0 = (int64_t)b * kBlock, c0 = (last ? C - kBlock : at0) + 2 * g * E;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = c0 + h * E;
#pragma unroll
        for (int m = 0; m < M; ++m)
          s.x[h][m] = SMALL ? load_each<DT, E>(x[m], c, C) : load_whole<DT, E>(x[m] + c);
        if constexpr (!W_T) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const elem *const row = w + (int64_t)min(r0 + 16 * j + i, a.rank - 1) * C;
            s.w[h][j] = SMALL ? load_each<DT, E>(row, c, C) : load_whole<DT, E>(row + c);
          }
        } else {
          const int r = r0 + i * NT;
          if (whole_ranks) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              s.rows[h][e] = load_whole<DT, NT>(w + (SMALL ? min(c + e, C - 1) : c + e) * a.rank + (r < a.rank ? r : 0));
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
              s.rows[h][e] = load_to_end<DT, NT>(w + (SMALL ? min(c + e, C - 1) : c + e) * a.rank, r, a.rank);
          }
          if constexpr (SMALL) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (c + e >= C) clear<DT, NT>(s.rows[h][e]);
          }
        }
      }
      if (last) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int shared = (int)(at0 - (c0 + h * E));
#pragma unroll
          for (int m = 0; m < M; ++m) clear_first<DT, E>(s.x[h][m], shared);
          if constexpr (!W_T) {
#pragma unroll
            for (int j = 0; j < NT; ++j) clear_first<DT, E>(s.w[h][j], shared);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (e < shared) clear<DT, NT>(s.rows[h][e]);
          }
        }
      }
    };
    auto multiply = [&](const DownStep<DT, NT, W_T, M> &s) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          u32x4 wf;
          if constexpr (W_T) wf = pick<DT, NT>(s.rows[h], j);
          else wf = frag_of<DT>(s.w[h][j]);
#pragma unroll
          for (int m = 0; m < M; ++m) acc[m][j] = mma<DT>(wf, frag_of<DT>(s.x[h][m]), acc[m][j]);
        }
    };
    // tiles start at different columns, so that rows a power of two apart do not meet at the same channels (65535 x
    // 4096, rank 16: forward 337 us, all from the first column 342; but dx of 8192 x 14336, rank 64, 174 and 163)
    const int b0 = part * part_blocks, nb = min(blocks, b0 + part_blocks) - b0;
    const int turn = nb > 0 ? (int)((uint32_t)at * 5u % (uint32_t)nb) : 0;
    auto block = [&](int b) { return b0 + (b + turn < nb ? b + turn : b + turn - nb); };
    DownStep<DT, NT, W_T, M> s0, s1;
    if (wave < nb) load(block(wave), s0);
    for (int b = wave; b < nb; b += 2 * WAVES) {
      if (b + WAVES < nb) load(block(b + WAVES), s1);
      multiply(s0);
      if (b + WAVES >= nb) break;
      if (b + 2 * WAVES < nb) load(block(b + 2 * WAVES), s0);
      multiply(s1);
    }
    __syncthreads();  // (of the last tile's reads)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[wave][16 * m + i][W_T ? (4 * g + q) * NT + j : 16 * j + 4 * g + q] = acc[m][j][q];
    __syncthreads();
    // the waves' sums, in their order: a thread takes E consecutive ranks of a row at a time
    const float s = a.scales ? a.scales[tile.x] : 1.0f;
    constexpr int kPer = RB / E;  // threads a row
    for (int it = threadIdx.x; it < kRows * kPer; it += kThreads) {
      const int row = it / kPer, r = it % kPer * E;
      float v[E];
      uint32_t mag = 0;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        v[k] = red[0][row][r + k];
#pragma unroll
        for (int t = 1; t < WAVES; ++t) v[k] += red[t][row][r + k];
        // (past the rank: zero, also where x is not finite)
        v[k] = r0 + r + k < a.rank ? s * v[k] : 0.0f;
        if (isfinite(v[k])) mag = max(mag, __float_as_uint(v[k]) & 0x7FFFFFFFu);
      }
      int e = 0;
      if constexpr (DT == F8LIN_FP16) {
#pragma unroll
        for (int off = 1; off < kPer; off <<= 1) mag = max(mag, (uint32_t)__shfl_xor((int)mag, off, 64));
        e = up_exponent(mag);
        if (a.h && row < tile.z && r == 0) a.exponents[(int64_t)(r0 / 64) * a.tokens + tile.y + row] = e;
      }
      if (row < tile.z && r0 + r < rp) {
        if (a.parts_out) {
          float *const to = a.parts_out + ((int64_t)part * a.tokens + tile.y + row) * rp + r0 + r;
#pragma unroll
          for (int k = 0; k < E; k += 4) *reinterpret_cast<v4f *>(to + k) = v4f{v[k], v[k + 1], v[k + 2], v[k + 3]};
        } else if (a.h) {
          // its place among the fragments of 16 rows, 1 KB for 16 ranks: 4 ranks a lane (32 ranks in the 16-bit types: 8 a
          // lane, the first four of them in the first KB, the others in the second)
          const int group = (at * tile_rows + first_row + row) / 16, rr = r0 + r;
          u32x4 *const to = reinterpret_cast<u32x4 *>(a.h) + (int64_t)group * (rp / 16) * 64 + row % 16;
          u32x4 o[E / 4];
#pragma unroll
          for (int k = 0; k < E; ++k) o[k / 4][k % 4] = __float_as_uint(DT == F8LIN_FP16 ? ldexpf(v[k], -e) : v[k]);
          u32x4 *const at4 = to + (E == 4 || rp == 16 ? rr / 16 * 64 + rr % 16 / 4 * 16 : rr / 32 * 128 + rr % 32 / 8 * 16);
          at4[0] = o[0];
          if constexpr (E == 8) at4[rp == 16 ? 16 : 64] = o[1];
        }
      }
      if (a.ht) {
#pragma unroll
        for (int k = 0; k < E; ++k) red[0][row][r + k] = v[k];  // (this thread's own)
      }
    }
    if (!a.parts_out && a.ht) {
      __syncthreads();
      for (int it = threadIdx.x; it < kRows * RB; it += kThreads) {
        const int row = it % kRows, r = it / kRows;
        if (row < tile.z && r0 + r < rp) a.ht[(int64_t)(r0 + r) * a.tokens + tile.y + row] = red[0][row][r];
      }
    }
  }
}

// Sums the parts that a split down product left, in their order, into H by
// rank.
__global__ __launch_bounds__(256) void lora_sum_kernel(const LoraDown a) {
  __shared__ float turn[16][17];
  if (plan_tile_count(a.plan, a.tokens, a.adapters) < 0) return;
  const int rp = lora_rank_pad(a.rank), tr = threadIdx.x & 15, tp = threadIdx.x >> 4;
  const int64_t ld = (int64_t)a.tokens * rp, rblocks = rp / 16;
  const int r = (int)(blockIdx.x % rblocks) * 16, p = (int)(blockIdx.x / rblocks) * 16;
  if (p + tp < a.tokens) {
    const float *const from = a.parts_out + (int64_t)(p + tp) * rp + r + tr;
    float v = from[0];
    for (int k = 1; k < a.parts; ++k) v += from[k * ld];
    turn[tp][tr] = v;
  }
  __syncthreads();
  if (p + tr < a.tokens) a.ht[(int64_t)(r + tp) * a.tokens + p + tr] = turn[tr][tp];
}

// ---------------------------------------------------------------- up

// Y[t][c] = base[t][c] + sum over r of H[position][r] * W(c, r), W (C, R) as
// rows, or (R, C) where W_T; base may be missing.  A wave takes 64 columns of
// up to 16 * M rows, a workgroup 256; lane (i, g) ends with row i of each
// group of 16 and, in operand tiles of 16 columns each, 16-byte pieces of
// columns that its neighbours of the same row continue to 64 bytes: in the
// 16-bit types row 4 p + q of tile j stands for column 32 (j / 2) + 8 p + 2 q
// + j % 2, in binary32 for 16 j + 4 p + q.

// W's fragments for KB ranks from r0 and 64 columns from c0 (SMALL: fewer may
// be there; WHOLE: the ranks are whole blocks).  KB = 32: 8 ranks a lane, 16: 4
// (binary32: always 16 ranks, 4 a lane).  What lies past the ranks is zero,
// whatever the memory holds: H is zero there.
template <int DT, int KB>
struct UpFrag {
  static constexpr int kPer = DT == F8LIN_FP32 ? 4 : KB / 4, kWords = DT == F8LIN_FP32 ? 4 : kPer / 2;
  uint32_t w[kWords];
};
template <int DT, int KB>
__device__ __forceinline__ v4f up_mma(const UpFrag<DT, KB> &f, const uint32_t *h, v4f c) {
  if constexpr (UpFrag<DT, KB>::kWords == 2) return mma16<DT>(u32x2{f.w[0], f.w[1]}, u32x2{h[0], h[1]}, c);
  else return mma<DT>(u32x4{f.w[0], f.w[1], f.w[2], f.w[3]}, u32x4{h[0], h[1], h[2], h[3]}, c);
}
template <int DT, bool W_T, bool SMALL, int KB, bool WHOLE>
__device__ __forceinline__ void up_weights(const typename MxElem<DT>::type *w, int rank, int64_t C, int64_t c0, int r0,
                                           UpFrag<DT, KB> (&wf)[4]) {
  constexpr bool F32 = DT == F8LIN_FP32;
  constexpr int P = UpFrag<DT, KB>::kPer, kWords = UpFrag<DT, KB>::kWords;  // ranks a lane, and their words
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, rg = r0 + P * g;
  if constexpr (!W_T) {
    // (columns past the end read the last one's: they are not stored)
    const typename MxElem<DT>::type *row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + (F32 ? 16 * j + i : 32 * (j >> 1) + 2 * i + (j & 1));
      row[j] = w + (SMALL ? min(c, C - 1) : c) * rank;
    }
    Few<DT, P> f[4];
    if (WHOLE || r0 + 4 * P <= rank) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_whole<DT, P>(row[j] + rg);
    } else if (rank >= P) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_to_end<DT, P>(row[j], rg, rank);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_each<DT, P>(row[j], rg, rank);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < kWords; ++k) wf[j].w[k] = f[j].w[k];
  } else if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + 16 * j + i;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const uint32_t v = w[(int64_t)(WHOLE ? rg + e : min(rg + e, rank - 1)) * C + (SMALL ? min(c, C - 1) : c)];
        wf[j].w[e] = WHOLE || rg + e < rank ? v : 0u;
      }
    }
  } else {
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      Few<F8LIN_BF16, 2> rows[P];
      const int64_t c = c0 + 32 * jj + 2 * i;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const typename MxElem<DT>::type *const from = w + (int64_t)(WHOLE ? rg + e : min(rg + e, rank - 1)) * C;
        rows[e] = SMALL ? load_each<F8LIN_BF16, 2>(from, c, C) : load_whole<F8LIN_BF16, 2>(from + c);
        rows[e].w[0] = WHOLE || rg + e < rank ? rows[e].w[0] : 0u;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < P; e += 4) {
          const u32x2 f = pick4<2>(rows[e], rows[e + 1], rows[e + 2], rows[e + 3], j);
          wf[2 * jj + j].w[e / 2] = f.x, wf[2 * jj + j].w[e / 2 + 1] = f.y;
        }
    }
  }
}
// The 64 columns of a wave: from c0, or for the last ones those that end with
// the row, of which only the ones from `own` on are stored (C >= 64).
struct UpCols {
  int64_t c0, own;
};
__device__ __forceinline__ UpCols up_cols(int64_t c0, int64_t C) {
  return UpCols{C >= 64 ? min(c0, C - 64) : c0, c0};
}
// base's pieces of one row.
template <int DT, bool SMALL>
__device__ __forceinline__ void up_base(const LoraUp &a, int64_t t, const UpCols &cols, u32x4 (&raw)[16 / kE<DT>]) {
  constexpr int E = kE<DT>;
  const int g = (threadIdx.x & 63) >> 4;
  const typename MxElem<DT>::type *const base = reinterpret_cast<const typename MxElem<DT>::type *>(a.base) + t * a.ldbase;
  if (!a.base) {
#pragma unroll
    for (int h = 0; h < 16 / E; ++h) raw[h] = u32x4{0, 0, 0, 0};
    return;
  }
#pragma unroll
  for (int h = 0; h < 16 / E; ++h) {
    const int64_t c = cols.c0 + 4 * E * h + E * g;
    raw[h] = frag_of<DT>(SMALL ? load_each<DT, E>(base, c, a.cols) : load_whole<DT, E>(base + c));
  }
}
// One row's pieces of y.
template <int DT, bool SMALL>
__device__ __forceinline__ void up_store(const LoraUp &a, int64_t t, bool adapted, const UpCols &cols,
                                         const u32x4 (&raw)[16 / kE<DT>], const v4f (&acc)[4]) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>;
  constexpr bool F32 = DT == F8LIN_FP32;
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int h = 0; h < 16 / E; ++h) {
    const int64_t c = cols.c0 + 4 * E * h + E * g;
    elem *const y = reinterpret_cast<elem *>(a.y) + t * a.ldy + c;
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t bits = F32 ? raw[h][e & 3] : (raw[h][e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      const float v = F32 ? acc[h & 3][e & 3] : acc[(2 * h + (e & 1)) & 3][e >> 1];
      f[e] = a.base ? elem_f32<DT>(bits) + v : v;
    }
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = F32 ? __float_as_uint(f[e]) : pack2<DT>(f[(2 * e) % E], f[(2 * e + 1) % E]);
    if (!adapted) v = raw[h];  // (base's bits)
    const bool whole = SMALL ? c + E <= a.cols : c >= cols.own;
    if (whole) {
      *reinterpret_cast<u32x4_u *>(y) = v;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (SMALL ? c + e < a.cols : c + e >= cols.own) y[e] = (elem)(F32 ? v[e & 3] : v[e >> 1] >> (16 * (e & 1)));
    }
  }
}
// Tiles of 64 rows, H in its final form.  Up to 64 ranks (NB blocks of KB): W
// stays in registers, the rows pass by in groups of 16, all their base on its
// way ahead; the tile's H comes through the LDS, once for the four waves, and
// becomes parts on that way.  NB = 0: any rank, 64 at a time, all rows' sums kept
// (8192 x 4096 to 14336, rank 128: forward 277 us, of two parts only and each
// wave with its own reads of H 286).

// A lane's ranks of one row of a block of KB, as the memory holds them.
template <int DT, int KB>
struct UpRaw {
  static constexpr int kPieces = DT != F8LIN_FP32 && KB == 32 ? 2 : 1;
  u32x4 w[kPieces];
};
template <int DT, int KB>
__device__ __forceinline__ UpRaw<DT, KB> up_raw(const u32x4 *h, int block) {
  UpRaw<DT, KB> r;
#pragma unroll
  for (int k = 0; k < UpRaw<DT, KB>::kPieces; ++k) r.w[k] = h[(block * UpRaw<DT, KB>::kPieces + k) * 64];
  return r;
}
// The same as operand fragments: part after part (binary32: itself).
template <int DT, int KB>
struct UpH {
  static constexpr int kWords = DT == F8LIN_FP32 ? 4 : kParts * KB / 8;
  uint32_t w[kWords];
};
template <int DT, int KB>
__device__ __forceinline__ UpH<DT, KB> up_split(const UpRaw<DT, KB> &r) {
  UpH<DT, KB> f;
  if constexpr (DT == F8LIN_FP32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f.w[k] = r.w[0][k];
  } else {
    float v[KB / 4];
#pragma unroll
    for (int k = 0; k < KB / 4; ++k) v[k] = __uint_as_float(r.w[k / 4][k % 4]);
    h_parts_of<DT, KB / 4>(v, f.w);
  }
  return f;
}
// Their place in the LDS: 16 bytes a lane at a time, the last of 16 ranks 8.
template <int DT, int KB>
struct UpShared {
  static constexpr int kWhole = UpH<DT, KB>::kWords / 4;
  u32x4 whole[kWhole][64];
  u32x2 half[UpH<DT, KB>::kWords % 4 ? 64 : 1];
  __device__ __forceinline__ void put(int lane, const UpH<DT, KB> &f) {
#pragma unroll
    for (int k = 0; k < kWhole; ++k) whole[k][lane] = u32x4{f.w[4 * k], f.w[4 * k + 1], f.w[4 * k + 2], f.w[4 * k + 3]};
    if constexpr (UpH<DT, KB>::kWords % 4) half[lane] = u32x2{f.w[4 * kWhole], f.w[4 * kWhole + 1]};
  }
  __device__ __forceinline__ UpH<DT, KB> get(int lane) const {
    UpH<DT, KB> f;
#pragma unroll
    for (int k = 0; k < 4 * kWhole; ++k) f.w[k] = whole[k / 4][lane][k % 4];
    if constexpr (UpH<DT, KB>::kWords % 4) f.w[4 * kWhole] = half[lane].x, f.w[4 * kWhole + 1] = half[lane].y;
    return f;
  }
};
template <int DT, int KB, bool CAREFUL>
__device__ __forceinline__ void up_products(const UpFrag<DT, KB> (&wf)[4], const UpH<DT, KB> &h, v4f (&acc)[4]) {
  constexpr int kAll = DT == F8LIN_FP32 ? 1 : kParts;
  if constexpr (!CAREFUL) {
    // (a part after the other: products that follow each other in one sum would wait)
#pragma unroll
    for (int k = 0; k < kAll; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = up_mma<DT, KB>(wf[j], h.w + k * (KB / 8), acc[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j] = up_mma<DT, KB>(wf[j], h.w, acc[j]);
      UpFrag<DT, KB> w;
#pragma unroll
      for (int e = 0; e < UpFrag<DT, KB>::kWords; ++e) w.w[e] = finite_of<DT>(wf[j].w[e]);
#pragma unroll
      for (int k = 1; k < kAll; ++k) acc[j] = up_mma<DT, KB>(w, h.w + k * (KB / 8), acc[j]);
      __builtin_amdgcn_sched_barrier(0);  // (one operand's copy at a time: the registers are the other path's)
    }
  }
}

// Blocks of ranks whose H is in the LDS at once.
template <int DT, int NB>
constexpr int up_blocks_at_once = NB > 0 ? NB : DT == F8LIN_FP32 ? 4 : 2;

template <int DT, bool W_T, int NB, int KB, bool SMALL, bool WHOLE>
__device__ __forceinline__ void up_tile(const LoraUp &a, const i32x4 tile, int at, const int *order, const UpCols cols,
                                        UpShared<DT, KB> (*shared)[up_blocks_at_once<DT, NB>]) {
  typedef typename MxElem<DT>::type elem;
  constexpr int kPieces = 16 / kE<DT>;
  constexpr int kRanks = DT == F8LIN_FP32 ? 16 : KB;  // of a block
  constexpr int kNB = up_blocks_at_once<DT, NB>;
  const int lane = threadIdx.x & 63, i = lane & 15, wave = threadIdx.x >> 6;
  const int64_t C = a.cols;
  const int rp = lora_rank_pad(a.rank);
  const bool adapted = tile.x < a.adapters;
  const elem *const w = reinterpret_cast<const elem *>(a.w) + (int64_t)tile.x * a.rank * C;
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  auto position = [&](int m) { return tile.y + min(16 * m + i, tile.z - 1); };
  const u32x4 *const from = reinterpret_cast<const u32x4 *>(a.h) + (int64_t)at * 4 * (rp / 16) * 64;
  const int h_ld = rp / 16 * 64;
  auto scale = [&](v4f (&acc)[4], int exponent) {
    if constexpr (DT == F8LIN_FP16) {
      const float f = ldexpf(1.0f, exponent);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] *= f;
    }
  };
  if (!adapted) {  // y is base
#pragma unroll 1
    for (int m = 0; 16 * m < tile.z; ++m) {
      const int64_t t = order[position(m)];
      u32x4 raw[kPieces];
      const v4f acc[4] = {zero, zero, zero, zero};
      up_base<DT, SMALL>(a, t, cols, raw);
      if (16 * m + i < tile.z) up_store<DT, SMALL>(a, t, false, cols, raw, acc);
    }
    return;
  }
  if constexpr (NB > 0) {
    UpFrag<DT, KB> wf[NB][4];
#pragma unroll
    for (int k = 0; k < NB; ++k) up_weights<DT, W_T, SMALL, KB, WHOLE>(w, a.rank, C, cols.c0, kRanks * k, wf[k]);
    u32x4 raw[4][kPieces];
    int64_t t[4];
    int exponent[4];
    const int groups = (tile.z + 15) >> 4;
    // the tile's H, read once by the workgroup, 16 rows a wave (what belongs to rows that are not there is whatever the
    // memory holds, and goes to no row that is)
    UpRaw<DT, KB> mine[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) mine[k] = up_raw<DT, KB>(from + wave * h_ld + lane, k);
    // (rows that are not there: the last one's)
#pragma unroll
    for (int m = 0; m < 4; ++m) t[m] = order[position(m)];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      up_base<DT, SMALL>(a, t[m], cols, raw[m]);
      if constexpr (DT == F8LIN_FP16) exponent[m] = a.exponents[position(m)];
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) shared[wave][k].put(lane, up_split<DT, KB>(mine[k]));
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m >= groups) break;
      v4f acc[4];
      auto products = [&](auto careful) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = zero;
#pragma unroll
        for (int k = 0; k < NB; ++k) up_products<DT, KB, careful>(wf[k], shared[m][k].get(lane), acc);
      };
      products(std::false_type{});
      if (DT != F8LIN_FP32 && __any(16 * m + i < tile.z && has_nan(acc))) products(std::true_type{});
      scale(acc, exponent[m]);
      if (16 * m + i < tile.z) up_store<DT, SMALL>(a, t[m], true, cols, raw[m], acc);
    }
  } else {
    constexpr bool kScaled = DT == F8LIN_FP16;  // 64 ranks share an exponent
    v4f sum[4][4];
    const u32x4 *const my = from + wave * h_ld + lane;
    const int blocks = rp / kRanks;
    UpRaw<DT, KB> mine[kNB];
    auto load = [&](int b0) {
#pragma unroll
      for (int k = 0; k < kNB; ++k)
        if (b0 + k < blocks) mine[k] = up_raw<DT, KB>(my, b0 + k);
    };
    auto products = [&](auto careful) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[m][j] = zero;
      load(0);
      for (int r0 = 0; r0 < rp; r0 += 64) {
        __syncthreads();  // (of the last ranks' reads)
#pragma unroll
        for (int k = 0; k < kNB; ++k)
          if (r0 / kRanks + k < blocks) shared[wave][k].put(lane, up_split<DT, KB>(mine[k]));
        load(r0 / kRanks + kNB);
        __syncthreads();
        v4f part[kScaled ? 4 : 1][4];
#pragma unroll
        for (int m = 0; m < (kScaled ? 4 : 1); ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[m][j] = zero;
        for (int r = r0; r < min(rp, r0 + 64); r += kRanks) {
          UpFrag<DT, KB> wf[4];
          up_weights<DT, W_T, SMALL, KB, WHOLE>(w, a.rank, C, cols.c0, r, wf);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            up_products<DT, KB, careful>(wf, shared[m][(r - r0) / kRanks].get(lane),
                                         kScaled ? part[m % (kScaled ? 4 : 1)] : sum[m]);
          }
        }
        if constexpr (kScaled) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            scale(part[m], a.exponents[(int64_t)(r0 / 64) * a.tokens + position(m)]);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[m][j] += part[m][j];
          }
        }
      }
    };
    products(std::false_type{});
    if constexpr (DT != F8LIN_FP32) {
      bool nan = false;
#pragma unroll
      for (int m = 0; m < 4; ++m) nan |= 16 * m + i < tile.z && has_nan(sum[m]);
      if (__syncthreads_or(nan)) products(std::true_type{});
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t t = order[position(m)];
      u32x4 raw[kPieces];
      up_base<DT, SMALL>(a, t, cols, raw);
      if (16 * m + i < tile.z) up_store<DT, SMALL>(a, t, true, cols, raw, sum[m]);
    }
  }
}

// (Waves a SIMD: the second pass of a sum with a NaN may not cost the first one registers.  8192 x 4096 to 14336 at
// rank 128: forward with three waves 277 us, with two 316.)
template <int DT, bool W_T, int NB, int KB, bool SMALL, bool WHOLE>
constexpr int up_waves = DT == F8LIN_FP32 || SMALL ? 1
                         : NB == 1                 ? (KB == 16 || WHOLE ? 4 : 3)
                         : NB == 2                 ? 3
                                                   : (DT == F8LIN_BF16 && (WHOLE || W_T) ? 3 : 1);
template <int DT, bool W_T, int NB, int KB, bool SMALL, bool WHOLE>
__global__ __launch_bounds__(256, (up_waves<DT, W_T, NB, KB, SMALL, WHOLE>)) void lora_up_kernel(const LoraUp a) {
  __shared__ UpShared<DT, KB> shared[4][up_blocks_at_once<DT, NB>];
  const int tiles = plan_tile_count(a.plan, a.tokens, a.adapters);
  const int64_t C = a.cols;
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  // (a wave past the columns takes the last ones, for the barriers' sake, and stores none of them)
  const int64_t c0 = (int64_t)blockIdx.x * 256 + 64 * (threadIdx.x >> 6);
  for (int at = blockIdx.y; at < tiles; at += gridDim.y) {
    const i32x4 tile = plan_tiles(a.plan, a.adapters)[at];
    up_tile<DT, W_T, NB, KB, SMALL, WHOLE>(a, tile, at, order, up_cols(c0, C), shared);
    __syncthreads();  // (of the tile's reads)
  }
}

// Tiles of 16 rows, H as the sums of its parts.
template <int DT, bool W_T, int G, int KB, bool SMALL, bool WHOLE>
__device__ __forceinline__ void up_few_tile(const LoraUp &a, const i32x4 tile, const int *order, int64_t c0) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>, P = UpFrag<DT, KB>::kPer;
  constexpr bool F32 = DT == F8LIN_FP32;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t C = a.cols;
  const int rp = lora_rank_pad(a.rank);
  const int64_t part_ld = (int64_t)a.tokens * rp;
  const bool adapted = tile.x < a.adapters;
  const int p = tile.y + min(i, tile.z - 1);
  const int64_t t = tile.z == 1 ? tile.w : order[p];
  u32x4 raw[G][16 / E];
#pragma unroll
  for (int k = 0; k < G; ++k) up_base<DT, SMALL>(a, t, up_cols(c0 + 64 * k, C), raw[k]);
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[G][4];
#pragma unroll
  for (int k = 0; k < G; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[k][j] = zero;
  if (adapted) {
    const elem *const w = reinterpret_cast<const elem *>(a.w) + (int64_t)tile.x * a.rank * C;
    auto products = [&](auto careful) {
      for (int r0 = 0; r0 < rp; r0 += 4 * P) {
        UpFrag<DT, KB> wf[G][4];
#pragma unroll
        for (int k = 0; k < G; ++k)
          up_weights<DT, W_T, SMALL, KB, WHOLE>(w, a.rank, C, up_cols(c0 + 64 * k, C).c0, r0, wf[k]);
        float hv[P];
#pragma unroll
        for (int e = 0; e < P; e += 4) {
          const float *const from = a.parts_in + (int64_t)p * rp + r0 + P * g + e;
          v4f s = *reinterpret_cast<const v4f *>(from);
#pragma unroll 4
          for (int k = 1; k < a.parts; ++k) s += *reinterpret_cast<const v4f *>(from + k * part_ld);
#pragma unroll
          for (int k = 0; k < 4; ++k) hv[e + k] = s[k];
        }
        if constexpr (F32) {
          uint32_t hw[P];
#pragma unroll
          for (int e = 0; e < P; ++e) hw[e] = __float_as_uint(hv[e]);
#pragma unroll
          for (int k = 0; k < G; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[k][j] = up_mma<DT, KB>(wf[k][j], hw, acc[k][j]);
        } else {
          uint32_t hw[kParts * P / 2];
          h_parts_of<F8LIN_BF16, P>(hv, hw);
#pragma unroll
          for (int k = 0; k < G; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              UpFrag<F8LIN_BF16, KB> f, left;  // (an fp16 operand as two)
              uint32_t h[P / 2];
#pragma unroll
              for (int e = 0; e < P / 2; ++e) {
                f.w[e] = wf[k][j].w[e], h[e] = hw[e];
                if constexpr (DT == F8LIN_FP16) split_f16(wf[k][j].w[e], f.w[e], left.w[e]);
                if constexpr (careful) h[e] = finite_of<F8LIN_BF16>(h[e]);
              }
              acc[k][j] = up_mma<F8LIN_BF16, KB>(f, hw, acc[k][j]);
              if constexpr (DT == F8LIN_FP16) acc[k][j] = up_mma<F8LIN_BF16, KB>(left, h, acc[k][j]);
              if constexpr (careful) {
#pragma unroll
                for (int e = 0; e < P / 2; ++e) f.w[e] = finite_of<F8LIN_BF16>(f.w[e]);
              }
#pragma unroll
              for (int part = 1; part < kParts; ++part) {
                acc[k][j] = up_mma<F8LIN_BF16, KB>(f, hw + part * (P / 2), acc[k][j]);
                if constexpr (DT == F8LIN_FP16) acc[k][j] = up_mma<F8LIN_BF16, KB>(left, hw + part * (P / 2), acc[k][j]);
              }
            }
        }
      }
    };
    products(std::false_type{});
    if constexpr (!F32) {
      bool nan = false;
#pragma unroll
      for (int k = 0; k < G; ++k) nan |= has_nan(acc[k]);
      if (__any(nan)) {
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[k][j] = zero;
        products(std::true_type{});
      }
    }
  }
  if (i < tile.z) {
#pragma unroll
    for (int k = 0; k < G; ++k)
      if (c0 + 64 * k < C) up_store<DT, SMALL>(a, t, adapted, up_cols(c0 + 64 * k, C), raw[k], acc[k]);
  }
}

template <int DT, bool W_T, int G, int KB, bool SMALL, bool WHOLE>
__global__ __launch_bounds__(256, DT != F8LIN_FP32 && !SMALL && G == 1 && (WHOLE || KB == 16) ? 4 : 1) void lora_up_few_kernel(const LoraUp a) {
  const int tiles = plan_tile_count(a.plan, a.tokens, a.adapters);
  const int64_t C = a.cols;
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 64 * G;
  if (c0 >= C) return;
  for (int at = blockIdx.y; at < tiles; at += gridDim.y) {
    const i32x4 tile = plan_tiles(a.plan, a.adapters)[at];
    up_few_tile<DT, W_T, G, KB, SMALL, WHOLE>(a, tile, order, c0);
  }
}

// ---------------------------------------------------------------- outer

// D_i(c, r) = sum over adapter i's positions p of X[order[p]][c] * H[p][r], as
// (R, C), or (C, R) where d_t.  A wave takes 16 * E columns (lane i the
// contiguous block of E at E * i, which become E operand tiles), 16 * NT ranks
// (NT: 1 or 2) and `chunk` sorted positions, which may hold several adapters.
// An adapter that lies within one chunk is written as it is; one that reaches
// over several leaves a binary32 partial sum for each (slot 2 * chunk, or 2 *
// chunk + 1 in the chunk where it begins), which lora_outer_join_kernel adds up.
// Each step's loads are on their way while the step before is multiplied.  (Two
// waves a SIMD in fp16, whose operands are pairs: with three, 21 registers went to
// memory, and both gradients of 949 tokens took 40.7 us instead of 36.9.)
template <int DT, int NT>
struct OuterStep {
  Few<DT, kE<DT>> rows[kE<DT>];
  u32x4 h[NT][kE<DT> / 4];
};
template <int DT, int NT, bool SMALL>
__global__ __launch_bounds__(256, NT == 1 && DT != F8LIN_FP16 ? 3 : 2) void lora_outer_kernel(const LoraOuter a) {
  typedef typename MxElem<DT>::type elem;
  constexpr int E = kE<DT>, kCols = 16 * E, kStep = 4 * E;
  __shared__ v4f join[4][E * NT][64];
  if (plan_tile_count(a.plan, a.tokens, a.adapters) < 0) return;
  const int *const starts = plan_starts(a.plan);
  const int *const order = plan_order(a.plan, a.tokens, a.adapters);
  const int *const owner = plan_owner(a.plan, a.tokens, a.adapters);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int rp = lora_rank_pad(a.rank);
  const int adapted = starts[a.adapters];
  int id = blockIdx.x;
  const bool second = id >= a.side[0].blocks * a.units;
  if (second) id -= a.side[0].blocks * a.units;
  const LoraOuterSide &side = second ? a.side[1] : a.side[0];
  // a workgroup's waves: `across` blocks of ranks of the same columns and tokens, times `split` parts of the tokens,
  // whose sums meet in the LDS, times blocks of columns; columns fastest: the workgroups of a chunk read the same H,
  // and rounds of 8 units, one an XCD, so that a row's columns are read through one L2
  const int across = a.across, split = a.split, side_by_side = 4 / (across * split);
  {
    const int per = 8 * side.blocks, round = id / per, in = id % per, n = min(8, a.units - 8 * round);
    id = (8 * round + in % n) * side.blocks + in / n;
  }
  const int64_t C = side.cols;
  // the wave's columns: the last ones end with the row, and only those from `own` on are stored
  const int64_t own = ((int64_t)(id % side.blocks) * side_by_side + wave / (across * split)) * kCols;
  const int64_t cw = SMALL ? own : min(own, C - kCols), c0 = cw + E * i;
  const int unit = id / side.blocks, chunk = unit % a.chunks;
  const int r0 = (unit / a.chunks * across + wave % across) * 16 * NT, turn = wave / across % split;
  if (split == 1 && own >= C) return;
  const int64_t first = (int64_t)chunk * a.chunk;
  const int end = (int)min((int64_t)adapted, first + a.chunk);
  const float *ht[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) ht[j] = side.ht + (int64_t)min(r0 + 16 * j + i, rp - 1) * a.tokens;  // (past the ranks: not stored)
  for (int p0 = (int)min((int64_t)adapted, first); p0 < end;) {
    const int ad = owner[p0], p1 = min(end, starts[ad + 1]);
    v4f acc[E][NT];
    auto clear_sums = [&] {
#pragma unroll
      for (int c = 0; c < E; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear_sums();
    // (nothing behind the adapter's tokens gets in, whatever it holds)
    auto load = [&](int p, OuterStep<DT, NT> &s) {
      const int at = p + g * E;
      const bool inside = p + kStep <= p1;
      const elem *row[E];
#pragma unroll
      for (int e = 0; e < E; ++e) row[e] = reinterpret_cast<const elem *>(side.x) + (int64_t)order[min(at + e, p1 - 1)] * side.ldx;
#pragma unroll
      for (int e = 0; e < E; ++e)
        s.rows[e] = SMALL ? load_each<DT, E>(row[e], c0, C) : load_whole<DT, E>(row[e] + c0);
      if (inside) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < E / 4; ++k) s.h[j][k] = *reinterpret_cast<const u32x4_u *>(ht[j] + at + 4 * k);
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float v = ht[j][min(at + e, p1 - 1)];
            s.h[j][e >> 2][e & 3] = at + e < p1 ? __float_as_uint(v) : 0u;
          }
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (at + e >= p1) clear<DT, E>(s.rows[e]);
      }
    };
    auto multiply = [&](const OuterStep<DT, NT> &s, auto careful) {
      u32x4 hp[NT][kParts];
      if constexpr (DT != F8LIN_FP32) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float v[E];
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = __uint_as_float(s.h[j][e >> 2][e & 3]);
          h_parts_of<F8LIN_BF16, E>(v, reinterpret_cast<uint32_t *>(hp[j]));
        }
      }
#pragma unroll
      for (int c = 0; c < E; ++c) {
        u32x4 xf = pick<DT, E>(s.rows, c);
        if constexpr (DT == F8LIN_FP32) {
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[c][j] = mma<DT>(xf, s.h[j][0], acc[c][j]);
        } else {
          u32x4 xl;
          if constexpr (DT == F8LIN_FP16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t hi, lo;
              split_f16(xf[e], hi, lo);
              xf[e] = hi, xl[e] = lo;
            }
          }
#pragma unroll
          for (int k = 0; k < kParts; ++k) {
            if constexpr (careful) {
#pragma unroll
              for (int e = 0; e < 4; ++e) xf[e] = k > 0 ? finite_of<F8LIN_BF16>(xf[e]) : xf[e];
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[c][j] = mma<F8LIN_BF16>(xf, hp[j][k], acc[c][j]);
              if constexpr (DT == F8LIN_FP16) {
                u32x4 h = hp[j][k];
                if constexpr (careful) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) h[e] = finite_of<F8LIN_BF16>(h[e]);
                }
                acc[c][j] = mma<F8LIN_BF16>(xl, h, acc[c][j]);
              }
            }
          }
          if constexpr (careful) __builtin_amdgcn_sched_barrier(0);  // (registers: a column at a time)
        }
      }
    };
    OuterStep<DT, NT> s0, s1;
    const int step = split * kStep, q0 = p0 + turn * kStep;
    if (q0 < p1) load(q0, s0);
    for (int p = q0; p < p1; p += 2 * step) {
      if (p + step < p1) load(p + step, s1);
      multiply(s0, std::false_type{});
      if (p + step >= p1) break;
      if (p + 2 * step < p1) load(p + 2 * step, s0);
      multiply(s1, std::false_type{});
    }
    if constexpr (DT != F8LIN_FP32) {
      bool nan = false;
#pragma unroll
      for (int c = 0; c < E; ++c) nan |= has_nan(acc[c]);
      if (__any(nan)) {
        clear_sums();
#pragma unroll 1
        for (int p = q0; p < p1; p += step) {
          load(p, s0);
          multiply(s0, std::true_type{});
        }
      }
    }
    // the token parts' sums, in their order
    if (split > 1) {
      __syncthreads();  // (of the last adapter's reads)
      if (turn > 0) {
#pragma unroll
        for (int c = 0; c < E; ++c)
#pragma unroll
          for (int j = 0; j < NT; ++j) join[wave][c * NT + j][lane] = acc[c][j];
      }
      __syncthreads();
      if (turn > 0) {
        p0 = p1;
        continue;
      }
      for (int t = 1; t < split; ++t)
#pragma unroll
        for (int c = 0; c < E; ++c)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[c][j] += join[wave + t * across][c * NT + j][lane];
    }
    // lane (i, g) holds rank r0 + 16 j + i of columns E * (4 g + q) + c of the wave's
    const bool whole = starts[ad] >= first && starts[ad + 1] <= first + a.chunk;
    const int slot = 2 * chunk + (starts[ad] >= first ? 1 : 0);
    const int64_t elems = (int64_t)a.rank * C;
    float *const part = side.part + (int64_t)slot * elems;
    elem *const d = reinterpret_cast<elem *>(side.d) + (int64_t)ad * elems;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = r0 + 16 * j + i;
      if (r >= a.rank) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = (int)cw + E * (4 * g + q), n = (int)min((int64_t)E, C - col), n0 = (int)own - col;
        // (a side has at most 256 * 2^22 elements: 32-bit offsets)
        uint32_t at = side.d_t ? (uint32_t)col * a.rank + r : (uint32_t)r * (uint32_t)C + col;
        const uint32_t step = side.d_t ? a.rank : 1;
        if (whole) {
#pragma unroll
          for (int c = 0; c < E; ++c, at += step)
            if (c >= n0 && c < n) d[at] = (elem)f32_to_elem(acc[c][j][q], DT);
        } else {
#pragma unroll
          for (int c = 0; c < E; ++c, at += step)
            if (c >= n0 && c < n) part[at] = acc[c][j][q];
        }
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

// How an outer product's four waves lie, and blocks of ranks beside them.
struct LoraOuterShape {
  int across, split, side_by_side, rblocks;
};
LoraOuterShape lora_outer_shape(int64_t tokens, int rank) {
  LoraOuterShape o;
  const int blocks = rank <= 16 ? 1 : (rank + 31) / 32;
  o.across = blocks > 2 ? 4 : blocks;
  o.rblocks = (blocks + o.across - 1) / o.across;
  // many tokens: waves side by side, so that a workgroup reads 1 KB of a row (65535 x 4096, rank 16: dA and dB with
  // their G 318 us, split over the tokens 341); else parts of the tokens, so that there are fewer chunks for the same
  // number of waves (4096 tokens of rank 32: 44 us, side by side 58)
  o.split = tokens >= 32768 ? 1 : 4 / o.across;
  o.side_by_side = 4 / (o.across * o.split);
  return o;
}

// Tiles along the grid's y (which the kernels stride over).
dim3 tile_grid(int64_t x, int max_tiles, int z) { return dim3((unsigned)x, (unsigned)std::min(max_tiles, 65535), (unsigned)z); }

template <int DT, bool W_T, int M, bool SMALL>
void down_rows(const LoraDown &a, hipStream_t s) {
  const int nt = rank_tiles(a.rank), rblocks = (a.rank + 16 * nt - 1) / (16 * nt);
  const dim3 grid = tile_grid(a.parts * (lora_tile(a.tokens) / (16 * M)), a.max_tiles, rblocks);
  if (nt == 1) lora_down_kernel<DT, 1, W_T, M, 4, SMALL><<<grid, 256, 0, s>>>(a);
  else if (nt == 2) lora_down_kernel<DT, 2, W_T, M, 4, SMALL><<<grid, 256, 0, s>>>(a);
  else lora_down_kernel<DT, 4, W_T, M, 4, SMALL><<<grid, 256, 0, s>>>(a);
}
template <int DT, bool W_T>
void down_typed(const LoraDown &a, hipStream_t s) {
  // 64 rows a workgroup read W once for four times the rows; fewer where that leaves the chip empty (70 tiles of rank
  // 32: 16 rows a workgroup 15 us, 64 rows 26; 135 of rank 64: 16 rows 42, 32 rows 27, 64 rows 35; 1029 of rank 16: 32
  // rows 98, 64 rows 92)
  const int64_t groups = (int64_t)a.max_tiles * ((a.rank + 63) / 64);
  if (a.cols < 8 * kE<DT>) down_rows<DT, W_T, 1, true>(a, s);
  else if (lora_tile(a.tokens) == 16 || groups < 128) down_rows<DT, W_T, 1, false>(a, s);
  else if (groups < 512) down_rows<DT, W_T, 2, false>(a, s);
  else down_rows<DT, W_T, 4, false>(a, s);
  if (a.parts_out && a.ht) {
    const int64_t grid = (int64_t)((a.tokens + 15) / 16) * (lora_rank_pad(a.rank) / 16);
    lora_sum_kernel<<<(unsigned)grid, 256, 0, s>>>(a);
  }
}
template <int DT, bool W_T, int NB, int KB>
void up_blocks(const LoraUp &a, const dim3 grid, hipStream_t s) {
  const bool whole = a.rank % (DT == F8LIN_FP32 ? 16 : KB) == 0;
  if (whole) lora_up_kernel<DT, W_T, NB, KB, false, true><<<grid, 256, 0, s>>>(a);
  else lora_up_kernel<DT, W_T, NB, KB, false, false><<<grid, 256, 0, s>>>(a);
}
template <int DT, bool W_T, int KB>
void up_few_blocks(const LoraUp &a, hipStream_t s) {
  auto grid = [&](int groups) { return tile_grid((a.cols + 256 * groups - 1) / (256 * groups), a.max_tiles, 1); };
  const bool whole = a.rank % (DT == F8LIN_FP32 ? 16 : KB) == 0;
  // two blocks of columns a wave where there are workgroups enough for either (64 tokens of as many adapters, 4096 to
  // 14336: forward with one 21.6 us, with two 21.2; dx 15.6 and 16.7)
  const bool many = (a.cols + 255) / 256 * a.max_tiles >= 1024;
  if (a.cols < 64) lora_up_few_kernel<DT, W_T, 1, KB, true, false><<<grid(1), 256, 0, s>>>(a);
  else if (!whole) lora_up_few_kernel<DT, W_T, 1, KB, false, false><<<grid(1), 256, 0, s>>>(a);
  else if (many) lora_up_few_kernel<DT, W_T, 2, KB, false, true><<<grid(2), 256, 0, s>>>(a);
  else lora_up_few_kernel<DT, W_T, 1, KB, false, true><<<grid(1), 256, 0, s>>>(a);
}
template <int DT, bool W_T>
void up_typed(const LoraUp &a, hipStream_t s) {
  constexpr int kTwo = DT == F8LIN_FP32 ? 2 : 1;  // (its blocks have 16 ranks)
  const dim3 grid = tile_grid((a.cols + 255) / 256, a.max_tiles, 1);
  if (a.parts_in) {
    if (a.rank <= 16) up_few_blocks<DT, W_T, 16>(a, s);
    else up_few_blocks<DT, W_T, 32>(a, s);
  } else if (a.cols < 64) {
    if (a.rank <= 16) lora_up_kernel<DT, W_T, 1, 16, true, false><<<grid, 256, 0, s>>>(a);
    else lora_up_kernel<DT, W_T, 0, 32, true, false><<<grid, 256, 0, s>>>(a);
  } else if (a.rank <= 16) {
    up_blocks<DT, W_T, 1, 16>(a, grid, s);
  } else if (a.rank <= 32) {
    up_blocks<DT, W_T, kTwo, 32>(a, grid, s);
  } else if (a.rank <= 64) {
    up_blocks<DT, W_T, 2 * kTwo, 32>(a, grid, s);
  } else {
    up_blocks<DT, W_T, 0, 32>(a, grid, s);
  }
}
template <int DT>
void outer_typed(LoraOuter a, hipStream_t s) {
  const LoraOuterShape shape = lora_outer_shape(a.tokens, a.rank);
  const int64_t cols = shape.side_by_side * 16 * kE<DT>;
  a.across = shape.across, a.split = shape.split;
  a.units = a.chunks * shape.rblocks;
  bool small = false;
  for (int i = 0; i < 2; ++i) {
    a.side[i].blocks = a.side[i].d ? (int)((a.side[i].cols + cols - 1) / cols) : 0;
    a.side[i].join_blocks = a.side[i].d ? (a.rank * a.side[i].cols + 1023) / 1024 : 0;
    small = small || (a.side[i].d && a.side[i].cols < 16 * kE<DT>);
  }
  const int64_t grid = (int64_t)(a.side[0].blocks + a.side[1].blocks) * a.units;
  if (grid > 0) {
    if (a.rank <= 16) {
      if (small) lora_outer_kernel<DT, 1, true><<<(unsigned)grid, 256, 0, s>>>(a);
      else lora_outer_kernel<DT, 1, false><<<(unsigned)grid, 256, 0, s>>>(a);
    } else {
      if (small) lora_outer_kernel<DT, 2, true><<<(unsigned)grid, 256, 0, s>>>(a);
      else lora_outer_kernel<DT, 2, false><<<(unsigned)grid, 256, 0, s>>>(a);
    }
  }
  const int64_t joins = (a.side[0].join_blocks + a.side[1].join_blocks) * a.adapters;
  if (joins > 0) lora_outer_join_kernel<DT><<<grid_of(joins), 256, 0, s>>>(a);
}

}  // namespace

int lora_parts(int64_t tokens, int adapters, int64_t cols, int rank) {
  if (!lora_split(tokens)) return 1;
  // enough workgroups for the chip, each with two 64-column blocks a wave at least (64 single tokens, 4096 columns: four
  // parts 6.0 us, two 7.8; more parts are more to read for the next kernel)
  const int64_t groups = std::max<int64_t>(1, lora_max_tiles(tokens, adapters)) * ((rank + 63) / 64);
  const int64_t want = (256 + groups - 1) / groups, most = (cols + 511) / 512;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), 8));
}

int lora_chunk(int64_t tokens, int64_t K, int64_t N, int rank) {
  // a partial sum is written and read in binary32 for every chunk: chunks of at least 16 * rank tokens (2048 at most)
  // keep that to a quarter of the data's bytes, at the price of workgroups where there are few features (4096 tokens,
  // 1024 x 1024, rank 128: 32 of them); else workgroups for the chip (dA and dB with their G, 65535 tokens of rank 16 in
  // 512 workgroups 318 us, in 1024 365; 8192 of rank 64 from 4096 to 14336, split over the tokens, in 1024 314, in 2048
  // 324)
  const LoraOuterShape o = lora_outer_shape(tokens, rank);
  const int64_t cols = 128 * o.side_by_side, per_chunk = ((K + cols - 1) / cols + (N + cols - 1) / cols) * o.rblocks;
  const int64_t chunks = std::max<int64_t>(1, (o.split == 1 ? 512 : 1024) / std::max<int64_t>(1, per_chunk));
  const int64_t each = std::max((tokens + chunks - 1) / chunks, (int64_t)16 * std::min(rank, 128));
  return (int)std::min<int64_t>(4096, std::max<int64_t>(128, (each + 127) / 128 * 128));
}

hipError_t launch_lora_plan(const void *index, bool wide, int tokens, int adapters, int *plan, hipStream_t stream) {
  if (adapters <= 255) lora_plan_kernel<16, 255><<<1, 1024, 0, stream>>>(index, wide, tokens, adapters, plan);
  else lora_plan_kernel<16, kLoraMaxAdapters><<<1, 1024, 0, stream>>>(index, wide, tokens, adapters, plan);
  return hipGetLastError();
}

hipError_t launch_lora_down(const LoraDown &a, int dtype, bool w_t, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  if (dtype == F8LIN_BF16) w_t ? down_typed<F8LIN_BF16, true>(a, stream) : down_typed<F8LIN_BF16, false>(a, stream);
  else if (dtype == F8LIN_FP16) w_t ? down_typed<F8LIN_FP16, true>(a, stream) : down_typed<F8LIN_FP16, false>(a, stream);
  else w_t ? down_typed<F8LIN_FP32, true>(a, stream) : down_typed<F8LIN_FP32, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_lora_up(const LoraUp &a, int dtype, bool w_t, hipStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return hipSuccess;
  if (dtype == F8LIN_BF16) w_t ? up_typed<F8LIN_BF16, true>(a, stream) : up_typed<F8LIN_BF16, false>(a, stream);
  else if (dtype == F8LIN_FP16) w_t ? up_typed<F8LIN_FP16, true>(a, stream) : up_typed<F8LIN_FP16, false>(a, stream);
  else w_t ? up_typed<F8LIN_FP32, true>(a, stream) : up_typed<F8LIN_FP32, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_lora_outer(const LoraOuter &a, int dtype, hipStream_t stream) {
  if (dtype == F8LIN_BF16) outer_typed<F8LIN_BF16>(a, stream);
  else if (dtype == F8LIN_FP16) outer_typed<F8LIN_FP16>(a, stream);
  else outer_typed<F8LIN_FP32>(a, stream);
  return hipGetLastError();
}

}  // namespace f8lin

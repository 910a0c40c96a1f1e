// MXFP4 product  C (M, N) = A (M, K) . B (N, K)^T (+ bias), operands as e2m1
// codes with an e8m0 scale per 32 elements of K, fp32 accumulation.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes four MX blocks of 32: lane l feeds
// the 16 code bytes and the one scale byte of block l / 16 of row l % 16, so
// a block's scale is applied by the matrix core and costs no instruction.
// The instruction runs on C^T (B as its first operand): lane l then holds
// columns 4 (l / 16) .. + 3 of row l % 16.
//
// Tiled kernel (four waves, 2 x 2, wave tile BM / 2 x BN / 2):
//   * A K block is 128 code bytes of a row (256 elements, two MFMA steps), in
//     two LDS stages filled by buffer_load ... lds; the scales come 16 bytes
//     of a row (two K blocks) at a time into a ring of two.
//   * Step 0 of a block runs from registers while step 1's fragments are read;
//     then one barrier says that the stage is free and that the next block is
//     resident; the rest of step 0 and step 1 copy the block after that and
//     read the next block's step-0 fragments.
//   * The copies follow a cursor of their own, two K blocks ahead, that walks
//     on into the next output tile: a tile's first blocks arrive while the one
//     before is finished and stored.
//   * Stores go straight from the accumulators: v_permlane16_swap of two
//     16-column blocks gives every lane eight adjacent columns.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

struct MxProblem {
  const uint8_t *a, *as, *b, *bs;
  void *c;           // splits > 1: splits x (M, N) fp32 partial products
  const void *bias;
  int64_t lda, lsa, ldb, lsb;
  int M, N, nb;      // nb: MX blocks of K
  int c_dtype, bias_dtype;
  int tiles_m, tiles_n, splits, group;
};
struct MxBatch {
  MxProblem p[kMxMaxGemms];
  int count;
};

__device__ __forceinline__ v8i frag8(const u32x4 &a) {
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
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

constexpr int kBlockBytes = 128;  // codes of a row in one K block: 256 elements, 8 MX blocks
constexpr int kBlocksPerK = kBlockBytes / 16;
constexpr int kXcds = 8;
constexpr int kCUs = 256;
// A tile's byte range is below 2^31 (at most 256 rows of 2^22 bytes), so this
// offset lies outside it, also with a row offset added.
constexpr int kOutOfRange = (int)0x80000000u;

constexpr int waitcnt(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

// (tile-row, tile-column) of a local tile index: groups of G tile-rows, each
// walked column by column, so that the tiles an XCD runs at once form a
// compact patch whose operand slices its L2 shares.
__device__ __forceinline__ void mx_tile_coords(int local, int G, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int gsize = G * tiles_n;
  const int grp = local / gsize, in = local % gsize;
  const int gm = min(G, tiles_m - grp * G);
  tm = grp * G + in % gm;
  tn = in / gm;
}

// One output tile (of one K range) of one problem.
struct Item {
  int pi, m0, n0, range;
  int kb0, nkb;  // first K block, number of K blocks (at least one)
  int nb;        // MX blocks from kb0 to the end of the range
};

template <int BM, int BN, int MINB>
__global__ __launch_bounds__(256, MINB) void mx_gemm_tiled_kernel(const MxBatch batch) {
  constexpr int MI = BM / 32, NJ = BN / 32;  // 16 x 16 blocks of a wave tile
  constexpr int NM = MI * NJ, NR = MI + NJ;  // MFMAs, and fragment reads, per step of 128 elements
  constexpr int NC = MI + NJ;                // 1 KB copies per wave and K block
  constexpr int OPA = BM * kBlockBytes, STB = OPA + BN * kBlockBytes;
  constexpr int SCA = BM * 16, SCB = SCA + BN * 16;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STB + 2 * SCB];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);

  // XCD x (workgroup index mod 8) owns a contiguous eighth of each problem's
  // item list; its workgroups take every wx-th item of it.
  const int xcd = (int)blockIdx.x % kXcds;
  const int nwg = (int)gridDim.x, wx = nwg / kXcds + (xcd < nwg % kXcds ? 1 : 0);
  auto share = [&](int i, int &st, int &ln) {
    const int T = i < batch.count ? batch.p[i].tiles_m * batch.p[i].tiles_n * batch.p[i].splits : 0;
    const int per = T / kXcds, rem = T % kXcds;
    st = xcd * per + min(xcd, rem);
    ln = per + (xcd < rem ? 1 : 0);
  };
  static_assert(kMxMaxGemms == 2, "two item lists");
  int st0, ln0, st1, ln1;
  share(0, st0, ln0);
  share(1, st1, ln1);
  const int total = ln0 + ln1;
  auto decode = [&](int it) {
    Item w;
    w.pi = it < ln0 ? 0 : 1;
    const int t = it < ln0 ? st0 + it : st1 + it - ln0;
    const MxProblem &P = batch.p[w.pi];
    const int per = P.tiles_m * P.tiles_n;
    w.range = t / per;
    int tm, tn;
    mx_tile_coords(t - w.range * per, P.group, P.tiles_m, P.tiles_n, tm, tn);
    w.m0 = tm * BM;
    w.n0 = tn * BN;
    // K ranges hold whole pairs of K blocks (16 bytes of scales)
    const int nkb = (P.nb + kBlocksPerK - 1) / kBlocksPerK, np = (nkb + 1) / 2;
    w.kb0 = w.range * np / P.splits * 2;
    const int end = min((w.range + 1) * np / P.splits * 2, nkb);
    w.nkb = end - w.kb0;
    w.nb = min(end * kBlocksPerK, P.nb) - w.kb0 * kBlocksPerK;
    return w;
  };
  int it = (int)blockIdx.x / kXcds;
  if (it >= total) return;

  // ---- Copies.  LDS slot s (16 bytes) of an operand's stage belongs to row
  // s / 8 and holds the row's place (s % 8) ^ ((row / 2) % 8); places p and
  // p + 4 (p < 4) hold chunks 2 p and 2 p + 1.  A lane's two steps read places
  // g and g + 4 -- free of bank conflicts -- and need the adjacent scale bytes
  // 2 g and 2 g + 1.  Copy k of a wave covers 8 of its rows; its chunk is one
  // of two per lane (k even / odd).
  int chunk[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = (lane >> 3) + 8 * e, p = (lane & 7) ^ ((row >> 1) & 7);
    chunk[e] = 2 * (p & 3) + (p >> 2);
  }
  int c_it = it, c_kb = 0, c_pair = 0;  // the cursor: item, K block of it, pairs of scales copied
  Item ci = decode(it);
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  int va[2], vb[2], vsa, vsb, step_a, step_b, step_sa, step_sb;
  auto set_copy_item = [&](bool live) {
    const MxProblem &P = batch.p[ci.pi];
    const int rows_a = min(BM, P.M - ci.m0), rows_b = min(BN, P.N - ci.n0);
    ra = __builtin_amdgcn_make_buffer_rsrc((void *)(P.a + ci.m0 * P.lda + ci.kb0 * kBlockBytes), (short)0,
                                           rows_a * (int)P.lda - ci.kb0 * kBlockBytes, 0x00020000);
    rb = __builtin_amdgcn_make_buffer_rsrc((void *)(P.b + ci.n0 * P.ldb + ci.kb0 * kBlockBytes), (short)0,
                                           rows_b * (int)P.ldb - ci.kb0 * kBlockBytes, 0x00020000);
    rsa = __builtin_amdgcn_make_buffer_rsrc((void *)(P.as + ci.m0 * P.lsa), (short)0, rows_a * (int)P.lsa, 0x00020000);
    rsb = __builtin_amdgcn_make_buffer_rsrc((void *)(P.bs + ci.n0 * P.lsb), (short)0, rows_b * (int)P.lsb, 0x00020000);
    step_a = 16 * (int)P.lda;
    step_b = 16 * (int)P.ldb;
    step_sa = 64 * (int)P.lsa;
    step_sb = 64 * (int)P.lsb;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      va[e] = live ? (wave * (BM / 4) + (lane >> 3) + 8 * e) * (int)P.lda + 16 * chunk[e] : kOutOfRange;
      vb[e] = live ? (wave * (BN / 4) + (lane >> 3) + 8 * e) * (int)P.ldb + 16 * chunk[e] : kOutOfRange;
    }
    vsa = live ? lane * (int)P.lsa : kOutOfRange;
    vsb = live ? lane * (int)P.lsb : kOutOfRange;
  };
  // offsets of the cursor's K block: chunks past the range's MX blocks lie
  // outside the buffer and read as zero codes
  int oa[2], ob[2];
  auto mask_copies = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool ok = c_kb * kBlocksPerK + chunk[e] < ci.nb;
      oa[e] = ok ? va[e] : kOutOfRange;
      ob[e] = ok ? vb[e] : kOutOfRange;
    }
  };
  // copy q (A: 0 .. MI - 1, then B) of the cursor's block into a stage
  auto copy = [&](int stage, int q) {
    const bool b = q >= MI;
    const int k = b ? q - MI : q;
    uint8_t *dst = smem + stage * STB + (b ? OPA + (wave * NJ + k) * 1024 : (wave * MI + k) * 1024);
    int v = b ? ob[k & 1] : oa[k & 1];
    if (k >> 1) {  // (opaque, so that no offset is held in a register of its own across the loop)
      const int st = (k >> 1) * (b ? step_b : step_a);
      asm volatile("v_add_u32 %0, %1, %2" : "=v"(v) : "s"(st), "v"(v));
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rb : ra, (lds_void *)dst, 16, v, c_kb * kBlockBytes, 0, 0);
  };
  // the scales of the cursor's block and the one after: 64 rows per copy
  auto copy_scales = [&]() {
    uint8_t *dst = smem + 2 * STB + (c_pair & 1) * SCB;
    const int so = (ci.kb0 + c_kb) * kBlocksPerK;
#pragma unroll
    for (int s0 = 0; s0 < (BM + BN) / 64; s0 += 4) {
      const int s = s0 + wave;
      if (s < BM / 64)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void *)(dst + s * 1024), 16, vsa + s * step_sa, so, 0, 0);
      else if (s < (BM + BN) / 64)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)(dst + s * 1024), 16, vsb + (s - BM / 64) * step_sb,
                                                 so, 0, 0);
    }
    ++c_pair;
  };
  auto advance = [&]() {
    if (++c_kb >= ci.nkb) {
      c_it += wx;
      c_kb = 0;
      if (c_it < total) ci = decode(c_it);
      set_copy_item(c_it < total);
    }
    mask_copies();
  };

  // ---- Fragments
  int base[2][2];  // [operand][step], within a stage
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int place = ((g + 4 * s) ^ ((r >> 1) & 7)) * 16;
    base[0][s] = (wm + r) * kBlockBytes + place;
    base[1][s] = OPA + (wn + r) * kBlockBytes + place;
  }
  const int sbase_a = 2 * STB + (wm + r) * 16 + 2 * g, sbase_b = 2 * STB + SCA + (wn + r) * 16 + 2 * g;
  u32x4 fa[2][MI], fb[2][NJ];
  int sa[MI], sb[NJ], sa_n[MI], sb_n[NJ];
  auto read = [&](int stage, int set, int k) {  // B's fragments first: the first MFMAs need them all
    const int b = k == 0 || k > NJ ? 0 : 1, f = k == 0 ? 0 : (b ? k - 1 : k - NJ);
    const u32x4 v = *reinterpret_cast<const u32x4 *>(smem + stage * STB + base[b][set] + f * 2048);
    if (b) fb[set][f] = v;
    else fa[set][f] = v;
  };
  auto read_scale = [&](int off, int k) {
    const int f = k < MI ? k : k - MI;
    const int v = *reinterpret_cast<const uint16_t *>(smem + (k < MI ? sbase_a : sbase_b) + off + f * 256);
    if (k < MI) sa_n[f] = v;
    else sb_n[f] = v;
  };
  v4f acc[MI][NJ];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };

  // scale bytes past the range's MX blocks may be anything (NaN among them): zero
  auto mask_scales = [&](int left) {
    if (left < kBlocksPerK) {
      const int have = left - 2 * g;
      const int m = have >= 2 ? 0xFFFF : (have == 1 ? 0xFF : 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) sa_n[i] &= m;
#pragma unroll
      for (int j = 0; j < NJ; ++j) sb_n[j] &= m;
    }
  };

  // ---- Output of a finished tile; returns whether exactly NST stores were issued by every wave
  constexpr int NST16 = NM / 2, NST32 = NM;
  auto store_tile = [&](const Item &w) -> int {
    const MxProblem &P = batch.p[w.pi];
    const int M = P.M, N = P.N;
    const bool partial = P.splits > 1;
    const int dt = partial ? F8LIN_FP32 : P.c_dtype;
    const bool inside = w.m0 + BM <= M && w.n0 + BN <= N;
    const int row0 = w.m0 + wm + r;
    if (P.bias && !partial) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int col = w.n0 + wn + 16 * j + 4 * g + v;
          const float b = col < N ? load_elem(P.bias, col, P.bias_dtype) : 0.0f;
#pragma unroll
          for (int i = 0; i < MI; ++i) acc[i][j][v] += b;
        }
    }
    if (dt == F8LIN_FP32) {
      float *c = reinterpret_cast<float *>(P.c) + (partial ? (int64_t)w.range * M * N : 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int row = row0 + 16 * i;
        float *cr = c + (int64_t)row * N + w.n0 + wn + 4 * g;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int left = N - (w.n0 + wn + 4 * g + 16 * j);
          if (inside || (row < M && left >= 4)) {
            *reinterpret_cast<u32x4_u *>(cr + 16 * j) = __builtin_bit_cast(u32x4, acc[i][j]);
          } else if (row < M) {
#pragma unroll
            for (int v = 0; v < 3; ++v)
              if (v < left) cr[16 * j + v] = acc[i][j][v];
          }
        }
      }
      return inside ? 2 : 0;
    }
    uint16_t *c = reinterpret_cast<uint16_t *>(P.c);
    auto put = [&](auto BF) {
      auto pack = [&](float x, float y) -> uint32_t {
        if constexpr (decltype(BF)::value)
          return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{x, y}, bf16x2_t));
        else
          return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y) << 16;
      };
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int row = row0 + 16 * i;
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          // lane group g: columns 8 (g / 2) .. + 7 of block j + g % 2
          const auto lo = __builtin_amdgcn_permlane16_swap(pack(acc[i][j][0], acc[i][j][1]),
                                                           pack(acc[i][j + 1][0], acc[i][j + 1][1]), false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(pack(acc[i][j][2], acc[i][j][3]),
                                                           pack(acc[i][j + 1][2], acc[i][j + 1][3]), false, false);
          const u32x4 o = {lo[0], hi[0], lo[1], hi[1]};
          const int col = w.n0 + wn + 16 * (j + (g & 1)) + 8 * (g >> 1);
          uint16_t *dst = c + (int64_t)row * N + col;
          if (inside || (row < M && col + 8 <= N)) {
            *reinterpret_cast<u32x4_u *>(dst) = o;
          } else if (row < M) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              if (col + v < N) dst[v] = (uint16_t)(o[v >> 1] >> (16 * (v & 1)));
          }
        }
      }
    };
    if (dt == F8LIN_BF16) put(std::true_type());
    else put(std::false_type());
    return inside ? 1 : 0;
  };

  // ---- Prologue: blocks 0 and 1 of the stream
  set_copy_item(true);
  mask_copies();
  copy_scales();
#pragma unroll
  for (int q = 0; q < NC; ++q) copy(0, q);
  advance();
  if (!(c_kb & 1)) copy_scales();
#pragma unroll
  for (int q = 0; q < NC; ++q) copy(1, q);
  advance();
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
  __builtin_amdgcn_s_barrier();
  Item cur = decode(it);
  it += wx;
  Item nxt = it < total ? decode(it) : cur;
  int kb = 0, stage = 0, r_pair = 0, stored = 0;
#pragma unroll
  for (int k = 0; k < NR; ++k) read(0, 0, k);
#pragma unroll
  for (int k = 0; k < NR; ++k) read_scale(0, k);
  mask_scales(cur.nb);
#pragma unroll
  for (int i = 0; i < MI; ++i) sa[i] = sa_n[i];
#pragma unroll
  for (int j = 0; j < NJ; ++j) sb[j] = sb_n[j];

  // Slots of a block's 2 NM MFMAs: step-1 fragments are read over the first
  // half of step 0; the barrier follows at slot TB; copies go out from there,
  // one every CG MFMAs; step 1 reads the next block's step-0 fragments and
  // scales.
  constexpr int TB = NM * 5 / 8;
  constexpr int CG = NM >= 64 ? 2 : 1;
  constexpr int RG = NM / 2 / NR;  // MFMAs per fragment read
  static_assert(RG >= 1 && TB + NC * CG < 2 * NM, "schedule");
  for (;;) {
   clear();
   for (kb = 0; kb < cur.nkb; ++kb) {
    const bool last = kb + 1 == cur.nkb;
    int q = 0;
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      const int i = t / NJ, j = t % NJ;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[0][j]), frag8(fa[0][i]), acc[i][j], 4, 4, 0,
                                                                   sb[j], 0, sa[i]);
      if (t % RG == 0 && t / RG < NR) read(stage, 1, t / RG);
      if (t == TB) {
        // this wave has read the whole stage and has its copies of the next
        // block (a tile stored in between: its stores may still be under way)
        if (stored == 0) __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
        else if (stored == 1) __builtin_amdgcn_s_waitcnt(waitcnt(NST16, 0));
        else __builtin_amdgcn_s_waitcnt(waitcnt(NST32 > 63 ? 63 : NST32, 0));
        stored = 0;
        __builtin_amdgcn_s_barrier();
        if (!(c_kb & 1)) copy_scales();
      }
      if (t > TB && (t - TB - 1) % CG == 0 && q < NC) copy(stage, q++);
      __builtin_amdgcn_sched_barrier(0);
    }
    const int nkb_next = last ? 0 : kb + 1;
    if (!(nkb_next & 1)) ++r_pair;
    const int soff = (r_pair & 1) * SCB + (nkb_next & 1) * 8;
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      const int i = t / NJ, j = t % NJ;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[1][j]), frag8(fa[1][i]), acc[i][j], 4, 4, 1,
                                                                   sb[j], 1, sa[i]);
      if (t % RG == 0 && t / RG < NR) {
        read(stage ^ 1, 0, t / RG);
        read_scale(soff, t / RG);
      }
      if ((NM + t - TB - 1) % CG == 0 && q < NC) copy(stage, q++);
      __builtin_amdgcn_sched_barrier(0);
    }
    advance();
    mask_scales(last ? nxt.nb : cur.nb - (kb + 1) * kBlocksPerK);
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = sa_n[i];
#pragma unroll
    for (int j = 0; j < NJ; ++j) sb[j] = sb_n[j];
    stage ^= 1;
   }
   stored = __builtin_amdgcn_readfirstlane(store_tile(cur));
   if (it >= total) break;
   cur = nxt;
   it += wx;
   if (it < total) nxt = decode(it);
  }
  // (the cursor's last copies fetch nothing but still write zeros into LDS)
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
}

// C = sum over ranges of the fp32 partial products, in range order (+ bias), rounded.
__global__ __launch_bounds__(256) void mx_split_reduce_kernel(const float *__restrict__ part, int splits, int64_t mn, int N,
                                                              void *c, int c_dtype, const void *bias, int bias_dtype) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < mn; i += (int64_t)gridDim.x * 256) {
    float s = part[i];
    for (int k = 1; k < splits; ++k) s += part[(int64_t)k * mn + i];
    if (bias) s += load_elem(bias, i % N, bias_dtype);
    store_elem(c, i, s, c_dtype);
  }
}

// K = 0: C is the bias, or zero.
__global__ __launch_bounds__(256) void mx_fill_kernel(void *c, int c_dtype, int64_t mn, int N, const void *bias,
                                                      int bias_dtype) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < mn; i += (int64_t)gridDim.x * 256)
    store_elem(c, i, bias ? load_elem(bias, i % N, bias_dtype) : 0.0f, c_dtype);
}

}  // namespace

size_t mx_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
bool mx_linear_fused(int64_t, int64_t, int64_t) { return false; }
hipError_t launch_mx_linear(const MxLinear &, hipStream_t) { return hipErrorInvalidValue; }

hipError_t launch_mx_gemms(const MxGemm *d, int count, void *, size_t, hipStream_t stream) {
  MxBatch b = {};
  int64_t big = 0;
  for (int i = 0; i < count; ++i) {
    if (d[i].M == 0 || d[i].N == 0) continue;
    if (d[i].K == 0) {
      const int64_t mn = d[i].M * d[i].N;
      mx_fill_kernel<<<(unsigned)std::min<int64_t>((mn + 255) / 256, 8192), 256, 0, stream>>>(
          d[i].c, d[i].c_dtype, mn, (int)d[i].N, d[i].bias, d[i].bias_dtype);
      continue;
    }
    MxProblem &p = b.p[b.count++];
    p = MxProblem{d[i].a.codes, d[i].a.scales, d[i].b.codes, d[i].b.scales, d[i].c,     d[i].bias,
                  d[i].a.ld,    d[i].a.scale_ld, d[i].b.ld,  d[i].b.scale_ld, (int)d[i].M, (int)d[i].N,
                  (int)((d[i].K + kMxBlock - 1) / kMxBlock), d[i].c_dtype, d[i].bias_dtype, 0, 0, 1, 4};
    big += ((d[i].M + 255) / 256) * ((d[i].N + 255) / 256);
  }
  if (b.count == 0) return hipGetLastError();
  const bool use_big = big >= kCUs;
  const int bm = use_big ? 256 : 128;
  int64_t tiles = 0;
  for (int i = 0; i < b.count; ++i) {
    MxProblem &p = b.p[i];
    p.tiles_m = (p.M + bm - 1) / bm;
    p.tiles_n = (p.N + bm - 1) / bm;
    tiles += (int64_t)p.tiles_m * p.tiles_n;
  }
  if (use_big)
    mx_gemm_tiled_kernel<256, 256, 1><<<(unsigned)std::min<int64_t>(tiles, kCUs), 256, 0, stream>>>(b);
  else
    mx_gemm_tiled_kernel<128, 128, 2><<<(unsigned)std::min<int64_t>(tiles, 2 * kCUs), 256, 0, stream>>>(b);
  return hipGetLastError();
}

}  // namespace f8lin

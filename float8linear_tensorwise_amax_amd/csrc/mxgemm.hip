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
//     two LDS stages (more in small tiles) filled by buffer_load ... lds; the
//     scales come 16 bytes of a row (two K blocks) at a time into a ring.
//   * Step 0 of a block runs from registers while step 1's fragments are read;
//     then one barrier says that the stage is free and that the next block is
//     resident; the rest of step 0 and step 1 copy the block after that and
//     read the next block's step-0 fragments.
//   * The copies follow a cursor of their own, two K blocks ahead, that walks
//     on into the next output tile: a tile's first blocks arrive while the one
//     before is finished and stored.
//   * Stores go straight from the accumulators: v_permlane16_swap of two
//     16-column blocks gives every lane eight adjacent columns.
// Measured (bf16 output, random codes): 8192^3 254 us (4.3 PFLOP/s), 65536 x
// 4096 x 4096 575 us (3.8), 4096 x 4096 x 65536 462 us (4.8), 4096^3 40 us.
// The matrix cores are busy for 56% of the cycles at 8192^3 and 45% at 8192 x
// 14336 x 4096, at 1.93 GHz of 2.4.  A K block of a 256 x 256 tile takes 1.75
// us, where its 128 MFMAs a wave of 16 cycles take 1.06; what each round of
// tiles costs besides (first loads, 128 KB of stores a tile) is 8.5 us, 23% of
// it at K = 4096.  Other spacings of the reads and copies in the K block were
// within 1%, waves set apart and skewed starts 1-4% slower.  256 x 256 with
// four waves reads least LDS per MFMA: 16 KB per 64 of them.
#include <algorithm>

#include "mx_common.h"

namespace f8lin {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

struct MxProblem {
  const uint8_t *a, *as, *b, *bs;
  void *c;
  const void *bias;
  int64_t lda, lsa, ldb, lsb;
  int M, N, nb;      // nb: MX blocks of K
  int c_dtype, bias_dtype;
  int nkb;           // K blocks of 128 bytes
  int tiles, group, group_log;  // output tiles, tile-rows per group (a power of two)
  // divisors: tiles per group, tile-rows of the last group
  int group_tiles, last_rows, last_group;
  uint32_t inv_group_tiles, inv_last_rows;
};
struct MxBatch {
  MxProblem p[kMxMaxGemms];
  int count;
};
typedef __attribute__((address_space(4))) MxBatch MxBatchArg;
typedef __attribute__((address_space(4))) MxProblem MxProblemArg;

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

// n / d for 0 <= n < 2^31 with inv = min(2^32 - 1, floor(2^32 / d)) from the
// host: the estimate is at most one too small.  (A tile's coordinates are
// worked out between two tiles, where nothing hides a division.)
__device__ __forceinline__ int div_by(int n, int d, uint32_t inv) {
  const int q = (int)(((uint64_t)(uint32_t)n * inv) >> 32);
  return n - q * d >= d ? q + 1 : q;
}

// One output tile of one problem.
struct Item {
  int pi, m0, n0;
  int nkb, nb;  // K blocks (at least one), MX blocks
};

template <int BM, int BN, int NS, int MINB, int DT>
__global__ __launch_bounds__(256, MINB) void mx_gemm_tiled_kernel(const MxBatch) {
  // The problems are read where the launch put them, through the scalar
  // cache (an argument indexed at run time would be copied to scratch).
  const MxBatchArg &batch = *(const MxBatchArg *)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int MI = BM / 32, NJ = BN / 32;  // 16 x 16 blocks of a wave tile
  constexpr int NM = MI * NJ, NR = MI + NJ;  // MFMAs, and fragment reads, per step of 128 elements
  constexpr int NC = MI + NJ;                // 1 KB copies per wave and K block
  constexpr int OPA = BM * kBlockBytes, STB = OPA + BN * kBlockBytes;
  constexpr int SCA = BM * 16, SCB = SCA + BN * 16;
  // pairs of K blocks whose scales are held: those of the NS - 1 blocks yet to
  // be read and of the one being copied, each of which may be a tile's only one
  constexpr int RING = NS <= 2 ? 2 : (NS <= 4 ? 4 : 8);
  static_assert(RING >= NS, "scale ring");
  constexpr int NSC = (BM + BN + 255) / 256;  // scale copies per wave and K block
  constexpr int NCP = NC + NSC;
  static_assert((NS - 1) * NCP <= 63, "vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * STB + (RING + 1) * SCB];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);

  // XCD x (workgroup index mod 8) owns a contiguous eighth of each problem's
  // item list; its workgroups take every wx-th item of it.
  const int xcd = (int)blockIdx.x % kXcds;
  const int nwg = (int)gridDim.x, wx = nwg / kXcds + (xcd < nwg % kXcds ? 1 : 0);
  auto share = [&](int i, int &st, int &ln) {
    const int T = i < batch.count ? batch.p[i].tiles : 0;
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
    const MxProblemArg &P = batch.p[w.pi];
    // groups of `group` tile-rows, each walked column by column, so that the
    // tiles an XCD runs at once form a compact patch whose operand slices its
    // L2 shares
    const int grp = div_by(t, P.group_tiles, P.inv_group_tiles), in = t - grp * P.group_tiles;
    const bool tail = grp == P.last_group;
    const int rows = tail ? P.last_rows : P.group;
    const int tn = tail ? div_by(in, P.last_rows, P.inv_last_rows) : in >> P.group_log;
    w.m0 = (grp * P.group + in - tn * rows) * BM;
    w.n0 = tn * BN;
    w.nkb = P.nkb;
    w.nb = P.nb;
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
    const MxProblemArg &P = batch.p[ci.pi];
    const int rows_a = min(BM, P.M - ci.m0), rows_b = min(BN, P.N - ci.n0);
    ra = __builtin_amdgcn_make_buffer_rsrc((void *)(P.a + ci.m0 * P.lda), (short)0, rows_a * (int)P.lda, 0x00020000);
    rb = __builtin_amdgcn_make_buffer_rsrc((void *)(P.b + ci.n0 * P.ldb), (short)0, rows_b * (int)P.ldb, 0x00020000);
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
  // The scales of the cursor's block and the one after, 64 rows per copy, into
  // the ring; at a pair's second block the same copies read nothing and land
  // in a spare slot, so that the loop holds no branch.
  auto copy_scales = [&]() {
    const bool even = !(c_kb & 1);
    uint8_t *dst = smem + NS * STB + (even ? (c_pair & (RING - 1)) * SCB : RING * SCB);
    const int so = c_kb * kBlocksPerK, odd = even ? 0 : kOutOfRange;
    if constexpr (BM == 256 && BN == 256) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void *)(dst + wave * 1024), 16, (vsa + wave * step_sa) | odd, so,
                                               0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)(dst + SCA + wave * 1024), 16,
                                               (vsb + wave * step_sb) | odd, so, 0, 0);
    } else {
      static_assert(BM + BN <= 256, "at most one copy per wave");
      // (a wave without rows of its own copies nothing into the spare slot, so
      // that every wave has issued as many copies)
      const bool b = wave >= BM / 64, none = wave >= (BM + BN) / 64;
      const int v = none ? kOutOfRange : b ? vsb + (wave - BM / 64) * step_sb : vsa + wave * step_sa;
      uint8_t *const to = none ? smem + NS * STB + RING * SCB : dst + wave * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rsb : rsa, (lds_void *)to, 16, v | odd, so, 0, 0);
    }
    c_pair += even ? 1 : 0;
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
  const int sbase_a = NS * STB + (wm + r) * 16 + 2 * g, sbase_b = NS * STB + SCA + (wn + r) * 16 + 2 * g;
  u32x4 fa[2][MI], fb[2][NJ];
  int sa_n[MI], sb_n[NJ];
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

  // ---- Output of a finished tile.  A tile that lies inside C issues exactly
  // NST stores per wave, which the next tile's first wait allows for; one on
  // the edge waits for its stores here.
  constexpr int NST = DT == F8LIN_FP32 ? NM : NM / 2;
  auto store_tile = [&](const Item &w, auto INSIDE) __attribute__((always_inline)) {
    constexpr bool inside = decltype(INSIDE)::value;
    const MxProblemArg &P = batch.p[w.pi];
    const int M = P.M, N = P.N;
    const int row0 = w.m0 + wm + r, col0 = w.n0 + wn;
    // One row pointer, moved on from row block to row block (opaque to the
    // compiler, which would otherwise hold an address for every store).
    constexpr int ES = DT == F8LIN_FP32 ? 4 : 2;
    const int lane_col = DT == F8LIN_FP32 ? 4 * g : 16 * (g & 1) + 8 * (g >> 1);
    const int left = N - col0 - lane_col;  // columns from this lane's first one to the edge
    int64_t at = (int64_t)(uintptr_t)P.c + ((int64_t)row0 * N + col0 + lane_col) * ES;
    const int64_t step = (int64_t)16 * N * ES;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const bool row_ok = inside || row0 + 16 * i < M;
      if constexpr (DT == F8LIN_FP32) {
        float *dst = reinterpret_cast<float *>((uintptr_t)at);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if (inside || (row_ok && left >= 16 * j + 4)) {
            *reinterpret_cast<u32x4_u *>(dst + 16 * j) = __builtin_bit_cast(u32x4, acc[i][j]);
          } else if (row_ok) {
#pragma unroll
            for (int v = 0; v < 3; ++v)
              if (left > 16 * j + v) dst[16 * j + v] = acc[i][j][v];
          }
        }
      } else {
        auto pack = [&](float x, float y) -> uint32_t {
          if constexpr (DT == F8LIN_BF16)
            return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{x, y}, bf16x2_t));
          else
            return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y) << 16;
        };
        uint16_t *dst = reinterpret_cast<uint16_t *>((uintptr_t)at);
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          // lane group g: columns 8 (g / 2) .. + 7 of block j + g % 2
          const auto lo = __builtin_amdgcn_permlane16_swap(pack(acc[i][j][0], acc[i][j][1]),
                                                           pack(acc[i][j + 1][0], acc[i][j + 1][1]), false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(pack(acc[i][j][2], acc[i][j][3]),
                                                           pack(acc[i][j + 1][2], acc[i][j + 1][3]), false, false);
          const u32x4 o = {lo[0], hi[0], lo[1], hi[1]};
          if (inside || (row_ok && left >= 16 * j + 8)) {
            *reinterpret_cast<u32x4_u *>(dst + 16 * j) = o;
          } else if (row_ok) {
#pragma unroll
            for (int v = 0; v < 7; ++v)
              if (left > 16 * j + v) dst[16 * j + v] = (uint16_t)(o[v >> 1] >> (16 * (v & 1)));
          }
        }
      }
      at += step;
      asm volatile("" : "+v"(at));
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!inside) __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
  };

  // ---- Prologue: the first NS blocks of the stream
  set_copy_item(true);
  mask_copies();
#pragma unroll 1
  for (int st = 0;;) {
    copy_scales();
#pragma unroll
    for (int q = 0; q < NC; ++q) copy(st, q);
    if (++st == NS) break;
    advance();
  }
  // (with two stages all of them: no stores follow these copies, and the first
  // block's wait, which allows for a tile's stores, would let the second
  // block's copies pass)
  __builtin_amdgcn_s_waitcnt(waitcnt(NS > 2 ? (NS - 1) * NCP : 0, 15));
  __builtin_amdgcn_s_barrier();
  Item cur = decode(it);
  it += wx;
  int stage = 0, r_pair = 0;
#pragma unroll
  for (int k = 0; k < NR; ++k) read(0, 0, k);
#pragma unroll
  for (int k = 0; k < NR; ++k) read_scale(0, k);

  // Slots of a block's 2 NM MFMAs: step-1 fragments are read over the first
  // half of step 0; the barrier follows at slot TB; copies go out from there,
  // one every CG MFMAs; step 1 reads the next block's step-0 fragments and
  // scales.
  constexpr int CG = NM >= 64 ? 5 : 1;
  constexpr int RG = NM / 2 / NR > 0 ? NM / 2 / NR : 1;  // MFMAs per fragment read
  constexpr int TB = NM * 9 / 16 > (NR - 1) * RG ? NM * 9 / 16 : (NR - 1) * RG;
  static_assert(TB < NM && TB + NC * CG < 2 * NM, "schedule");
  auto block = [&](int kb) __attribute__((always_inline)) {
    // (everything that branches comes first: the compiler moves MFMAs across
    // branches, away from the reads and copies they are to run next to)
    advance();
    mask_scales(cur.nb - kb * kBlocksPerK);
    int sa[MI], sb[NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = sa_n[i];
#pragma unroll
    for (int j = 0; j < NJ; ++j) sb[j] = sb_n[j];
    int after = kb + 1;
    asm volatile("" : "+s"(after));  // (opaque: no copy of the loop for the last block)
    const int nkb_next = after == cur.nkb ? 0 : after;
    int q = 0;
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      const int i = t / NJ, j = t % NJ;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[0][j]), frag8(fa[0][i]), acc[i][j], 4, 4, 0,
                                                                   sb[j], 0, sa[i]);
      if (t % RG == 0 && t / RG < NR) read(stage, 1, t / RG);
      if (t == TB) {
        // This wave has read the whole stage and has its copies of the next
        // block.  With two stages, in a tile's first block only the last
        // tile's stores came after those copies, so they may still be under
        // way.  (The branch is out of the compiler's sight: it would move
        // MFMAs across one.)
        if constexpr (NS > 2) __builtin_amdgcn_s_waitcnt(waitcnt((NS - 2) * NCP, 0));
        else asm volatile(
            "s_waitcnt vmcnt(%1) lgkmcnt(0)\n\t"
            "s_cmp_eq_u32 %0, 0\n\t"
            "s_cbranch_scc1 .Lfirst%=\n\t"
            "s_waitcnt vmcnt(0)\n"
            ".Lfirst%=:"
            :
            : "s"(kb), "n"(NST > 63 ? 63 : NST)
            : "scc", "memory");
        __builtin_amdgcn_s_barrier();
        copy_scales();
      }
      if (t > TB && (t - TB - 1) % CG == 0 && q < NC) copy(stage, q++);
      __builtin_amdgcn_sched_barrier(0);
    }
    r_pair += nkb_next & 1 ? 0 : 1;
    const int soff = (r_pair & (RING - 1)) * SCB + (nkb_next & 1) * 8;
    const int next = stage + 1 == NS ? 0 : stage + 1;
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      const int i = t / NJ, j = t % NJ;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[1][j]), frag8(fa[1][i]), acc[i][j], 4, 4, 1,
                                                                   sb[j], 1, sa[i]);
      if (t % RG == 0 && t / RG < NR) {
        read(next, 0, t / RG);
        read_scale(soff, t / RG);
      }
      if ((NM + t - TB - 1) % CG == 0 && q < NC) copy(stage, q++);
      __builtin_amdgcn_sched_barrier(0);
    }
    stage = next;
  };
  for (;;) {
    // the sums start from the bias
    {
      const MxProblemArg &P = batch.p[cur.pi];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        v4f init = {0.0f, 0.0f, 0.0f, 0.0f};
        if (P.bias) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int col = cur.n0 + wn + 16 * j + 4 * g + v;
            init[v] = col < P.N ? load_elem(P.bias, col, P.bias_dtype) : 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = init;
      }
    }
    for (int kb = 0; kb < cur.nkb; ++kb) block(kb);
    if (cur.m0 + BM <= batch.p[cur.pi].M && cur.n0 + BN <= batch.p[cur.pi].N)
      store_tile(cur, std::true_type());
    else
      store_tile(cur, std::false_type());
    if (it >= total) break;
    cur = decode(it);
    it += wx;
  }
  // (the cursor's last copies fetch nothing but still write zeros into LDS)
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
}

// ---- Few rows (M <= 64): bound by reading B once.  A workgroup of NW waves
// owns NT x 16 rows of B (output columns), so that many workgroups stream B; the
// waves split K in 128-byte blocks (wave w takes blocks w, w + NW, ...), load
// operands straight into registers, U blocks in flight, and their partial
// sums meet in LDS (1 x 14336 x 4096: 9.7 us or 3.2 TB/s; a read of 32 MB alone
// takes 10 us here).  FUSED (X not yet quantised, M <= 16): every workgroup
// quantises X into LDS itself while its first loads of B are under way.
struct MxSkinny {
  const uint8_t *a, *as, *b, *bs;
  const void *x;
  void *c;
  const void *bias;
  int64_t lda, lsa, ldb, lsb, ldx;
  int M, N, K, nb, nkb;
  int c_dtype, bias_dtype;
};


// LDS strides of the quantised X: rows 16 bytes apart from a multiple of 128
// (bank conflicts), scales after all codes.
__host__ __device__ constexpr int fused_row(int nkb) { return nkb * kBlockBytes + 16; }
__host__ __device__ constexpr int fused_scale_row(int nkb) { return nkb * kBlocksPerK; }
// log2 of the threads that quantise a row together: 32 items a K block
__host__ __device__ constexpr int fused_row_log(int nkb, int waves) {
  int l = 5;
  while ((32 << (l - 5)) < 32 * nkb && (32 << (l - 5)) < 64 * waves) ++l;
  return l;
}
__host__ __device__ constexpr int fused_bytes(int M, int nkb) { return M * (fused_row(nkb) + fused_scale_row(nkb)); }

template <int MT, int NT, int NW, bool FUSED, int XDT, int RULE>
__global__ __launch_bounds__(64 * NW) void mx_skinny_kernel(const MxSkinny P) {
  constexpr int U = MT <= 2 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16 * NT;
  const int rows_b = min(16 * NT, P.N - n0);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void *)(P.b + n0 * P.ldb), (short)0,
                                                                      rows_b * (int)P.ldb, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc((void *)(P.bs + n0 * P.lsb), (short)0,
                                                                       rows_b * (int)P.lsb, 0x00020000);
  __amdgpu_buffer_rsrc_t ra, rsa;
  if constexpr (!FUSED) {
    ra = __builtin_amdgcn_make_buffer_rsrc((void *)P.a, (short)0, P.M * (int)P.lda, 0x00020000);
    rsa = __builtin_amdgcn_make_buffer_rsrc((void *)P.as, (short)0, P.M * (int)P.lsa, 0x00020000);
  }
  // chunks g and 4 + g of block kb of a row (four lanes read 64 bytes in a
  // row) and the block's eight scale bytes; chunks past K lie outside the
  // buffer
  auto load = [&](__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rss, int ld, int ls, int row, int kb, u32x4(&f)[2],
                  u32x2 &sc) {
    const int c = kb * kBlocksPerK + g;
    const int o = row * ld + c * 16;
    f[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, c < P.nb ? o : kOutOfRange, 0, 0));
    f[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, c + 4 < P.nb ? o + 64 : kOutOfRange, 0, 0));
    sc = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                                       rss, kb < P.nkb ? row * ls + kb * kBlocksPerK : kOutOfRange, 0, 0));
  };
  // this lane's two scale bytes, in bytes 0 and 1; zero past K
  const uint32_t pick = 0x0C0C0400u + 0x0101u * g;
  auto scale = [&](const u32x2 &sc, int kb) {
    const int left = P.nb - kb * kBlocksPerK - g;
    uint32_t sel = pick;
    if (left <= 4) sel = left <= 0 ? 0x0C0C0C0Cu : (sel & 0xFFu) | 0x0C0C0C00u;
    return (int)__builtin_amdgcn_perm(sc.y, sc.x, sel);
  };
  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 fb[U][NT][2], fa[FUSED ? 1 : U][MT][2];
  u32x2 sb[U][NT], sa[FUSED ? 1 : U][MT];
  auto load_all = [&](int kb0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) load(rb, rsb, (int)P.ldb, (int)P.lsb, 16 * n + r, kb0 + NW * u, fb[u][n], sb[u][n]);
      if constexpr (!FUSED) {
#pragma unroll
        for (int m = 0; m < MT; ++m) load(ra, rsa, (int)P.lda, (int)P.lsa, 16 * m + r, kb0 + NW * u, fa[u][m], sa[u][m]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all U blocks in flight before the first use
  };
  int kb0 = wave;
  load_all(kb0);
  const int xrow = fused_row(P.nkb), xsrow = fused_scale_row(P.nkb);
  uint8_t *const xs = dyn + P.M * xrow;
  if constexpr (FUSED) {
    typedef typename MxElem<XDT>::type elem;
    // eight values each, a block per quad; several rows at once where they are short
    const int row_log = fused_row_log(P.nkb, NW), row_threads = 1 << row_log;
    for (int m = (int)threadIdx.x >> row_log; m < P.M; m += (64 * NW) >> row_log) {
      const elem *x = reinterpret_cast<const elem *>(P.x) + m * P.ldx;
      for (int i = (int)threadIdx.x & (row_threads - 1); i < P.nkb * kBlocksPerK * 4; i += row_threads) {
        const Raw8<XDT> v = load_raw8<XDT>(x + 8 * i, P.K - 8 * i);
        const int e = mx_scale_byte<RULE>(mag_f32_bits<XDT>(quad_max(raw_mag<XDT>(v))));
        *reinterpret_cast<uint32_t *>(dyn + m * xrow + 4 * i) = e == kMxNan ? 0u : raw_codes<XDT>(v, mx_scale_f32(e));
        if ((i & 3) == 0) xs[m * xsrow + (i >> 2)] = (uint8_t)e;
      }
    }
    __syncthreads();
  }
  for (;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + NW * u;
      int sbu[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) sbu[n] = scale(sb[u][n], kb);
      if constexpr (FUSED) {
        fa[0][0][0] = fa[0][0][1] = u32x4{0, 0, 0, 0};
        sa[0][0] = u32x2{0, 0};
        if (r < P.M && kb < P.nkb) {
          const u32x4 *src = reinterpret_cast<const u32x4 *>(dyn + r * xrow + kb * kBlockBytes + 16 * g);
          fa[0][0][0] = src[0];
          fa[0][0][1] = src[4];
          sa[0][0] = *reinterpret_cast<const u32x2 *>(xs + r * xsrow + kb * kBlocksPerK);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int ua = FUSED ? 0 : u;
        const int sau = scale(sa[ua][m], kb);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[u][n][0]), frag8(fa[ua][m][0]), acc[m][n],
                                                                       4, 4, 0, sbu[n], 0, sau);
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag8(fb[u][n][1]), frag8(fa[ua][m][1]), acc[m][n],
                                                                       4, 4, 1, sbu[n], 1, sau);
        }
      }
    }
    kb0 += NW * U;
    if (kb0 >= P.nkb) break;
    load_all(kb0);
  }
  __syncthreads();  // (the quantised X is read by all: the partial sums take its place)
  v4f *red = reinterpret_cast<v4f *>(dyn);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[((wave * MT + m) * NT + n) * 64 + lane] = acc[m][n];
  __syncthreads();
  for (int i = wave; i < MT * NT; i += NW) {
    const int m = i / NT, n = i % NT;
    v4f t = red[i * 64 + lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) t += red[(w * MT * NT + i) * 64 + lane];
    const int row = 16 * m + r, col = n0 + 16 * n + 4 * g;
    if (row < P.M) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (col + v < P.N) {
          const float b = P.bias ? load_elem(P.bias, col + v, P.bias_dtype) : 0.0f;
          store_elem(P.c, (int64_t)row * P.N + col + v, t[v] + b, P.c_dtype);
        }
    }
  }
}

// K = 0: C is the bias, or zero.
__global__ __launch_bounds__(256) void mx_fill_kernel(void *c, int c_dtype, int64_t mn, int N, const void *bias,
                                                      int bias_dtype) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < mn; i += (int64_t)gridDim.x * 256)
    store_elem(c, i, bias ? load_elem(bias, i % N, bias_dtype) : 0.0f, c_dtype);
}

void set_tiles(MxProblem &p, int bm, int bn, int group_log) {
  const int tm = (p.M + bm - 1) / bm, tn = (p.N + bn - 1) / bn;
  auto inv = [](int d) { return (uint32_t)std::min<uint64_t>(0xFFFFFFFFull, (1ull << 32) / (uint64_t)d); };
  p.tiles = tm * tn;
  p.group_log = group_log;
  p.group = 1 << group_log;
  p.group_tiles = p.group * tn;
  p.last_rows = tm % p.group ? tm % p.group : p.group;
  p.last_group = (tm - 1) >> group_log;
  p.inv_group_tiles = inv(p.group_tiles);
  p.inv_last_rows = inv(p.last_rows);
}

template <int BM, int BN, int NS, int MINB>
void launch_tiled(const MxBatch &b, int dt, int64_t tiles, hipStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, MINB * kCUs);
  if (dt == F8LIN_FP32)
    mx_gemm_tiled_kernel<BM, BN, NS, MINB, F8LIN_FP32><<<grid, 256, 0, stream>>>(b);
  else if (dt == F8LIN_BF16)
    mx_gemm_tiled_kernel<BM, BN, NS, MINB, F8LIN_BF16><<<grid, 256, 0, stream>>>(b);
  else
    mx_gemm_tiled_kernel<BM, BN, NS, MINB, F8LIN_FP16><<<grid, 256, 0, stream>>>(b);
}

// Waves per workgroup: eight where few workgroups have a contraction of more
// than two rounds of loads (products back to back, cold weights; 1 x 4096 x
// 14336 with X quantised inside 10.3 us, with four 11.9 us; 48 x 8192 x 4096
// 11.0 us, with four 12.4 us; 16 x 4800 x 1600 5.9 us, with four 4.9 us; 51 x
// 4800 x 1600 6.7 us, with four 6.4 us; 4 x 4096 x 4096, X inside, 7.1 us, with
// the four that the rule takes 7.6 us).
int skinny_waves(int64_t grid, int64_t nkb, int MT) { return grid <= 2 * kCUs && nkb >= (MT <= 2 ? 32 : 16) ? 8 : 4; }

// Blocks of 16 columns per workgroup: several share what is read of A, but the
// time is that of the CU with the most blocks (products back to back, cold
// weights; 16 rows: 9216 x 4096 with three 8.8 us, one 11.3 us, two 11.4 us;
// 14336 x 4096 with four 10.5 us, two 11.6 us, one 14.0 us, three 14.4 us; 51
// rows: 8192 x 4096 with two 11.2 us, one 16.3 us).  Several workgroups that
// fit on a CU at once count as rounds all the same, which short contractions
// do not bear out: 51 x 4800 x 1600 with the two that the rule takes 6.4 us,
// with one 6.1 us; 33 x 4800 x 1600 6.1 and 5.9 us; 64 x 6400 x 1600 6.8 and
// 7.0 us; 16 x 4800 x 1600 4.9 and 5.1 us.
int skinny_blocks(int N, int MT, int most) {
  int best = 1;
  int64_t least = 0;
  for (int nt = 1; nt <= most; ++nt) {
    const int64_t rounds = ((N + 16 * nt - 1) / (16 * nt) + kCUs - 1) / kCUs, cost = rounds * (2 * nt + MT);
    if (nt == 1 || cost < least) best = nt, least = cost;
  }
  return best;
}

template <int MT, int NT, bool FUSED, int XDT, int RULE>
void launch_skinny_nw(const MxSkinny &k, hipStream_t stream) {
  const unsigned grid = (unsigned)((k.N + 16 * NT - 1) / (16 * NT));
  const size_t x = FUSED ? fused_bytes(k.M, k.nkb) : 0;
  if (skinny_waves(grid, k.nkb, MT) == 8)
    mx_skinny_kernel<MT, NT, 8, FUSED, XDT, RULE><<<grid, 512, std::max<size_t>(x, 8 * MT * NT * 1024), stream>>>(k);
  else
    mx_skinny_kernel<MT, NT, 4, FUSED, XDT, RULE><<<grid, 256, std::max<size_t>(x, 4 * MT * NT * 1024), stream>>>(k);
}

// Few enough rows for the skinny kernel: up to 64, or fewer where 64 x 64 tiles
// would fill the chip as well (in us, with X's quantisation: 64 x 8192 x 4096
// 15.3, tiled 16.4; 64 x 9216 x 4096 18.4, 16.4; 32 x 11000 x 11000 27.3, 27.6;
// 32 x 14336 x 4096 18.2, 16.3).
bool skinny(const MxProblem &p) {
  return p.M <= 16 || (p.M <= 32 && p.N <= 48 * kCUs) || (p.M <= 64 && p.N <= 32 * kCUs);
}

void launch_skinny(const MxProblem &p, hipStream_t stream) {
  MxSkinny k = {};
  k.a = p.a, k.as = p.as, k.b = p.b, k.bs = p.bs, k.c = p.c, k.bias = p.bias;
  k.lda = p.lda, k.lsa = p.lsa, k.ldb = p.ldb, k.lsb = p.lsb;
  k.M = p.M, k.N = p.N, k.nb = p.nb, k.nkb = p.nkb;
  k.c_dtype = p.c_dtype, k.bias_dtype = p.bias_dtype;
  const int mt = (p.M + 15) / 16;
  const int nt = skinny_blocks(p.N, mt, mt == 1 ? 4 : (mt == 2 ? 3 : 2));
  if (mt == 1) {
    if (nt == 1) launch_skinny_nw<1, 1, false, 0, 0>(k, stream);
    else if (nt == 2) launch_skinny_nw<1, 2, false, 0, 0>(k, stream);
    else if (nt == 3) launch_skinny_nw<1, 3, false, 0, 0>(k, stream);
    else launch_skinny_nw<1, 4, false, 0, 0>(k, stream);
  } else if (mt == 2) {
    if (nt == 1) launch_skinny_nw<2, 1, false, 0, 0>(k, stream);
    else if (nt == 2) launch_skinny_nw<2, 2, false, 0, 0>(k, stream);
    else launch_skinny_nw<2, 3, false, 0, 0>(k, stream);
  } else {
    if (nt == 1) launch_skinny_nw<4, 1, false, 0, 0>(k, stream);
    else launch_skinny_nw<4, 2, false, 0, 0>(k, stream);
  }
}

// The tile a problem takes: 0: 256 x 256, one workgroup per CU; 1: 128 x 128,
// two per CU; 2: the same, one per CU with four stages; 3: 64 x 64, one per CU
// with eight stages.  The one whose estimated time is least: rounds of
// workgroups times a cost per round (prologue and stores) and per K block, in
// microseconds as measured (bf16 output):
//   4096 x 4096 x 4096       0:  40   1: 49   2: 57   3: 110
//   4096 x 4096 x 256        0:  17   1: 14   2: 19   3:  29
//   2048 x 4096 x 4096       0:  36   1: 27   2: 32   3:  58
//   256 x 4096 x 4096        0:  32   1: 17   2: 18   3:  13
//   1600 x 1600 x 12288      0:  74   1: 44   2: 38   3:  59
int tile_for(const MxProblem &p) {
  auto rounds = [&](int b, int slots) {
    const int64_t tiles = (int64_t)((p.M + b - 1) / b) * ((p.N + b - 1) / b);
    return (double)((tiles + slots - 1) / slots);
  };
  const double k = p.nkb;
  const bool spread = rounds(128, kCUs) <= 1.0;  // at most one 128 x 128 tile per CU
  const double t[4] = {5.5 + rounds(256, kCUs) * (8.5 + 1.75 * k),
                       3.0 + (spread ? 3.5 + 0.75 * k : rounds(128, 2 * kCUs) * (4.4 + 1.15 * k)),
                       4.0 + rounds(128, kCUs) * (3.5 + 0.68 * k), 4.5 + rounds(64, kCUs) * (1.7 + 0.36 * k)};
  return (int)(std::min_element(t, t + 4) - t);
}

// Problems of one output type and tile in one launch.
void launch_batch(MxBatch &b, int tile, int dt, hipStream_t stream) {
  const int bm = tile == 0 ? 256 : tile < 3 ? 128 : 64;
  int64_t tiles = 0;
  for (int i = 0; i < b.count; ++i) {
    // groups of 4 tile-rows; of 8 with small tiles, and in long runs of big
    // ones (65536 x 4096 x 4096: 576 us, with 4 586 us; 8192^3: 256 and 252 us)
    const bool many = (int64_t)((b.p[i].M + 255) / 256) * ((b.p[i].N + 255) / 256) >= 8 * kCUs;
    set_tiles(b.p[i], bm, bm, tile == 0 && !many ? 2 : 3);
    tiles += b.p[i].tiles;
  }
  if (tile == 0) launch_tiled<256, 256, 2, 1>(b, dt, tiles, stream);
  else if (tile == 1) launch_tiled<128, 128, 2, 2>(b, dt, tiles, stream);
  else if (tile == 2) launch_tiled<128, 128, 4, 1>(b, dt, tiles, stream);
  else launch_tiled<64, 64, 8, 1>(b, dt, tiles, stream);
}

}  // namespace

// Whether X is quantised by every workgroup of the product itself.  That saves
// a launch and costs every workgroup the whole of X's arithmetic: the passes
// that its threads make over a row's items, and one more, for all rows (more
// where a SIMD runs more than four of its waves).  In us, fused and with a
// launch of its own (and the count that the rule takes):
//   1 x 4096 x 4096   5.6, 7.7 (3)     4 x 4096 x 4096   7.5, 8.0 (12)
//   6 x 4800 x 1600   7.2, 7.5 (12)    8 x 4800 x 1600   8.2, 7.6 (16)
//   2 x 4096 x 14336 12.0, 13.7 (10)   4 x 4096 x 14336 15.2, 13.8 (20)
//   2 x 28672 x 4096 18.6, 20.4 (11)   4 x 28672 x 4096 22.1, 20.2 (21)
bool mx_linear_fused(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > 16) return false;
  const int64_t nkb = (K + 8 * kBlocksPerK * 4 - 1) / (8 * kBlocksPerK * 4), grid = (N + 15) / 16;
  const int waves = skinny_waves(grid, nkb, 1);
  const int64_t at_once = (64 * waves) >> fused_row_log((int)nkb, waves);
  const int64_t passes = (M + at_once - 1) / at_once * ((32 * nkb + 64 * waves - 1) / (64 * waves) + 1);
  return passes * std::max<int64_t>(4 * kCUs, grid) <= 12 * 4 * kCUs;
}

hipError_t launch_mx_linear(const MxLinear &l, hipStream_t stream) {
  MxSkinny k = {};
  k.x = l.x, k.ldx = l.ldx, k.b = l.w.codes, k.bs = l.w.scales, k.ldb = l.w.ld, k.lsb = l.w.scale_ld;
  k.c = l.y, k.c_dtype = l.y_dtype, k.bias = l.bias, k.bias_dtype = l.bias_dtype;
  k.M = (int)l.M, k.N = (int)l.N, k.K = (int)l.K;
  k.nb = (int)((l.K + kMxBlock - 1) / kMxBlock), k.nkb = (k.nb + kBlocksPerK - 1) / kBlocksPerK;
#define F8_MX_L(DT)                                              \
  if (l.rule == F8LIN_MX_CEIL)                                   \
    launch_skinny_nw<1, 1, true, DT, F8LIN_MX_CEIL>(k, stream);     \
  else                                                           \
    launch_skinny_nw<1, 1, true, DT, F8LIN_MX_FLOOR>(k, stream)
  if (l.x_dtype == F8LIN_BF16) {
    F8_MX_L(F8LIN_BF16);
  } else if (l.x_dtype == F8LIN_FP16) {
    F8_MX_L(F8LIN_FP16);
  } else {
    F8_MX_L(F8LIN_FP32);
  }
#undef F8_MX_L
  return hipGetLastError();
}

hipError_t launch_mx_gemms(const MxGemm *d, int count, hipStream_t stream) {
  bool any = false;
  MxBatch b = {};
  int tile[kMxMaxGemms], dt[kMxMaxGemms];
  for (int i = 0; i < count; ++i) {
    if (d[i].M == 0 || d[i].N == 0) continue;
    any = true;
    if (d[i].K == 0) {
      const int64_t mn = d[i].M * d[i].N;
      mx_fill_kernel<<<(unsigned)std::min<int64_t>((mn + 255) / 256, 8192), 256, 0, stream>>>(
          d[i].c, d[i].c_dtype, mn, (int)d[i].N, d[i].bias, d[i].bias_dtype);
      continue;
    }
    MxProblem &p = b.p[b.count];
    p.a = d[i].a.codes;
    p.as = d[i].a.scales;
    p.b = d[i].b.codes;
    p.bs = d[i].b.scales;
    p.c = d[i].c;
    p.bias = d[i].bias;
    p.lda = d[i].a.ld;
    p.lsa = d[i].a.scale_ld;
    p.ldb = d[i].b.ld;
    p.lsb = d[i].b.scale_ld;
    p.M = (int)d[i].M;
    p.N = (int)d[i].N;
    p.nb = (int)((d[i].K + kMxBlock - 1) / kMxBlock);
    p.nkb = (p.nb + kBlocksPerK - 1) / kBlocksPerK;
    p.c_dtype = d[i].c_dtype;
    p.bias_dtype = d[i].bias_dtype;
    if (skinny(p)) {
      launch_skinny(p, stream);
    } else {
      tile[b.count] = tile_for(p);
      dt[b.count++] = d[i].c_dtype;
    }
  }
  if (b.count == 2 && (tile[0] != tile[1] || dt[0] != dt[1])) {
    MxBatch second = {};
    second.p[0] = b.p[1];
    second.count = b.count = 1;
    launch_batch(second, tile[1], dt[1], stream);
  }
  if (b.count > 0) launch_batch(b, tile[0], dt[0], stream);
  return any ? hipGetLastError() : hipSuccess;
}

}  // namespace f8lin

// The low-rank adapters' launchers and the layout of their plan.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace f8lin {

constexpr int kLoraMaxAdapters = 2047;   // of a plan: 16 waves' counts of each fit the LDS
constexpr int kLoraMaxRank = 256;
constexpr int kLoraMagic = 0x4C6F5241;

// Ranks of H: 16, or blocks of 32.
__host__ __device__ inline int lora_rank_pad(int rank) { return rank <= 16 ? 16 : (rank + 31) / 32 * 32; }
// Rows of a tile: few tokens are mostly single ones of many adapters, or need
// more workgroups than 64-row tiles give (1024 tokens of 4 adapters, 4096 x
// 4096, rank 16: forward 14.0 us in 16-row tiles, 18.4 in 64-row ones; 2048
// tokens 21.1 and 21.6; 4096 of rank 32 42 and 32).
__host__ __device__ inline int lora_tile(int64_t tokens) { return tokens <= 1024 ? 16 : 64; }
__host__ __device__ inline int64_t lora_max_tiles(int64_t tokens, int64_t adapters) {
  const int64_t groups = tokens < adapters + 1 ? tokens : adapters + 1, rows = lora_tile(tokens);
  // (a group's last tile may be short; a token is in one tile)
  const int64_t most = (tokens + rows - 1) / rows + groups;
  return most < tokens ? most : tokens;
}
// Words before the tiles, and before the tokens' order.
__host__ __device__ inline int64_t lora_tiles_at(int64_t adapters) { return (4 + adapters + 2 + 3) / 4 * 4; }
__host__ __device__ inline int64_t lora_order_at(int64_t tokens, int64_t adapters) {
  return lora_tiles_at(adapters) + 4 * lora_max_tiles(tokens, adapters);
}
__host__ __device__ inline int64_t lora_plan_words(int64_t tokens, int64_t adapters) {
  return lora_order_at(tokens, adapters) + 2 * tokens;
}

struct LoraDown {
  const int *plan;
  int tokens, adapters, rank, max_tiles;
  const void *x;  // (tokens, cols)
  int64_t ldx, cols;
  const void *w;        // (adapters, rank, cols) or (adapters, cols, rank)
  const float *scales;  // (adapters) or null
  // H in binary32 where the later products look for it: in the order of the up
  // product's operand fragments, a tile after the other, max_tiles x 64 x
  // rank_pad (h; with fp16 data times 2^-e, beside its exponents e, one for 64
  // ranks of a position: rank / 64 rounded up x tokens), and by rank, rank_pad x
  // tokens (ht); either may be null.  Only with lora_split: parts_out, the parts'
  // sums, parts x tokens x rank_pad, in place of h.
  uint32_t *h;
  float *ht;
  int *exponents;
  float *parts_out;
  int parts;
};
struct LoraUp {
  const int *plan;
  int tokens, adapters, rank, max_tiles;
  const uint32_t *h;  // as left by down, or null:
  const int *exponents;
  const float *parts_in;  // the parts' sums
  int parts;
  const void *w;  // (adapters, cols, rank) or (adapters, rank, cols)
  const void *base;
  int64_t ldbase, cols;
  void *y;
  int64_t ldy;
};
struct LoraOuterSide {
  const void *x;  // (tokens, cols)
  int64_t ldx, cols;
  const float *ht;  // H by rank
  void *d;         // (adapters, rank, cols), or (adapters, cols, rank) where d_t; null: not computed
  int d_t;
  float *part;  // 2 * chunks x rank x cols
  int blocks;   // (set by the launch)
  int64_t join_blocks;
};
struct LoraOuter {
  const int *plan;
  int tokens, adapters, rank;
  int chunk, chunks;  // sorted positions a workgroup takes, and how many such
  LoraOuterSide side[2];
  int units, across, split;  // (set by the launch)
};

// Whether H passes between the products as sums of parts (16-row tiles), into
// how many parts the columns of a down product are then split, and the
// positions of an outer product's chunk.
inline bool lora_split(int64_t tokens) { return lora_tile(tokens) == 16; }
int lora_parts(int64_t tokens, int adapters, int64_t cols, int rank);
int lora_chunk(int64_t tokens, int64_t K, int64_t N, int rank);
hipError_t launch_lora_plan(const void *index, bool wide, int tokens, int adapters, int *plan, hipStream_t stream);
hipError_t launch_lora_down(const LoraDown &a, int dtype, bool w_t, hipStream_t stream);
hipError_t launch_lora_up(const LoraUp &a, int dtype, bool w_t, hipStream_t stream);
hipError_t launch_lora_outer(const LoraOuter &a, int dtype, hipStream_t stream);

}  // namespace f8lin

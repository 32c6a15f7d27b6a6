// Kernel arguments of the attention over shared prefixes, shared by its C-ABI
// layer (paged.cpp) and its kernels (shared.cu).
#pragma once

#include "paged.h"

namespace sfi {

constexpr int kMaxTiles = kMaxBatch / 2;  // of a launch: a group that shares has two sequences at least
constexpr int kTileRows = 256;            // query rows of a tile

// Up to 2 x 128 / G sequences of one group.
struct SharedTile {
  int32_t b0, seqs;  // its sequences
  int32_t lead;      // the group's first sequence, whose pages are read
  int32_t n;         // positions that they share
};

// What the first kernel leaves for the others.
struct SharedPlan {
  int32_t n_tiles;
  int32_t alone;    // != 0: some sequence shares nothing
  long long total;  // key blocks of all KV heads in all tiles
  long long own[kMaxBatch + 1];  // tiles of a KV head in the own positions of the sequences before each
  long long start[kMaxTiles + 1];  // key blocks of all KV heads in the tiles before each
  SharedTile tile[kMaxTiles];
};

struct SharedArgs {
  // 3-D maps: [sequence][head][d] of q, boxes of 64 elements of d, G heads and 128 / G sequences;
  // of the pool's rows (64 elements of d, row, 64-element block of d), boxes of `box` rows
  CUtensorMap tmq, tmk, tmv;
  int32_t box;        // 8, 16, 24 or 48, which divides the page size; 0: no maps of k and v
  int32_t pool_rows;  // rows of the maps: what lies behind reads as zero
  int32_t tok;        // sequences of 128 query rows: 128 / G
  int32_t max_tiles;  // that the plan may have
  int32_t n_groups;
  const int32_t* cu_group;
  const int32_t* shared_pages;
  int32_t* skip;      // [B]
  SharedPlan* plan;
  float* states;      // [grid + tiles * H_kv][d + 2][256]
  PagedAttnArgs own;  // the sequences' own positions (geo.skip is set)
};

// Flags groups that are wrong, and nothing else (a batch of one, where no group can share).
cudaError_t launch_check_groups(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared_attn(const SharedArgs& a, int D, bool use_tma, int grid, cudaStream_t st);

}  // namespace sfi

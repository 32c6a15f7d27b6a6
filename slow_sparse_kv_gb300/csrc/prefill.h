// Kernel arguments of the prompt attention, shared by its C-ABI layer
// (paged.cpp) and its kernel (prefill.cu).
#pragma once

#include "sfi_internal.h"

namespace sfi {

constexpr int kPrefillMaxGroup = 16;  // query heads per KV head, at most
constexpr int kPrefillMaxGrid = 256;  // CTAs of a launch, at most
constexpr int kMaxParts = 8;          // parts that a tile is cut into, at most
constexpr int kSplitWaves = 8;        // waves of tiles below which the last one's may be cut
constexpr int kSplitKeys = 1024;      // keys in all below which none is

// A pair of 128-row tiles: 2 x 128 / G tokens of one (sequence, KV head).
struct PrefillTile {
  int rows;    // tokens it has (0: no tile, the end)
  int g;       // KV head
  int q0;      // first query row
  int k0, nk;  // the sequence's first key row and its number of keys
  int seen;    // keys that the first token sees (may be negative: none, and none for some after it)
  int n[2];    // key blocks of each half
  int slot;    // where a part of a tile leaves its state, -1: a whole tile
};

struct PrefillArgs {
  // 3-D maps [row][head][d] of q, k and v, boxes of 64 elements of d with a
  // 128-byte swizzle: G heads x 128 / G rows of q, 1 head x 128 rows of k and v
  CUtensorMap tmq, tmk, tmv;
  // the same of out, boxes of G heads x 32 / G rows (where G divides 32)
  CUtensorMap tmo;
  void* out;
  float* lse;  // [total_q][H_q] or null
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t out_stride;
  int32_t B, H_q, H_kv, G, total_q, total_k;
  int32_t tok;      // tokens per 128-row query tile: 128 / G
  float scale_log2; // log2(e) / sqrt(d)
  uint32_t* status;
  uint32_t* next;  // [2]: next tile, CTAs that ran out; zero between launches
  int32_t* span;   // [B] scratch: CTA tiles of each sequence and KV head
  int32_t* lvl;    // [B] scratch: the level of its first one
  int32_t* cut_count;  // [2]: how many tiles are cut, into how many parts
  PrefillTile* cuts;   // [kPrefillMaxGrid] those tiles
  float* partials;  // [kPrefillMaxGrid][256][d + 2] states of the parts of tiles; null: none is cut
  long long wait_cycles;
};

cudaError_t launch_prefill(const PrefillArgs& a, int D, cudaStream_t st);

}  // namespace sfi

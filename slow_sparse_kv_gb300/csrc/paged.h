// Kernel arguments of the paged-cache calls, shared by their C-ABI layer
// (paged.cpp) and their kernels (paged_attn.cu, pages.cu).
#pragma once

#include "sfi_internal.h"

namespace sfi {

constexpr int kPagedMaxGrid = 256;  // CTAs of a paged-attention launch, at most

// Geometry of a paged cache on the device.
struct PagedGeo {
  int32_t B, H_kv, P, n_pages, max_pages;
  int64_t page_stride;  // elements (bytes of an 8-bit pool)
  int32_t* table;
  int32_t* len;
  uint32_t* status;
  uint32_t* refused;  // a bit for each sequence that an extension left as it was
  const int32_t* skip;  // pages at the start of each sequence that are left out; null: none
};

struct PagedAttnArgs {
  // bf16 pools with page_size a multiple of 16: 3-D maps (64 elements of d,
  // row, 64-element block of d) of the pool's rows, boxes of 16 rows
  CUtensorMap tmk, tmv;
  PagedGeo geo;
  const void* q;
  const void* k;
  const void* v;
  float* out;
  float* lse;  // nullable
  int32_t H_q, G;
  float scale_log2;   // log2(e) / sqrt(d)
  float* partials;    // [grid + B * H_kv][G][d + 2]
  long long wait_cycles;
  // 8-bit pools
  int32_t scale_at;   // bytes from a page's start to its scales
  int32_t box;        // rows of the maps' boxes (where there are maps): 32 or 16
};

// The same over an 8-bit pool.  use_tma: the maps are set, 3-D maps (d bytes, row of a page, page)
// with a swizzle of d bytes.
cudaError_t launch_paged_attn_q8(const PagedAttnArgs& a, int D, bool e4m3, bool q_f32, bool use_tma, int grid,
                                 cudaStream_t st);

// use_tma: the maps are set
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int D, bool f32, bool use_tma, int grid,
                              cudaStream_t st);

// The same for bf16 pools without the join, each warp with a share of its own: the pieces of all
// units that hold anything lie in partials, [warps of the grid + B * H_kv][G][d + 2].
constexpr int kPagedWarps = 8;  // of a CTA, that attend
cudaError_t launch_paged_pieces(const PagedAttnArgs& a, int D, bool use_tma, int grid, cudaStream_t st);

struct AppendArgs {
  PagedGeo geo;
  const uint8_t* k_new;
  const uint8_t* v_new;
  uint8_t* k;
  uint8_t* v;
  int64_t k_stride, v_stride;  // bytes
  int64_t page_bytes;
  const int32_t* cu;  // null: one row per sequence
  int32_t total;
  int32_t row_bytes;  // of one head
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t st);

// The same into an 8-bit pool: row_bytes is that of codes, the strides are bytes of the new rows.
struct QuantArgs : AppendArgs {
  int32_t scale_at;  // bytes from a page's start to its scales
};
cudaError_t launch_append_q8(const QuantArgs& a, bool f32, bool e4m3, cudaStream_t st);

// Sequences named by the host, passed by value.
struct SeqList {
  int16_t id[kMaxBatch];
};

// Rows of pages to move, in every layer, of k and of v.
struct PageMove {
  uint8_t* k;
  uint8_t* v;
  int64_t layer_bytes, page_bytes;  // strides
  int32_t n_layers, H_kv, P, row_bytes, n_pages;
  int32_t whole;     // bytes of a page
  int32_t scale_at;  // 8-bit pools: bytes from a page's start to its scales; 0: none
  uint32_t* status;
};

// fresh: [n_pages] device scratch
cudaError_t launch_extend(const PagedGeo& g, int32_t* ref, const int32_t* n_new, int32_t* fresh,
                          cudaStream_t st);
// jobs: [n] device scratch (source page, new page, rows)
cudaError_t launch_fork(const PagedGeo& g, int32_t* ref, const SeqList& src, const SeqList& dst,
                        int n, const PageMove& mv, int4* jobs, cudaStream_t st);
cudaError_t launch_free(const PagedGeo& g, int32_t* ref, const SeqList& seqs, int n, cudaStream_t st);
// map, holes, moved: [n_pages] device scratch; n_moved: [1]
cudaError_t launch_compact(const PagedGeo& g, int32_t* ref, int32_t* new_id, const PageMove& mv,
                           int32_t* map, int32_t* holes, int32_t* moved, int32_t* n_moved,
                           cudaStream_t st);
cudaError_t launch_page_copy(const PageMove& mv, const int32_t* src, const int32_t* dst, int n,
                             cudaStream_t st);

}  // namespace sfi

// Kernel arguments of the norm and rotation of query and key heads, shared by
// their C-ABI layer (rope.cpp) and their kernel (rope.cu).
#pragma once

#include "sfi_internal.h"

namespace sfi {

struct RopeArgs {
  const void* q;
  const void* k;
  const void* wq;  // null: ones
  const void* wk;
  void* q_out;
  void* k_out;
  const int32_t* pos;  // null where nothing is rotated
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements
  int32_t total, H_q, H_kv;
  int32_t rot;         // dimensions that are rotated, a multiple of 8
  int32_t pos_offset;
  int32_t norm;        // != 0: RMS norm
  int32_t parts;       // warps that share a row (set by the launcher)
  float eps;
  uint64_t freq[64];   // turns a position, in units of 2^-64, modulo 1
};

// next: pairs of neighbours (2i, 2i + 1); else (i, i + rot / 2)
cudaError_t launch_rope(const RopeArgs& a, int D, bool f32, bool next, cudaStream_t st);

}  // namespace sfi

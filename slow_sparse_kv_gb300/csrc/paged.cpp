// C ABI of the prompt attention and of the paged KV cache: host-side
// validation, workspace plans and dispatch.  Every check happens before
// anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "prefill.h"
#include "sfi_internal.h"

namespace sfi {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool misaligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

sfi_status check_heads(int H_q, int H_kv, int D) {
  if (H_kv < 1 || H_q < 1 || H_q % H_kv != 0)
    return fail(SFI_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", H_q, H_kv);
  if (H_q / H_kv > kPrefillMaxGroup)
    return fail(SFI_ERR_UNSUPPORTED, "query heads per KV head must be 1 to %d (got %d)", kPrefillMaxGroup, H_q / H_kv);
  if (D != 64 && D != 128) return fail(SFI_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", D);
  return SFI_OK;
}

sfi_status check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(SFI_ERR_WORKSPACE, "workspace is NULL");
  if (ws_bytes < need)
    return fail(SFI_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return fail(SFI_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return SFI_OK;
}

// A row stride in elements: 0 stands for rows without gaps.
sfi_status row_stride(const char* name, int64_t stride, int64_t row, int64_t* out) {
  *out = stride == 0 ? row : stride;
  if (*out < row || *out % 8 != 0)
    return fail(SFI_ERR_INVALID_ARG, "%s (%lld) must be 0, or at least a row of %lld elements and a multiple of 8",
                name, (long long)stride, (long long)row);
  if (*out >= (int64_t(1) << 38)) return fail(SFI_ERR_CAPACITY, "%s (%lld) exceeds 2^38 elements", name, (long long)stride);
  return SFI_OK;
}

sfi_status check_packed(const sfi_packed_layout* L) {
  if (!L) return fail(SFI_ERR_INVALID_ARG, "layout is NULL");
  if (L->batch < 1) return fail(SFI_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", L->batch);
  if (L->batch > kMaxBatch) return fail(SFI_ERR_CAPACITY, "batch %d exceeds the limit %d", L->batch, kMaxBatch);
  sfi_status s = check_heads(L->n_q_heads, L->n_kv_heads, L->head_dim);
  if (s != SFI_OK) return s;
  if (L->dtype != SFI_BF16) return fail(SFI_ERR_UNSUPPORTED, "prompt attention takes bf16 (dtype %d)", L->dtype);
  if (L->total_q < 0 || L->total_k < 0)
    return fail(SFI_ERR_INVALID_ARG, "total_q and total_k must be >= 0 (got %d, %d)", L->total_q, L->total_k);
  if (!L->cu_q || !L->cu_k) return fail(SFI_ERR_INVALID_ARG, "cu_q and cu_k must be device pointers");
  const int tok = 128 / (L->n_q_heads / L->n_kv_heads);
  if (((long long)L->total_q / (2 * tok) + L->batch) * L->n_kv_heads > 0x7fffffffLL)
    return fail(SFI_ERR_CAPACITY, "total_q %d with %d KV heads exceeds the grid", L->total_q, L->n_kv_heads);
  return SFI_OK;
}

// [rows][heads][D] with `stride` elements between rows, boxes of `bh` heads x `br` rows.
bool encode_heads(CUtensorMap* m, const void* base, int D, int heads, int rows, int64_t stride, int bh, int br) {
  const uint64_t dims[3] = {uint64_t(D), uint64_t(heads), uint64_t(rows)};
  const uint64_t st[2] = {uint64_t(D) * 2, uint64_t(stride) * 2};
  const uint32_t box[3] = {64, uint32_t(bh), uint32_t(br)};
  return encode_bf16_3d(m, base, dims, st, box);
}

}  // namespace
}  // namespace sfi

using namespace sfi;

extern "C" {

size_t sfi_prefill_attn_workspace_size(const sfi_packed_layout* L) {
  return check_packed(L) == SFI_OK ? 256 : 0;  // the status word
}

sfi_status sfi_prefill_attn(const sfi_packed_layout* L, const void* q, const void* k, const void* v, void* out,
                            float* lse_out, void* ws, size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_packed(L);
  if (s != SFI_OK) return s;
  const int D = L->head_dim, G = L->n_q_heads / L->n_kv_heads;
  int64_t qs, ks, vs, os;
  if ((s = row_stride("q_stride", L->q_stride, int64_t(L->n_q_heads) * D, &qs)) != SFI_OK) return s;
  if ((s = row_stride("k_stride", L->k_stride, int64_t(L->n_kv_heads) * D, &ks)) != SFI_OK) return s;
  if ((s = row_stride("v_stride", L->v_stride, int64_t(L->n_kv_heads) * D, &vs)) != SFI_OK) return s;
  if ((s = row_stride("out_stride", L->out_stride, int64_t(L->n_q_heads) * D, &os)) != SFI_OK) return s;
  if ((s = check_workspace(ws, ws_bytes, 256)) != SFI_OK) return s;
  if (L->total_q == 0) return SFI_OK;
  if (!q || !out || (L->total_k > 0 && (!k || !v)))
    return fail(SFI_ERR_INVALID_ARG, "q, k, v and out must be set");
  if (misaligned16(q) || misaligned16(out) || (L->total_k > 0 && (misaligned16(k) || misaligned16(v))))
    return fail(SFI_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
  PrefillArgs a;
  std::memset(&a, 0, sizeof(a));
  a.out = out;
  a.lse = lse_out;
  a.cu_q = L->cu_q;
  a.cu_k = L->cu_k;
  a.out_stride = os;
  a.B = L->batch;
  a.H_q = L->n_q_heads;
  a.H_kv = L->n_kv_heads;
  a.G = G;
  a.total_q = L->total_q;
  a.total_k = L->total_k;
  a.tok = 128 / G;
  a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(D)));
  a.status = static_cast<uint32_t*>(ws);
  a.wait_cycles = wait_limit_cycles();
  bool ok = encode_heads(&a.tmq, q, D, L->n_q_heads, L->total_q, qs, G, a.tok);
  if (L->total_k > 0)  // without keys the kernel loads neither
    ok = ok && encode_heads(&a.tmk, k, D, L->n_kv_heads, L->total_k, ks, 1, 128) &&
         encode_heads(&a.tmv, v, D, L->n_kv_heads, L->total_k, vs, 1, 128);
  if (!ok) return fail(SFI_ERR_CUDA, "encoding the tensor maps of q, k and v failed");
  const cudaError_t e = launch_prefill(a, D, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
  return SFI_OK;
}

}  // extern "C"

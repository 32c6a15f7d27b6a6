// C ABI of the prompt attention and of the paged KV cache: host-side
// validation, workspace plans and dispatch.  Every check happens before
// anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged.h"
#include "prefill.h"
#include "sfi_internal.h"

namespace sfi {
namespace {

// The prompt attention's workspace: the status word, the counters of the tiles, two
// numbers for each sequence, and where tiles may be cut along their keys, the
// states of their parts.
// (Bytes 384 to 512 belong to the paged calls, which may use the same workspace.)
constexpr size_t kRefusedAt = 384;
constexpr size_t kPrefillWs = 512 + 8 * kMaxBatch;
constexpr size_t kCutWs = 256 + kPrefillMaxGrid * 64;  // the cut tiles
static_assert(sizeof(PrefillTile) <= 64, "kCutWs");
bool may_cut(const sfi_packed_layout* L) {
  const int span = 2 * (128 / (L->n_q_heads / L->n_kv_heads));
  // (there are at least total_q / span tiles for each KV head, if the sequences
  // hold all rows)
  return L->total_k >= kSplitKeys &&
         (long long)L->total_q / span * L->n_kv_heads < (long long)kSplitWaves * kPrefillMaxGrid;
}
size_t prefill_ws(const sfi_packed_layout* L) {
  return kPrefillWs + (may_cut(L) ? kCutWs + size_t(kPrefillMaxGrid) * 256 * (L->head_dim + 2) * 4 : 0);
}

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

// A row stride in elements, in units of 16 bytes: 0 stands for rows without gaps.
sfi_status row_stride(const char* name, int64_t stride, int64_t row, int64_t unit, int64_t* out) {
  *out = stride == 0 ? row : stride;
  if (*out < row || *out % unit != 0)
    return fail(SFI_ERR_INVALID_ARG, "%s (%lld) must be 0, or at least a row of %lld elements and a multiple of %lld",
                name, (long long)stride, (long long)row, (long long)unit);
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

int64_t elem_bytes(int dtype) { return dtype == SFI_F32 ? 4 : 2; }

// Elements between pages (page_stride, or a page where it is 0).
int64_t page_elems(const sfi_paged_layout* L) {
  return L->page_stride ? L->page_stride : int64_t(L->n_kv_heads) * L->page_size * L->head_dim;
}

// Rows of d elements from the pool's first to its last.
int64_t pool_rows(const sfi_paged_layout* L) {
  return (L->n_pages - 1) * (page_elems(L) / L->head_dim) + int64_t(L->n_kv_heads) * L->page_size;
}

sfi_status check_paged(const sfi_paged_layout* L) {
  if (!L) return fail(SFI_ERR_INVALID_ARG, "layout is NULL");
  if (L->batch < 1) return fail(SFI_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", L->batch);
  if (L->batch > kMaxBatch) return fail(SFI_ERR_CAPACITY, "batch %d exceeds the limit %d", L->batch, kMaxBatch);
  const sfi_status s = check_heads(L->n_q_heads, L->n_kv_heads, L->head_dim);
  if (s != SFI_OK) return s;
  if (L->dtype != SFI_F32 && L->dtype != SFI_BF16)
    return fail(SFI_ERR_UNSUPPORTED, "dtype must be SFI_F32 or SFI_BF16 (got %d)", L->dtype);
  if ((long long)L->batch * L->n_kv_heads > kMaxUnits)
    return fail(SFI_ERR_CAPACITY, "batch * n_kv_heads = %lld exceeds the limit %d", (long long)L->batch * L->n_kv_heads,
                kMaxUnits);
  if (L->page_size < 1 || L->n_pages < 1 || L->max_pages < 1)
    return fail(SFI_ERR_INVALID_ARG, "page_size, n_pages and max_pages must be >= 1 (got %d, %d, %d)", L->page_size,
                L->n_pages, L->max_pages);
  if (L->page_size > 1024 || L->n_pages > (1 << 24) || (long long)L->max_pages * L->page_size > (1LL << 30))
    return fail(SFI_ERR_CAPACITY,
                "page_size <= 1024, n_pages <= 2^24, max_pages * page_size <= 2^30 (got %d, %d, %lld)", L->page_size,
                L->n_pages, (long long)L->max_pages * L->page_size);
  const int64_t page = int64_t(L->n_kv_heads) * L->page_size * L->head_dim;
  if (L->page_stride != 0 && (L->page_stride < page || L->page_stride % L->head_dim != 0))
    return fail(SFI_ERR_INVALID_ARG,
                "page_stride (%lld) must be 0, or at least a page of %lld elements and a multiple of head_dim",
                (long long)L->page_stride, (long long)page);
  if (page * 4 >= (1LL << 31)) return fail(SFI_ERR_CAPACITY, "a page of %lld elements is too large", (long long)page);
  if (page_elems(L) >= (1LL << 38) || pool_rows(L) >= (1LL << 31))
    return fail(SFI_ERR_CAPACITY, "the pool spans 2^31 rows of head_dim elements or more");
  if (!L->page_table || !L->len) return fail(SFI_ERR_INVALID_ARG, "page_table and len must be device pointers");
  return SFI_OK;
}

// What the paged calls keep in their workspace.
struct PagedPlan {
  size_t partials, jobs, map, holes, moved, n_moved, total;
};

PagedPlan plan_paged(const sfi_paged_layout* L) {
  const size_t units = size_t(L->batch) * L->n_kv_heads, G = L->n_q_heads / L->n_kv_heads;
  PagedPlan p;
  // the status word, the prompt attention's counters, which may share the workspace, and
  // the bits of the refused sequences, which it leaves alone
  static_assert(kRefusedAt % 4 == 0 && kRefusedAt + kMaxBatch / 8 <= 512, "refused");
  size_t off = 512;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  p.partials = take((units + kPagedMaxGrid) * G * (L->head_dim + 2) * 4);
  p.jobs = take(size_t(kMaxBatch) * sizeof(int4));
  p.map = take(size_t(L->n_pages) * 4);
  p.holes = take(size_t(L->n_pages) * 4);
  p.moved = take(size_t(L->n_pages) * 4);
  p.n_moved = take(4);
  p.total = off;
  return p;
}

PagedGeo geo_of(const sfi_paged_layout* L, void* ws) {
  return PagedGeo{L->batch,  L->n_kv_heads, L->page_size, L->n_pages,
                  L->max_pages, page_elems(L), L->page_table, L->len, static_cast<uint32_t*>(ws),
                  reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kRefusedAt)};
}

sfi_status check_store(const sfi_paged_layout* L, const sfi_page_store* S, bool rows) {
  if (!S) return fail(SFI_ERR_INVALID_ARG, "store is NULL");
  if (!S->ref) return fail(SFI_ERR_INVALID_ARG, "ref must be a device pointer");
  if (!rows) return SFI_OK;
  if (!S->k || !S->v) return fail(SFI_ERR_INVALID_ARG, "k and v must be set");
  if (misaligned16(S->k) || misaligned16(S->v)) return fail(SFI_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (S->n_layers < 1) return fail(SFI_ERR_INVALID_ARG, "n_layers must be >= 1 (got %d)", S->n_layers);
  if (S->n_layers > 4096) return fail(SFI_ERR_CAPACITY, "n_layers %d exceeds the limit 4096", S->n_layers);
  if (S->layer_stride < 0 || S->layer_stride % L->head_dim != 0 || (S->n_layers > 1 && S->layer_stride == 0))
    return fail(SFI_ERR_INVALID_ARG, "layer_stride (%lld) must be a positive multiple of head_dim",
                (long long)S->layer_stride);
  if (S->layer_stride >= (1LL << 42)) return fail(SFI_ERR_CAPACITY, "layer_stride exceeds 2^42 elements");
  return SFI_OK;
}

PageMove move_of(const sfi_paged_layout* L, const sfi_page_store* S, void* ws) {
  const int64_t e = elem_bytes(L->dtype);
  PageMove m;
  m.k = static_cast<uint8_t*>(S->k);
  m.v = static_cast<uint8_t*>(S->v);
  m.layer_bytes = S->layer_stride * e;
  m.page_bytes = page_elems(L) * e;
  m.n_layers = S->n_layers;
  m.H_kv = L->n_kv_heads;
  m.P = L->page_size;
  m.row_bytes = int(L->head_dim * e);
  m.n_pages = L->n_pages;
  m.status = static_cast<uint32_t*>(ws);
  return m;
}

// A host list of n sequences, each in [0, batch), none twice if `distinct`.
sfi_status take_list(const char* name, const int32_t* v, int n, int batch, bool distinct, SeqList* out) {
  bool seen[kMaxBatch] = {};
  for (int i = 0; i < n; ++i) {
    if (v[i] < 0 || v[i] >= batch) return fail(SFI_ERR_INVALID_ARG, "%s: no sequence %d (batch %d)", name, v[i], batch);
    if (distinct && seen[v[i]]) return fail(SFI_ERR_INVALID_ARG, "%s: sequence %d is listed twice", name, v[i]);
    seen[v[i]] = true;
    out->id[i] = int16_t(v[i]);
  }
  return SFI_OK;
}

sfi_status check_list_size(int n, int batch) {
  if (n < 0 || n > batch) return fail(SFI_ERR_INVALID_ARG, "n must lie in [0, batch] (got %d)", n);
  return SFI_OK;
}

}  // namespace
}  // namespace sfi

using namespace sfi;

extern "C" {

size_t sfi_prefill_attn_workspace_size(const sfi_packed_layout* L) {
  return check_packed(L) == SFI_OK ? prefill_ws(L) : 0;
}

sfi_status sfi_prefill_attn(const sfi_packed_layout* L, const void* q, const void* k, const void* v, void* out,
                            float* lse_out, void* ws, size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_packed(L);
  if (s != SFI_OK) return s;
  const int D = L->head_dim, G = L->n_q_heads / L->n_kv_heads;
  int64_t qs, ks, vs, os;
  if ((s = row_stride("q_stride", L->q_stride, int64_t(L->n_q_heads) * D, 8, &qs)) != SFI_OK) return s;
  if ((s = row_stride("k_stride", L->k_stride, int64_t(L->n_kv_heads) * D, 8, &ks)) != SFI_OK) return s;
  if ((s = row_stride("v_stride", L->v_stride, int64_t(L->n_kv_heads) * D, 8, &vs)) != SFI_OK) return s;
  if ((s = row_stride("out_stride", L->out_stride, int64_t(L->n_q_heads) * D, 8, &os)) != SFI_OK) return s;
  if ((s = check_workspace(ws, ws_bytes, prefill_ws(L))) != SFI_OK) return s;
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
  a.next = a.status + 64;
  a.span = reinterpret_cast<int32_t*>(a.status + 128);
  a.lvl = a.span + kMaxBatch;
  if (may_cut(L)) {
    char* const cut = static_cast<char*>(ws) + kPrefillWs;
    a.cut_count = reinterpret_cast<int32_t*>(cut);
    a.cuts = reinterpret_cast<PrefillTile*>(cut + 256);
    a.partials = reinterpret_cast<float*>(cut + kCutWs);
  }
  a.wait_cycles = wait_limit_cycles();
  bool ok = encode_heads(&a.tmq, q, D, L->n_q_heads, L->total_q, qs, G, a.tok);
  if (32 % G == 0) ok = ok && encode_heads(&a.tmo, out, D, L->n_q_heads, L->total_q, os, G, 32 / G);
  if (L->total_k > 0)  // without keys the kernel loads neither
    ok = ok && encode_heads(&a.tmk, k, D, L->n_kv_heads, L->total_k, ks, 1, 128) &&
         encode_heads(&a.tmv, v, D, L->n_kv_heads, L->total_k, vs, 1, 128);
  if (!ok) return fail(SFI_ERR_CUDA, "encoding the tensor maps of q, k and v failed");
  const cudaError_t e = launch_prefill(a, D, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
  return SFI_OK;
}

size_t sfi_paged_workspace_size(const sfi_paged_layout* L) {
  return check_paged(L) == SFI_OK ? plan_paged(L).total : 0;
}

sfi_status sfi_paged_attn(const sfi_paged_layout* L, const void* q, const void* k, const void* v, float* out,
                          float* lse_out, void* ws, size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if (!q || !k || !v || !out) return fail(SFI_ERR_INVALID_ARG, "q, k, v and out must be set");
  if (misaligned16(q) || misaligned16(k) || misaligned16(v))
    return fail(SFI_ERR_INVALID_ARG, "q, k and v must be 16-byte aligned");
  const PagedPlan p = plan_paged(L);
  if ((s = check_workspace(ws, ws_bytes, p.total)) != SFI_OK) return s;
  const int D = L->head_dim;
  char* w = static_cast<char*>(ws);
  PagedAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.geo = geo_of(L, ws);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse_out;
  a.H_q = L->n_q_heads;
  a.G = L->n_q_heads / L->n_kv_heads;
  a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(D)));
  a.partials = reinterpret_cast<float*>(w + p.partials);
  a.wait_cycles = wait_limit_cycles();
  // A tile of 16 positions that lies in one page is one box per tensor; other
  // page sizes are gathered row by row.
  bool use_tma = false;
  if (L->dtype == SFI_BF16 && L->page_size % 16 == 0) {
    const uint64_t dims[3] = {64, uint64_t(pool_rows(L)), uint64_t(D / 64)};
    const uint64_t st[2] = {uint64_t(D) * 2, 128};
    const uint32_t box[3] = {64, 16, uint32_t(D / 64)};
    use_tma = encode_bf16_3d(&a.tmk, k, dims, st, box) && encode_bf16_3d(&a.tmv, v, dims, st, box);
    if (!use_tma) return fail(SFI_ERR_CUDA, "encoding the tensor maps of k and v failed");
  }
  const int grid = std::min(device_sm_count(), kPagedMaxGrid);
  const cudaError_t e = launch_paged_attn(a, D, L->dtype == SFI_F32, use_tma, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return SFI_OK;
}

sfi_status sfi_paged_append(const sfi_paged_layout* L, int32_t total_new, const void* k_new, const void* v_new,
                            int64_t k_stride, int64_t v_stride, const int32_t* cu_new, void* k, void* v, void* ws,
                            size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if (total_new < 0) return fail(SFI_ERR_INVALID_ARG, "total_new must be >= 0 (got %d)", total_new);
  if (!cu_new && total_new != L->batch)
    return fail(SFI_ERR_INVALID_ARG, "without cu_new there is a row for each of the %d sequences (got %d)", L->batch,
                total_new);
  const int64_t e = elem_bytes(L->dtype), row = int64_t(L->n_kv_heads) * L->head_dim;
  int64_t ks, vs;
  if ((s = row_stride("k_stride", k_stride, row, 16 / e, &ks)) != SFI_OK) return s;
  if ((s = row_stride("v_stride", v_stride, row, 16 / e, &vs)) != SFI_OK) return s;
  if ((s = check_workspace(ws, ws_bytes, plan_paged(L).total)) != SFI_OK) return s;
  if (!k || !v || (total_new > 0 && (!k_new || !v_new)))
    return fail(SFI_ERR_INVALID_ARG, "k_new, v_new, k and v must be set");
  if (misaligned16(k) || misaligned16(v) || (total_new > 0 && (misaligned16(k_new) || misaligned16(v_new))))
    return fail(SFI_ERR_INVALID_ARG, "k_new, v_new, k and v must be 16-byte aligned");
  if (total_new == 0) return SFI_OK;
  AppendArgs a;
  a.geo = geo_of(L, ws);
  a.k_new = static_cast<const uint8_t*>(k_new);
  a.v_new = static_cast<const uint8_t*>(v_new);
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.k_stride = ks * e;
  a.v_stride = vs * e;
  a.page_bytes = page_elems(L) * e;
  a.cu = cu_new;
  a.total = total_new;
  a.row_bytes = int(L->head_dim * e);
  const cudaError_t err = launch_append(a, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err, "append launch");
  return SFI_OK;
}

sfi_status sfi_pages_extend(const sfi_paged_layout* L, const sfi_page_store* S, const int32_t* n_new, void* ws,
                            size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if ((s = check_store(L, S, false)) != SFI_OK) return s;
  const PagedPlan p = plan_paged(L);
  if ((s = check_workspace(ws, ws_bytes, p.total)) != SFI_OK) return s;
  int32_t* const fresh = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + p.holes);
  const cudaError_t e = launch_extend(geo_of(L, ws), S->ref, n_new, fresh, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "extend launch");
  return SFI_OK;
}

sfi_status sfi_pages_fork(const sfi_paged_layout* L, const sfi_page_store* S, const int32_t* src, const int32_t* dst,
                          int32_t n, void* ws, size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if ((s = check_store(L, S, true)) != SFI_OK) return s;
  if ((s = check_list_size(n, L->batch)) != SFI_OK) return s;
  if (n > 0 && (!src || !dst)) return fail(SFI_ERR_INVALID_ARG, "src and dst must be set");
  SeqList from, to;
  if ((s = take_list("src", src, n, L->batch, false, &from)) != SFI_OK) return s;
  if ((s = take_list("dst", dst, n, L->batch, true, &to)) != SFI_OK) return s;
  bool is_dst[kMaxBatch] = {};
  for (int i = 0; i < n; ++i) is_dst[dst[i]] = true;
  for (int i = 0; i < n; ++i)
    if (is_dst[src[i]]) return fail(SFI_ERR_INVALID_ARG, "sequence %d is a source and a destination", src[i]);
  const PagedPlan p = plan_paged(L);
  if ((s = check_workspace(ws, ws_bytes, p.total)) != SFI_OK) return s;
  if (n == 0) return SFI_OK;
  int4* const jobs = reinterpret_cast<int4*>(static_cast<char*>(ws) + p.jobs);
  const cudaError_t e = launch_fork(geo_of(L, ws), S->ref, from, to, n, move_of(L, S, ws), jobs,
                                    static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fork launch");
  return SFI_OK;
}

sfi_status sfi_pages_free(const sfi_paged_layout* L, const sfi_page_store* S, const int32_t* seqs, int32_t n, void* ws,
                          size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if ((s = check_store(L, S, false)) != SFI_OK) return s;
  if ((s = check_list_size(n, L->batch)) != SFI_OK) return s;
  if (n > 0 && !seqs) return fail(SFI_ERR_INVALID_ARG, "seqs must be set");
  SeqList list;
  if ((s = take_list("seqs", seqs, n, L->batch, true, &list)) != SFI_OK) return s;
  if ((s = check_workspace(ws, ws_bytes, plan_paged(L).total)) != SFI_OK) return s;
  if (n == 0) return SFI_OK;
  const cudaError_t e = launch_free(geo_of(L, ws), S->ref, list, n, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "free launch");
  return SFI_OK;
}

sfi_status sfi_pages_compact(const sfi_paged_layout* L, const sfi_page_store* S, int32_t* new_id, void* ws,
                             size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if ((s = check_store(L, S, true)) != SFI_OK) return s;
  const PagedPlan p = plan_paged(L);
  if ((s = check_workspace(ws, ws_bytes, p.total)) != SFI_OK) return s;
  char* w = static_cast<char*>(ws);
  const cudaError_t e = launch_compact(geo_of(L, ws), S->ref, new_id, move_of(L, S, ws),
                                       reinterpret_cast<int32_t*>(w + p.map), reinterpret_cast<int32_t*>(w + p.holes),
                                       reinterpret_cast<int32_t*>(w + p.moved),
                                       reinterpret_cast<int32_t*>(w + p.n_moved), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "compaction launch");
  return SFI_OK;
}

sfi_status sfi_pages_copy(const sfi_paged_layout* L, const sfi_page_store* S, const int32_t* src, const int32_t* dst,
                          int32_t n, void* ws, size_t ws_bytes, sfi_stream stream) {
  sfi_status s = check_paged(L);
  if (s != SFI_OK) return s;
  if ((s = check_store(L, S, true)) != SFI_OK) return s;
  if (n < 0 || n > L->n_pages) return fail(SFI_ERR_INVALID_ARG, "n must lie in [0, n_pages] (got %d)", n);
  if (n > 0 && (!src || !dst)) return fail(SFI_ERR_INVALID_ARG, "src and dst must be device pointers");
  if ((s = check_workspace(ws, ws_bytes, plan_paged(L).total)) != SFI_OK) return s;
  if (n == 0) return SFI_OK;
  const cudaError_t e = launch_page_copy(move_of(L, S, ws), src, dst, n, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
  return SFI_OK;
}

}  // extern "C"

// C ABI of the norm and rotation of query and key heads: host-side validation,
// the frequencies as fractions of a turn, dispatch.  Every check happens before
// anything is enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "rope.h"
#include "sfi_internal.h"

namespace sfi {
namespace {

constexpr int kMaxHeads = 4096;

bool misaligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

sfi_status row_stride(const char* name, int64_t stride, int64_t row, int64_t unit, int64_t* out) {
  *out = stride == 0 ? row : stride;
  if (*out < row || *out % unit != 0)
    return fail(SFI_ERR_INVALID_ARG, "%s (%lld) must be 0, or at least a row of %lld elements and a multiple of %lld",
                name, (long long)stride, (long long)row, (long long)unit);
  if (*out >= (int64_t(1) << 38)) return fail(SFI_ERR_CAPACITY, "%s (%lld) exceeds 2^38 elements", name, (long long)stride);
  return SFI_OK;
}

// inv_freq / 2 pi modulo 1, in units of 2^-64: 1 / 2 pi as the sum of two doubles, and the product
// with both and its rounding error, so that it is off by less than 2^-100 of itself.
uint64_t turns_of(double inv_freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double p = inv_freq * kHi, rest = std::fma(inv_freq, kHi, -p) + inv_freq * kLo;
  const double whole = std::ldexp(p - std::trunc(p), 64);  // below 2^64 in magnitude, and exact
  const uint64_t x = whole < 0 ? 0 - static_cast<uint64_t>(-whole) : static_cast<uint64_t>(whole);
  const double y = std::ldexp(rest, 64);
  return std::fabs(y) < 9.2e18 ? x + static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(y))) : x;
}

}  // namespace
}  // namespace sfi

using namespace sfi;

extern "C" {

sfi_status sfi_qk_norm_rope(const sfi_rotary_layout* L, const void* q, const void* k, const void* q_weight,
                            const void* k_weight, void* q_out, void* k_out, sfi_stream stream) {
  if (!L) return fail(SFI_ERR_INVALID_ARG, "layout is NULL");
  if (L->total < 0) return fail(SFI_ERR_INVALID_ARG, "total must be >= 0 (got %d)", L->total);
  if (L->n_q_heads < 0 || L->n_kv_heads < 0 || (L->n_q_heads == 0 && L->n_kv_heads == 0))
    return fail(SFI_ERR_INVALID_ARG, "n_q_heads (%d) and n_kv_heads (%d) must be >= 0, and one of them positive",
                L->n_q_heads, L->n_kv_heads);
  if (L->n_q_heads > kMaxHeads || L->n_kv_heads > kMaxHeads)
    return fail(SFI_ERR_CAPACITY, "n_q_heads and n_kv_heads must be <= %d (got %d, %d)", kMaxHeads, L->n_q_heads,
                L->n_kv_heads);
  const int D = L->head_dim;
  if (D != 64 && D != 128) return fail(SFI_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", D);
  if (L->dtype != SFI_F32 && L->dtype != SFI_BF16)
    return fail(SFI_ERR_UNSUPPORTED, "dtype must be SFI_F32 or SFI_BF16 (got %d)", L->dtype);
  if (L->rotary_dim < 0 || L->rotary_dim > D || L->rotary_dim % 8 != 0)
    return fail(SFI_ERR_INVALID_ARG, "rotary_dim must be a multiple of 8 in [0, head_dim] (got %d)", L->rotary_dim);
  if (L->rotary_dim > 0 && !L->inv_freq) return fail(SFI_ERR_INVALID_ARG, "inv_freq (host) must be set");
  if (L->norm && !(L->eps >= 0.f && std::isfinite(L->eps)))
    return fail(SFI_ERR_INVALID_ARG, "eps must be >= 0 and finite (got %g)", double(L->eps));
  if (!L->norm && (q_weight || k_weight)) return fail(SFI_ERR_INVALID_ARG, "weights without a norm");
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int i = 0; i < L->rotary_dim / 2; ++i) {
    if (!(std::fabs(L->inv_freq[i]) <= 0x1p32))  // (beyond, the turns' fraction would lose bits)
      return fail(SFI_ERR_INVALID_ARG, "inv_freq[%d] (%g) must lie in [-2^32, 2^32]", i, L->inv_freq[i]);
    a.freq[i] = turns_of(L->inv_freq[i]);
  }
  const int unit = L->dtype == SFI_F32 ? 4 : 8;
  const int64_t rq = int64_t(L->n_q_heads) * D, rk = int64_t(L->n_kv_heads) * D;
  sfi_status s;
  if ((s = row_stride("q_stride", L->q_stride, rq, unit, &a.q_stride)) != SFI_OK) return s;
  if ((s = row_stride("k_stride", L->k_stride, rk, unit, &a.k_stride)) != SFI_OK) return s;
  if ((s = row_stride("q_out_stride", L->q_out_stride, rq, unit, &a.q_out_stride)) != SFI_OK) return s;
  if ((s = row_stride("k_out_stride", L->k_out_stride, rk, unit, &a.k_out_stride)) != SFI_OK) return s;
  if (L->total == 0) return SFI_OK;
  if (L->rotary_dim > 0 && !L->pos) return fail(SFI_ERR_INVALID_ARG, "pos must be a device pointer");
  if ((rq > 0 && (!q || !q_out)) || (rk > 0 && (!k || !k_out)))
    return fail(SFI_ERR_INVALID_ARG, "q, q_out (with query heads) and k, k_out (with KV heads) must be set");
  if ((rq > 0 && (misaligned16(q) || misaligned16(q_out) || misaligned16(q_weight))) ||
      (rk > 0 && (misaligned16(k) || misaligned16(k_out) || misaligned16(k_weight))))
    return fail(SFI_ERR_INVALID_ARG, "q, k, their weights and outputs must be 16-byte aligned");
  if ((rq > 0 && q == q_out && a.q_stride != a.q_out_stride && L->total > 1) ||
      (rk > 0 && k == k_out && a.k_stride != a.k_out_stride && L->total > 1))
    return fail(SFI_ERR_INVALID_ARG, "in place, rows and outputs have the same stride");
  a.q = q;
  a.k = k;
  a.wq = q_weight;
  a.wk = k_weight;
  a.q_out = q_out;
  a.k_out = k_out;
  a.pos = L->pos;
  a.total = L->total;
  a.H_q = L->n_q_heads;
  a.H_kv = L->n_kv_heads;
  a.rot = L->rotary_dim;
  a.pos_offset = L->pos_offset;
  a.norm = L->norm != 0;
  a.eps = L->eps;
  const cudaError_t e = launch_rope(a, D, L->dtype == SFI_F32, L->interleaved != 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotation launch");
  return SFI_OK;
}

}  // extern "C"

// The paged cache's bookkeeping and copies: storing new rows, extending, forking,
// freeing and compacting sequences, copying pages.
//
// The bookkeeping (tables, lengths, reference counts) is a few kilobytes of
// integers: one CTA does it, so that allocation needs no atomics between CTAs
// and its result does not depend on their order.  It is bound by the latency
// of a few dependent reads.  The copies are bound by HBM (read and write each
// row once) and run on all SMs in slices of 16 KB, 64 bytes in flight a thread.
// Measured (GPU time of a launch that finds nothing in L2): extending 64 sequences
// 3.7 us, freeing 3.6, a fork's plan 6.0 and its copies 6.6 (16 pages, 8 layers), a
// compaction's plan 4.6 and its moves of 352 MB 52 (6.77 TB/s), a token's rows for
// 64 sequences 6.0, a prompt batch's 267 MB 37 to 39.  Into a cache in 8 bits: 37000 positions of 8 heads
// of 128 in bf16 (231 MB) as e4m3 in 39.5, 5.8 TB/s (the issue slots are nearly as full: the rounding comes
// next after HBM), as int8 in 48, bound by the rounding; from fp32 (383 MB) in 60, 6.4 TB/s; a token's
// rows for 64 sequences 4.8.  (A token's first heads read before its sequence is looked up: 41.3, 52, 62, 5.9.)
// Free pages are looked for from the lowest on, 4096 counts a round of 0.9 us: extending
// 64 sequences takes 3.7 us where the first round finds them, 18 with the low 95% of
// 65000 pages taken, 223 of 10^6 and 4.2 ms of 2^24.
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "pdl.cuh"

namespace sfi {
namespace {

constexpr int kPlan = 1024;       // threads of a bookkeeping CTA
constexpr int kCopy = 256;        // threads of a copying CTA
constexpr int kSlice = 16 * 1024; // bytes that a copying CTA moves at a time
static_assert(kPlan >= kMaxBatch, "a thread for every sequence");

// Inclusive sum over the CTA (kPlan threads); `part` is 32 shared entries.
__device__ __forceinline__ long long block_scan(long long x, long long* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the entries of an earlier scan have been read
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long y = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    part[lane] = y;
  }
  __syncthreads();
  return x + (warp > 0 ? part[warp - 1] : 0);
}

// The first `want` free pages in ascending order, into fresh[0..); returns
// how many there are (at most want).
__device__ __forceinline__ int find_free(const int32_t* ref, int n_pages, long long want, int32_t* fresh,
                                         long long* part) {
  long long got = 0;
  for (int p0 = 0; p0 < n_pages && got < want; p0 += 4 * kPlan) {
    const int p = p0 + 4 * threadIdx.x;
    bool free[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free[i] = p + i < n_pages && ref[p + i] == 0;
      n += free[i];
    }
    long long at = got + block_scan(n, part) - n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free[i]) {
        if (at < want) fresh[at] = p + i;
        ++at;
      }
    got += part[31];
  }
  __syncthreads();
  return int(min(got, want));
}

__device__ __forceinline__ int pages_of(int n, int P) { return n / P + (n % P != 0); }

// Sequence b is no longer one that an extension refused.
__device__ __forceinline__ void forget_refusal(const PagedGeo& g, int b) { atomicAnd(g.refused + (b >> 5), ~(1u << (b & 31))); }

__global__ void __launch_bounds__(kPlan) extend_kernel(PagedGeo g, int32_t* ref, const int32_t* n_new,
                                                       int32_t* fresh) {
  __shared__ long long part[32];
  __shared__ int need[kMaxBatch], have[kMaxBatch];
  __shared__ long long at[kMaxBatch];
  const int b = threadIdx.x, warp = b >> 5, lane = b & 31;
  const int cap = g.max_pages * g.P;
  pdl_launch();
  pdl_wait();
  int n = 0, more = 0, want = 0;
  uint32_t flags = 0;
  if (b < g.B) {
    n = g.len[b];
    more = n_new ? n_new[b] : (n > 0 ? 1 : 0);
    if (n < 0 || n > cap || more < 0) {
      flags = SFI_DEV_LEN_OVER_CAP;
      more = n = 0;
    } else if (more > cap - n) {
      flags = SFI_DEV_NO_PAGES;
      more = 0;
    } else {
      want = pages_of(n + more, g.P) - pages_of(n, g.P);
    }
    have[b] = pages_of(n, g.P);
  }
  need[b] = want;
  const long long end = block_scan(want, part);
  at[b] = end - want;
  const long long total = part[31];
  __syncthreads();
  const int found = find_free(ref, g.n_pages, min(total, (long long)g.n_pages), fresh, part);
  if (found < total) {
    // too few: in order, whoever still fits
    if (b == 0) {
      int left = found;
      for (int i = 0; i < g.B; ++i) {
        at[i] = found - left;
        if (need[i] > left) need[i] = -1;
        else left -= need[i];
      }
    }
    __syncthreads();
    if (b < g.B && need[b] < 0) {
      flags |= SFI_DEV_NO_PAGES;
      more = 0;
    }
  }
  if (b < g.B && more > 0) g.len[b] = n + more;
  if (flags) set_status(g.status, flags);
  // whom an append has to leave out: who asked and was refused, until it is served
  const uint32_t bad = __ballot_sync(kFull, flags != 0), served = __ballot_sync(kFull, more > 0);
  if (lane == 0) {
    if (served) atomicAnd(g.refused + warp, ~served);
    if (bad) atomicOr(g.refused + warp, bad);
  }
  for (int s = warp; s < g.B; s += kPlan / 32)
    for (int i = lane; i < need[s]; i += 32) {
      const int p = fresh[at[s] + i];
      g.table[int64_t(s) * g.max_pages + have[s] + i] = p;
      ref[p] = 1;
    }
}

__global__ void __launch_bounds__(kPlan) fork_kernel(PagedGeo g, int32_t* ref, const __grid_constant__ SeqList src,
                                                     const __grid_constant__ SeqList dst, int n, int4* jobs) {
  __shared__ long long part[32];
  __shared__ int32_t fresh[kMaxBatch];
  __shared__ int full[kMaxBatch];  // first the pages that the source holds; then the full ones to share
  __shared__ bool outside[kMaxBatch];  // a page of the source lies outside the pool
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  pdl_launch();
  pdl_wait();
  int len = 0, need = 0, s = 0, t = 0;
  uint32_t flags = 0;
  bool in = false;
  if (i < n) {
    s = src.id[i], t = dst.id[i];
    len = g.len[s];
    if (len < 0 || len > g.max_pages * g.P) flags = SFI_DEV_LEN_OVER_CAP;
    else if (g.len[t] != 0) flags = SFI_DEV_BAD_INDEX;
    else in = true;
    full[i] = in ? pages_of(len, g.P) : 0;
  }
  __syncthreads();
  // (a warp reads the first pages of four pairs at once: 100 forks of 300 positions 10.8 us,
  // pair by pair 11.9)
  constexpr int W = kPlan / 32, AT_ONCE = 4;
  for (int j0 = warp; j0 < n; j0 += AT_ONCE * W) {
    int page[AT_ONCE];
#pragma unroll
    for (int e = 0; e < AT_ONCE; ++e) {
      const int j = j0 + e * W;
      page[e] = j < n && lane < full[j] ? g.table[int64_t(src.id[j]) * g.max_pages + lane] : 0;
    }
#pragma unroll
    for (int e = 0; e < AT_ONCE; ++e) {
      const int j = j0 + e * W;
      if (j >= n) break;
      const int32_t* const from = g.table + int64_t(src.id[j]) * g.max_pages;
      bool bad = uint32_t(page[e]) >= uint32_t(g.n_pages);
      for (int k = 32 + lane; k < full[j]; k += 32) bad |= uint32_t(from[k]) >= uint32_t(g.n_pages);
      bad = __any_sync(kFull, bad);
      if (lane == 0) outside[j] = bad;
    }
  }
  __syncthreads();
  if (i < n) {
    if (outside[i]) {
      flags = SFI_DEV_BAD_INDEX;
      in = false;
    }
    need = in && len % g.P != 0;
  }
  const int rank = int(block_scan(need, part)) - need;
  const int total = int(part[31]);
  __syncthreads();
  const int found = find_free(ref, g.n_pages, total, fresh, part);
  if (i < n) {
    if (need && rank >= found) {
      flags |= SFI_DEV_NO_PAGES;
      in = false;
    }
    full[i] = in ? len / g.P : 0;
    int4 job = make_int4(0, 0, 0, 0);
    if (in && need) {
      const int to = fresh[rank];
      job = make_int4(g.table[int64_t(s) * g.max_pages + len / g.P], to, len % g.P, 0);
      g.table[int64_t(t) * g.max_pages + len / g.P] = to;
      ref[to] = 1;
    }
    jobs[i] = job;
    if (in) g.len[t] = len, forget_refusal(g, t);
    if (flags) set_status(g.status, flags);
  }
  __syncthreads();
  for (int j = warp; j < n; j += kPlan / 32) {
    const int32_t* const from = g.table + int64_t(src.id[j]) * g.max_pages;
    int32_t* const to = g.table + int64_t(dst.id[j]) * g.max_pages;
    for (int k = lane; k < full[j]; k += 32) {
      const int p = from[k];
      to[k] = p;
      atomicAdd(ref + p, 1);
    }
  }
}

__global__ void __launch_bounds__(kCopy) free_kernel(PagedGeo g, int32_t* ref, const __grid_constant__ SeqList seqs) {
  pdl_launch();
  pdl_wait();
  const int b = seqs.id[blockIdx.x];
  const int n = g.len[b];
  if (n < 0 || n > g.max_pages * g.P) {
    if (threadIdx.x == 0) set_status(g.status, SFI_DEV_LEN_OVER_CAP);
    return;
  }
  int32_t* const row = g.table + int64_t(b) * g.max_pages;
  for (int i = threadIdx.x; i < pages_of(n, g.P); i += kCopy) {
    const int p = row[i];
    row[i] = -1;
    // (a count that is zero gets back what was taken off, whatever the order of the
    // decrements; between the two it may read as less)
    bool bad = p < 0 || p >= g.n_pages;
    if (!bad && atomicSub(ref + p, 1) <= 0) {
      atomicAdd(ref + p, 1);
      bad = true;
    }
    if (bad) set_status(g.status, SFI_DEV_BAD_INDEX);
  }
  __syncthreads();
  if (threadIdx.x == 0) g.len[b] = 0, forget_refusal(g, b);
}

// x / y for 0 <= x, 0 < y: in 32 bits where they do (a tenth of the time).
__device__ __forceinline__ long long div_fast(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)(uint32_t(x) / uint32_t(y)) : x / y;
}

// Bytes [0, n) from src to dst (both 16-byte aligned), by one CTA.
__device__ __forceinline__ void copy_slice(uint8_t* dst, const uint8_t* src, int n) {
  const uint4* const s = reinterpret_cast<const uint4*>(src);
  uint4* const d = reinterpret_cast<uint4*>(dst);
  n >>= 4;
  for (int i = threadIdx.x; i < n; i += 4 * kCopy) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopy < n) v[k] = __ldcs(s + i + k * kCopy);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopy < n) __stcs(d + i + k * kCopy, v[k]);
  }
}

// Item `item` of a whole page's copy: a page is one run of `bytes` in each
// (layer, k or v), cut into `slices`.
__device__ __forceinline__ void copy_page_item(const PageMove& mv, int bytes, int slices, int src, int dst, int item) {
  const int sl = item % slices, lk = item / slices;
  const int64_t off = int64_t(lk >> 1) * mv.layer_bytes + int64_t(sl) * kSlice;
  uint8_t* const pool = ((lk & 1) ? mv.v : mv.k) + off;
  copy_slice(pool + dst * mv.page_bytes, pool + src * mv.page_bytes, min(kSlice, bytes - sl * kSlice));
}

// The partly filled pages of forks: job (source, new page, rows); rows of one
// head are one run.
__global__ void __launch_bounds__(kCopy) fork_copy_kernel(const __grid_constant__ PageMove mv, const int4* jobs, int n) {
  pdl_launch();
  pdl_wait();
  const int slices = (mv.P * mv.row_bytes + kSlice - 1) / kSlice;
  const long long per = (long long)mv.n_layers * 2 * mv.H_kv * slices, items = per * n;
  for (long long x = blockIdx.x; x < items; x += gridDim.x) {
    const long long i = div_fast(x, per);
    const int4 job = jobs[i];
    uint32_t y = uint32_t(x - i * per);
    const int sl = int(y % slices);
    y /= slices;
    const int h = int(y % mv.H_kv);
    y /= mv.H_kv;
    const int bytes = job.z * mv.row_bytes - sl * kSlice;
    if (bytes <= 0) continue;
    if (mv.scale_at && sl == 0) {
      uint8_t* const scales = ((y & 1) ? mv.v : mv.k) + (y >> 1) * mv.layer_bytes + mv.scale_at + int64_t(h) * mv.P * 4;
      for (int r = threadIdx.x; r < job.z; r += kCopy)
        reinterpret_cast<float*>(scales + job.y * mv.page_bytes)[r] =
            reinterpret_cast<const float*>(scales + job.x * mv.page_bytes)[r];
    }
    uint8_t* const pool = ((y & 1) ? mv.v : mv.k) + (y >> 1) * mv.layer_bytes + int64_t(h) * mv.P * mv.row_bytes +
                          int64_t(sl) * kSlice;
    copy_slice(pool + job.y * mv.page_bytes, pool + job.x * mv.page_bytes, min(kSlice, bytes));
  }
}

__global__ void __launch_bounds__(kCopy) page_copy_kernel(const __grid_constant__ PageMove mv, const int32_t* src,
                                                          const int32_t* dst, int n) {
  pdl_launch();
  pdl_wait();
  const int bytes = mv.whole, slices = (bytes + kSlice - 1) / kSlice;
  const int per = mv.n_layers * 2 * slices;
  for (long long x = blockIdx.x; x < (long long)per * n; x += gridDim.x) {
    const int i = int(div_fast(x, per)), from = src[i], to = dst[i];
    if (from < 0 || from >= mv.n_pages || to < 0 || to >= mv.n_pages) {
      if (threadIdx.x == 0) set_status(mv.status, SFI_DEV_BAD_INDEX);
    } else if (from != to) {
      copy_page_item(mv, bytes, slices, from, to, int(x - (long long)i * per));
    }
  }
}

// The plan of a compaction: which used page at or past n_live goes to which
// free page before it.  Every CTA counts the pages before its own part for
// itself (the counts are small and stay in L2), so that one launch does.
//   map[p]: p for a page that stays, -1 for a free one, -2 - r for the r-th that moves
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const int32_t* ref, int n_pages, int chunk, int32_t* map,
                                                             int32_t* holes, int32_t* moved, int32_t* n_moved) {
  __shared__ long long part[32];
  pdl_launch();
  pdl_wait();
  const int lo = blockIdx.x * chunk, hi = min(lo + chunk, n_pages);
  int all = 0, before = 0;
  for (int p = threadIdx.x; p < n_pages; p += kPlan) {
    const int live = ref[p] != 0;
    all += live;
    before += live && p < lo;
  }
  block_scan(all, part);
  const int n_live = int(part[31]);
  block_scan(before, part);
  int run = int(part[31]);  // used pages before the CTA's part
  int low = 0;              // used pages before n_live
  for (int p = threadIdx.x; p < n_live; p += kPlan) low += ref[p] != 0;
  block_scan(low, part);
  low = int(part[31]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_moved = n_live - low;
  for (int p0 = lo; p0 < hi; p0 += kPlan) {
    const int p = p0 + threadIdx.x;
    const int live = p < hi && ref[p] != 0;
    const int r = run + int(block_scan(live, part)) - live;  // used pages before p
    run += int(part[31]);
    if (p >= hi) continue;
    int to = -1;
    if (p < n_live) {
      if (live) to = p;
      else holes[p - r] = p;
    } else if (live) {
      moved[r - low] = p;
      to = -2 - (r - low);
    }
    map[p] = to;
  }
}

// The moves, and the counts, tables and ids that follow them.
__global__ void __launch_bounds__(kCopy) compact_kernel(const __grid_constant__ PageMove mv, PagedGeo g, int32_t* ref,
                                                        int32_t* new_id, const int32_t* map, const int32_t* holes,
                                                        const int32_t* moved, const int32_t* n_moved) {
  pdl_launch();
  pdl_wait();
  const int n = *n_moved;
  const long long tid = (long long)blockIdx.x * kCopy + threadIdx.x, all = (long long)gridDim.x * kCopy;
  for (long long i = tid; i < n; i += all) {
    const int from = moved[i], to = holes[i];
    ref[to] = ref[from];
    ref[from] = 0;
  }
  if (new_id)
    for (long long p = tid; p < g.n_pages; p += all) {
      const int m = map[p];
      new_id[p] = m < -1 ? holes[-2 - m] : m;
    }
  for (int b = blockIdx.x; b < g.B; b += gridDim.x) {
    const int len = g.len[b];
    if (len < 0 || len > g.max_pages * g.P) {
      if (threadIdx.x == 0) set_status(g.status, SFI_DEV_LEN_OVER_CAP);
      continue;
    }
    int32_t* const row = g.table + int64_t(b) * g.max_pages;
    for (int i = threadIdx.x; i < pages_of(len, g.P); i += kCopy) {
      const int p = row[i];
      const int m = p >= 0 && p < g.n_pages ? map[p] : -1;
      if (m == -1) set_status(g.status, SFI_DEV_BAD_INDEX);  // held, but outside the pool or counted free
      else if (m < -1) row[i] = holes[-2 - m];
    }
  }
  const int bytes = mv.whole, slices = (bytes + kSlice - 1) / kSlice;
  const int per = mv.n_layers * 2 * slices;
  for (long long x = blockIdx.x; x < (long long)per * n; x += gridDim.x) {
    const int i = int(div_fast(x, per));
    copy_page_item(mv, bytes, slices, moved[i], holes[i], int(x - (long long)i * per));
  }
}

// Row t of the new ones, the `back`-th last of the m of sequence b, by one warp.
__device__ __forceinline__ void append_row(const AppendArgs& a, int b, int m, int back, int t, int cap, int lane) {
  const PagedGeo& g = a.geo;
  const int n = g.len[b];
  const uint32_t refused = g.refused[b >> 5] >> (b & 31) & 1;  // (read beside the length, not behind its check)
  if ((n < 0) | (n > cap) | (m > n) | refused) return;
  const int pos = n - back;
  const int page = g.table[int64_t(b) * g.max_pages + pos / g.P];
  if (page < 0 || page >= g.n_pages) {
    if (lane == 0) set_status(g.status, SFI_DEV_BAD_INDEX);
    return;
  }
  const int per = a.row_bytes / 16;  // chunks of a head's row: 8, 16 or 32
  const int chunks = g.H_kv * per;
  const uint4* const ks = reinterpret_cast<const uint4*>(a.k_new + t * a.k_stride);
  const uint4* const vs = reinterpret_cast<const uint4*>(a.v_new + t * a.v_stride);
  const int64_t at = page * a.page_bytes + int64_t(pos % g.P) * a.row_bytes;
  for (int i = lane; i < chunks; i += 64) {
    uint4 k[2], v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (i + 32 * e < chunks) k[e] = __ldcs(ks + i + 32 * e), v[e] = __ldcs(vs + i + 32 * e);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = i + 32 * e;
      if (x >= chunks) break;
      const int64_t to = at + int64_t(x / per) * g.P * a.row_bytes + (x % per) * 16;
      *reinterpret_cast<uint4*>(a.k + to) = k[e];
      *reinterpret_cast<uint4*>(a.v + to) = v[e];
    }
  }
}

// 8 elements of a row as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = __ldcs(reinterpret_cast<const float4*>(p)), v[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = v[0].x, x[1] = v[0].y, x[2] = v[0].z, x[3] = v[0].w, x[4] = v[1].x, x[5] = v[1].y, x[6] = v[1].z, x[7] = v[1].w;
  }
  // The largest magnitude over the row's LPH lanes, as its bits (those of an infinity or a NaN are
  // larger than any number's).
  template <int LPH>
  __device__ __forceinline__ uint32_t top() const {
    float x[8];
    get(x);
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
    for (int w = 1; w < LPH; w <<= 1) t = max(t, __shfl_xor_sync(kFull, t, w));
    return t;
  }
};
template <>
struct Eight<bf16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const { Unpack<bf16_t>::run(v, x); }
  // (two at a time: magnitudes compare as 16-bit numbers)
  template <int LPH>
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
#pragma unroll
    for (int w = 1; w < LPH; w <<= 1) t = __vmaxu2(t, __shfl_xor_sync(kFull, t, w));
    return max(t & 0xffff0000u, t << 16);
  }
};

// Codes of 8 elements of a row whose largest magnitude is `top` (bits), and the row's scale.
//
// int8: x / s is rounded as if it were exact.  n = rint(x * (1 / s)) is off by one at most, and
// only next to a tie; e = x - n s is exact in fp32 (a multiple of the smaller of both
// last places, below s in magnitude), so comparing it with s / 2 decides: half of the maximum
// is such a tie in every row (63.5), and the rounded quotient would put it on either side.
// rint by an addition of 1.5 * 2^23, whose last byte is then the code.
// e4m3: the scale is a power of two, so x / s is exact and the conversion rounds once.
// Rows whose maximum lies outside [2^-60, 2^100] take a longer way: there 1 / s or e could leave
// fp32's normal numbers.
template <bool E4M3>
__device__ __noinline__ uint2 quantise_far(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                           uint32_t top, float* scale) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  if (top >= 0x7f800000u) {
    *scale = __uint_as_float(0x7fc00000u);
    return make_uint2(0, 0);
  }
  const float amax = __uint_as_float(top);
  uint32_t w[2] = {0, 0};
  if constexpr (E4M3) {
    const bool tiny = amax < 0x1p-126f;  // (scaled up to read its exponent)
    const uint32_t bits = tiny ? __float_as_uint(amax * 0x1p64f) : top;
    const int k = int(bits >> 23) - 127 - (tiny ? 64 : 0) - 8 + ((bits & 0x7fffffu) > 0x600000u);
    const float s = amax == 0.f || k < -149 ? 0.f : k < -126 ? __uint_as_float(1u << (k + 149)) : __uint_as_float(uint32_t(k + 127) << 23);
    *scale = s;
    if (s == 0.f) return make_uint2(0, 0);
    const int k0 = -k / 2, k1 = -k - k0;  // (1 / s may be beyond fp32)
    const float f0 = __uint_as_float(uint32_t(k0 + 127) << 23), f1 = __uint_as_float(uint32_t(k1 + 127) << 23);
    for (int i = 0; i < 4; ++i) {
      uint16_t c;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x[2 * i + 1] * f0 * f1), "f"(x[2 * i] * f0 * f1));
      w[i / 2] |= uint32_t(c) << (i % 2 * 16);
    }
  } else {
    float s = amax / 127.f;
    *scale = s;
    if (s == 0.f) return make_uint2(0, 0);
    const float up = amax < 0x1p-60f ? 0x1p80f : 1.f;  // both sides of the quotient, so that nothing underflows
    s *= up;
    const float inv = 1.f / s, half = 0.5f * s;
    for (int i = 0; i < 8; ++i) {
      const float y = x[i] * up;
      float n = rintf(y * inv);
      const float e = fmaf(-n, s, y);
      if (fabsf(e) > half || (fabsf(e) == half && (int(n) & 1))) n += copysignf(1.f, e);
      n = fminf(fmaxf(n, -127.f), 127.f);  // (a subnormal scale may be much too small)
      w[i / 4] |= (uint32_t(int(n)) & 0xffu) << (i % 4 * 8);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <bool E4M3>
__device__ __forceinline__ uint2 quantise(const float (&x)[8], uint32_t top, float* scale) {
  if (top < 0x21800000u || top > 0x71800000u)  // 2^-60, 2^100
    return quantise_far<E4M3>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], top, scale);
  uint32_t w[2];
  if constexpr (E4M3) {
    // amax = m 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8: s = 2^k, k = e - 8, or e - 7 where m > 1.75
    const uint32_t k = (top + 0x1fffffu) >> 23;  // e + 127, + 1
    *scale = __uint_as_float((k - 8) << 23);
    const float f = __uint_as_float((254 + 8 - k) << 23);
    const uint64_t ff = pair(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t p = mul2(pair(x[4 * i], x[4 * i + 1]), ff), q = mul2(pair(x[4 * i + 2], x[4 * i + 3]), ff);
      asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
          "mov.b32 %0, {l, h};\n\t}"
          : "=r"(w[i])
          : "f"(lo(p)), "f"(hi(p)), "f"(lo(q)), "f"(hi(q)));
    }
  } else {
    constexpr float BIG = 12582912.f;
    // max / 127 by the rounded reciprocal and one correction by the remainder, which rounds the quotient
    // correctly (Markstein's theorem; all 2^23 significands were compared).  1 / s may be off.
    constexpr float kInv = 1.f / 127.f;
    const float amax = __uint_as_float(top), s0 = amax * kInv, s = fmaf(fmaf(-s0, 127.f, amax), kInv, s0);
    const float inv = __fdividef(1.f, s), half = 0.5f * s;
    *scale = s;
    float t[8], worst = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t p = pair(x[2 * i], x[2 * i + 1]), z = fma2(p, pair(inv, inv), pair(BIG, BIG));
      const uint64_t n = add2(z, pair(-BIG, -BIG)), e = fma2(n, pair(-s, -s), p);
      t[2 * i] = lo(z), t[2 * i + 1] = hi(z);
      worst = fmaxf(worst, fmaxf(fabsf(lo(e)), fabsf(hi(e))));
    }
    if (worst >= half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = t[i] - BIG, e = fmaf(-n, s, x[i]);
        if (fabsf(e) > half || (fabsf(e) == half && (__float_as_uint(t[i]) & 1))) t[i] += copysignf(1.f, e);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                         __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040), 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

// A token's rows into an 8-bit pool: d / 8 lanes a head, K and V of `AHEAD` heads read at once.
template <typename T, bool E4M3, int D>
struct Quant : QuantArgs {};

template <typename T, bool E4M3, int D>
__device__ __forceinline__ void append_row(const Quant<T, E4M3, D>& a, int b, int m, int back, int t, int cap, int lane) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, AHEAD = 2;
  const PagedGeo& g = a.geo;
  const int n = g.len[b];
  const uint32_t refused = g.refused[b >> 5] >> (b & 31) & 1;
  if ((n < 0) | (n > cap) | (m > n) | refused) return;
  const int pos = n - back;
  const int page = g.table[int64_t(b) * g.max_pages + pos / g.P];
  if (page < 0 || page >= g.n_pages) {
    if (lane == 0) set_status(g.status, SFI_DEV_BAD_INDEX);
    return;
  }
  const T* const src[2] = {reinterpret_cast<const T*>(a.k_new + t * a.k_stride),
                           reinterpret_cast<const T*>(a.v_new + t * a.v_stride)};
  const int64_t at = page * a.page_bytes;
  uint8_t* const dst[2] = {a.k + at, a.v + at};
  const int in = pos % g.P, u = lane % LPH;
  for (int h0 = lane / LPH; h0 - lane / LPH < g.H_kv; h0 += AHEAD * HPW) {
    Eight<T> r[AHEAD][2];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int h = h0 + i * HPW;
        if (h < g.H_kv) r[i][y].load(src[y] + h * D + u * 8);
        else r[i][y].clear();
      }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t top = r[i][y].template top<LPH>();
        float x[8], scale;
        r[i][y].get(x);
        const uint2 codes = quantise<E4M3>(x, top, &scale);
        const int h = h0 + i * HPW;
        if (h >= g.H_kv) continue;
        const int64_t row = int64_t(h) * g.P + in;
        *reinterpret_cast<uint2*>(dst[y] + row * D + u * 8) = codes;
        if (u == 0) *reinterpret_cast<float*>(dst[y] + a.scale_at + row * 4) = scale;
      }
  }
}

// New rows into their pages: a warp takes one token's K and V, for each sequence that
// holds the token: one, where the offsets ascend; where some do not, those that are in
// order are stored all the same, so all pairs are looked through (by each warp for its
// token up to 32 sequences, else by the CTA for its eight; a search by halves would miss
// some).  A sequence that an extension refused holds the length from before it: the rows
// would go over its last ones, which may lie in pages that others share, so it is left
// out.  The last CTA only looks for what is to be flagged.
template <typename Args>
constexpr int kAppendCtas = 1;  // on an SM at least: registers for more rows on their way
template <typename T, bool E4M3, int D>
constexpr int kAppendCtas<Quant<T, E4M3, D>> = sizeof(T) == 2 ? 6 : 5;
template <typename Args>
__global__ void __launch_bounds__(kCopy, kAppendCtas<Args>) append_kernel(const __grid_constant__ Args a) {
  constexpr int kWarps = kCopy / 32;
  __shared__ uint32_t mask[kMaxBatch / 32];  // sequences with rows among the CTA's tokens
  static_assert(kMaxBatch / 32 == 32, "a lane for every word");
  const PagedGeo& g = a.geo;
  pdl_launch();
  pdl_wait();
  const int cap = g.max_pages * g.P;
  if (blockIdx.x == gridDim.x - 1) {
    for (int b = threadIdx.x; b < g.B; b += kCopy) {
      const int n = g.len[b];
      bool bad = n < 0 || n > cap, refused = g.refused[b >> 5] >> (b & 31) & 1;
      if (a.cu) {
        const int c0 = a.cu[b], c1 = a.cu[b + 1];
        refused = refused && c0 < c1;
        bad = bad || c0 < 0 || c1 < c0 || c1 > a.total || (c1 - c0 > n && !refused);
      }
      if (bad || refused) set_status(g.status, (bad ? SFI_DEV_LEN_OVER_CAP : 0u) | (refused ? SFI_DEV_NO_PAGES : 0u));
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * kWarps, t = t0 + warp;
  // of the pairs that are in order, does b's hold some of the rows [from, from + n)?
  auto holds = [&](int b, int from, int n) {
    if (b >= g.B) return false;
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    return c0 >= 0 && c1 <= a.total && c0 < c1 && c0 - from < n && c1 > from;
  };
  uint32_t word;  // the lane's 32 sequences
  if (!a.cu) {
    word = lane == t >> 5 ? 1u << (t & 31) : 0;
  } else if (g.B <= 32) {
    const uint32_t in = __ballot_sync(kFull, holds(lane, t, 1));
    word = lane == 0 ? in : 0;
  } else {
#pragma unroll
    for (int w = warp; w < 32; w += kWarps) {
      const uint32_t in = __ballot_sync(kFull, holds(w * 32 + lane, t0, kWarps));
      if (lane == 0) mask[w] = in;
    }
    __syncthreads();
    word = mask[lane];
  }
  if (t >= a.total) return;
  for (uint32_t words = __ballot_sync(kFull, word != 0); words; words &= words - 1) {
    const int w = __ffs(words) - 1;
    for (uint32_t bits = __shfl_sync(kFull, word, w); bits; bits &= bits - 1) {
      const int b = w * 32 + __ffs(bits) - 1;
      const int c0 = a.cu ? a.cu[b] : t, c1 = a.cu ? a.cu[b + 1] : t + 1;
      if (t >= c0 && t < c1) append_row(a, b, c1 - c0, c1 - t, t, cap, lane);
    }
  }
}

// CTAs of a copy of at most `items` slices: eight to an SM keep HBM busy.
int copy_grid(long long items) {
  const long long most = 8LL * device_sm_count();
  return int(items < 1 ? 1 : items < most ? items : most);
}

long long page_slices(const PageMove& mv) {
  return (long long)mv.n_layers * 2 * ((mv.whole + kSlice - 1LL) / kSlice);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  return launch_pdl(append_kernel<AppendArgs>, dim3((a.total - 1) / (kCopy / 32) + 2), kCopy, 0, st, a);
}

template <typename T, bool E4M3, int D>
static cudaError_t launch_quant(const QuantArgs& a, cudaStream_t st) {
  return launch_pdl(append_kernel<Quant<T, E4M3, D>>, dim3((a.total - 1) / (kCopy / 32) + 2), kCopy, 0, st,
                    Quant<T, E4M3, D>{a});
}

cudaError_t launch_append_q8(const QuantArgs& a, bool f32, bool e4m3, cudaStream_t st) {
  if (a.row_bytes == 64) {
    if (f32) return e4m3 ? launch_quant<float, true, 64>(a, st) : launch_quant<float, false, 64>(a, st);
    return e4m3 ? launch_quant<bf16_t, true, 64>(a, st) : launch_quant<bf16_t, false, 64>(a, st);
  }
  if (f32) return e4m3 ? launch_quant<float, true, 128>(a, st) : launch_quant<float, false, 128>(a, st);
  return e4m3 ? launch_quant<bf16_t, true, 128>(a, st) : launch_quant<bf16_t, false, 128>(a, st);
}

cudaError_t launch_extend(const PagedGeo& g, int32_t* ref, const int32_t* n_new, int32_t* fresh, cudaStream_t st) {
  return launch_pdl(extend_kernel, dim3(1), kPlan, 0, st, g, ref, n_new, fresh);
}

cudaError_t launch_fork(const PagedGeo& g, int32_t* ref, const SeqList& src, const SeqList& dst, int n,
                        const PageMove& mv, int4* jobs, cudaStream_t st) {
  const cudaError_t e = launch_pdl(fork_kernel, dim3(1), kPlan, 0, st, g, ref, src, dst, n, jobs);
  if (e != cudaSuccess) return e;
  const long long slices = ((long long)mv.P * mv.row_bytes + kSlice - 1) / kSlice;
  return launch_pdl(fork_copy_kernel, dim3(copy_grid(slices * mv.H_kv * 2 * mv.n_layers * n)), kCopy, 0, st, mv, jobs, n);
}

cudaError_t launch_free(const PagedGeo& g, int32_t* ref, const SeqList& seqs, int n, cudaStream_t st) {
  return launch_pdl(free_kernel, dim3(n), kCopy, 0, st, g, ref, seqs);
}

cudaError_t launch_compact(const PagedGeo& g, int32_t* ref, int32_t* new_id, const PageMove& mv, int32_t* map,
                           int32_t* holes, int32_t* moved, int32_t* n_moved, cudaStream_t st) {
  // parts of whole rounds of a CTA, at most one CTA to an SM
  const int rounds = (g.n_pages + kPlan - 1) / kPlan, sms = device_sm_count();
  const int chunk = (rounds + sms - 1) / sms * kPlan;
  const cudaError_t e = launch_pdl(compact_plan_kernel, dim3((g.n_pages + chunk - 1) / chunk), kPlan, 0, st, ref,
                                   g.n_pages, chunk, map, holes, moved, n_moved);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_kernel, dim3(copy_grid(page_slices(mv) * g.n_pages)), kCopy, 0, st, mv, g, ref, new_id, map,
                    holes, moved, n_moved);
}

cudaError_t launch_page_copy(const PageMove& mv, const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
  return launch_pdl(page_copy_kernel, dim3(copy_grid(page_slices(mv) * n)), kCopy, 0, st, mv, src, dst, n);
}

}  // namespace sfi

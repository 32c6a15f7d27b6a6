// What the attentions of one token over a paged cache have in common: the line of
// tiles and how it is cut into shares, the lookup of a tile's unit, the states of
// pieces and the kernel that joins them.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.h"
#include "pdl.cuh"
#include "tc5_attn.cuh"

namespace sfi {
namespace {

constexpr int kWarps = kPagedWarps;                    // that attend
constexpr int kThreads = kWarps * 32;        // of them
constexpr int kProducers = 4;                // warps that copy
constexpr int kAllThreads = kThreads + kProducers * 32;
constexpr int kAttendRegs = 216, kCopyRegs = 72;  // of 168 each at launch: 2 * 216 + 72 = 3 * 168

// Tiles of one KV head in the sequences before each, in shared memory.
struct Line {
  long long pre[kMaxBatch + 1];
  long long part[kWarps];
};

// How the line of `total` tiles is cut: into shares of equal size, one for each of
// `grid` CTAs.  (With the last quarter of each share as three smaller items, taken
// from a counter, the CTAs end closer together: 492 us instead of 500 for 32 sequences
// of 4096 to 65536, 161.5 instead of 163 for 8 x 32768; but each item costs a merge, a
// longer join and registers: 60 instead of 53 us for 64 x 1000, 150 instead of 133 for
// 8 x ~24000 with 16 heads a group, 189 instead of 176 for 8 x 32768 in fp32 with d = 64.)
struct Cut {
  long long total, per, wide;  // tiles of a share; those before `wide` belong to shares with one more
  int shares, extra;           // extra: shares with one tile more

  // few tiles: fewer shares, of at least `least` (a tile for each warp)
  __device__ __forceinline__ Cut(long long total_, int grid, int least = kWarps) {
    total = total_;
    const long long most = (total + least - 1) / least;
    shares = most < grid ? int(most) : grid;
    // (a 64-bit division takes ~10 times as long)
    per = shares <= 0 ? 0 : total < (1LL << 31) ? (long long)(uint32_t(total) / uint32_t(shares)) : total / shares;
    extra = shares > 0 ? int(total - per * shares) : 0;
    wide = extra * (per + 1);
  }
  __device__ __forceinline__ long long start(int share) const { return share * per + min(share, extra); }
  // the share that holds tile x
  __device__ __forceinline__ int holder(long long x) const {
    if (total < (1LL << 31))
      return x < wide ? int(uint32_t(x) / uint32_t(per + 1)) : extra + int(uint32_t(x - wide) / uint32_t(per));
    return int(x < wide ? x / (per + 1) : extra + (x - wide) / per);
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 16 bytes, of which `bytes` (0 or 16) are read and the rest are zero.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// A place in the line of tiles: the unit (sequence b, KV head g) whose tiles
// are [begin, end).
struct Unit {
  int b, g;
  long long begin, end;
};

__device__ __forceinline__ void unit_next(Unit& u, const Line& ln, int B, int H_kv) {
  if (++u.g == H_kv) {
    u.g = 0;
    ++u.b;
  }
  u.begin = u.end;
  if (u.b < B) u.end += ln.pre[u.b + 1] - ln.pre[u.b];  // else the line's end
}

// The unit that holds tile x (x below the line's end).
__device__ __forceinline__ Unit unit_at(long long x, const Line& ln, int B, int H_kv) {
  int lo = 0, hi = B;  // last b with pre[b] * H_kv <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ln.pre[mid] * H_kv <= x) lo = mid;
    else hi = mid;
  }
  const long long nt = ln.pre[lo + 1] - ln.pre[lo];
  const long long in = x - ln.pre[lo] * H_kv;
  Unit u;
  u.b = lo;
  u.g = in < (1LL << 31) ? int(uint32_t(in) / uint32_t(nt)) : int(in / nt);
  u.begin = ln.pre[lo] * H_kv + u.g * nt;
  u.end = u.begin + nt;
  return u;
}

// Pages at the start of sequence b that are left out (SKIP: geo.skip is set).
template <bool SKIP>
__device__ __forceinline__ int skipped(const PagedGeo& geo, int b) { return SKIP ? geo.skip[b] : 0; }

// Fills `ln` (the first kThreads threads of a CTA); `flag` reports lengths out of
// range.
template <int TR, bool SKIP = false>
__device__ __forceinline__ void scan_lengths(const PagedGeo& geo, Line& ln, bool flag) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = geo.B, cap = geo.max_pages * geo.P;
  auto tiles = [&](int b) {
    int n = b < B ? geo.len[b] : 0;
    if (n < 0 || n > cap) {
      if (flag) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
      n = n < 0 ? 0 : cap;
    }
    if (SKIP && b < B) n -= skipped<SKIP>(geo, b) * geo.P;
    return (n + TR - 1) / TR;
  };
  auto scan = [&](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  if (B <= 32) {
    if (warp == 0) {
      const long long run = scan(tiles(lane));
      if (lane < B) ln.pre[lane + 1] = run;
      if (lane == 0) ln.pre[0] = 0;
    }
    __syncthreads();
    return;
  }
  // (what lies behind the last sequence counts nothing, so the threads behind
  // kThreads do no harm)
  constexpr int PER = kMaxBatch / kThreads;
  int nt[PER];
  long long mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += nt[i] = tiles(tid * PER + i);
  const long long run = scan(mine);
  if (lane == 31 && warp < kWarps) ln.part[warp] = run;
  __syncthreads();
  long long before = run - mine;
  for (int w = 0; w < min(warp, kWarps); ++w) before += ln.part[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < B) ln.pre[b] = before;
    before += nt[i];
    if (b == B - 1) ln.pre[B] = before;
  }
  __syncthreads();
}

__device__ __forceinline__ void attend_sync() { named_bar_sync(1, kThreads); }

// The first tile from `from` on whose number is r modulo m (a power of two).
__device__ __forceinline__ long long first_of(long long from, int r, int m) { return from + ((r - from) & (m - 1)); }

// Joins the pieces of each unit that has several, in their order:
//   out = sum_w f_w o_w / sum_w f_w l_w,  f_w = 2^(c (m_w - max m)).
// Up to 16 pieces: a thread for each output.  More: 32 outputs a CTA, the pieces
// dealt over its warps, and the warps' sums joined.  Bound by the latency of two or
// three reads from L2.
struct Joined {
  float m = -INFINITY, l = 0.f, o = 0.f;
  // N pieces from `p` on, `step` floats apart, of which `n` are there; output d
  template <int N>
  __device__ __forceinline__ void add(const float* p, int64_t step, int n, int d, int D, float c) {
    float mv[N], lv[N], ov[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      mv[e] = e < n ? __ldcg(p + e * step + D) : -INFINITY;
      lv[e] = e < n ? __ldcg(p + e * step + D + 1) : 0.f;
      ov[e] = e < n ? __ldcg(p + e * step + d) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) add(mv[e], lv[e], ov[e], c);
  }
  __device__ __forceinline__ void add(float m_, float l_, float o_, float c) {
    if (m_ == -INFINITY && l_ == 0.f) return;  // saw only scores of -infinity, or nothing
    const float top = fmaxf(m, m_), f = ex2((m - top) * c), f_ = ex2((m_ - top) * c);
    const bool none = m == -INFINITY && l == 0.f;
    l = (none ? 0.f : f * l) + f_ * l_;
    o = (none ? 0.f : f * o) + f_ * o_;
    m = top;
  }
  __device__ __forceinline__ void put(const PagedAttnArgs& a, int64_t qrow, int h, int d, int D, float c) const {
    a.out[qrow + h * D + d] = l == 0.f ? 0.f : o / l;
    if (d == 0 && a.lse) a.lse[qrow / D + h] = (m * c + log2f(l)) * 0.6931471805599453f;
  }
};

// By CTA (bx, by) of nx x ny; SKIP: single pieces too, and no units of which something is left out.
template <int TR, int D, bool SKIP = false>
__device__ __forceinline__ void join_units(const PagedAttnArgs& a, const Line& ln, const Cut& cut, int bx, int nx, int by,
                                           int ny) {
  constexpr int AHEAD = 8;  // pieces read at a time
  __shared__ float part[3][kWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.geo;
  const int B = geo.B, H_kv = geo.H_kv, G = a.G;
  const float c = a.scale_log2;
  const int64_t step = int64_t(G) * (D + 2);
  for (int unit = bx; unit < B * H_kv; unit += nx) {
    const int b = unit / H_kv, g = unit - b * H_kv;
    const long long nt = ln.pre[b + 1] - ln.pre[b], begin = ln.pre[b] * H_kv + g * nt;
    if (nt == 0 || skipped<SKIP>(geo, b) > 0) continue;
    const int first = cut.holder(begin), pieces = cut.holder(begin + nt - 1) - first + 1;
    if (pieces == 1 && !SKIP) continue;
    const int64_t qrow = (int64_t(b) * a.H_q + int64_t(g) * G) * D;
    const float* const p = a.partials + (first + unit) * step;
    if (pieces <= 2 * AHEAD) {
      for (int i = by * kThreads + tid; i < G * D; i += ny * kThreads) {
        const int h = i / D, d = i - h * D;
        Joined j;
        for (int w = 0; w < pieces; w += AHEAD) j.add<AHEAD>(p + h * (D + 2) + w * step, step, pieces - w, d, D, c);
        j.put(a, qrow, h, d, D, c);
      }
      continue;
    }
    for (int y = by; y < G * (D / 32); y += ny) {
      const int h = y / (D / 32), d = y % (D / 32) * 32 + lane;
      // warp w takes the w-th eighth of the pieces
      const int share = (pieces + kWarps - 1) / kWarps, w1 = min(pieces, (warp + 1) * share);
      Joined j;
      for (int w = warp * share; w < w1; w += AHEAD) j.add<AHEAD>(p + h * (D + 2) + w * step, step, w1 - w, d, D, c);
      part[0][warp][lane] = j.m;
      part[1][warp][lane] = j.l;
      part[2][warp][lane] = j.o;
      __syncthreads();
      if (warp == 0) {
        j = Joined();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) j.add(part[0][w][lane], part[1][w][lane], part[2][w][lane], c);
        j.put(a, qrow, h, d, D, c);
      }
      __syncthreads();
    }
  }
}

template <int TR, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int grid) {
  __shared__ Line ln;
  pdl_launch();
  pdl_wait();
  scan_lengths<TR>(a.geo, ln, false);
  join_units<TR, D>(a, ln, Cut(ln.pre[a.geo.B] * a.geo.H_kv, grid), blockIdx.x, gridDim.x, blockIdx.y, gridDim.y);
}

// The joining kernel behind a launch of `grid` CTAs: a CTA for each unit, and for each 32
// outputs of it while that is no more than four CTAs to an SM.
template <int TR, int D>
cudaError_t launch_join(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  const int units = a.geo.B * a.geo.H_kv, most = 4 * grid, y = a.G * (D / 32);
  return launch_pdl(paged_join_kernel<TR, D>,
                    dim3(units < most ? units : most, units >= most ? 1 : most / units < y ? most / units : y),
                    kThreads, 0, st, a, grid);
}

}  // namespace
}  // namespace sfi

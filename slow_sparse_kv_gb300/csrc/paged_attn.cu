// Attention of one new token over a paged KV cache, split over its length.
//
// A tile is 16 (fp32: 8) consecutive positions of one (sequence, KV head).  All
// tiles of all sequences stand in one line, sequence by sequence and head by
// head, and the line is cut, whatever the lengths, into a share for each CTA.  Four
// warps look up pages, 32 tiles at a time, and copy ahead, across the borders of
// sequences, into rings of 24 KB for each of the eight warps that attend (a warp that
// looked up and copied for itself waited for the table's reads before each tile: 1.8
// times as long).  A tile's place in the line says which warp takes it.
// Bound by HBM: 2 d e bytes a position and 4 d G flops, G <= 16.  Measured, 32 / 8
// heads of 128 in pages of 16: 8 x 32768 positions (1.07 GB) in 164 us, 6.56 TB/s,
// where a copy reaches 6.78; fp32, 4 x 32768, 165 us; 32 sequences of 4096 to
// 65536 (2.57 GB) in 379 us, 6.79 TB/s; 256 x 300 (0.31 GB) in 70 us; one of 700 in
// 9.1 us, the two launches.
//
// What a CTA saw of one (sequence, KV head) is a piece, a softmax state (m, l,
// o), merged over the warps through shared memory.  The only piece of its unit is
// normalised and written; others go to the workspace, and a second small kernel,
// launched early and waiting for the first one's end, joins them in the order of
// the line.  (Joined by whichever CTA came last, each piece cost a fence and an
// atomic, 2000 clocks; with pieces of single warps the joins took longer than the
// merges.)
//
// bf16: S^T = K Q^T by mma.sync with the 16 positions as M and the group's heads
// as N (8 columns; two tiles of them for G > 8), O^T += V^T P^T with P moved to
// the B operand by movmatrix.  The output is fp32, so P is not rounded to bf16
// but split into three bf16 terms (24 bits in all), at the price of two more
// products with V; each tile's product starts from zero and is added to o in
// fp32, because the tensor cores truncate where they add (with two terms and one
// long chain of MMAs the output's error was 1.5e-6 at 700 positions and 4.3e-6 at
// 32768).  tcgen05 would leave 128 - G of its 128 rows empty; the kernel waits for
// HBM either way.
// fp32: CUDA cores, d spread over the lanes, dots by transpose-reduction, products and
// sums in pairs (f32x2; without: 4 x 32768, 16 heads a group 379 us against 349, 8 heads 194
// against 180, d = 64 with 4 heads, 8 x 32768, 176 against 170; 4 heads of 128, which
// HBM bounds, 161 against 165).
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "pdl.cuh"

namespace sfi {
namespace {

constexpr int kWarps = 8;                    // that attend
constexpr int kThreads = kWarps * 32;        // of them
constexpr int kProducers = 4;                // warps that copy
constexpr int kAllThreads = kThreads + kProducers * 32;
constexpr int kAttendRegs = 216, kCopyRegs = 72;  // of 168 each at launch: 2 * 216 + 72 = 3 * 168
constexpr int kRingBytes = 196608;
constexpr float kGrow = 8.0f;                // growth of the maximum (log2) that moves m

enum Load { kTma, kCpAsync, kBulk };

template <typename T, int D, int NT>
struct Cfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int TR = F32 ? 8 : 16;                  // positions per tile
  static constexpr int ROW = D * int(sizeof(T));           // bytes of a row
  static constexpr int HALF = TR * ROW;                    // K part of a stage, then V's
  static constexpr int STAGES = kRingBytes / kWarps / (2 * HALF);  // a warp's: 3 of 8 KB, 6 of 4 KB
  static constexpr int SLOTS = kWarps * STAGES;
  static constexpr int HEADS = NT * 8;                     // heads that the registers hold
  static constexpr int MH = 4;                             // heads merged at a time
  static constexpr int MROW = D + 4;                       // floats of a merged head: o, m, l
  static constexpr int SMEM = 1024 + kRingBytes + kWarps * MH * MROW * 4;
};

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

  __device__ __forceinline__ Cut(long long total_, int grid) {
    total = total_;
    // few tiles: fewer shares, of a tile for each warp at least
    const long long most = (total + kWarps - 1) / kWarps;
    shares = most < grid ? int(most) : grid;
    per = shares > 0 ? total / shares : 0;
    extra = shares > 0 ? int(total - per * shares) : 0;
    wide = extra * (per + 1);
  }
  __device__ __forceinline__ long long start(int share) const { return share * per + min(share, extra); }
  // the share that holds tile x
  __device__ __forceinline__ int holder(long long x) const {
    if (total < (1LL << 31))  // (a 64-bit division takes ~10 times as long)
      return x < wide ? int(uint32_t(x) / uint32_t(per + 1)) : extra + int(uint32_t(x - wide) / uint32_t(per));
    return int(x < wide ? x / (per + 1) : extra + (x - wide) / per);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Four fp32 values of shared memory as two pairs.
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(addr));
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

// Fills `ln` (the first kThreads threads of a CTA); `flag` reports lengths out of
// range.
template <int TR>
__device__ __forceinline__ void scan_lengths(const PagedGeo& geo, Line& ln, bool flag) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = geo.B, cap = geo.max_pages * geo.P;
  auto tiles = [&](int b) {
    int n = b < B ? geo.len[b] : 0;
    if (n < 0 || n > cap) {
      if (flag) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
      n = n < 0 ? 0 : cap;
    }
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

// What the warps of a CTA share besides the ring.
struct Shared {
  Line ln;
  uint64_t full[48], empty[48];                           // of each slot of the ring
  volatile int abort;
  uint64_t merge_free;                                    // the warps' states have been read
};

// The first tile from `from` on whose number is r modulo m (a power of two).
__device__ __forceinline__ long long first_of(long long from, int r, int m) { return from + ((r - from) & (m - 1)); }

// The copying warps: warp `p` takes the tiles of the attending warps p and p + 4.
template <typename T, int D, int NT, Load LD>
__device__ __forceinline__ void copy_tiles(const PagedAttnArgs& a, Shared& sh, long long from, long long to,
                                           uint32_t ring, int p) {
  using C = Cfg<T, D, NT>;
  constexpr int TR = C::TR;
  const PagedGeo& geo = a.geo;
  const int lane = threadIdx.x & 31, P = geo.P, H_kv = geo.H_kv, cap = geo.max_pages * P;
  const T* const kp = static_cast<const T*>(a.k);
  const T* const vp = static_cast<const T*>(a.v);
  bool ok = true;
  const long long first[2] = {first_of(from, p, kWarps), first_of(from, p + kProducers, kWarps)};
  for (long long x0 = first_of(from, p, kProducers); x0 < to && ok; x0 += kProducers * 32) {
    // 32 tiles: each lane finds the place and the page of its own
    const long long x = x0 + kProducers * lane;
    const bool mine = x < to;
    Unit u{0, 0, 0, 0};
    int t = 0, n = 0;
    int page[LD == kBulk ? TR : 1];
    if (mine) {
      u = unit_at(x, sh.ln, geo.B, H_kv);
      t = int(x - u.begin);
      n = min(geo.len[u.b], cap);
    }
    const int32_t* const row = geo.table + int64_t(u.b) * geo.max_pages;
    if (LD != kCpAsync) {
      bool bad = false;
#pragma unroll
      for (int r = 0; r < (LD == kBulk ? TR : 1); ++r) {
        const int pos = t * TR + r;
        page[r] = mine && pos < n ? row[pos / P] : 0;  // (fp32: mostly the same entry)
        if (page[r] < 0 || page[r] >= geo.n_pages) bad = true, page[r] = 0;
      }
      if (bad) set_status(geo.status, SFI_DEV_BAD_INDEX);
    }
    // fp32: the lane's rows, and where they go on in another page
    int rows = 0, in0 = 0;
    uint32_t starts = 0;
    if (LD == kBulk) {
      rows = min(TR, n - t * TR);
      in0 = t * TR % P;
      int in = in0;
#pragma unroll
      for (int r = 1; r < TR; ++r) {
        in = in + 1 == P ? 0 : in + 1;
        if (in == 0 && r < rows) starts |= 1u << r;
      }
    }
    const int64_t at0 = page[0] * geo.page_stride + (int64_t(u.g) * P + in0) * D;
    const int row0 = LD == kTma ? int(page[0] * (geo.page_stride / D) + u.g * P + t * TR % P) : 0;
    const int count = int(min(32LL, (to - x0 + kProducers - 1) / kProducers));
    // kCpAsync: the i-th tile's row of this lane (lane % TR): its page, and where in it,
    // -1 for no row.  A tile's pages are read while the one before it is copied (waited
    // for before each tile: 136 us against 129 for 8 x ~24000 positions in pages of 20).
    int pg = 0, in = -1;
    auto row_of = [&](int i) {
      const int ut = __shfl_sync(kFull, t, i), ug = __shfl_sync(kFull, u.g, i), un = __shfl_sync(kFull, n, i);
      const int32_t* const urow = geo.table + int64_t(__shfl_sync(kFull, u.b, i)) * geo.max_pages;
      const int pos = ut * TR + lane % TR;
      pg = pos < un ? urow[pos / P] : 0;
      in = pos < un ? ug * P + pos % P : -1;
    };
    if (LD == kCpAsync) row_of(0);
    for (int i = 0; i < count && ok; ++i) {
      const long long xi = x0 + kProducers * i;
      const int w = int(xi >> 2) & 1;  // which of the two warps
      const uint32_t y = uint32_t(xi - first[w]) / kWarps;
      const int slot = (p + w * kProducers) * C::STAGES + int(y % C::STAGES);
      const uint32_t use = y / C::STAGES;
      if (use > 0) ok = warp_ctrl_wait(smem_addr(&sh.empty[slot]), (use - 1) & 1, &sh.abort, geo.status);
      if (!ok) break;
      const uint32_t dst = ring + slot * 2 * C::HALF, bar = smem_addr(&sh.full[slot]);
      if constexpr (LD == kTma) {
        if (lane == i) {
          mbar_arrive_expect_tx(bar, 2 * C::HALF);
          tma_load_3d(dst, &a.tmk, 0, row0, 0, bar);
          tma_load_3d(dst + C::HALF, &a.tmv, 0, row0, 0, bar);
        }
      } else if constexpr (LD == kBulk) {
        if (lane == i) {
          // runs of rows that lie in one page
          mbar_arrive_expect_tx(bar, uint32_t(rows) * 2 * C::ROW);
          const uint32_t bytes = uint32_t(min(P - in0, rows)) * C::ROW;
          bulk_load(dst, kp + at0, bytes, bar);
          bulk_load(dst + C::HALF, vp + at0, bytes, bar);
          if (starts) {
#pragma unroll
            for (int r = 1; r < TR; ++r) {
              if (!(starts >> r & 1)) continue;
              const uint32_t more = uint32_t(min(P, rows - r)) * C::ROW;
              const int64_t at = page[r] * geo.page_stride + int64_t(u.g) * P * D;
              bulk_load(dst + r * C::ROW, kp + at, more, bar);
              bulk_load(dst + C::HALF + r * C::ROW, vp + at, more, bar);
            }
          }
        }
      } else {
        // 16-byte chunks of single rows, in the layout that the maps' swizzle gives
        constexpr int CH = C::ROW / 16;  // chunks of a row
        if (pg < 0 || pg >= geo.n_pages) {
          set_status(geo.status, SFI_DEV_BAD_INDEX);
          pg = 0;
        }
        const int at = in < 0 ? -1 : int(pg * (geo.page_stride / D) + in);  // of the pool's rows, below 2^31
        if (i + 1 < count) row_of(i + 1);
#pragma unroll
        for (int j = 0; j < TR * CH / 32; ++j) {
          const int r = (j * 32 + lane) / CH, ch = lane % CH;
          const int from_row = __shfl_sync(kFull, at, r);
          const int64_t ra = int64_t(max(from_row, 0)) * D + ch * 8;
          const uint32_t some = from_row >= 0 ? 16 : 0;
          const uint32_t dr = dst + (ch / 8) * (TR * 128) + r * 128 + ((ch & 7) ^ (r & 7)) * 16;
          cp_async16_zfill(dr, kp + ra, some);
          cp_async16_zfill(dr + C::HALF, vp + ra, some);
        }
        cp_async_arrive_noinc(bar);
      }
    }
    __syncwarp();
  }
  // No copy may be in flight when the CTA exits: the attending warps wait for
  // every tile, unless one of these warps gave up (after seconds, in which all
  // earlier copies have landed).
  if (!ok) sh.abort = 2;
  if (LD == kCpAsync) asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int D, int NT, Load LD>
__global__ void __launch_bounds__(kAllThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<T, D, NT>;
  constexpr bool F32 = C::F32;
  constexpr int TR = C::TR;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u;
  float* const merge = reinterpret_cast<float*>(smem_raw + (ring - smem_addr(smem_raw)) + kRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.geo;
  const int B = geo.B, H_kv = geo.H_kv, G = a.G;
  const int cap = geo.max_pages * geo.P;

  if (tid < C::SLOTS) {
    mbar_init(smem_addr(&sh.full[tid]), LD == kCpAsync ? 32 : 1);
    mbar_init(smem_addr(&sh.empty[tid]), 1);
  } else if (tid == 96) {
    mbar_init(smem_addr(&sh.merge_free), kWarps);
    sh.abort = 0;
  }
  fence_mbar_init();
  // (this kernel starts while the one before it on the stream drains, and the
  // joining kernel while this one drains; each waits for the results before it)
  pdl_launch();
  pdl_wait();
  scan_lengths<TR>(geo, sh.ln, blockIdx.x == 0);
  const Line& ln = sh.ln;
  const long long total = ln.pre[B] * H_kv;

  // sequences that hold nothing
  for (int u = blockIdx.x; u < B * H_kv; u += gridDim.x) {
    const int b = u / H_kv, g = u - b * H_kv;
    if (ln.pre[b + 1] != ln.pre[b]) continue;
    const int64_t row = int64_t(b) * a.H_q + int64_t(g) * G;
    for (int i = tid; i < G * D; i += kAllThreads) a.out[row * D + i] = 0.f;
    if (a.lse && tid < G) a.lse[row + tid] = -INFINITY;
  }
  // this CTA's share of the line (a CTA beyond the shares has none)
  const Cut cut(total, gridDim.x);
  const int share = blockIdx.x;
  const long long from = share < cut.shares ? cut.start(share) : total;
  const long long to = share < cut.shares ? cut.start(share + 1) : total;

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    copy_tiles<T, D, NT, LD>(a, sh, from, to, ring, warp - kWarps);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAttendRegs));
    const float c = a.scale_log2;
    uint32_t y = 0;       // this warp's tiles so far
    uint32_t merges = 0;  // and rounds of merging
    constexpr int NS = F32 ? NT * 2 : NT;  // (see the state below)
    constexpr int NE = F32 ? 1 : 2;
    constexpr int KS = D / 16;
    constexpr int LPR = D / 4, RPP = 32 / LPR;  // fp32: lanes per row, rows per pass
    const int li = lane % LPR, half = lane / LPR;
    // the lane's part of a unit's queries, and the sequence's length
    uint32_t qb[F32 ? 1 : NT][KS][2];
    // (fp32 with more than 8 heads: both q and o would not fit, so the queries are read
    // from L1 again for each tile: 379 us instead of 639 for 4 x 32768, 16 heads a group,
    // when that was measured)
    constexpr bool Q_REGS = NT == 1;
    uint64_t qf[F32 && Q_REGS ? NS * 4 : 1][2];
    auto load_unit = [&](const Unit& u) {
      const int64_t qrow = (int64_t(u.b) * a.H_q + int64_t(u.g) * G) * D;
      if constexpr (!F32) {
        const uint32_t* qw = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + qrow);
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          const int head = h * 8 + (lane >> 2);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qb[h][kk][e] = head < G ? qw[(head * D + kk * 16 + e * 8) / 2 + (lane & 3)] : 0u;
        }
      } else if constexpr (Q_REGS) {
#pragma unroll
        for (int h = 0; h < NS * 4; ++h) {
          ulonglong2 w = make_ulonglong2(0, 0);
          if (h < G) w = reinterpret_cast<const ulonglong2*>(static_cast<const T*>(a.q) + qrow + h * D)[li];
          qf[h][0] = w.x, qf[h][1] = w.y;
        }
      }
      return min(geo.len[u.b], cap);
    };
    if (from < to) {
      long long x = first_of(from, warp, kWarps);  // this warp's next tile
      Unit u = unit_at(from, ln, B, H_kv);
      int n = load_unit(u);
      while (true) {
        const long long pe = min(u.end, to);
        const int b = u.b, g = u.g;
        const int64_t qrow = (int64_t(b) * a.H_q + int64_t(g) * G) * D;

        // state: bf16 head 2 (lane % 4) + e of column tile h, in every lane with the same lane % 4;
        // fp32 head 4 h + lane % 4
        float m[NS][NE], l[NS][NE];
#pragma unroll
        for (int h = 0; h < NS; ++h)
#pragma unroll
          for (int e = 0; e < NE; ++e) m[h][e] = -INFINITY, l[h][e] = 0.f;

        float o[F32 ? 1 : KS][F32 ? 1 : NT][4];
        uint64_t of[F32 ? NS * 4 : 1][2];  // fp32: a pair of dimensions each
        if constexpr (!F32) {
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int h = 0; h < NT; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[kk][h][e] = 0.f;
        } else {
#pragma unroll
          for (int h = 0; h < NS * 4; ++h) of[h][0] = of[h][1] = 0;
        }

        for (; x < pe; x += kWarps) {
          const int slot = warp * C::STAGES + int(y % C::STAGES);
          const uint32_t use = y / C::STAGES;
          ++y;
          const int left = n - int(x - u.begin) * TR;  // rows of the tile that count
          const bool ok = warp_pipe_wait(smem_addr(&sh.full[slot]), use & 1, &sh.abort, geo.status, a.wait_cycles);
          if (!ok) {
            // the stage is given back once its rows have landed, without them
            if (sh.abort != 2) mbar_wait(smem_addr(&sh.full[slot]), use & 1);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.empty[slot]));
            continue;
          }
          const uint32_t ks = ring + slot * 2 * C::HALF, vs = ks + C::HALF;

          if constexpr (!F32) {
            float s[NT][4];
#pragma unroll
            for (int h = 0; h < NT; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
            {
              const int r = lane & 15, hi = lane >> 4;
#pragma unroll
              for (int kk = 0; kk < KS; ++kk) {
                uint32_t k0, k1, k2, k3;
                ldsm_x4(ks + (kk / 4) * (TR * 128) + r * 128 + ((((kk & 3) * 2 + hi) ^ (r & 7)) * 16), k0, k1, k2, k3);
#pragma unroll
                for (int h = 0; h < NT; ++h) mma_bf16_16816(s[h], k0, k1, k2, k3, qb[h][kk][0], qb[h][kk][1]);
              }
            }
            const int r0 = lane >> 2;
            const bool in0 = r0 < left, in1 = r0 + 8 < left;
            uint32_t pw[NT][3][2];  // P^T in three bf16 terms
#pragma unroll
            for (int h = 0; h < NT; ++h) {
              float top[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                s[h][e] = in0 ? s[h][e] : -INFINITY;
                s[h][2 + e] = in1 ? s[h][2 + e] : -INFINITY;
                top[e] = fmaxf(s[h][e], s[h][2 + e]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], w));
              }
              const bool g0 = (top[0] - m[h][0]) * c > kGrow, g1 = (top[1] - m[h][1]) * c > kGrow;
              if (__any_sync(kFull, g0 || g1)) {
                const float f0 = g0 ? ex2((m[h][0] - top[0]) * c) : 1.f, f1 = g1 ? ex2((m[h][1] - top[1]) * c) : 1.f;
                if (g0) m[h][0] = top[0];
                if (g1) m[h][1] = top[1];
                l[h][0] *= f0;
                l[h][1] *= f1;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                  o[kk][h][0] *= f0, o[kk][h][1] *= f1;
                  o[kk][h][2] *= f0, o[kk][h][3] *= f1;
                }
              }
              const float b0 = m[h][0] == -INFINITY ? 0.f : m[h][0] * c, b1 = m[h][1] == -INFINITY ? 0.f : m[h][1] * c;
              const float p0 = ex2(fmaf(s[h][0], c, -b0)), p1 = ex2(fmaf(s[h][1], c, -b1));
              const float p2 = ex2(fmaf(s[h][2], c, -b0)), p3 = ex2(fmaf(s[h][3], c, -b1));
              l[h][0] += p0 + p2;
              l[h][1] += p1 + p3;
              float r0 = p0, r1 = p1, r2 = p2, r3 = p3;
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                const uint32_t w0 = pack_bf16x2(r0, r1), w1 = pack_bf16x2(r2, r3);
                pw[h][e][0] = movmatrix_trans(w0);
                pw[h][e][1] = movmatrix_trans(w1);
                r0 -= __uint_as_float(w0 << 16), r1 -= __uint_as_float(w0 & 0xffff0000u);
                r2 -= __uint_as_float(w1 << 16), r3 -= __uint_as_float(w1 & 0xffff0000u);
              }
            }
            // rows behind the sequence's end may hold anything: 0 * NaN is not 0
            const int vr = 2 * (lane & 3);
            const uint32_t m0 = (vr < left ? 0xffffu : 0u) | (vr + 1 < left ? 0xffff0000u : 0u);
            const uint32_t m1 = (vr + 8 < left ? 0xffffu : 0u) | (vr + 9 < left ? 0xffff0000u : 0u);
            const int r = (lane & 7) + (lane >> 4) * 8, hi = (lane >> 3) & 1;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              uint32_t v0, v1, v2, v3;
              ldsm_x4_trans(vs + (kk / 4) * (TR * 128) + r * 128 + ((((kk & 3) * 2 + hi) ^ (r & 7)) * 16), v0, v1, v2, v3);
              if (left < TR) v0 &= m0, v1 &= m0, v2 &= m1, v3 &= m1;
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 2; e >= 0; --e) mma_bf16_16816(d, v0, v1, v2, v3, pw[h][e][0], pw[h][e][1]);  // small terms first
#pragma unroll
                for (int e = 0; e < 4; ++e) o[kk][h][e] += d[e];
              }
            }
          } else {
            constexpr int PASS = TR / RPP;
#pragma unroll
            for (int h = 0; h < NS; ++h) {
              if (h * 4 >= G) break;
              float v[PASS * 4];
              uint64_t qt[4][2];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (Q_REGS) {
                  qt[e][0] = qf[h * 4 + e][0], qt[e][1] = qf[h * 4 + e][1];
                } else {
                  ulonglong2 w = make_ulonglong2(0, 0);
                  if (h * 4 + e < G)
                    w = reinterpret_cast<const ulonglong2*>(static_cast<const T*>(a.q) + qrow + (h * 4 + e) * D)[li];
                  qt[e][0] = w.x, qt[e][1] = w.y;
                }
              }
#pragma unroll
              for (int i = 0; i < PASS; ++i) {
                uint64_t k0, k1;
                lds_pairs(ks + (i * RPP + half) * C::ROW + li * 16, k0, k1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint64_t t = fma2(k1, qt[e][1], mul2(k0, qt[e][0]));
                  v[i * 4 + e] = lo(t) + hi(t);
                }
              }
              // lane li of a row group: the dot of pass li / 4 and head 4 h + li % 4
              transpose_reduce<LPR>(v, li);
              const int row = (li >> 2) * RPP + half;
              const float s = row < left ? v[0] : -INFINITY;
              float top = s;
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
              const bool grow = (top - m[h][0]) * c > kGrow;
              if (__any_sync(kFull, grow)) {
                const float f = grow ? ex2((m[h][0] - top) * c) : 1.f;
                if (grow) m[h][0] = top;
                l[h][0] *= f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float fe = __shfl_sync(kFull, f, e);
                  of[h * 4 + e][0] = mul2(of[h * 4 + e][0], pair(fe, fe));
                  of[h * 4 + e][1] = mul2(of[h * 4 + e][1], pair(fe, fe));
                }
              }
              const float p = ex2(fmaf(s, c, -(m[h][0] == -INFINITY ? 0.f : m[h][0] * c)));
              l[h][0] += p;
#pragma unroll
              for (int i = 0; i < PASS; ++i) {
                uint64_t v0, v1;
                lds_pairs(vs + (i * RPP + half) * C::ROW + li * 16, v0, v1);
                if (i * RPP + half >= left) v0 = v1 = 0;  // 0 * NaN is not 0
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float pe_ = __shfl_sync(kFull, p, half * LPR + i * 4 + e);
                  of[h * 4 + e][0] = fma2(pair(pe_, pe_), v0, of[h * 4 + e][0]);
                  of[h * 4 + e][1] = fma2(pair(pe_, pe_), v1, of[h * 4 + e][1]);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.empty[slot]));
        }

        // the next unit of the share; its queries are on their way during the merge
        Unit next = u;
        do unit_next(next, ln, B, H_kv);
        while (next.begin < to && next.end == next.begin);
        const bool more = next.begin < to;
        if (more) n = load_unit(next);

        // ---- the piece: the warps' states merged, MH heads at a time.  A warp writes
        // when all have read the round before, which they mostly have long since,
        // so that a round is one wait for all.  (With factors by 32 threads between two
        // more of them, and the next queries loaded behind it: 106 us against 84 for
        // 256 x 300 positions, 93 against 88 for 131072.)
        const bool alone = u.begin >= from && u.end <= to;  // the unit's only piece
        float* const slot = a.partials + (share + b * H_kv + g) * int64_t(G) * (D + 2);
#pragma unroll
        for (int h0 = 0; h0 < C::HEADS; h0 += C::MH) {
          if (h0 >= G) break;
          if (merges > 0) warp_ctrl_wait(smem_addr(&sh.merge_free), (merges - 1) & 1, &sh.abort, geo.status);
          ++merges;
          float* const mine = merge + warp * C::MH * C::MROW;
          if constexpr (!F32) {
            const int h = h0 / 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = l[h][e];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(kFull, t, w);
              const int at = h * 8 + 2 * (lane & 3) + e - h0;  // this lane's head
              if (at < 0 || at >= C::MH) continue;
              float* const row = mine + at * C::MROW;
              if (lane < 4) row[D] = m[h][e], row[D + 1] = t;
#pragma unroll
              for (int kk = 0; kk < KS; ++kk) {
                row[kk * 16 + (lane >> 2)] = o[kk][h][e];
                row[kk * 16 + 8 + (lane >> 2)] = o[kk][h][2 + e];
              }
            }
          } else {
            const int h = h0 / 4;
            float t = l[h][0];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(kFull, t, w);
            if (lane < 4) mine[lane * C::MROW + D] = m[h][0], mine[lane * C::MROW + D + 1] = t;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float x_ = y & 1 ? hi(of[h * 4 + e][y / 2]) : lo(of[h * 4 + e][y / 2]);
                if (RPP == 2) x_ += __shfl_xor_sync(kFull, x_, 16);
                if (half == 0) mine[e * C::MROW + li * 4 + y] = x_;
              }
            }
          }
          attend_sync();
          for (int i = tid; i < min(C::MH, G - h0) * D; i += kThreads) {
            const int h = i / D, d = i - h * D;
            float2 ml[kWarps];
            float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              ml[w] = *reinterpret_cast<const float2*>(merge + (w * C::MH + h) * C::MROW + D);
              M = fmaxf(M, ml[w].x);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              // (a warp that saw nothing, or only scores of -infinity, adds nothing)
              const bool none = ml[w].x == -INFINITY && ml[w].y == 0.f;
              const float f = ex2((ml[w].x - M) * c);
              L += none ? 0.f : f * ml[w].y;
              O += none ? 0.f : f * merge[(w * C::MH + h) * C::MROW + d];
            }
            if (alone) {
              a.out[qrow + (h0 + h) * D + d] = L == 0.f ? 0.f : O / L;
              if (d == 0 && a.lse) a.lse[qrow / D + h0 + h] = (M * c + log2f(L)) * 0.6931471805599453f;
            } else {
              float* const p = slot + (h0 + h) * (D + 2);
              p[d] = O;
              if (d == 0) p[D] = M, p[D + 1] = L;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.merge_free));
        }
        if (!more) break;
        u = next;
      }
    }
  }
}

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

template <int TR, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int grid) {
  constexpr int AHEAD = 8;  // pieces read at a time
  __shared__ Line ln;
  __shared__ float part[3][kWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.geo;
  const int B = geo.B, H_kv = geo.H_kv, G = a.G;
  const float c = a.scale_log2;
  pdl_launch();
  pdl_wait();
  scan_lengths<TR>(geo, ln, false);
  const Cut cut(ln.pre[B] * H_kv, grid);
  const int64_t step = int64_t(G) * (D + 2);
  for (int unit = blockIdx.x; unit < B * H_kv; unit += gridDim.x) {
    const int b = unit / H_kv, g = unit - b * H_kv;
    const long long nt = ln.pre[b + 1] - ln.pre[b], begin = ln.pre[b] * H_kv + g * nt;
    if (nt == 0) continue;
    const int first = cut.holder(begin), pieces = cut.holder(begin + nt - 1) - first + 1;
    if (pieces == 1) continue;
    const int64_t qrow = (int64_t(b) * a.H_q + int64_t(g) * G) * D;
    const float* const p = a.partials + (first + unit) * step;
    if (pieces <= 2 * AHEAD) {
      for (int i = blockIdx.y * kThreads + tid; i < G * D; i += gridDim.y * kThreads) {
        const int h = i / D, d = i - h * D;
        Joined j;
        for (int w = 0; w < pieces; w += AHEAD) j.add<AHEAD>(p + h * (D + 2) + w * step, step, pieces - w, d, D, c);
        j.put(a, qrow, h, d, D, c);
      }
      continue;
    }
    for (int y = blockIdx.y; y < G * (D / 32); y += gridDim.y) {
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

template <typename T, int D, int NT, Load LD>
cudaError_t launch_t(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<T, D, NT>;
  auto* const kernel = paged_attn_kernel<T, D, NT, LD>;
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, allowed);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kernel, dim3(grid), kAllThreads, C::SMEM, st, a);
  if (e2 != cudaSuccess) return e2;
  // a CTA for each unit, and for each 32 outputs of it while that is no more
  // than four CTAs to an SM
  const int units = a.geo.B * a.geo.H_kv, most = 4 * grid, y = a.G * (D / 32);
  return launch_pdl(paged_join_kernel<C::TR, D>,
                    dim3(units < most ? units : most, units >= most ? 1 : most / units < y ? most / units : y),
                    kThreads, 0, st, a, grid);
}

template <int D, int NT>
cudaError_t launch_n(const PagedAttnArgs& a, bool f32, bool use_tma, int grid, cudaStream_t st) {
  if (f32) return launch_t<float, D, NT, kBulk>(a, grid, st);
  return use_tma ? launch_t<bf16_t, D, NT, kTma>(a, grid, st) : launch_t<bf16_t, D, NT, kCpAsync>(a, grid, st);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int D, bool f32, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64) return a.G <= 8 ? launch_n<64, 1>(a, f32, use_tma, grid, st) : launch_n<64, 2>(a, f32, use_tma, grid, st);
  return a.G <= 8 ? launch_n<128, 1>(a, f32, use_tma, grid, st) : launch_n<128, 2>(a, f32, use_tma, grid, st);
}

}  // namespace sfi

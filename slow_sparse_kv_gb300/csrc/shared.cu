// Attention of one new token for sequences of which groups share their first pages:
// the shared positions are read once for a group, not once for each sequence.
//
// For sequence b of a group that shares n0 positions, softmax over all positions is joined
// from two states (m, l, o): over [0, n0), with the group's other sequences, and over
// [n0, len[b]), by itself, which is paged_attn.cu's kernel with the first pages left out.
//   out = sum_w f_w o_w / sum_w f_w l_w,  f_w = 2^(c (m_w - max m)),  c = log2(e) / sqrt(d)
//
// The shared part is a matrix product: the group's queries of a KV head, members x G rows,
// against n0 keys.  A tile is 2 x 128 such rows; all tiles' blocks of 48 keys, KV head by KV
// head, stand in one line, which is cut into a share of equal size for each CTA.  In a CTA, as
// in prefill.cu: S = Q K^T (tcgen05.mma from shared memory into tensor memory), softmax
// statistics with a thread for each row, P over S's columns, O += P V; the two halves of
// a tile alternate, so that the tensor cores work on one while the other's softmax runs.
// (A tile of 128 rows or fewer is taken by both halves, each with every other block.)
// The output is fp32, so P is kept in three bf16 terms (24 bits: nothing is lost), at the price
// of two more products with V.  (With two terms and a product's sums in tensor memory
// from a piece's first block to its last the outputs were off by 2e-6 to 5e-6, now by 2.4e-7 to 7.4e-7.)
// Bytes: 4 d n0 a group and KV head; flops 4 d for each row and key, 8 d with all three terms.
// From some 100 rows on the tensor cores bound it, below HBM does.
//
// Three launches: the shared part, the sequences' own part, and one that joins the states of
// both.  Measured, 32 / 8 heads of 128: 64 sequences behind 32768 positions, 16 to 1024 of
// their own, 96 us: 61 (0.56 PFLOP/s as the formula counts, 1.13 with the terms; the tensor
// pipe is active for 55% of the cycles; 7 before the first product, 4 for taking sums out of
// tensor memory), 19 and 14; that these run one after another is what is left to gain.  5 groups of
// 9 behind 6000 positions in pages of 24: 62 us (32, 12 and 14).  6 sequences, 8 / 2 heads of 64,
// behind 600 positions: 18 us (6.5, 4.3 and 5.3).  sfi_paged_attn on the same sequences is faster where less than
// 0.25 GB is saved: 2 behind 8192 28 us and 15, 4 behind 32768 60 and 47, 16 behind 8192 29 and 49, 64 behind
// 512 29 each, behind 32768 86 and 615 (100 own positions each, in a row of calls).
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged_line.cuh"
#include "pdl.cuh"
#include "shared.h"
#include "tc5.cuh"
#include "tc5_attn.cuh"

namespace sfi {
namespace {

constexpr int kSharedThreads = 384;  // 2 softmax warpgroups; two loading warps, an MMA warp, one for the plan
constexpr int kRows = 128;           // query rows of a half tile
constexpr int kKeys = 48;            // keys of a block
// Tensor memory: three regions of a block's scores and, over and behind them, its P, which the
// steps take in turn, so that scores are ready when a half comes to them; and both halves'
// sums.  (Blocks of 64 keys leave room for two regions only, and each half then waits for its own
// products before its next scores.)
constexpr int kRegions = 3, kRegion = 80, kSums = 256;
constexpr int kTerms = 3;            // bf16 terms of P
constexpr int kChain = 4;            // blocks of a half whose products with V are added in tensor memory
constexpr float kGrow = 8.0f;        // growth of the maximum (log2) that moves m
constexpr int kJoinCols = 16;        // columns of an item of the join
constexpr int kJoinCtas = 2;         // its CTAs on an SM
constexpr int kOwnTile = 16;         // positions of a tile of paged_attn.cu's kernel in bf16

template <int D>
struct SCfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t QTILE = kRows * 128 * HALVES;  // bytes of 128 rows
  static constexpr uint32_t TILE = kKeys * 128 * HALVES;   // and of a block of K or V
  static constexpr int STAGES = 5;                         // pairs of them in flight
  static constexpr uint32_t SMEM = 1024 + 2 * QTILE + STAGES * 2 * TILE;
  static constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 504 - 2 * SOFTMAX_REGS;
};

// Where term e of the z-th 16 keys of a block's P lies behind the block's scores' first column,
// 8 columns each: that of the first 32 keys where their own scores were and behind them all.
__host__ __device__ constexpr int term_at(int z, int e) {
  return z < 2 ? (z * 3 + e < 4 ? 8 * (z * 3 + e) : 48 + 8 * (z * 3 + e - 4)) : (e < 2 ? 32 + 8 * e : 64);
}

// ---- the shared part
struct SharedMem {
  uint64_t q_full, q_empty;
  // A stage is a pair: K of a block and V of the one before, since the scores run ahead; the first
  // pair of a piece has no V, the last one no K.
  uint64_t kv_full[5], kv_empty[5], drained;
  // Scores run ahead of the softmax threads, and these ahead of the products: a barrier for each
  // region.  None may be two phases ahead of who waits for it, nor one behind: it would look
  // like the other.  The halves take the steps in turn, so who waits for the scores of step s
  // has seen those of s - 2, behind which those of s - 3, the region's last ones, were complete;
  // and a region's next scores and P come behind its last products.
  uint64_t s_full[kRegions], p_ready[kRegions], o_full[kRegions];
  uint32_t tmem;
  volatile int abort;
  // the plan, and what it is made of
  long long total;
  int n_tiles;
  long long start[kMaxTiles + 1];
  SharedTile tile[kMaxTiles];
  int cu[kMaxBatch + 1], pages[kMaxBatch];
  bool bad[kMaxBatch];
};

// The group of sequence b: the last one that begins at or before it, if it holds it; -1: none.
__device__ __forceinline__ int group_of(const SharedMem& sh, int n, int b) {
  int lo = 0, hi = n;  // (as many groups begin at or before b as lie below `lo`)
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sh.cu[mid] <= b) lo = mid + 1;
    else hi = mid;
  }
  return lo > 0 && b < sh.cu[lo] ? lo - 1 : -1;
}

// Pages that group i shares (one sequence alone would gain nothing).
__device__ __forceinline__ int shares_of(const SharedMem& sh, int i) {
  return !sh.bad[i] && sh.cu[i + 1] - sh.cu[i] > 1 ? sh.pages[i] : 0;
}

// Which sequences share what, as tiles, made by every CTA for itself; returns the number of groups,
// 0 if their offsets are out of order: then all sequences are by themselves.  So are those of a
// group whose number of pages is out of range or more than a member holds: the result does not
// depend on what is shared, only the time does.  (Loops are not unrolled: this runs once, and its
// instructions take longer to come than to run.)
__device__ __forceinline__ int make_plan(const SharedArgs& a, SharedMem& sh, bool first) {
  const PagedGeo& geo = a.own.geo;
  const int tid = threadIdx.x, lane = tid & 31, n = a.n_groups, B = geo.B, cap = geo.max_pages * geo.P;
  const int len0 = tid < B ? geo.len[tid] : 0;
#pragma unroll 1
  for (int i = tid; i <= n; i += kSharedThreads) {
    sh.cu[i] = a.cu_group[i];
    if (i == n) break;
    const int pages = a.shared_pages[i];
    sh.bad[i] = pages < 0 || pages > geo.max_pages;
    sh.pages[i] = pages;
    if (sh.bad[i] && first) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
  }
  __syncthreads();
  bool wrong = false;
#pragma unroll 1
  for (int i = tid; i < n; i += kSharedThreads) wrong |= sh.cu[i] < 0 || sh.cu[i] > sh.cu[i + 1] || sh.cu[i + 1] > B;
  const int groups = __syncthreads_or(wrong) ? 0 : n;
  if (groups < n && first && tid == 0) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
#pragma unroll 1
  for (int b = tid; b < B; b += kSharedThreads) {
    const int g = group_of(sh, groups, b), len = b == tid ? len0 : geo.len[b];
    if (g < 0 || sh.pages[g] <= 0) continue;
    if (len < 0 || len > cap || len < (long long)sh.pages[g] * geo.P) {
      if (first) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
      sh.bad[g] = true;
    }
  }
  __syncthreads();
  if (tid < 32) {
    int t0 = 0;  // tiles and blocks of the groups before
    long long x0 = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < groups; i0 += 32) {
      const int i = i0 + lane, pages = i < groups ? shares_of(sh, i) : 0;
      const int tiles = pages > 0 ? (sh.cu[i + 1] - sh.cu[i] + 2 * a.tok - 1) / (2 * a.tok) : 0;
      const long long blocks = (long long)((pages * geo.P + kKeys - 1) / kKeys) * geo.H_kv;
      int t = tiles;
      long long x = tiles * blocks;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int t1 = __shfl_up_sync(kFull, t, o);
        const long long x1 = __shfl_up_sync(kFull, x, o);
        if (lane >= o) t += t1, x += x1;
      }
      int at = t0 + t - tiles;
      long long start = x0 + x - tiles * blocks;
      t0 += __shfl_sync(kFull, t, 31);
      x0 += __shfl_sync(kFull, x, 31);
#pragma unroll 1
      for (int y = 0; y < tiles; ++y, ++at, start += blocks) {
        const int b0 = sh.cu[i] + y * 2 * a.tok;
        sh.tile[at] = SharedTile{b0, min(2 * a.tok, sh.cu[i + 1] - b0), sh.cu[i], pages * geo.P};
        sh.start[at] = start;
      }
    }
    if (lane == 0) sh.n_tiles = t0, sh.total = sh.start[t0] = x0;
  }
  __syncthreads();
  return groups;
}

// Flags what is wrong with the groups where nothing can be shared (one CTA).
__global__ void __launch_bounds__(kSharedThreads) check_groups_kernel(const __grid_constant__ SharedArgs a) {
  __shared__ SharedMem sh;
  pdl_launch();
  pdl_wait();
  make_plan(a, sh, true);
}

// Leaves the plan for the kernels behind (one warp of the first CTA, beside the others' work).
__device__ __forceinline__ void publish_plan(const SharedArgs& a, const SharedMem& sh, int groups) {
  const PagedGeo& geo = a.own.geo;
  const int lane = threadIdx.x & 31, cap = geo.max_pages * geo.P;
#pragma unroll 1
  for (int i = lane; i <= sh.n_tiles; i += 32) {
    a.plan->start[i] = sh.start[i];
    if (i < sh.n_tiles) a.plan->tile[i] = sh.tile[i];
  }
  bool alone = false;
  long long before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < geo.B; b0 += 32) {
    const int b = b0 + lane, g = b < geo.B ? group_of(sh, groups, b) : -1, skip = g < 0 ? 0 : shares_of(sh, g);
    const int len = b < geo.B ? min(max(geo.len[b], 0), cap) : 0;
    if (b < geo.B) a.skip[b] = skip;
    alone |= b < geo.B && skip == 0;
    const int tiles = b < geo.B ? (len - skip * geo.P + kOwnTile - 1) / kOwnTile : 0;
    long long x = tiles;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long x1 = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += x1;
    }
    if (b < geo.B) a.plan->own[b + 1] = before + x;
    before += __shfl_sync(kFull, x, 31);
  }
  alone = __any_sync(kFull, alone);
  if (lane == 0) a.plan->own[0] = 0, a.plan->n_tiles = sh.n_tiles, a.plan->total = sh.total, a.plan->alone = alone;
}

// The pieces of a CTA's share of the line: blocks [j0, j1) of KV head g of tile t.
struct Walk {
  long long x, to;
  int t, g, nb, j0, j1;
  SharedTile tile;

  __device__ __forceinline__ Walk(const SharedMem& sh, int n_tiles, int H_kv, long long from, long long to_) {
    x = from;
    to = to_;
    if (x >= to) return;
    int lo = 0, hi = n_tiles;  // last tile that begins at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.start[mid] <= x) lo = mid;
      else hi = mid;
    }
    t = lo;
    load(sh);
    const long long in = x - sh.start[t];
    g = in < (1LL << 31) ? int(uint32_t(in) / uint32_t(nb)) : int(in / nb);
    j0 = int(in - (long long)g * nb);
    j1 = int(min((long long)nb, j0 + (to - x)));
  }
  __device__ __forceinline__ void load(const SharedMem& sh) {
    tile = sh.tile[t];
    nb = (tile.n + kKeys - 1) / kKeys;
  }
  __device__ __forceinline__ bool more() const { return x < to; }
  __device__ __forceinline__ void next(const SharedMem& sh, int H_kv) {
    x += j1 - j0;
    if (x >= to) return;
    j0 = 0;
    if (++g == H_kv) {
      g = 0;
      ++t;
      load(sh);
    }
    j1 = int(min((long long)nb, to - x));
  }
};

// The probabilities of 16 keys: p = 2^(c s - c m), summed in fp32, as three bf16
// terms, pairs of keys in a word.  Each term is the upper half of what is left, cut and not
// rounded: 8 bits each, 24 in all, so that nothing is lost.
__device__ __forceinline__ void exp_terms(const uint32_t* s, uint64_t cc, uint64_t mm, uint64_t (&sum)[4], uint32_t (&w)[kTerms][8]) {
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint64_t y = fma2(pair(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), cc, mm);
    uint64_t p = pair(ex2(lo(y)), ex2(hi(y)));
    sum[x & 3] = add2(sum[x & 3], p);
#pragma unroll
    for (int e = 0; e < kTerms; ++e) {
      const uint32_t p0 = uint32_t(p), p1 = uint32_t(p >> 32);
      w[e][x] = __byte_perm(p0, p1, 0x7632);
      if (e + 1 < kTerms)  // (p is not negative)
        p = add2(p, pair(__uint_as_float((p0 & 0xffff0000u) | 0x80000000u), __uint_as_float((p1 & 0xffff0000u) | 0x80000000u)));
    }
  }
}

template <int D, bool TMA>
__global__ void __launch_bounds__(kSharedThreads, 1) shared_attn_kernel(const __grid_constant__ SharedArgs a) {
  using C = SCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ SharedMem sh;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.own.geo;
  const int G = a.own.G, H_kv = geo.H_kv;
  const long long wait_cycles = a.own.wait_cycles;

  if (warp == 9) {
    if (lane == 0) {
      sh.abort = 0;
      mbar_init(smem_addr(&sh.q_full), 1);
      mbar_init(smem_addr(&sh.q_empty), 1);
      for (int i = 0; i < kRegions; ++i) {
        mbar_init(smem_addr(&sh.s_full[i]), 1);
        mbar_init(smem_addr(&sh.p_ready[i]), 128);
        mbar_init(smem_addr(&sh.o_full[i]), 1);
      }
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(smem_addr(&sh.kv_full[i]), TMA ? 1 : 2);  // (without maps, a warp for K and one for V)
        mbar_init(smem_addr(&sh.kv_empty[i]), 1);
      }
      mbar_init(smem_addr(&sh.drained), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tc5::alloc(smem_addr(&sh.tmem), 512);
    tc5::fence_before();
  }
  if (tid < 3) {
    const CUtensorMap* const map = tid == 0 ? &a.tmq : tid == 1 ? &a.tmk : &a.tmv;
    if (tid == 0 || TMA) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  pdl_launch();
  pdl_wait();
  const int groups = make_plan(a, sh, blockIdx.x == 0);
  const int n_tiles = sh.n_tiles;
  tc5::fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t q_sm = base, kv_sm = base + 2 * C::QTILE;
  auto wait_for = [&](uint64_t* bar, int use) {
    return wait(smem_addr(bar), use & 1, sh, geo.status, wait_cycles);
  };
  const Cut cut(sh.total, gridDim.x, 1);
  const int share = blockIdx.x;
  const long long from = share < cut.shares ? cut.start(share) : 0, to = share < cut.shares ? cut.start(share + 1) : 0;
  auto halves = [&](const SharedTile& t) { return t.seqs > a.tok ? 2 : 1; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 8 || (warp == 10 && !TMA)) {
      // ---- loads: each piece's Q, then its pairs of K and V through the ring.  With maps one
      // warp: a lane looks up the page of its box, some blocks at a time, and loads it.  Without,
      // a warp for K and one for V copy row by row.
      const bool keys = warp == 8;
      int st = 0, uses = 0, q_uses = 0;  // the next stage, and the times that the ring has gone round
      int pending = -1;                  // the stage whose copies have not been waited for (!TMA)
      bool ok = true;
      auto landed = [&](int left) {  // all but the last `left` groups of copies
        if (left) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        // (the tensor cores read through the async proxy)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.kv_full[pending]));
        pending = -1;
      };
      for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
        if (keys) {
          if (q_uses > 0) ok = __all_sync(kFull, wait_for(&sh.q_empty, q_uses - 1));
          if (!ok) break;
          if (lane == 0) {
            const int nh = halves(w.tile);
            mbar_arrive_expect_tx(smem_addr(&sh.q_full), uint32_t(nh * a.tok * G) * 128 * C::HALVES);
            for (int i = 0; i < nh; ++i)
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(q_sm + i * C::QTILE + h * (kRows * 128), &a.tmq, h * 64, w.g * G, w.tile.b0 + i * a.tok, smem_addr(&sh.q_full));
          }
          ++q_uses;
        }
        const int32_t* const table = geo.table + int64_t(w.tile.lead) * geo.max_pages;
        auto page_of = [&](int pos) {
          int page = pos < w.tile.n ? table[pos / geo.P] : 0;
          if (page < 0 || page >= geo.n_pages) {
            set_status(geo.status, SFI_DEV_BAD_INDEX);
            page = 0;
          }
          return page;
        };
        if constexpr (TMA) {
          const int boxes = kKeys / a.box, ahead = 32 / boxes;
          int rows = 0, last = 0, left = 0;  // rows of `left` blocks, a lane for each box; the last block's
          for (int j = w.j0; j <= w.j1 && ok; ++j) {
            if (j < w.j1 && left == 0) {
              const int pos = j * kKeys + lane * a.box;
              // (rows behind the shared ones: zeros, since 0 * NaN is not 0)
              rows = pos < w.tile.n ? int(page_of(pos) * (geo.page_stride / D) + w.g * geo.P + pos % geo.P) : a.pool_rows;
              left = ahead;
            }
            const int row = __shfl_sync(kFull, rows, min((ahead - left) * boxes + lane % boxes, 31));
            if (uses > 0) ok = __all_sync(kFull, wait_for(&sh.kv_empty[st], uses - 1));
            if (!ok) break;
            const uint32_t bar = smem_addr(&sh.kv_full[st]), dst = kv_sm + st * 2 * C::TILE + lane * a.box * 128;
            if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE * ((j < w.j1) + (j > w.j0)));
            __syncwarp();
            if (lane < boxes)
              for (int h = 0; h < C::HALVES; ++h) {
                if (j < w.j1) tma_load_3d(dst + h * (kKeys * 128), &a.tmk, 0, row, h, bar);
                if (j > w.j0) tma_load_3d(dst + C::TILE + h * (kKeys * 128), &a.tmv, 0, last, h, bar);
              }
            last = row;
            --left;
            if (++st == C::STAGES) st = 0, ++uses;
          }
        } else {
          constexpr int CH = D / 8;  // 16-byte chunks of a row
          const uint8_t* const pool = static_cast<const uint8_t*>(keys ? a.own.k : a.own.v);
          for (int y = w.j0; y <= w.j1; ++y) {
            const int j = keys ? y : y - 1;  // the block
            const bool there = j >= w.j0 && j < w.j1;
            int64_t at[2];  // bytes from the pool's start to rows lane and lane + 32, -1: no row
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int pos = j * kKeys + lane + 32 * i;
              const bool in = there && pos < w.tile.n && lane + 32 * i < kKeys;
              const int64_t row = page_of(in ? pos : w.tile.n) * geo.page_stride + (int64_t(w.g) * geo.P + pos % geo.P) * D;
              at[i] = in ? row * 2 : -1;
            }
            if (uses > 0 && !__all_sync(kFull, mbar_test_wait(smem_addr(&sh.kv_empty[st]), (uses - 1) & 1))) {
              // (whoever has to free it may wait for what is pending)
              if (pending >= 0) landed(0);
              ok = __all_sync(kFull, wait_for(&sh.kv_empty[st], uses - 1));
            }
            if (!ok) break;
            if (there) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll 8
                for (int z = 0; z < (i == 0 ? CH : CH * (kKeys - 32) / 32); ++z) {
                  const int r = (z * 32 + lane) / CH, ch = lane % CH;  // of these 32 rows
                  const int64_t src = __shfl_sync(kFull, at[i], r);
                  const uint32_t dst = kv_sm + (st * 2 + !keys) * C::TILE + (ch >> 3) * (kKeys * 128) + (32 * i + r) * 128 + (((ch & 7) ^ (r & 7)) << 4);
                  cp_async16_zfill(dst, pool + max(src, int64_t(0)) + (src >= 0 ? ch * 16 : 0), src >= 0 ? 16 : 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (pending >= 0) landed(1);
            pending = st;
            if (++st == C::STAGES) st = 0, ++uses;
          }
          // (the next piece's Q waits for this one's last scores, and so for its last K)
          if (pending >= 0) landed(0);
        }
      }
      // no copy may be in flight when the CTA exits (after a wait that gave up, some may
      // never have been waited for)
      if (!TMA && pending >= 0) landed(0);
      if (q_uses > 0) mbar_wait(smem_addr(&sh.q_full), (q_uses - 1) & 1);
      if (TMA)
        for (int y = 0; y < C::STAGES; ++y) {
          const int last = y < st ? uses : uses - 1;  // the stage's last use
          if (last >= 0) mbar_wait(smem_addr(&sh.kv_full[y]), last & 1);
        }
    } else if (warp == 9) {
      // ---- products, all of them from one lane
      if (tc5::elect()) {
        // The tensor cores hold only a few products in waiting (some 200 clocks), so what lies
        // between one step's and the next's is kept short: stages, regions and phases are counted
        // up and not divided, a step has one wait for P, done while the step before is multiplied,
        // and there is one commit for the scores and one for a pair of K and V.  (With a wait and
        // a commit for each of K, V and the two parts of P: 1400 clocks a step, of which 910 are
        // products.)
        constexpr uint32_t kIdS = tc5::idesc_bf16(kRows, kKeys, false);
        constexpr uint32_t kIdO = tc5::idesc_bf16(kRows, D, true);
        const uint32_t full = smem_addr(&sh.kv_full[0]), empty = smem_addr(&sh.kv_empty[0]);
        const uint32_t s_full = smem_addr(&sh.s_full[0]), p_ready = smem_addr(&sh.p_ready[0]), o_full = smem_addr(&sh.o_full[0]);
        const uint64_t q_desc = tc5::desc_sw128(q_sm, 16, 1024), k_desc = tc5::desc_sw128(kv_sm, 16, 1024),
                       v_desc = tc5::desc_sw128(kv_sm + C::TILE, kKeys * 128, 1024);
        auto await = [&](uint32_t bar, uint32_t parity) { return wait(bar, parity, sh, geo.status, wait_cycles); };
        uint32_t ks = 0, k_ph = 0, vs = 0;             // the stages of the next K and V
        uint32_t rs = 0, rp = 0, p_ph = 0;             // the regions of the next scores and P
        uint32_t s_half = 0, half = 0, q_ph = 0;       // the halves of the next scores and P
        bool ok = true;
        for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
          // Steps of a piece: block k / 2 for a half where both halves have rows, else block k,
          // both halves having the same rows.  The halves take the steps in turn, over all pieces.
          const bool two = halves(w.tile) == 2;
          const int n = (w.j1 - w.j0) << two;
          // Scores of the next step: whether it is the first of its block's steps, and the last.
          auto scores = [&](bool begins, bool ends) {  // S = Q K^T
            if (begins) ok = ok && await(full + ks * 8, k_ph);
            if (!ok) return;
            const uint64_t qd = q_desc + (two && s_half ? C::QTILE >> 4 : 0), kd = k_desc + ks * (2 * C::TILE >> 4);
            const uint32_t d = tmem + rs * kRegion;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc5::mma_ss(d, qd + (((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4),
                          kd + (((kk / 4) * (kKeys * 128) + (kk % 4) * 32) >> 4), kIdS, kk > 0);
            tc5::commit(s_full + rs * 8);
            if (ends) {
              const bool wraps = ks + 1 == C::STAGES;
              ks = wraps ? 0 : ks + 1;
              k_ph ^= wraps;
            }
            rs = rs + 1 == kRegions ? 0 : rs + 1;
            s_half ^= 1;
          };
          uint32_t chain = 0;  // steps since the sums were begun, of both halves
          // Products with V of the next step, and whether it is the last of its block's.
          auto products = [&](bool ends) {  // O (+)= P V
            const uint64_t vd = v_desc + vs * (2 * C::TILE >> 4);
            const uint32_t d = tmem + kSums + half * 128, p = tmem + rp * kRegion;
            tc5::fence_after();
#pragma unroll
            for (int z = 0; z < kKeys / 16; ++z)
#pragma unroll
              for (int e = kTerms - 1; e >= 0; --e)  // small terms first
                tc5::mma_ts(d, p + term_at(z, e), vd + z * (2048 >> 4), kIdO, chain > 1 || z > 0 || e + 1 < kTerms);
            if (ends) {
              tc5::commit(empty + vs * 8);
              vs = vs + 1 == C::STAGES ? 0 : vs + 1;
            }
            chain = chain + 1 == 2 * kChain ? 0 : chain + 1;
            half ^= 1;
            const bool wraps = rp + 1 == kRegions;
            rp = wraps ? 0 : rp + 1;
            p_ph ^= wraps;
          };
          // A step with more behind it: P of the next one mostly lies there already; if not, the
          // scores go first.
          auto step = [&](bool ends, bool s_begins, bool s_ends) {
            products(ends);
            const bool there = mbar_test_wait(p_ready + rp * 8, p_ph);
            scores(s_begins, s_ends);
            if (!there) ok = ok && await(p_ready + rp * 8, p_ph);
          };
          ok = await(smem_addr(&sh.q_full), q_ph);
          q_ph ^= 1;
          // (a region is free: the products with the P that lay there were issued before)
          for (int k = 0; k < min(n, kRegions); ++k) scores(!two || (k & 1) == 0, !two || (k & 1));
          tc5::commit(empty + vs * 8);  // the first pair, which has no V
          vs = vs + 1 == C::STAGES ? 0 : vs + 1;
          if (n <= kRegions) tc5::commit(smem_addr(&sh.q_empty));
          ok = ok && await(p_ready + rp * 8, p_ph);
          // (without a branch but for waits: one costs as much as an MMA)
          int k = 0;
          if (two) {
            for (; k + kRegions + 1 < n && ok; k += 2) {
              step(false, false, true);
              step(true, true, false);
            }
          } else {
            for (; k + kRegions < n && ok; ++k) step(true, true, true);
          }
          for (; k < n && ok; ++k) {
            if (two ? k == n - 2 : k == n - 1) {  // the last pair, which has no K
              ok = await(full + ks * 8, k_ph);
              if (++ks == C::STAGES) ks = 0, k_ph ^= 1;
              if (!ok) break;
            }
            const uint32_t region = rp;
            products(!two || (k & 1));
            if (k + kRegions < n) scores((k & 1) != 0, (k & 1) == 0);
            // (who waits for these products otherwise waits for scores that were issued behind them)
            else tc5::commit(o_full + region * 8);
            if (k + kRegions + 1 == n || (k + kRegions == n && !two)) {
              if (n > kRegions) tc5::commit(smem_addr(&sh.q_empty));
            }
            if (k + 1 < n) ok = ok && await(p_ready + rp * 8, p_ph);
          }
        }
        // the products in flight end before tensor memory is freed, whether or
        // not a softmax warp still waits for them
        tc5::commit(smem_addr(&sh.drained));
        mbar_wait(smem_addr(&sh.drained), 0);
      }
      __syncwarp();
    } else if (warp == 11 && blockIdx.x == 0) {
      publish_plan(a, sh, groups);
    }
  } else {
    // ---- softmax, sums and states of half i: one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int i = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // 32 * (warp % 4) in the lane field
    const uint32_t o_tm = tmem + kSums + i * 128 + lanes;
    const float c = a.own.scale_log2;
    int done = 0;            // steps of the pieces before
    uint32_t o_ph = 0;       // bit r: parity of the region's next commit of sums
    bool ok = true;
    for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
      const bool two = halves(w.tile) == 2;
      const int n = (w.j1 - w.j0) << two;
      float m = -INFINITY, l = 0.f;
      uint64_t o[D / 2];
#pragma unroll
      for (int x = 0; x < D / 2; ++x) o[x] = 0;
      // the products with V of the last few blocks, from tensor memory (the tensor cores truncate
      // where they add; here it is fp32)
      auto add_sums = [&] {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t v[16];
          tc5::ld16(o_tm + 16 * x, v);
          tc5::wait_ld();
          pin(v);
#pragma unroll
          for (int y = 0; y < 8; ++y)
            o[8 * x + y] = add2(o[8 * x + y], pair(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])));
        }
      };
      // The products of step k are complete once the scores of step k + 3 are, which were issued
      // behind them, or their own commit has arrived, where there are no such scores.
      auto summed = [&](int k) {
        const uint32_t step = done + k, reg = step % kRegions;
        if (k + kRegions < n) return __all_sync(kFull, wait_for(&sh.s_full[reg], step / kRegions + 1));
        return __all_sync(kFull, wait_for(&sh.o_full[reg], o_ph >> reg & 1));
      };
      const int k0 = (i - done) & 1;
      int chain = 0;  // blocks whose products are in tensor memory
      for (int k = k0; k < n; k += 2) {
        const int j = w.j0 + (k >> two), lim = w.tile.n - j * kKeys;
        const uint32_t step = done + k, reg = step % kRegions, s_tm = tmem + reg * kRegion + lanes;
        ok = __all_sync(kFull, wait_for(&sh.s_full[reg], step / kRegions));
        if (!ok) break;
        tc5::fence_after();
        // (32 scores and 16, these again for their exponentials: registers are short)
        uint32_t s[32];
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        {
          uint32_t t[16];
          tc5::ld16(s_tm + 32, t);
          tc5::ld32(s_tm, s);
          tc5::wait_ld();
          pin(t);
          pin(s);
          if (lim < kKeys) {
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = x < lim ? s[x] : 0xff800000u;
#pragma unroll
            for (int x = 0; x < 16; ++x) t[x] = 32 + x < lim ? t[x] : 0xff800000u;
          }
#pragma unroll
          for (int x = 0; x < 16; x += 2)
            mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(t[x]), __uint_as_float(t[x + 1]));
        }
#pragma unroll
        for (int x = 0; x < 32; x += 2)
          mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        const bool grow = (top - m) * c > kGrow, any = __any_sync(kFull, grow);
        if (chain == kChain || (any && chain > 0)) {
          ok = summed(k - 2);
          if (!ok) break;
          tc5::fence_after();
        }
        if (chain == kChain) add_sums(), chain = 0;
        if (any) {
          const float f = grow ? ex2((m - top) * c) : 1.f;
          if (grow) m = top;
          l *= f;
#pragma unroll
          for (int x = 0; x < D / 2; ++x) o[x] = mul2(o[x], pair(f, f));
          if (chain > 0) {
#pragma unroll 1
            for (int x = 0; x < D / 16; ++x) {
              uint32_t v[16];
              tc5::ld16(o_tm + 16 * x, v);
              tc5::wait_ld();
              pin(v);
#pragma unroll
              for (int y = 0; y < 16; ++y) v[y] = __float_as_uint(__uint_as_float(v[y]) * f);
              tc5::st16(o_tm + 16 * x, v);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : -m * c;
        const uint64_t cc = pair(c, c), mm = pair(mc, mc);
        uint64_t sum[4] = {0, 0, 0, 0};
        hand_over(smem_addr(&sh.p_ready[reg]), [&] {
#pragma unroll
          for (int z = 0; z < kKeys / 16; ++z) {
            if (z == 2) {
              uint32_t t[16];
              tc5::ld16(s_tm + 32, t);
              tc5::wait_ld();
              pin(t);
#pragma unroll
              for (int x = 0; x < 16; ++x) s[x] = 32 + x < lim ? t[x] : 0xff800000u;
            }
            uint32_t p[kTerms][8];
            exp_terms(s + (z & 1) * 16, cc, mm, sum, p);
#pragma unroll
            for (int e = 0; e < kTerms; ++e) tc5::st8(s_tm + term_at(z, e), p[e]);
          }
        });
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += lo(sum[0]) + hi(sum[0]);
        ++chain;
      }
      if (ok && chain > 0) {
        ok = summed(n - 1 - ((n - 1 - k0) & 1));
        tc5::fence_after();
        if (ok) add_sums();
      }
      if (!ok) break;
      // the commits of this piece's last steps
      for (int k = max(0, n - kRegions); k < n; ++k) o_ph ^= 1u << (done + k) % kRegions;
      done += n;
      // the piece's state (rows side by side, so that the lanes' stores are)
      float* const st = a.states + int64_t(share + w.t * H_kv + w.g) * (kTileRows * (D + 2)) + i * kRows + r;
      if (r < a.tok * G && (two ? i : 0) * a.tok + r / G < w.tile.seqs) {
#pragma unroll
        for (int x = 0; x < D / 2; ++x) st[2 * x * kTileRows] = lo(o[x]), st[(2 * x + 1) * kTileRows] = hi(o[x]);
        st[D * kTileRows] = m, st[(D + 1) * kTileRows] = l;
      }
    }
    tc5::fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc5::fence_after();
    tc5::dealloc(tmem, 512);
  }
}

// ---- the join
// Items of 32 rows of a tile and 16 columns.  First the states of the shared part, a lane a row,
// as these states lie, and the pieces dealt over the warps; then, through shared memory, the
// warps' states and those of the sequences' own positions, 8 lanes a row, as those lie.  Then
// the pieces of sequences that share nothing.
// Bound by latency: a few dependent reads from L2, about 1000 clocks each, so reads that do
// not depend on one another are issued together, and nothing is computed again that the first
// kernel could leave.  (All pieces by each warp, 8 columns of 64 each, and a lane a row for the own
// positions too, where each read touches 32 lines: 25 us for 256 rows of 20 pieces.)
struct State {
  float m = -INFINITY, l = 0.f;
  // Takes in N states; returns the factors of what it was and of theirs: -1 for one that saw only
  // scores of -infinity, or nothing, and adds nothing.  Any other's is its weight, which may be 0 in
  // fp32: its finite sums then add nothing, and its NaNs and infinities reach the result, since 0
  // times one is NaN.  (A floor under the weights would let large finite sums through: 2^-126 of 5e37.)
  static __device__ __forceinline__ float factor(float m, float l, float top, float c) {
    return m == -INFINITY && l == 0.f ? -1.f : ex2((m - top) * c);
  }
  template <int N>
  __device__ __forceinline__ float take(const float (&mv)[N], const float (&lv)[N], float (&f)[N], float c) {
    float top = m;
#pragma unroll
    for (int w = 0; w < N; ++w) top = fmaxf(top, mv[w]);
    const float was = factor(m, l, top, c);
    l = was < 0.f ? 0.f : l * was;
#pragma unroll
    for (int w = 0; w < N; ++w) {
      f[w] = factor(mv[w], lv[w], top, c);
      l = f[w] < 0.f ? l : fmaf(f[w], lv[w], l);
    }
    m = top;
    return was;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, kJoinCtas) shared_join_kernel(const __grid_constant__ SharedArgs a, int grid, int ny) {
  constexpr int AHEAD = 3, OWN = 4;  // states that a thread reads at a time
  constexpr int STEP = kTileRows * (D + 2);
  __shared__ Line ln;
  __shared__ float o_sh[kWarps][kJoinCols][33], ml_sh[kWarps][2][32];
  const PagedGeo& geo = a.own.geo;
  const int H_kv = geo.H_kv, G = a.own.G, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float c = a.own.scale_log2;
  pdl_launch();
  pdl_wait();
  const int n_tiles = a.plan->n_tiles, alone = a.plan->alone;
  const Cut shared(a.plan->total, grid, 1), own(a.plan->own[geo.B] * H_kv, grid * kPagedWarps, 1);
  // (32-row blocks that all tiles have first: they are spread over the SMs)
  const int columns = n_tiles * H_kv * (D / kJoinCols), items = columns * (kTileRows / 32);
  for (int y = blockIdx.x; y < items; y += gridDim.x) {
    const int block = y / columns, in = y - block * columns, unit = in / (D / kJoinCols), t = unit / H_kv, g = unit - t * H_kv;
    const int d0 = in % (D / kJoinCols) * kJoinCols;
    const SharedTile tile = a.plan->tile[t];
    const long long start = a.plan->start[t];
    const int half = block * 32 / kRows;
    // the row at place x of the block: its sequence of the tile, -1 for none, and head of the group
    auto seq_of = [&](int x, int& head) {
      const int r = (block * 32 + x) % kRows, tt = r / G, seq = half * a.tok + tt;
      head = r - tt * G;
      return tt < a.tok && seq < tile.seqs ? seq : -1;
    };
    int head;
    const bool valid = seq_of(lane, head) >= 0;
    if (!__syncthreads_or(valid)) continue;  // (and what an item before left in shared memory has been read)
    // whose row this thread writes, and where its own positions lie in their line
    const int seq = seq_of(tid >> 3, head), b = tile.b0 + max(seq, 0);
    const long long own0 = a.plan->own[b], own1 = a.plan->own[b + 1];
    {
      const int nb = (tile.n + kKeys - 1) / kKeys;
      const long long begin = start + (long long)g * nb;
      const int first = shared.holder(begin), pieces = shared.holder(begin + nb - 1) - first + 1;
      // (a tile of one half has two states of each row in a piece)
      const bool both = tile.seqs <= a.tok;
      const int n = valid ? both ? 2 * pieces : pieces : 0;
      const float* const p = a.states + int64_t(first + unit) * STEP + block * 32 + lane;
      State st;
      float o[kJoinCols];
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
#pragma unroll 1
      for (int w0 = warp; w0 < n; w0 += AHEAD * kWarps) {
        float mv[AHEAD], lv[AHEAD], f[AHEAD], v[AHEAD][kJoinCols];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const int w = w0 + k * kWarps;
          const float* const q = p + (both ? int64_t(w >> 1) * STEP + (w & 1) * kRows : int64_t(w) * STEP);
          const bool there = w < n;
          mv[k] = there ? __ldcg(q + D * kTileRows) : -INFINITY;
          lv[k] = there ? __ldcg(q + (D + 1) * kTileRows) : 0.f;
#pragma unroll
          for (int e = 0; e < kJoinCols; ++e) v[k][e] = there ? __ldcg(q + (d0 + e) * kTileRows) : 0.f;
        }
        const float was = st.take(mv, lv, f, c);
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) {
          o[e] = was < 0.f ? 0.f : o[e] * was;
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) o[e] = f[k] < 0.f ? o[e] : fmaf(f[k], v[k][e], o[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) o_sh[warp][e][lane] = o[e];
      ml_sh[warp][0][lane] = st.m, ml_sh[warp][1][lane] = st.l;
    }
    __syncthreads();
    if (seq < 0) continue;
    const int row = tid >> 3, col = 2 * (tid & 7);
    State st;
    float2 o = make_float2(0.f, 0.f);
    {
      float mv[kWarps], lv[kWarps], f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mv[w] = ml_sh[w][0][row], lv[w] = ml_sh[w][1][row];
      st.take(mv, lv, f, c);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (!(f[w] < 0.f)) o.x = fmaf(f[w], o_sh[w][col][row], o.x), o.y = fmaf(f[w], o_sh[w][col + 1][row], o.y);
    }
    const long long nt = own1 - own0, o0 = own0 * H_kv + g * nt;
    if (nt > 0) {
      const int first = own.holder(o0), n = own.holder(o0 + nt - 1) - first + 1;
      const float* p = a.own.partials + ((first + int64_t(b) * H_kv + g) * G + head) * (D + 2);
      const int64_t step = int64_t(G) * (D + 2);
#pragma unroll 1
      for (int w0 = 0; w0 < n; w0 += OWN, p += OWN * step) {
        float mv[OWN], lv[OWN], f[OWN];
        float2 v[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
          const bool there = w0 + k < n;
          const float2 ml = there ? __ldcg(reinterpret_cast<const float2*>(p + k * step + D)) : make_float2(-INFINITY, 0.f);
          mv[k] = ml.x, lv[k] = ml.y;
          v[k] = there ? __ldcg(reinterpret_cast<const float2*>(p + k * step + d0 + col)) : make_float2(0.f, 0.f);
        }
        const float was = st.take(mv, lv, f, c);
        o.x = was < 0.f ? 0.f : o.x * was, o.y = was < 0.f ? 0.f : o.y * was;
#pragma unroll
        for (int k = 0; k < OWN; ++k)
          if (!(f[k] < 0.f)) o.x = fmaf(f[k], v[k].x, o.x), o.y = fmaf(f[k], v[k].y, o.y);
      }
    }
    const int64_t to = int64_t(b) * a.own.H_q + g * G + head;
    const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
    *reinterpret_cast<float2*>(a.own.out + to * D + d0 + col) = make_float2(o.x * inv, o.y * inv);
    if (d0 + col == 0 && a.own.lse) a.own.lse[to] = (st.m * c + log2f(st.l)) * 0.6931471805599453f;
  }
  if (!alone) return;
  __syncthreads();
  scan_lengths<kOwnTile, true>(geo, ln, false);
  const int nx = gridDim.x / ny;
  if (int(blockIdx.x) < nx * ny) join_units<kOwnTile, D, true>(a.own, ln, own, blockIdx.x % nx, nx, blockIdx.x / nx, ny);
}

template <int D, bool TMA>
cudaError_t launch_shared(const SharedArgs& a, bool own_tma, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(shared_attn_kernel<D, TMA>), int(SCfg<D>::SMEM), allowed);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(shared_attn_kernel<D, TMA>, dim3(grid), kSharedThreads, SCfg<D>::SMEM, st, a)) != cudaSuccess) return e;
  if ((e = launch_paged_pieces(a.own, D, own_tma, grid, st)) != cudaSuccess) return e;
  // CTAs for the items that there may be, or for 32 outputs of a unit each, while all of them
  // find room at once
  const long long most = (long long)kJoinCtas * grid, units = (long long)a.own.geo.B * a.own.geo.H_kv, y = a.own.G * (D / 32);
  const long long items = (long long)a.max_tiles * a.own.geo.H_kv * (kTileRows / 32 * (D / kJoinCols)), pieces = units * y;
  const int ctas = int(items < most && pieces < most ? (items < pieces ? pieces : items) : most);
  const int ny = int(units >= ctas ? 1 : ctas / units < y ? ctas / units : y);
  return launch_pdl(shared_join_kernel<D>, dim3(ctas), kThreads, 0, st, a, grid, ny);
}

}  // namespace

cudaError_t launch_check_groups(const SharedArgs& a, cudaStream_t st) {
  return launch_pdl(check_groups_kernel, dim3(1), kSharedThreads, 0, st, a);
}

cudaError_t launch_shared_attn(const SharedArgs& a, int D, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64) return a.box ? launch_shared<64, true>(a, use_tma, grid, st) : launch_shared<64, false>(a, use_tma, grid, st);
  return a.box ? launch_shared<128, true>(a, use_tma, grid, st) : launch_shared<128, false>(a, use_tma, grid, st);
}

}  // namespace sfi

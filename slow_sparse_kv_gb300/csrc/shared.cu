// Attention of one new token for sequences of which groups share their first pages:
// the shared positions are read once for a group, not once for each sequence.
//
// For sequence b of a group that shares n0 positions, softmax over all positions is joined
// from two states (m, l, o): over [0, n0), with the group's other sequences, and over
// [n0, len[b]), by itself, which is paged_attn.cu's kernel with the first pages left out.
//   out = sum_w f_w o_w / sum_w f_w l_w,  f_w = 2^(c (m_w - max m)),  c = log2(e) / sqrt(d)
//
// The shared part is a matrix product: the group's queries of a KV head, members x G rows,
// against n0 keys.  A tile is 2 x 128 such rows; all tiles' blocks of 128 keys, KV head by KV
// head, stand in one line, which is cut into a share of equal size for each CTA.  In a CTA, as
// in prefill.cu: S = Q K^T (tcgen05.mma from shared memory into tensor memory), softmax
// statistics with a thread for each row, P over S's columns, O += P V; the two halves of
// a tile alternate, so that the tensor cores work on one while the other's softmax runs.
// The output is fp32, so P is kept in two bf16 terms (16 bits), at the price of a second
// product with V.
// Bytes: 4 d n0 a group and KV head; flops 4 d (6 d with the second term) for each row and key.
// From 64 rows on about the tensor cores bound it, below HBM does.
//
// Four launches: the plan (which tiles, from the device's group offsets and lengths), the
// shared part, the sequences' own part, and one that joins the states of both.
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

constexpr int kSharedThreads = 384;  // 2 softmax warpgroups; two loading warps, an MMA warp, one that idles
constexpr int kRows = 128;           // query rows of a half tile
constexpr int kKeys = 64;            // keys of a block
constexpr int kParts = 2;            // P of a block is handed over in halves, of 32 keys
constexpr int kTerms = 3;            // bf16 terms of P
constexpr int kChain = 4;            // blocks of a half whose products with V are added in tensor memory
constexpr float kGrow = 8.0f;        // growth of the maximum (log2) that moves m
constexpr int kPlan = 1024;          // threads of the plan
template <int D>
constexpr int kJoinBlocks = kTileRows / 32 * (D / 32);  // CTAs' worth of a tile and KV head in the join
constexpr int kOwnTile = 16;         // positions of a tile of paged_attn.cu's kernel in bf16

template <int D>
struct SCfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t QTILE = kRows * 128 * HALVES;  // bytes of 128 rows
  static constexpr uint32_t TILE = kKeys * 128 * HALVES;   // and of a block of K or V
  static constexpr int STAGES = 8;                         // of them in flight
  static constexpr uint32_t SMEM = 1024 + 2 * QTILE + STAGES * TILE;
  static constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 504 - 2 * SOFTMAX_REGS;
};

// Where term e of half h of a block's P lies behind the block's scores' first column: the
// first half's next to the second half's scores, which are read again after it.
__host__ __device__ constexpr int term_at(int h, int e) { return h == 0 ? (e == 0 ? 0 : 48 + 16 * e) : 16 * (e + 1); }

// ---- the plan
// Inclusive sum over the CTA (kPlan threads).
__device__ __forceinline__ long long plan_scan(long long x, long long* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
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

// Which sequences share what, as tiles.  Offsets that are out of order leave all sequences
// by themselves; so does, for its group, a number of pages that is out of range or more
// than a member holds: the result does not depend on what is shared, only the time does.
__global__ void __launch_bounds__(kPlan) shared_plan_kernel(const __grid_constant__ SharedArgs a) {
  __shared__ int cu[kMaxBatch + 1], pages[kMaxBatch];
  __shared__ bool bad[kMaxBatch];
  __shared__ long long part[32];
  const PagedGeo& geo = a.own.geo;
  const int i = threadIdx.x, n = a.n_groups, B = geo.B, cap = geo.max_pages * geo.P;
  pdl_launch();
  pdl_wait();
  if (i <= n) cu[i] = a.cu_group[i];
  if (i == 0 && n == kPlan) cu[n] = a.cu_group[n];
  int mine = 0;
  if (i < n) {
    mine = a.shared_pages[i];
    if (mine < 0 || mine > geo.max_pages) {
      set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
      mine = 0;
    }
    pages[i] = mine;
    bad[i] = false;
  }
  const int len = i < B ? geo.len[i] : 0;
  __syncthreads();
  const bool out_of_order = i < n && (cu[i] < 0 || cu[i] > cu[i + 1] || cu[i + 1] > B);
  const bool none = __syncthreads_or(out_of_order);
  if (none && i == 0) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
  // the group of sequence i: the last one that begins at or before it, if it holds it
  int group = -1;
  if (!none && i < B) {
    int lo = 0, hi = n;  // (as many groups begin at or before i as lie below `lo`)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= i) lo = mid + 1;
      else hi = mid;
    }
    group = lo - 1;
    if (group >= 0 && i >= cu[group + 1]) group = -1;
    if (group >= 0 && pages[group] > 0 && (len < 0 || len > cap || len < (long long)pages[group] * geo.P)) {
      set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
      bad[group] = true;
    }
  }
  __syncthreads();
  const int members = !none && i < n ? cu[i + 1] - cu[i] : 0;
  // (one sequence alone would gain nothing)
  const int shares = members > 1 && !bad[i] ? pages[i] : 0;
  if (i < n) pages[i] = shares;
  __syncthreads();
  const int skip = i < B && group >= 0 ? pages[group] : 0;
  if (i < B) a.skip[i] = skip;
  const bool alone = __syncthreads_or(i < B && skip == 0);
  const int tiles = shares > 0 ? (members + 2 * a.tok - 1) / (2 * a.tok) : 0;
  const long long blocks = (shares * (long long)geo.P + kKeys - 1) / kKeys * geo.H_kv;
  const int first = int(plan_scan(tiles, part)) - tiles;
  const int all = int(part[31]);
  const long long start = plan_scan(tiles * blocks, part) - tiles * blocks;
  for (int t = 0; t < tiles; ++t) {
    SharedTile tile;
    tile.b0 = cu[i] + t * 2 * a.tok;
    tile.seqs = min(2 * a.tok, cu[i + 1] - tile.b0);
    tile.lead = cu[i];
    tile.n = shares * geo.P;
    a.plan->tile[first + t] = tile;
    a.plan->start[first + t] = start + t * blocks;
  }
  if (i == 0) {
    a.plan->n_tiles = all;
    a.plan->alone = alone;
    a.plan->total = a.plan->start[all] = part[31];
  }
}

// ---- the shared part
struct SharedMem {
  uint64_t q_full[2], q_empty[2], s_full[2], o_full[2], p_ready[2][kParts];
  uint64_t kv_full[8], kv_empty[8], drained;
  uint32_t tmem;
  volatile int abort;
  long long start[kMaxTiles + 1];
  SharedTile tile[kMaxTiles];
};

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
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_addr(&sh.q_full[i]), 1);
        mbar_init(smem_addr(&sh.q_empty[i]), 1);
        mbar_init(smem_addr(&sh.s_full[i]), 1);
        mbar_init(smem_addr(&sh.o_full[i]), 1);
        for (int h = 0; h < kParts; ++h) mbar_init(smem_addr(&sh.p_ready[i][h]), 128);
      }
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(smem_addr(&sh.kv_full[i]), 1);
        mbar_init(smem_addr(&sh.kv_empty[i]), 1);
      }
      mbar_init(smem_addr(&sh.drained), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tc5::alloc(smem_addr(&sh.tmem), 512);
    tc5::fence_before();
  }
  pdl_launch();
  pdl_wait();
  const int n_tiles = a.plan->n_tiles;
  for (int t = tid; t <= n_tiles; t += kSharedThreads) {
    sh.start[t] = a.plan->start[t];
    if (t < n_tiles) sh.tile[t] = a.plan->tile[t];
  }
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t q_sm = base, kv_sm = base + 2 * C::QTILE;
  auto stage = [&](int x) { return x % C::STAGES; };
  auto wait_for = [&](uint64_t* bar, int use) {
    return wait(smem_addr(bar), use & 1, sh, geo.status, wait_cycles);
  };
  const Cut cut(a.plan->total, gridDim.x, 1);
  const int share = blockIdx.x;
  const long long from = share < cut.shares ? cut.start(share) : 0, to = share < cut.shares ? cut.start(share + 1) : 0;
  auto halves = [&](const SharedTile& t) { return t.seqs > a.tok ? 2 : 1; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 8 || (warp == 10 && !TMA)) {
      // ---- loads: each piece's Q, then K_j, V_j, K_j+1, .. through the ring.  With maps one
      // warp: a lane looks up the page of its box, a block ahead, and loads it.  Without,
      // a warp for K and one for V copy row by row.
      const bool keys = warp == 8;
      int x = 0, q_uses[2] = {0, 0};
      int pending = -1;  // the stage use whose copies have not been waited for (!TMA)
      bool ok = true;
      auto landed = [&](int left) {  // all but the last `left` groups of copies
        if (left) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        // (the tensor cores read through the async proxy)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.kv_full[stage(pending)]));
      };
      for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
        if (keys) {
          for (int i = 0; i < halves(w.tile) && ok; ++i) {
            if (q_uses[i] > 0) ok = __all_sync(kFull, wait_for(&sh.q_empty[i], q_uses[i] - 1));
            if (!ok) break;
            if (lane == 0) {
              const uint32_t bar = smem_addr(&sh.q_full[i]);
              mbar_arrive_expect_tx(bar, uint32_t(a.tok * G) * 128 * C::HALVES);
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(q_sm + i * C::QTILE + h * (kRows * 128), &a.tmq, h * 64, w.g * G, w.tile.b0 + i * a.tok, bar);
            }
            ++q_uses[i];
          }
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
          // the pages of `ahead` blocks at a time: a lane for each box
          const int boxes = kKeys / a.box, ahead = 32 / boxes;
          int rows = 0;
          for (int j = w.j0; j < w.j1 && ok; ++j) {
            const int in = (j - w.j0) % ahead;
            if (in == 0) {
              const int pos = j * kKeys + lane * a.box;
              // (rows behind the shared ones: zeros, since 0 * NaN is not 0)
              rows = pos < w.tile.n ? int(page_of(pos) * (geo.page_stride / D) + w.g * geo.P + pos % geo.P) : a.pool_rows;
            }
            const int row = __shfl_sync(kFull, rows, in * boxes + lane % boxes);
            for (int y = 0; y < 2; ++y, ++x) {
              if (x >= C::STAGES) ok = __all_sync(kFull, wait_for(&sh.kv_empty[stage(x)], x / C::STAGES - 1));
              if (!ok) break;
              const uint32_t bar = smem_addr(&sh.kv_full[stage(x)]);
              if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE);
              __syncwarp();
              if (lane < boxes)
                for (int h = 0; h < C::HALVES; ++h)
                  tma_load_3d(kv_sm + stage(x) * C::TILE + h * (kKeys * 128) + lane * a.box * 128, y ? &a.tmv : &a.tmk, 0, row, h, bar);
            }
          }
        } else {
          constexpr int CH = D / 8;  // 16-byte chunks of a row
          const uint8_t* const pool = static_cast<const uint8_t*>(keys ? a.own.k : a.own.v);
          for (int j = w.j0; j < w.j1; ++j, x += 2) {
            const int y = x + (keys ? 0 : 1);
            int64_t at[kKeys / 32];  // bytes from the pool's start to rows lane + 32 i, -1: no row
#pragma unroll
            for (int i = 0; i < kKeys / 32; ++i) {
              const int pos = j * kKeys + lane + 32 * i;
              const int64_t row = page_of(pos) * geo.page_stride + (int64_t(w.g) * geo.P + pos % geo.P) * D;
              at[i] = pos < w.tile.n ? row * 2 : -1;
            }
            const int before = y / C::STAGES - 1;  // the stage's last use
            if (y >= C::STAGES && !__all_sync(kFull, mbar_test_wait(smem_addr(&sh.kv_empty[stage(y)]), before & 1))) {
              // (whoever has to free it may wait for what is pending)
              if (pending >= 0) landed(0), pending = -1;
              ok = __all_sync(kFull, wait_for(&sh.kv_empty[stage(y)], before));
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kKeys / 32; ++i)
#pragma unroll 8
              for (int z = 0; z < CH; ++z) {
                const int r = (z * 32 + lane) / CH, ch = lane % CH;  // of these 32 rows
                const int64_t src = __shfl_sync(kFull, at[i], r);
                const uint32_t dst = kv_sm + stage(y) * C::TILE + (ch >> 3) * (kKeys * 128) + (32 * i + r) * 128 + (((ch & 7) ^ (r & 7)) << 4);
                cp_async16_zfill(dst, pool + max(src, int64_t(0)) + (src >= 0 ? ch * 16 : 0), src >= 0 ? 16 : 0);
              }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (pending >= 0) landed(1);
            pending = y;
          }
          // (the next piece's Q waits for this one's last scores, and so for its last K)
          if (pending >= 0) landed(0), pending = -1;
        }
      }
      // no copy may be in flight when the CTA exits (after a wait that gave up, some may
      // never have been waited for)
      if (!TMA && pending >= 0) landed(0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (q_uses[i] > 0) mbar_wait(smem_addr(&sh.q_full[i]), (q_uses[i] - 1) & 1);
      if (TMA)
        for (int y = max(0, x - C::STAGES); y < x; ++y)
          mbar_wait(smem_addr(&sh.kv_full[stage(y)]), (y / C::STAGES) & 1);
    } else if (warp == 9) {
      // ---- products, all of them from one lane
      if (tc5::elect()) {
        constexpr uint32_t kIdS = tc5::idesc_bf16(kRows, kKeys, false);
        constexpr uint32_t kIdO = tc5::idesc_bf16(kRows, D, true);
        int x = 0, tiles[2] = {0, 0}, steps[2] = {0, 0};  // x: blocks of the pieces before
        bool ok = true;
        auto full = [&](int y) { return wait_for(&sh.kv_full[stage(y)], y / C::STAGES); };
        for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
          // Steps of a piece: step k is half k % 2 with block k / 2 where both halves have
          // rows; else both halves have the same rows and take the blocks in turn.
          const int nh = halves(w.tile), n = (w.j1 - w.j0) * nh;
          auto block = [&](int k) { return x + (nh == 2 ? k >> 1 : k); };
          auto scores = [&](int k) {  // S_i = Q_i K^T
            const int i = k & 1, y = 2 * block(k);
            ok = ok && full(y);
            if (!ok) return;
            const uint64_t qd = tc5::desc_sw128(q_sm + (nh == 2 ? i : 0) * C::QTILE, 16, 1024);
            const uint64_t kd = tc5::desc_sw128(kv_sm + stage(y) * C::TILE, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc5::mma_ss(tmem + i * 128, qd + (((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4),
                          kd + (((kk / 4) * (kKeys * 128) + (kk % 4) * 32) >> 4), kIdS, kk > 0);
            tc5::commit(smem_addr(&sh.s_full[i]));
            if (nh == 1 || i == 1) tc5::commit(smem_addr(&sh.kv_empty[stage(y)]));
            if (nh == 2 ? k + 2 >= n : k + 1 == n) tc5::commit(smem_addr(&sh.q_empty[nh == 2 ? i : 0]));
          };
          for (int i = 0; i < nh; ++i) ok = ok && wait_for(&sh.q_full[i], tiles[i]++);
          // (S_i's columns are free: the products with P_i, which lay there, were issued before)
          scores(0);
          if (n > 1) scores(1);
          for (int k = 0; k < n && ok; ++k) {
            const bool fresh = (k >> 1) % kChain == 0;  // the half's sums have been read
            const int i = k & 1, y = 2 * block(k) + 1;
            ok = full(y);
            const uint64_t vd = tc5::desc_sw128(kv_sm + stage(y) * C::TILE, kKeys * 128, 1024);
#pragma unroll
            for (int h = 0; h < kParts; ++h) {  // O_i (+)= P_i V, the parts of P as they come
              ok = ok && wait_for(&sh.p_ready[i][h], steps[i]);
              if (!ok) break;
              tc5::fence_after();
#pragma unroll
              for (int k16 = h * (kKeys / kParts / 16); k16 < (h + 1) * (kKeys / kParts / 16); ++k16)
#pragma unroll
                for (int e = kTerms - 1; e >= 0; --e)  // small terms first
                  tc5::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + term_at(h, e) + (k16 & 1) * 8, vd + k16 * (2048 >> 4), kIdO,
                              !fresh || k16 > 0 || e + 1 < kTerms);
            }
            ++steps[i];
            if (!ok) break;
            if ((k >> 1) % kChain == kChain - 1 || k + 2 >= n) tc5::commit(smem_addr(&sh.o_full[i]));
            if (nh == 1 || i == 1) tc5::commit(smem_addr(&sh.kv_empty[stage(y)]));
            if (k + 2 < n) scores(k + 2);
          }
          x += w.j1 - w.j0;
        }
        // the products in flight end before tensor memory is freed, whether or
        // not a softmax warp still waits for them
        tc5::commit(smem_addr(&sh.drained));
        mbar_wait(smem_addr(&sh.drained), 0);
      }
      __syncwarp();
    }
  } else {
    // ---- softmax, sums and states of half i: one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int i = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // 32 * (warp % 4) in the lane field
    const uint32_t s_tm = tmem + i * 128 + lanes, o_tm = tmem + 256 + i * 128 + lanes;
    const uint32_t p_bar = smem_addr(&sh.p_ready[i][0]);
    const float c = a.own.scale_log2;
    int steps = 0, sums = 0;
    bool ok = true;
    for (Walk w(sh, n_tiles, H_kv, from, to); w.more() && ok; w.next(sh, H_kv)) {
      const int nh = halves(w.tile), every = nh == 2 ? 1 : 2;
      float m = -INFINITY, l = 0.f;
      uint64_t o[D / 2];
#pragma unroll
      for (int x = 0; x < D / 2; ++x) o[x] = 0;
      int k = 0;  // blocks of this half
      for (int j = w.j0 + (nh == 2 ? 0 : i); j < w.j1; j += every, ++k, ++steps) {
        ok = __all_sync(kFull, wait_for(&sh.s_full[i], steps));
        if (!ok) break;
        tc5::fence_after();
        // (32 scores at a time, the first ones again for their exponentials: registers are short)
        const int lim = w.tile.n - j * kKeys;
        uint32_t s[32];
        auto load = [&](int h) {
          tc5::ld32(s_tm + 32 * h, s);
          tc5::wait_ld();
          pin(s);
          if (lim < kKeys) {
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = 32 * h + x < lim ? s[x] : 0xff800000u;
          }
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          load(h);
#pragma unroll
          for (int x = 0; x < 32; x += 2)
            mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        const bool grow = (top - m) * c > kGrow;
        if (__any_sync(kFull, grow)) {
          const float f = grow ? ex2((m - top) * c) : 1.f;
          if (grow) m = top;
          l *= f;
#pragma unroll
          for (int x = 0; x < D / 2; ++x) o[x] = mul2(o[x], pair(f, f));
          if (k % kChain != 0) {
            // (the products of the block before are complete: they were issued before these scores)
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
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          if (h > 0) load(h);
          hand_over(p_bar + 8 * h, [&] {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t p[kTerms][8];
              exp_terms(s + z * 16, cc, mm, sum, p);
#pragma unroll
              for (int e = 0; e < kTerms; ++e) tc5::st8(s_tm + term_at(h, e) + z * 8, p[e]);
            }
          });
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += lo(sum[0]) + hi(sum[0]);
        // the products with V of a few blocks, added here in fp32 (the tensor cores truncate
        // where they add)
        if (k % kChain != kChain - 1 && j + every < w.j1) continue;
        ok = __all_sync(kFull, wait_for(&sh.o_full[i], sums++));
        if (!ok) break;
        tc5::fence_after();
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          uint32_t v[32];
          tc5::ld32(o_tm + 32 * x, v);
          tc5::wait_ld();
          pin(v);
#pragma unroll
          for (int y = 0; y < 16; ++y)
            o[16 * x + y] = add2(o[16 * x + y], pair(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])));
        }
      }
      if (!ok) break;
      // the piece's state (rows side by side, so that the lanes' stores are)
      float* const st = a.states + int64_t(share + w.t * H_kv + w.g) * (kTileRows * (D + 2)) + i * kRows + r;
      if (r < a.tok * G && (nh == 2 ? i : 0) * a.tok + r / G < w.tile.seqs) {
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
// The first `tile_ctas` CTAs take 32 rows of a tile and 32 columns each, a lane a row, a warp 4
// columns: the states of the shared part in the line's order, then those of the
// sequence's own positions.  The others join the pieces of sequences that share nothing.
template <int D>
__global__ void __launch_bounds__(kThreads) shared_join_kernel(const __grid_constant__ SharedArgs a, int grid, int tile_ctas, int ny) {
  constexpr int PER = 4, AHEAD = 8;  // columns of a thread; states read at a time
  __shared__ Line ln;
  const PagedGeo& geo = a.own.geo;
  const int H_kv = geo.H_kv, G = a.own.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float c = a.own.scale_log2;
  pdl_launch();
  pdl_wait();
  const int n_tiles = a.plan->n_tiles;
  const long long total = a.plan->total, items = (long long)n_tiles * H_kv * kJoinBlocks<D>;
  if (int(blockIdx.x) >= tile_ctas ? !a.plan->alone : blockIdx.x >= items) return;
  scan_lengths<kOwnTile>(geo, ln, false);
  const Cut own(ln.pre[geo.B] * H_kv, grid * kPagedWarps, 1);
  if (int(blockIdx.x) >= tile_ctas) {
    const int x = blockIdx.x - tile_ctas, nx = (gridDim.x - tile_ctas) / ny;
    join_units<kOwnTile, D>(a.own, ln, own, true, x % nx, nx, x / nx, ny);
    return;
  }
  const Cut shared(total, grid, 1);
  for (long long y = blockIdx.x; y < items; y += tile_ctas) {
    const int unit = int(y / kJoinBlocks<D>), t = unit / H_kv, g = unit - t * H_kv, at = int(y % (kTileRows / 32)) * 32 + lane;
    const int d = int(y % kJoinBlocks<D>) / (kTileRows / 32) * 32 + warp * PER;
    const SharedTile tile = a.plan->tile[t];
    const long long start = a.plan->start[t];
    const int i = at / kRows, r = at % kRows, tt = r / G, seq = i * a.tok + tt;
    if (tt >= a.tok || seq >= tile.seqs) continue;
    float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    // states from `p` on, `step` floats apart (odd ones another `odd`); columns `col` floats apart
    auto add = [&](const float* p, int64_t step, int odd, int pieces, int64_t col) {
      for (int w0 = 0; w0 < pieces; w0 += AHEAD) {
        float mv[AHEAD], lv[AHEAD], v[AHEAD][PER], top = m;
#pragma unroll
        for (int w = 0; w < AHEAD; ++w) {
          const bool in = w0 + w < pieces;
          const float* const s = odd ? p + ((w0 + w) >> 1) * step + (w & 1) * odd : p + (w0 + w) * step;
          mv[w] = in ? __ldcg(s + D * col) : -INFINITY;
          lv[w] = in ? __ldcg(s + (D + 1) * col) : 0.f;
#pragma unroll
          for (int e = 0; e < PER; ++e) v[w][e] = in ? __ldcg(s + (d + e) * col) : 0.f;
        }
#pragma unroll
        for (int w = 0; w < AHEAD; ++w) top = fmaxf(top, mv[w]);
        const bool none = m == -INFINITY && l == 0.f;
        const float f = none ? 0.f : ex2((m - top) * c);
        l = none ? 0.f : l * f;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = none ? 0.f : o[e] * f;
#pragma unroll
        for (int w = 0; w < AHEAD; ++w) {
          if (mv[w] == -INFINITY && lv[w] == 0.f) continue;  // saw only scores of -infinity, or nothing
          const float fw = ex2((mv[w] - top) * c);
          l = fmaf(fw, lv[w], l);
#pragma unroll
          for (int e = 0; e < PER; ++e) o[e] = fmaf(fw, v[w][e], o[e]);
        }
        m = top;
      }
    };
    const int nb = (tile.n + kKeys - 1) / kKeys;
    const long long begin = start + (long long)g * nb;
    const int first = shared.holder(begin), pieces = shared.holder(begin + nb - 1) - first + 1;
    // (a tile of one half has two states of each row in a piece)
    const bool both = tile.seqs <= a.tok;
    add(a.states + int64_t(first + unit) * (kTileRows * (D + 2)) + at, kTileRows * (D + 2), both ? kRows : 0, both ? 2 * pieces : pieces, kTileRows);
    const int b = tile.b0 + seq, hh = r - tt * G;
    const long long nt = ln.pre[b + 1] - ln.pre[b], b0 = ln.pre[b] * H_kv + g * nt;
    if (nt > 0) {
      const int f2 = own.holder(b0), n2 = own.holder(b0 + nt - 1) - f2 + 1;
      add(a.own.partials + (f2 + int64_t(b) * H_kv + g) * (int64_t(G) * (D + 2)) + hh * (D + 2), int64_t(G) * (D + 2), 0, n2, 1);
    }
    const int64_t row = int64_t(b) * a.own.H_q + g * G + hh;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<float4*>(a.own.out + row * D + d) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    if (d == 0 && a.own.lse) a.own.lse[row] = (m * c + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool TMA>
cudaError_t launch_shared(const SharedArgs& a, bool own_tma, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(shared_attn_kernel<D, TMA>), int(SCfg<D>::SMEM), allowed);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(shared_plan_kernel, dim3(1), kPlan, 0, st, a)) != cudaSuccess) return e;
  if ((e = launch_pdl(shared_attn_kernel<D, TMA>, dim3(grid), kSharedThreads, SCfg<D>::SMEM, st, a)) != cudaSuccess) return e;
  if ((e = launch_paged_pieces(a.own, D, own_tma, grid, st)) != cudaSuccess) return e;
  const int units = a.own.geo.B * a.own.geo.H_kv, most = 4 * grid, y = a.own.G * (D / 32);
  const int nx = units < most ? units : most, ny = units >= most ? 1 : most / units < y ? most / units : y;
  const long long blocks = (long long)a.max_tiles * a.own.geo.H_kv * kJoinBlocks<D>;
  const int tile_ctas = int(blocks < 2 * most ? blocks : 2 * most);
  return launch_pdl(shared_join_kernel<D>, dim3(tile_ctas + nx * ny), kThreads, 0, st, a, grid, tile_ctas, ny);
}

}  // namespace

cudaError_t launch_shared_attn(const SharedArgs& a, int D, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64) return a.box ? launch_shared<64, true>(a, use_tma, grid, st) : launch_shared<64, false>(a, use_tma, grid, st);
  return a.box ? launch_shared<128, true>(a, use_tma, grid, st) : launch_shared<128, false>(a, use_tma, grid, st);
}

}  // namespace sfi

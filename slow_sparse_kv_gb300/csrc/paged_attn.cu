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
// SOLO (the own positions behind a shared prefix, few for each sequence): the line is cut into
// a share for each warp, whose state is a piece by itself, so that nothing is merged in
// the CTA; shared.cu joins the pieces (64 sequences of 16 to 1024 positions: 17 us, 43 before).
// fp32: CUDA cores, d spread over the lanes, dots by transpose-reduction, products and
// sums in pairs (f32x2; without: 4 x 32768, 16 heads a group 379 us against 349, 8 heads 194
// against 180, d = 64 with 4 heads, 8 x 32768, 176 against 170; 4 heads of 128, which
// HBM bounds, 161 against 165).
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "paged_line.cuh"
#include "pdl.cuh"

namespace sfi {
namespace {

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

// Four fp32 values of shared memory as two pairs.
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(addr));
}

// What the warps of a CTA share besides the ring.
struct Shared {
  Line ln;
  uint64_t full[48], empty[48];                           // of each slot of the ring
  volatile int abort;
  uint64_t merge_free;                                    // the warps' states have been read
};

// A run of tiles.
struct Run {
  long long from, to;
};

// The run of attending warp w, where each warp has a share of its own (neighbouring shares
// lie in neighbouring CTAs, so that a few tiles are spread over the SMs).
__device__ __forceinline__ Run warp_run(const Cut& cut, int w) {
  const int share = w * gridDim.x + blockIdx.x;
  return share < cut.shares ? Run{cut.start(share), cut.start(share + 1)} : Run{0, 0};
}

// The copying warps: warp `p` takes the tiles of the attending warps p and p + 4: every
// fourth one of the CTA's share [from, to), or with SOLO those of the two warps' own shares
// in turn.
template <typename T, int D, int NT, Load LD, bool SOLO>
__device__ __forceinline__ void copy_tiles(const PagedAttnArgs& a, Shared& sh, const Cut& cut, long long from, long long to,
                                           uint32_t ring, int p) {
  using C = Cfg<T, D, NT>;
  constexpr int TR = C::TR;
  const PagedGeo& geo = a.geo;
  const int lane = threadIdx.x & 31, P = geo.P, H_kv = geo.H_kv, cap = geo.max_pages * P;
  const T* const kp = static_cast<const T*>(a.k);
  const T* const vp = static_cast<const T*>(a.v);
  bool ok = true;
  const long long first[2] = {first_of(from, p, kWarps), first_of(from, p + kProducers, kWarps)};
  Run runs[2] = {{0, 0}, {0, 0}};
  if (SOLO) {
    runs[0] = warp_run(cut, p), runs[1] = warp_run(cut, p + kProducers);
    to = 2 * max(runs[0].to - runs[0].from, runs[1].to - runs[1].from);
  }
  constexpr int STEP = SOLO ? 1 : kProducers;
  for (long long x0 = SOLO ? 0 : first_of(from, p, kProducers); x0 < to && ok; x0 += STEP * 32) {
    // 32 tiles: each lane finds the place and the page of its own
    const long long x = SOLO ? runs[lane & 1].from + ((x0 + lane) >> 1) : x0 + kProducers * lane;
    const bool mine = SOLO ? x < runs[lane & 1].to : x < to;
    Unit u{0, 0, 0, 0};
    int t = 0, n = 0;
    int page[LD == kBulk ? TR : 1];
    if (mine) {
      u = unit_at(x, sh.ln, geo.B, H_kv);
      t = int(x - u.begin);
      n = min(geo.len[u.b], cap) - skipped<SOLO>(geo, u.b) * P;
    }
    const int32_t* const row = geo.table + int64_t(u.b) * geo.max_pages + skipped<SOLO>(geo, u.b);
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
    const int count = int(min(32LL, (to - x0 + STEP - 1) / STEP));
    // kCpAsync: the i-th tile's row of this lane (lane % TR): its page, and where in it,
    // -1 for no row.  A tile's pages are read while the one before it is copied (waited
    // for before each tile: 136 us against 129 for 8 x ~24000 positions in pages of 20).
    int pg = 0, in = -1;
    auto row_of = [&](int i) {
      const int ut = __shfl_sync(kFull, t, i), ug = __shfl_sync(kFull, u.g, i), un = __shfl_sync(kFull, n, i);
      const int ub = __shfl_sync(kFull, u.b, i);
      const int32_t* const urow = geo.table + int64_t(ub) * geo.max_pages + skipped<SOLO>(geo, ub);
      const int pos = ut * TR + lane % TR;
      pg = pos < un ? urow[pos / P] : 0;
      in = pos < un ? ug * P + pos % P : -1;
    };
    if (LD == kCpAsync) row_of(0);
    for (int i = 0; i < count && ok; ++i) {
      const long long xi = x0 + STEP * i;
      const int w = SOLO ? int(xi) & 1 : int(xi >> 2) & 1;  // which of the two warps
      const uint32_t y = SOLO ? uint32_t(xi >> 1) : uint32_t(xi - first[w]) / kWarps;
      if (SOLO && !__shfl_sync(kFull, mine, i)) {
        if (LD == kCpAsync && i + 1 < count) row_of(i + 1);
        continue;
      }
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

template <typename T, int D, int NT, Load LD, bool SOLO>
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
  scan_lengths<TR, SOLO>(geo, sh.ln, blockIdx.x == 0);
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
  const Cut cut = SOLO ? Cut(total, gridDim.x * kWarps, 1) : Cut(total, gridDim.x);
  const int share = blockIdx.x;
  const long long from = share < cut.shares ? cut.start(share) : total;
  const long long to = share < cut.shares ? cut.start(share + 1) : total;

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    copy_tiles<T, D, NT, LD, SOLO>(a, sh, cut, from, to, ring, warp - kWarps);
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
      return min(geo.len[u.b], cap) - skipped<SOLO>(geo, u.b) * geo.P;
    };
    const Run run = SOLO ? warp_run(cut, warp) : Run{from, to};
    constexpr int STEP = SOLO ? 1 : kWarps;
    if (run.from < run.to) {
      long long x = SOLO ? run.from : first_of(run.from, warp, kWarps);  // this warp's next tile
      Unit u = unit_at(run.from, ln, B, H_kv);
      int n = load_unit(u);
      while (true) {
        const long long pe = min(u.end, run.to);
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

        for (; x < pe; x += STEP) {
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
        while (next.begin < run.to && next.end == next.begin);
        const bool more = next.begin < run.to;
        if (more) n = load_unit(next);

        if constexpr (SOLO && !F32) {
          // the warp's state is a piece by itself
          float* const slot = a.partials + (warp * int(gridDim.x) + share + b * H_kv + g) * int64_t(G) * (D + 2);
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = l[h][e];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(kFull, t, w);
              const int head = h * 8 + 2 * (lane & 3) + e;
              if (head >= G) continue;
              float* const row = slot + head * (D + 2);
              if (lane < 4) row[D] = m[h][e], row[D + 1] = t;
#pragma unroll
              for (int kk = 0; kk < KS; ++kk) {
                row[kk * 16 + (lane >> 2)] = o[kk][h][e];
                row[kk * 16 + 8 + (lane >> 2)] = o[kk][h][2 + e];
              }
            }
          if (!more) break;
          u = next;
          continue;
        }
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

template <typename T, int D, int NT, Load LD, bool SOLO>
cudaError_t launch_t(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<T, D, NT>;
  auto* const kernel = paged_attn_kernel<T, D, NT, LD, SOLO>;
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, allowed);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kernel, dim3(grid), kAllThreads, C::SMEM, st, a);
  if (e2 != cudaSuccess || SOLO) return e2;
  return launch_join<C::TR, D>(a, grid, st);
}

template <int D, int NT>
cudaError_t launch_n(const PagedAttnArgs& a, bool f32, bool use_tma, int grid, cudaStream_t st) {
  if (f32) return launch_t<float, D, NT, kBulk, false>(a, grid, st);
  return use_tma ? launch_t<bf16_t, D, NT, kTma, false>(a, grid, st) : launch_t<bf16_t, D, NT, kCpAsync, false>(a, grid, st);
}

template <int D, int NT>
cudaError_t launch_solo(const PagedAttnArgs& a, bool use_tma, int grid, cudaStream_t st) {
  return use_tma ? launch_t<bf16_t, D, NT, kTma, true>(a, grid, st) : launch_t<bf16_t, D, NT, kCpAsync, true>(a, grid, st);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int D, bool f32, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64) return a.G <= 8 ? launch_n<64, 1>(a, f32, use_tma, grid, st) : launch_n<64, 2>(a, f32, use_tma, grid, st);
  return a.G <= 8 ? launch_n<128, 1>(a, f32, use_tma, grid, st) : launch_n<128, 2>(a, f32, use_tma, grid, st);
}

cudaError_t launch_paged_pieces(const PagedAttnArgs& a, int D, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64) return a.G <= 8 ? launch_solo<64, 1>(a, use_tma, grid, st) : launch_solo<64, 2>(a, use_tma, grid, st);
  return a.G <= 8 ? launch_solo<128, 1>(a, use_tma, grid, st) : launch_solo<128, 2>(a, use_tma, grid, st);
}

}  // namespace sfi

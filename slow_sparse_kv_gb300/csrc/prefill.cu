// Causal attention over packed prompts (bf16, grouped heads) on the
// fifth-generation tensor cores.
//
// One CTA to an SM takes tile after tile: 2 x 128 query rows of one (sequence,
// KV head); a row is one (token, query head of the group), so a tile holds
// 128 / G tokens times the G heads that share the KV head, and K and V are read
// once for all of them.  The tiles come from a shared counter, the long ones
// first; loads run ahead into the next tile, so that its first products start
// while the last one's output is written.
// For each block of 128 keys: S = Q K^T (tcgen05.mma from shared memory into
// tensor memory), softmax statistics with one thread per row, P in bf16 over
// S's columns in tensor memory, O += P V (P from tensor memory).  The two
// tiles alternate: while one's softmax runs, the tensor cores work on the
// other's products.  Tensor memory: S0/P0, S1/P1, O0, O1 (4 x 128 columns).
//
// With d = 128 bound by the tensor cores (4 d flops per row and visible key; active for
// 75% of the cycles of a launch over 8192 tokens).  With d = 64 by the serial chain of a
// half: scores, row maximum, exponentials, P over the scores' columns, its last products,
// and only then the next scores.  A pair of blocks takes 1.33 us, nearly the 1.4 of
// d = 128, though its products halved; tensor pipe, exponentials and issue slots are
// active for 41, 41 and 50% of the cycles (6 x 4096 tokens, 32 / 8 heads).
// Measured, 32 / 8 heads of 128: 16384 tokens in 1.32 to 1.36 ms (1.62 to 1.66 PFLOP/s; a
// library's matrix product reaches 1.88), 3 chunks of ~900 tokens after ~10000 in 309 us
// (1.46), 16 prompts of 260 to 4000 tokens in 310 us (1.31); with d = 64, 0.73 to 0.77
// (8192 tokens, 16 / 4 heads) and 0.98 (6 x 4096, 32 / 8).  A tile's start and output
// take another 2 us.  (A warpgroup of its own for the output was tried: 176 registers
// for the softmax threads instead of 216, and a tile's products wait for the output of
// both halves of the last one, 239 us against 223 for set B and no gain for long ones.)
// Set B, here and below, on which the steps were compared: 16 other prompts, of 85 to
// 3521 tokens, 17592 in all, 32 / 8 heads of 128, calls back to back with nothing
// flushed between; 216 us now.
//
// Online softmax: out = sum_j 2^(c (s_j - m)) v_j / sum_j 2^(c (s_j - m)) with
// c = log2(e) / sqrt(d) holds for any m, so m only follows the row maximum when
// that has grown by more than 8 in the exponent (P then stays below 2^8, fp32
// sums far from overflow, bf16's relative rounding the same); O is rescaled in
// tensor memory only then.
#include <cuda_runtime.h>

#include <atomic>

#include "f32x2.cuh"
#include "pdl.cuh"
#include "prefill.h"
#include "tc5.cuh"
#include "tc5_attn.cuh"

namespace sfi {
namespace {

constexpr int kThreads = 384;  // 2 softmax warpgroups; a load, an MMA, a scheduling and a cleaning warp
constexpr int kRows = 128;     // query rows per tile
constexpr int kKeys = 128;     // keys per block
// P of a block is handed over in parts, the first 64 keys, then twice 32: the
// products start early and the scores behind them wait for a short last part.  (Set B:
// 218 us; in halves 224, 96 and 32 keys 226, whole 231.)
constexpr int kParts = 3;
__host__ __device__ constexpr int part_end(int part) { return part == 0 ? 64 : part == 1 ? 96 : kKeys; }
constexpr float kGrow = 8.0f;  // growth of the maximum (log2) that moves m

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t TILE = kRows * 128 * HALVES;  // bytes of a 128-row tile
  static constexpr int STAGES = D == 128 ? 4 : 6;         // K and V blocks in flight
  static constexpr uint32_t OUT = 8 * 32 * 128;           // 32 rows of 64 outputs for each softmax warp
  static constexpr uint32_t SMEM = 1024 + (2 + STAGES) * TILE + OUT;
  // Registers a thread: launched with 168; the softmax threads hold a whole row of
  // scores, the third warpgroup gives up what they take.  (d = 128: 208 and 88
  // against 216 and 72, set B 220 against 224 us; d = 64: 186 against
  // 180, 8192 tokens; with 200 the row spills, 233 us.)
  static constexpr int SOFTMAX_REGS = D == 128 ? 208 : 216, OTHER_REGS = 504 - 2 * SOFTMAX_REGS;
};

using Tile = PrefillTile;

constexpr int kTileReaders = 11;  // loads, MMAs, the cleaning warp, 8 softmax warps

struct Shared {
  uint64_t q_full[2], q_empty[2], s_full[2], o_full[2], p_ready[2][kParts], tile_full[2], tile_empty[2];
  uint64_t kv_full[6], kv_empty[6], drained;
  // The cleaned last V blocks, one barrier after the other: the cleaning warp may be
  // done with two tiles of which the MMA lane has waited for neither (a short one
  // behind another, both in the ring), and a barrier two phases ahead looks like one
  // that is still to come.  More than two it cannot be ahead: a tile is handed out when
  // the one two before it has been given back by the softmax warps, behind its output
  // and so behind the products with its last V block.
  uint64_t v_clean[2];
  Tile tile[2];
  uint32_t tmem;
  volatile int abort;
};

__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// Part H of a block's probabilities: p = 2^(c s - c m) summed in fp32 (four
// pairs of sums) and rounded to bf16 pairs in s's first half.
template <int H>
__device__ __forceinline__ void exp_part(uint32_t (&s)[kKeys], uint64_t cc, uint64_t mm, uint64_t (&sum)[4]) {
#pragma unroll
  for (int x = H ? part_end(H - 1) / 2 : 0; x < part_end(H) / 2; ++x) {
    const uint64_t y = fma2(pair(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), cc, mm);
    const float p0 = ex2(lo(y)), p1 = ex2(hi(y));
    sum[x & 3] = add2(sum[x & 3], pair(p0, p1));
    s[x] = pack_bf16x2(p0, p1);
  }
}

// Which tile has which rank (one warp).  Levels stand for the keys that a tile
// sees, in units of its tokens: sequence b has its tiles at levels lvl[b] ..
// lvl[b] + span[b] - 1.  Ranks go from the highest level down, so that the long
// tiles start first; within a level by sequence, and the KV heads of a tile are
// neighbours.  A CTA asks for growing ranks, so the walk goes on from where it
// stood.
struct Seq {
  int q0, nq, k0, nk;  // first row and rows, of q and of k
};
struct Ranks {
  const PrefillArgs& a;
  // (up to 32 sequences stay in registers, a lane each: reading them back from
  // memory for every step of the search took 10 to 15 us at a kernel's start, and for
  // a tile's offsets another 0.4)
  Seq one = {0, 0, 0, 0};
  int span1 = 0, lvl1 = 0;
  bool bad = false;  // this lane's offsets are out of order
  int level, before, here;  // the level it stands at, tiles above it and on it

  // Stands above the highest level.
  __device__ __forceinline__ explicit Ranks(const PrefillArgs& a_) : a(a_) {
    const int lane = threadIdx.x & 31;
    if (a.B <= 32 && lane < a.B) bad = !sequence(a, lane, &one, &span1, &lvl1);
    int t = 0;
    each([&](int, int span, int lvl) { t = max(t, span > 0 ? lvl + span : 0); });
    level = __reduce_max_sync(kFull, t);
    before = here = 0;
  }
  // rows, CTA tiles and first level of sequence b; false if its offsets are out of order
  static __device__ __forceinline__ bool sequence(const PrefillArgs& a, int b, Seq* s, int* span, int* lvl) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1], tokens = 2 * a.tok;
    const bool ok = q0 >= 0 && q0 <= q1 && q1 <= a.total_q && k0 >= 0 && k0 <= k1 && k1 <= a.total_k;
    *s = Seq{q0, q1 - q0, k0, k1 - k0};
    *span = ok ? (q1 - q0 + tokens - 1) / tokens : 0;
    *lvl = ok ? max(0, (k1 - k0) - (q1 - q0)) / tokens : 0;
    return ok;
  }
  // the rows of sequence b, one that is in order
  __device__ __forceinline__ Seq rows_of(int b) const {
    if (a.B <= 32)
      return Seq{__shfl_sync(kFull, one.q0, b), __shfl_sync(kFull, one.nq, b), __shfl_sync(kFull, one.k0, b),
                 __shfl_sync(kFull, one.nk, b)};
    return Seq{a.cu_q[b], a.cu_q[b + 1] - a.cu_q[b], a.cu_k[b], a.cu_k[b + 1] - a.cu_k[b]};
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31;
    if (a.B <= 32) f(lane, span1, lvl1);
    else
      for (int b = lane; b < a.B; b += 32) f(b, a.span[b], a.lvl[b]);
  }
  // tiles on levels tau and above
  __device__ __forceinline__ int from(int tau) const {
    int n = 0;
    each([&](int, int span, int lvl) { n += min(max(lvl + span - tau, 0), span); });
    return __reduce_add_sync(kFull, n);
  }
  // sequence and tile of a rank below from(0), for growing ranks
  __device__ __forceinline__ void find(int rank, int* seq, int* tile) {
    const int lane = threadIdx.x & 31;
    if (rank >= before + here) {
      // the level with from(level + 1) <= rank < from(level), below this one
      int lo = 0, hi = level;
      if (level > 0 && from(level - 1) > rank) lo = level - 1;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from(mid) > rank) lo = mid;
        else hi = mid;
      }
      level = lo;
      before = from(lo + 1);
      here = from(lo) - before;
    }
    int left = rank - before;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int span = a.B <= 32 ? span1 : b < a.B ? a.span[b] : 0, lvl = a.B <= 32 ? lvl1 : b < a.B ? a.lvl[b] : 0;
      const uint32_t in = __ballot_sync(kFull, lvl <= level && level < lvl + span);
      if (left < __popc(in)) {
        // the lane with `left` set bits below its own
        const bool me = (in >> lane & 1) && __popc(in & ((1u << lane) - 1)) == left;
        const int at = __ffs(__ballot_sync(kFull, me)) - 1;
        *seq = b0 + at;
        *tile = level - __shfl_sync(kFull, lvl, at);
        return;
      }
      left -= __popc(in);
    }
  }
};

__device__ __forceinline__ Tile make_tile(const PrefillArgs& a, int g, const Seq& seq, int tile) {
  Tile t;
  const int span = 2 * a.tok, first = tile * span, nq = seq.nq;
  t.g = g;
  t.k0 = seq.k0;
  t.nk = seq.nk;
  t.slot = -1;
  t.q0 = seq.q0 + first;
  t.rows = min(span, nq - first);
  t.seen = t.nk - nq + first + 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tokens = min(t.rows, (i + 1) * a.tok);  // the half's last one sees seen + tokens - 1
    t.n[i] = t.rows > i * a.tok ? (max(0, min(t.seen + tokens - 1, t.nk)) + kKeys - 1) / kKeys : 0;
  }
  return t;
}

// Which tiles are cut along their keys.  A few waves of tiles of about the same
// length (the next chunks of long prompts, say) leave most SMs idle in the last
// one: its tiles, the last `tiles` ranks, are then cut into `parts` of at least 4
// key blocks, so that all SMs get one.  (A whole prompt's last tiles are its short
// ones and fill the gaps as they are.)
struct Split {
  long long total;  // tiles, -1: too many for ranks of 31 bits
  long long first;  // ranks from here on are cut
  int tiles, parts;
};

__device__ __forceinline__ Split split_of(const PrefillArgs& a, Ranks r, int grid) {  // one warp
  Split s;
  // (offsets that descend between two sequences let both hold the same rows, and so have
  // more tiles than the call has reckoned with by its rows; 2^32, which this sum could
  // not show, would take 270 GB of queries)
  const int tiles = r.from(0);
  s.total = s.first = (long long)tiles * a.H_kv;
  s.tiles = 0;
  s.parts = 1;
  if (tiles < 0 || s.total > 0x7fffffffLL) {
    s.total = -1;
    s.first = 0;
    return s;
  }
  if (a.partials == nullptr || s.total == 0 || s.total >= kSplitWaves * grid) return s;
  // (below 2^31: kSplitWaves * grid)
  const int rest = int(uint32_t(s.total) % uint32_t(grid));
  if (rest == 0) return s;
  int seq = 0, tile = 0;
  r.find(0, &seq, &tile);
  const Tile longest = make_tile(a, 0, r.rows_of(seq), tile);
  r.find(int(uint32_t(s.total - 1) / uint32_t(a.H_kv)), &seq, &tile);
  const Tile shortest = make_tile(a, 0, r.rows_of(seq), tile);
  const int most = max(longest.n[0], longest.n[1]), least = max(shortest.n[0], shortest.n[1]);
  if (s.total > grid && 2 * least < most) return s;
  const int parts = min(min(kMaxParts, grid / rest), (s.total > grid ? least : most) / 4);
  if (parts < 2) return s;
  s.tiles = rest;
  s.first = s.total - rest;
  s.parts = parts;
  return s;
}

// The part of a tile as a tile of its own, whose keys begin with the part's.
__device__ __forceinline__ void take_part(Tile& t, int part, int parts, int slot) {
  const int n = max(t.n[0], t.n[1]), j0 = int((long long)n * part / parts), j1 = int((long long)n * (part + 1) / parts);
#pragma unroll
  for (int i = 0; i < 2; ++i) t.n[i] = max(0, min(t.n[i], j1) - j0);
  t.k0 += j0 * kKeys;
  t.nk -= j0 * kKeys;
  t.seen -= j0 * kKeys;
  t.slot = slot;
}

// The state of a tile pair's 256 rows: o as [D][256], then m and l.
template <int D>
__device__ __forceinline__ float* slot_of(const PrefillArgs& a, int slot) {
  return a.partials + int64_t(slot) * (2 * kRows * (D + 2));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 9) {
    if (lane == 0) {
      sh.abort = 0;
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_addr(&sh.q_full[i]), 1);
        mbar_init(smem_addr(&sh.q_empty[i]), 1);
        mbar_init(smem_addr(&sh.s_full[i]), 1);
        mbar_init(smem_addr(&sh.o_full[i]), 1);
        for (int h = 0; h < kParts; ++h) mbar_init(smem_addr(&sh.p_ready[i][h]), 128);
        mbar_init(smem_addr(&sh.tile_full[i]), 1);
        mbar_init(smem_addr(&sh.tile_empty[i]), kTileReaders);
      }
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(smem_addr(&sh.kv_full[i]), 1);
        mbar_init(smem_addr(&sh.kv_empty[i]), 2);  // its last product, and the cleaning warp
      }
      for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&sh.v_clean[i]), 1);
      mbar_init(smem_addr(&sh.drained), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tc5::alloc(smem_addr(&sh.tmem), 512);
    tc5::fence_before();
  }
  pdl_launch();
  pdl_wait();
  if (a.B > 32)
    for (int b = tid; b < a.B; b += kThreads) {
      Seq seq;
      int span, lvl;
      const bool ok = Ranks::sequence(a, b, &seq, &span, &lvl);
      if (!ok && blockIdx.x == 0) set_status(a.status, SFI_DEV_LEN_OVER_CAP);
      // (every CTA writes the same values and reads its own)
      a.span[b] = span, a.lvl[b] = lvl;
    }
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t q_sm = base, kv_sm = base + 2 * C::TILE;
  auto stage = [&](int x) { return x % C::STAGES; };
  auto wait_for = [&](uint64_t* bar, int use) {
    return wait(smem_addr(bar), use & 1, sh, a.status, a.wait_cycles);
  };
  // The k-th tile of this CTA, once it is there; one without rows ends the walk.
  auto take = [&](int k, Tile& t) {
    if (!wait_for(&sh.tile_full[k & 1], k >> 1)) return false;
    t = sh.tile[k & 1];
    return true;
  };
  auto taken = [&](int k) { mbar_arrive(smem_addr(&sh.tile_empty[k & 1])); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 8 && lane == 0) {
      // ---- loads: each tile's Q, then K_0, V_0, K_1, V_1, ... through the ring
      int x = 0, q_uses[2] = {0, 0};
      bool ok = true;
      Tile t;
      for (int k = 0; ok && take(k, t); ++k) {
        taken(k);
        if (t.rows == 0) break;
        const int n = max(t.n[0], t.n[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || t.n[i] == 0) continue;
          if (q_uses[i] > 0) ok = wait_for(&sh.q_empty[i], q_uses[i] - 1);
          if (!ok) continue;
          const uint32_t bar = smem_addr(&sh.q_full[i]);
          mbar_arrive_expect_tx(bar, uint32_t(a.tok * a.G) * 128 * C::HALVES);
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(q_sm + i * C::TILE + h * (kRows * 128), &a.tmq, h * 64, t.g * a.G, t.q0 + i * a.tok, bar);
          ++q_uses[i];
        }
        for (int y = 0; y < 2 * n && ok; ++y) {
          if (x >= C::STAGES) ok = wait_for(&sh.kv_empty[stage(x)], x / C::STAGES - 1);
          if (!ok) break;
          const uint32_t bar = smem_addr(&sh.kv_full[stage(x)]);
          mbar_arrive_expect_tx(bar, C::TILE);
          const void* map = (y & 1) ? &a.tmv : &a.tmk;
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(kv_sm + stage(x) * C::TILE + h * (kKeys * 128), map, h * 64, t.g, t.k0 + (y >> 1) * kKeys, bar);
          ++x;
        }
      }
      // no copy may be in flight when the CTA exits (after a wait that gave
      // up, some may never have been waited for)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (q_uses[i] > 0) mbar_wait(smem_addr(&sh.q_full[i]), (q_uses[i] - 1) & 1);
      for (int y = max(0, x - C::STAGES); y < x; ++y)
        mbar_wait(smem_addr(&sh.kv_full[stage(y)]), (y / C::STAGES) & 1);
    } else if (warp == 9) {
      // ---- products, all of them from one lane: a warp-wide vote or
      // __syncwarp between MMAs costs more than their issue
      if (tc5::elect()) {
        constexpr uint32_t kIdS = tc5::idesc_bf16(kRows, kKeys, false);
        constexpr uint32_t kIdO = tc5::idesc_bf16(kRows, D, true);
        int x = 0, tiles[2] = {0, 0}, blocks[2] = {0, 0}, cleaned = 0;
        auto full = [&](int y) { return wait_for(&sh.kv_full[stage(y)], y / C::STAGES); };
        auto scores = [&](int i, int y, bool last) {  // S_i = Q_i K^T
          const uint64_t qd = tc5::desc_sw128(q_sm + i * C::TILE, 16, 1024);
          const uint64_t kd = tc5::desc_sw128(kv_sm + stage(y) * C::TILE, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = ((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4;
            tc5::mma_ss(tmem + i * 128, qd + at, kd + at, kIdS, kk > 0);
          }
          tc5::commit(smem_addr(&sh.s_full[i]));
          if (last) tc5::commit(smem_addr(&sh.q_empty[i]));
        };
        bool ok = true;
        Tile t;
        for (int k = 0; ok && take(k, t); ++k) {
          taken(k);
          if (t.rows == 0) break;
          const int n = max(t.n[0], t.n[1]);
          if (n == 0) continue;
          ok = full(x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || t.n[i] == 0) continue;
            ok = wait_for(&sh.q_full[i], tiles[i]++);
            // (S_i's columns are free: the last tile's products with P_i, which
            // lay there, were issued before)
            if (!ok) continue;
            scores(i, x, t.n[i] == 1);
            if (i == 1 || t.n[1] == 0) tc5::commit(smem_addr(&sh.kv_empty[stage(x)]));
          }
          auto v_landed = [&](int j, int y) {
            if ((j + 1) * kKeys <= t.nk) return full(y);
            const int c = cleaned++;
            return wait_for(&sh.v_clean[c & 1], c >> 1);
          };
          for (int j = 0; j < n && ok; ++j, x += 2) {
            ok = v_landed(j, x + 1);
            const uint64_t vd = tc5::desc_sw128(kv_sm + stage(x + 1) * C::TILE, kKeys * 128, 1024);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= t.n[i]) continue;
              const bool last = i == 1 || j >= t.n[1];  // of the halves that use V_j
#pragma unroll
              for (int h = 0; h < kParts; ++h) {  // O_i += P_i V, the parts of P as they come
                ok = ok && wait_for(&sh.p_ready[i][h], blocks[i]);
                if (!ok) break;
                tc5::fence_after();
#pragma unroll
                for (int k16 = h ? part_end(h - 1) / 16 : 0; k16 < part_end(h) / 16; ++k16)
                  tc5::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k16 * 8, vd + k16 * (2048 >> 4), kIdO,
                              j > 0 || k16 > 0);
              }
              ++blocks[i];
              if (!ok) continue;
              if (last) tc5::commit(smem_addr(&sh.kv_empty[stage(x + 1)]));
              if (j + 1 < t.n[i]) {
                ok = full(x + 2);
                if (!ok) continue;
                scores(i, x + 2, j + 2 == t.n[i]);
                if (i == 1 || j + 1 >= t.n[1]) tc5::commit(smem_addr(&sh.kv_empty[stage(x + 2)]));
              } else {
                tc5::commit(smem_addr(&sh.o_full[i]));
              }
            }
          }
        }
        // the products in flight end before tensor memory is freed, whether or
        // not a softmax warp still waits for them
        tc5::commit(smem_addr(&sh.drained));
        mbar_wait(smem_addr(&sh.drained), 0);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---- which tiles: the CTA's own index first, then by a shared counter
      long long rank = blockIdx.x;
      Ranks ranks(a);
      const Split split = split_of(a, ranks, gridDim.x);
      if (blockIdx.x == 0 && lane == 0 && a.partials != nullptr) a.cut_count[0] = split.tiles, a.cut_count[1] = split.parts;
      if (blockIdx.x == 0 && (ranks.bad || split.total < 0)) set_status(a.status, SFI_DEV_LEN_OVER_CAP);
      for (int k = 0;; ++k) {
        Tile t;
        t.rows = 0;
        if (rank < split.first + (long long)split.tiles * split.parts) {
          // (the parts of a tile have neighbouring ranks)
          const int cut = rank < split.first ? 0 : int(rank - split.first);
          const int whole = int(rank < split.first ? rank : split.first + cut / split.parts);
          int seq = 0, tile = 0;
          ranks.find(whole / a.H_kv, &seq, &tile);
          t = make_tile(a, whole % a.H_kv, ranks.rows_of(seq), tile);
          if (rank >= split.first) {
            if (lane == 0 && cut % split.parts == 0) a.cuts[cut / split.parts] = t;
            take_part(t, cut % split.parts, split.parts, cut);
          }
        }
        if (k > 1 && !__all_sync(kFull, wait_for(&sh.tile_empty[k & 1], (k >> 1) - 1))) break;
        if (lane == 0) {
          sh.tile[k & 1] = t;
          mbar_arrive(smem_addr(&sh.tile_full[k & 1]));  // (release: the tile is visible to who waits)
        }
        __syncwarp();
        if (t.rows == 0) break;
        if (lane == 0) rank = gridDim.x + (long long)atomicAdd(a.next, 1u);
        rank = __shfl_sync(kFull, rank, 0);
      }
      // the last CTA to run out leaves the counters at zero
      if (lane == 0 && atomicAdd(a.next + 1, 1u) == gridDim.x - 1) {
        a.next[0] = 0;
        a.next[1] = 0;
      }
    } else if (warp == 11) {
      // ---- the rows of a sequence's last V block that lie behind it belong to
      // nobody or to the next one: P is zero there, but 0 * NaN is not
      int x = 0, cleaned = 0;
      bool ok = true;
      Tile t;
      for (int k = 0; ok && __all_sync(kFull, take(k, t)); ++k) {
        __syncwarp();
        if (lane == 0) taken(k);
        if (t.rows == 0) break;
        const int n = max(t.n[0], t.n[1]);
        for (int y = 0; y < 2 * n && ok; ++y, ++x) {
          ok = __all_sync(kFull, wait_for(&sh.kv_full[stage(x)], x / C::STAGES));
          if (!ok) break;
          if (y == 2 * n - 1 && n * kKeys > t.nk) {
            const uint32_t v_sm = kv_sm + stage(x) * C::TILE;
            for (int z = (t.nk - (n - 1) * kKeys) * 8 + lane; z < kKeys * 8; z += 32)
              for (int h = 0; h < C::HALVES; ++h)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_sm + h * (kKeys * 128) + z * 16), "r"(0)
                             : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.v_clean[cleaned & 1]));
            ++cleaned;
          }
          if (lane == 0) mbar_arrive(smem_addr(&sh.kv_empty[stage(x)]));
        }
      }
    }
  } else {
    // ---- softmax and output of tile half i: one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int i = warp >> 2;
    const int r = tid & 127;
    const int tt = r / a.G;                           // token of the tile
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // 32 * (warp % 4) in the lane field
    const uint32_t s_tm = tmem + i * 128 + lanes, o_tm = tmem + 256 + i * 128 + lanes;
    const uint32_t p_bar = smem_addr(&sh.p_ready[i][0]);
    const float c = a.scale_log2;
    const uint32_t out_sm = base + (2 + C::STAGES) * C::TILE + warp * (32 * 128);
    int blocks = 0, tiles = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!__all_sync(kFull, wait_for(&sh.tile_full[k & 1], k >> 1))) break;
      const Tile& t = sh.tile[k & 1];  // (given back behind the output: registers are short here)
      if (t.rows == 0) break;
      const int n_it = t.n[i];
      const int row = i * a.tok + tt;  // of the tile pair's tokens
      const bool valid = tt < a.tok && row < t.rows;
      const int limit = valid ? max(0, min(t.seen + row, t.nk)) : 0;  // keys this row sees
      const int open = max(0, min(t.seen + i * a.tok, t.nk));         // keys every valid row sees
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n_it; ++j) {
        ok = __all_sync(kFull, wait_for(&sh.s_full[i], blocks++));
        if (!ok) break;
        tc5::fence_after();
        uint32_t s[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tc5::ld32(s_tm + 32 * x, s + 32 * x);
        tc5::wait_ld();
        pin(s);
        if ((j + 1) * kKeys > open) {
          const int lim = limit - j * kKeys;
#pragma unroll
          for (int x = 0; x < 128; ++x) s[x] = x < lim ? s[x] : 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 128; x += 2)
          mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        if (j == 0) {
          m = top;
        } else {
          const bool grow = (top - m) * c > kGrow;
          if (__any_sync(kFull, grow)) {
            // PV of block j - 1 is complete: it was issued before these scores
            // (16 columns at a time: the scores of the block are in registers)
            const float f = grow ? ex2((m - top) * c) : 1.f;
            if (grow) m = top;
            l *= f;
#pragma unroll 1
            for (int x = 0; x < D / 16; ++x) {
              uint32_t o[16];
              tc5::ld16(o_tm + 16 * x, o);
              tc5::wait_ld();
              pin(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc5::st16(o_tm + 16 * x, o);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : -m * c;
        const uint64_t cc = pair(c, c), mm = pair(mc, mc);
        uint64_t sum[4] = {0, 0, 0, 0};
        exp_part<0>(s, cc, mm, sum);
        hand_over(p_bar, [&] { tc5::st32(s_tm, s); });
        exp_part<1>(s, cc, mm, sum);
        hand_over(p_bar + 8, [&] { tc5::st16(s_tm + 32, s + 32); });
        exp_part<2>(s, cc, mm, sum);
        hand_over(p_bar + 16, [&] { tc5::st16(s_tm + 48, s + 48); });
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += lo(sum[0]) + hi(sum[0]);
      }
      if (ok && n_it > 0) ok = __all_sync(kFull, wait_for(&sh.o_full[i], tiles++));
      if (!ok) break;
      tc5::fence_after();
      if (t.slot >= 0) {
        // a part of a tile: the state as it is (rows side by side, so that the
        // lanes' stores are), for the joining kernel
        float* const st = slot_of<D>(a, t.slot) + i * kRows + r;
        for (int x = 0; x < (n_it > 0 ? D / 16 : 0); ++x) {
          uint32_t o[16];
          tc5::ld16(o_tm + 16 * x, o);
          tc5::wait_ld();
          pin(o);
#pragma unroll
          for (int y = 0; y < 16; ++y) st[(16 * x + y) * (2 * kRows)] = __uint_as_float(o[y]);
        }
        st[D * (2 * kRows)] = m;
        st[(D + 1) * (2 * kRows)] = l;
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) taken(k);
        continue;
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
      const int h = t.g * a.G + r - tt * a.G;
      const int64_t at = int64_t(t.q0) + row;
      // where this thread's row goes, -1: nowhere
      const int64_t to = valid ? 2 * (at * a.out_stride + int64_t(h) * D) : -1;
      const bool none = limit == 0;  // no key: nothing was written for the row, or for others' sake only
      // Out through shared memory, 64 columns at a time, by TMA where the warp's 32
      // rows are whole tokens of the tile, and else with 8 lanes to 128 bytes.
      // (Stores from registers, a row to a lane or rows by 8 lanes, hold up the
      // load/store unit, and with it every wait of the CTA, for 3000 clocks.  A loop,
      // not unrolled: this code runs once a tile, and fetching it costs more than
      // running it; 220 -> 216 us for set B.)
      const bool whole = 32 % a.G == 0 && __all_sync(kFull, valid);
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t o[32];
        if (n_it > 0) {
          tc5::ld32(o_tm + 32 * x, o);
          tc5::wait_ld();
          pin(o);
        }
        if (x % 2 == 0) {  // the copy that read the buffer last is done
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = none ? 0u : pack_bf16x2(__uint_as_float(o[8 * y + 2 * e]) * inv, __uint_as_float(o[8 * y + 2 * e + 1]) * inv);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           out_sm + lane * 128 + (((x % 2 * 4 + y) ^ (lane & 7)) * 16)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        if (x % 2 == 0) continue;
        if (whole) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&a.tmo, out_sm, x / 2 * 64, t.g * a.G, t.q0 + i * a.tok + (warp & 3) * 32 / a.G);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {
          __syncwarp();
#pragma unroll 1
          for (int y = 0; y < 8; ++y) {
            const int rr = y * 4 + (lane >> 3), ch = lane & 7;
            const int64_t dst = __shfl_sync(kFull, to, rr);
            const uint4 w = lds128(out_sm + rr * 128 + ((ch ^ (rr & 7)) * 16));
            if (dst >= 0) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + dst + 128 * (x / 2) + 16 * ch) = w;
          }
          __syncwarp();
        }
      }
      // (the next tile's first P says that O_i has been read)
      tc5::fence_before();
      if (valid && a.lse) a.lse[at * a.H_q + h] = limit == 0 ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
      __syncwarp();
      if (lane == 0) taken(k);
    }
    // (shared memory outlives the copies out of it)
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    tc5::fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc5::fence_after();
    tc5::dealloc(tmem, 512);
  }
}

// Joins the parts of the tiles that were cut, in order:
//   out = sum_w f_w o_w / sum_w f_w l_w,  f_w = 2^(c (m_w - max m)).
// A CTA takes 32 rows of a tile pair and 64 columns, a lane a row, a warp 8 columns.
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const __grid_constant__ PrefillArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  pdl_wait();
  if (int(blockIdx.x) >= a.cut_count[0]) return;
  const int parts = a.cut_count[1];
  const Tile t = a.cuts[blockIdx.x];
  const float c = a.scale_log2;
  const int at = blockIdx.y * 32 + lane, i = at / kRows, r = at % kRows, tt = r / a.G;
  const int row = i * a.tok + tt;
  if (tt >= a.tok || row >= t.rows) return;
  // (after a wait that gave up, the tile may be one that an earlier call left)
  if (t.q0 < 0 || t.q0 >= a.total_q - row || t.g < 0 || t.g >= a.H_kv || parts > kMaxParts) return;
  const float* const p = slot_of<D>(a, blockIdx.x * parts) + at;
  constexpr int64_t STEP = 2 * kRows * (D + 2);
  float f[kMaxParts], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int w = 0; w < kMaxParts; ++w) {
    f[w] = w < parts ? __ldcg(p + w * STEP + D * (2 * kRows)) : -INFINITY;
    M = fmaxf(M, f[w]);
  }
#pragma unroll
  for (int w = 0; w < kMaxParts; ++w) {
    const float l = w < parts ? __ldcg(p + w * STEP + (D + 1) * (2 * kRows)) : 0.f;
    // (a part that saw no key, or only scores of -infinity, adds nothing)
    const bool none = f[w] == -INFINITY && l == 0.f;
    f[w] = none ? -1.f : ex2((f[w] - M) * c);
    L += none ? 0.f : f[w] * l;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  constexpr int PER = 8;  // columns of a thread
  const int d = blockIdx.z * 64 + warp * PER;
  float o[PER];
#pragma unroll
  for (int y = 0; y < PER; ++y) o[y] = 0.f;
#pragma unroll
  for (int w0 = 0; w0 < kMaxParts; w0 += 4) {
    float v[4][PER];  // 32 reads in flight
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int y = 0; y < PER; ++y) v[w][y] = w0 + w < parts ? __ldcg(p + (w0 + w) * STEP + (d + y) * (2 * kRows)) : 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int y = 0; y < PER; ++y) o[y] = f[w0 + w] == -1.f ? o[y] : fmaf(f[w0 + w], v[w][y], o[y]);
  }
  const int h = t.g * a.G + r - tt * a.G;
  const int64_t q = int64_t(t.q0) + row;
  uint4 v;
  v.x = pack_bf16x2(o[0] * inv, o[1] * inv);
  v.y = pack_bf16x2(o[2] * inv, o[3] * inv);
  v.z = pack_bf16x2(o[4] * inv, o[5] * inv);
  v.w = pack_bf16x2(o[6] * inv, o[7] * inv);
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + 2 * (q * a.out_stride + int64_t(h) * D + d)) = v;
  if (d == 0 && a.lse) a.lse[q * a.H_q + h] = (M * c + log2f(L)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(prefill_kernel<D>), int(Cfg<D>::SMEM), allowed);
  if (e != cudaSuccess) return e;
  // total / span <= sum_b ceil(n_b / span) <= total / span + B, if the sequences
  // hold all rows
  const long long least = (long long)a.total_q / (2 * a.tok) * a.H_kv, most = least + (long long)a.B * a.H_kv;
  const int sms = device_sm_count() < kPrefillMaxGrid ? device_sm_count() : kPrefillMaxGrid;
  PrefillArgs b = a;
  // No tile is cut, and no joining kernel needed (45 -> 40 us for 2048 tokens), with
  //  - many waves of tiles;
  //  - one wave that takes more than half of the SMs: no tile would get two;
  //  - more tiles than SMs and no more keys than queries: some sequence has no context,
  //    and its first tile is too short to be cut with the others.
  if (least >= (long long)kSplitWaves * sms || (2 * least > sms && (most <= sms || a.total_k <= a.total_q)))
    b.partials = nullptr;
  // (which tiles are cut depends on the grid: the SMs' number wherever some may be)
  const int grid = b.partials != nullptr || most > sms ? sms : int(most);
  const cudaError_t e2 = launch_pdl(prefill_kernel<D>, dim3(grid), kThreads, Cfg<D>::SMEM, st, b);
  if (e2 != cudaSuccess || b.partials == nullptr) return e2;
  return launch_pdl(prefill_join_kernel<D>, dim3(grid, 2 * kRows / 32, D / 64), 256, 0, st, b);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, int D, cudaStream_t st) {
  return D == 64 ? launch_t<64>(a, st) : launch_t<128>(a, st);
}

}  // namespace sfi

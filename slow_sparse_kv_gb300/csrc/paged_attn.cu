// Attention of one new token over a paged KV cache, split over its length.
//
// A tile is 16 (fp32: 8) consecutive positions of one (sequence, KV head).  All
// tiles of all sequences stand in one line, sequence by sequence and head by
// head; CTA c of C takes the c-th of C equal parts of the line, whatever the
// lengths, and its warp w the tiles whose number is w modulo 8.  Each warp
// keeps its own ring of tiles in shared memory, filled by its own copies some
// tiles ahead across the borders of sequences, so that the memory pipe never
// waits for the arithmetic.  Bound by HBM: 2 d e bytes a position and 4 d G
// flops, G <= 16.
//
// At the end of a piece (the CTA's part of one (sequence, KV head)) the warps'
// softmax states (m, l, o) are merged through shared memory; a piece that is
// not the whole unit goes to the workspace, and the CTA that counts the unit's
// last piece joins them, in the order of the line, so that the result does not
// depend on who comes last.
//
// bf16: S^T = K Q^T by mma.sync with the 16 positions as M and the group's heads
// as N (8 columns; two tiles of them for G > 8), O^T += V^T P^T with P moved to
// the B operand by movmatrix.  The output is fp32, so P is not rounded to bf16
// but split into two bf16 terms (what is lost is below 2^-17 of p), at the price
// of a second product with V.  tcgen05 would leave 128 - G of its 128 rows
// empty; the kernel waits for HBM either way.
// fp32: CUDA cores, d spread over the lanes, dots by transpose-reduction.
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.h"

namespace sfi {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStageBytes = 24576;  // ring of one warp
constexpr float kGrow = 8.0f;       // growth of the maximum (log2) that moves m

enum Load { kTma, kCpAsync, kBulk };

template <typename T, int D, int NT>
struct Cfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int TR = F32 ? 8 : 16;                  // positions per tile
  static constexpr int ROW = D * int(sizeof(T));           // bytes of a row
  static constexpr int HALF = TR * ROW;                    // K part of a stage, then V's
  static constexpr int STAGES = kStageBytes / (2 * HALF);  // 3 for 8 KB tiles, 6 for 4 KB
  static constexpr int HEADS = NT * 8;                     // heads that the registers hold
  static constexpr int MH = 4;                             // heads merged at a time
  static constexpr int MROW = D + 4;                       // floats of a merged head: o, m, l
  static constexpr int SMEM = 1024 + kWarps * kStageBytes + kWarps * MH * MROW * 4;
};

struct Shared {
  uint64_t full[kWarps][6];
  volatile int abort;
  int last;
  long long pre[kMaxBatch + 1];  // tiles of one KV head in the sequences before b
  long long part[kWarps];
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

__device__ __forceinline__ void unit_next(Unit& u, const Shared& sh, int B, int H_kv) {
  if (++u.g == H_kv) {
    u.g = 0;
    ++u.b;
  }
  u.begin = u.end;
  if (u.b < B) u.end += sh.pre[u.b + 1] - sh.pre[u.b];  // else the line's end
}

// The unit that holds tile x (x below the line's end).
__device__ __forceinline__ Unit unit_at(long long x, const Shared& sh, int B, int H_kv) {
  int lo = 0, hi = B;  // last b with pre[b] * H_kv <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.pre[mid] * H_kv <= x) lo = mid;
    else hi = mid;
  }
  const long long nt = sh.pre[lo + 1] - sh.pre[lo];
  Unit u;
  u.b = lo;
  u.g = int((x - sh.pre[lo] * H_kv) / nt);
  u.begin = sh.pre[lo] * H_kv + u.g * nt;
  u.end = u.begin + nt;
  return u;
}

template <typename T, int D, int NT, Load LD>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<T, D, NT>;
  constexpr bool F32 = C::F32;
  constexpr int TR = C::TR;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  float* const merge = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)) + kWarps * kStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.geo;
  const int B = geo.B, H_kv = geo.H_kv, P = geo.P, G = a.G;
  const int cap = geo.max_pages * P;

  // ---- tiles before each sequence
  {
    constexpr int PER = kMaxBatch / kThreads;
    int nt[PER];
    long long mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid * PER + i;
      int n = b < B ? geo.len[b] : 0;
      if (n < 0 || n > cap) {
        if (blockIdx.x == 0) set_status(geo.status, SFI_DEV_LEN_OVER_CAP);
        n = n < 0 ? 0 : cap;
      }
      nt[i] = (n + TR - 1) / TR;
      mine += nt[i];
    }
    long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) sh.part[warp] = run;
    if (tid == 0) sh.abort = 0;
    if (lane == 0 && LD != kCpAsync) {
      for (int i = 0; i < C::STAGES; ++i) mbar_init(smem_addr(&sh.full[warp][i]), 1);
      fence_mbar_init();
    }
    __syncthreads();
    long long before = run - mine;
    for (int w = 0; w < warp; ++w) before += sh.part[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid * PER + i;
      if (b < B) sh.pre[b] = before;
      before += nt[i];
      if (b == B - 1) sh.pre[B] = before;
    }
    __syncthreads();
  }
  const long long total = sh.pre[B] * H_kv;

  // sequences that hold nothing
  for (int u = blockIdx.x; u < B * H_kv; u += gridDim.x) {
    const int b = u / H_kv, g = u - b * H_kv;
    if (sh.pre[b + 1] != sh.pre[b]) continue;
    const int64_t row = int64_t(b) * a.H_q + int64_t(g) * G;
    for (int i = tid; i < G * D; i += kThreads) a.out[row * D + i] = 0.f;
    if (a.lse && tid < G) a.lse[row + tid] = -INFINITY;
  }
  // parts of a tile for each warp at least
  const long long parts = min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
  if (blockIdx.x >= parts) return;
  const long long T0 = blockIdx.x * total / parts, T1 = (blockIdx.x + 1) * total / parts;

  const uint32_t ring = base + warp * kStageBytes;
  const T* const kp = static_cast<const T*>(a.k);
  const T* const vp = static_cast<const T*>(a.v);
  const float c = a.scale_log2;

  // ---- this warp's copies: tile `ld` of unit `lu`, into stage ls
  const long long first = T0 + ((warp - T0) % kWarps + kWarps) % kWarps;
  long long ld = first;
  int ls = 0;
  Unit lu = unit_at(T0, sh, B, H_kv);
  int page = 0;  // of this lane's row of tile ld
  auto fetch_page = [&]() {
    if (ld >= T1) return;
    while (ld >= lu.end) unit_next(lu, sh, B, H_kv);
    const int pos = int(ld - lu.begin) * TR + (LD == kTma ? 0 : lane % TR);
    const int n = min(geo.len[lu.b], cap);
    page = pos < n ? geo.table[int64_t(lu.b) * geo.max_pages + pos / P] : 0;
  };
  auto issue = [&]() {  // tile ld, whose page is known; then looks up the next one's
    if (ld >= T1) {
      if (LD == kCpAsync) asm volatile("cp.async.commit_group;" ::: "memory");
      return;
    }
    if (page < 0 || page >= geo.n_pages) {
      set_status(geo.status, SFI_DEV_BAD_INDEX);
      page = 0;
    }
    const int t = int(ld - lu.begin);
    const uint32_t dst = ring + ls * 2 * C::HALF;
    const uint32_t bar = smem_addr(&sh.full[warp][ls]);
    if constexpr (LD == kTma) {
      if (lane == 0) {
        const int row = int(page * (geo.page_stride / D) + lu.g * P + t * TR % P);
        mbar_arrive_expect_tx(bar, 2 * C::HALF);
        tma_load_3d(dst, &a.tmk, 0, row, 0, bar);
        tma_load_3d(dst + C::HALF, &a.tmv, 0, row, 0, bar);
      }
    } else {
      const int n = min(geo.len[lu.b], cap);
      const int pos = t * TR + lane % TR;
      const int in = pos % P;
      const int64_t at = page * geo.page_stride + (int64_t(lu.g) * P + in) * D;
      if constexpr (LD == kBulk) {
        // runs of rows that lie in one page, one lane each
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(min(TR, n - t * TR)) * 2 * C::ROW);
        __syncwarp();
        if (lane < TR && pos < n && (lane == 0 || in == 0)) {
          const uint32_t bytes = uint32_t(min(min(P - in, TR - lane), n - pos)) * C::ROW;
          bulk_load(dst + lane * C::ROW, kp + at, bytes, bar);
          bulk_load(dst + C::HALF + lane * C::ROW, vp + at, bytes, bar);
        }
      } else {
        // 16-byte chunks, in the layout that the maps' swizzle gives
        constexpr int CH = C::ROW / 16;  // chunks of a row
#pragma unroll
        for (int i = 0; i < TR * CH / 32; ++i) {
          const int r = (i * 32 + lane) / CH, ch = lane % CH;
          const int64_t ra = __shfl_sync(kFull, at, r) + ch * 8;
          const uint32_t some = t * TR + r < n ? 16 : 0;
          const uint32_t to = dst + (ch / 8) * (TR * 128) + r * 128 + ((ch & 7) ^ (r & 7)) * 16;
          cp_async16_zfill(to, kp + ra, some);
          cp_async16_zfill(to + C::HALF, vp + ra, some);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    }
    ls = ls + 1 == C::STAGES ? 0 : ls + 1;
    ld += kWarps;
    fetch_page();
  };
  fetch_page();
  for (int i = 0; i < C::STAGES - 1; ++i) issue();

  // ---- the CTA's pieces
  long long x = first;  // this warp's next tile to compute
  int cs = 0;
  uint32_t phase = 0;
  for (Unit u = unit_at(T0, sh, B, H_kv); u.begin < T1; unit_next(u, sh, B, H_kv)) {
    if (u.end == u.begin) continue;
    const long long pe = min(u.end, T1);
    const int n = min(geo.len[u.b], cap);
    const int64_t qrow = (int64_t(u.b) * a.H_q + int64_t(u.g) * G) * D;

    // state: bf16 head 2 (lane % 4) + e of column tile h, in every lane with the same lane % 4;
    // fp32 head 4 h + lane % 4
    constexpr int NS = F32 ? NT * 2 : NT;
    constexpr int NE = F32 ? 1 : 2;
    float m[NS][NE], l[NS][NE];
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int e = 0; e < NE; ++e) m[h][e] = -INFINITY, l[h][e] = 0.f;

    // per-lane operands
    constexpr int KS = D / 16;
    uint32_t qb[F32 ? 1 : NT][KS][2];
    float o[F32 ? 1 : KS][F32 ? 1 : NT][4];
    float qf[F32 ? NS * 4 : 1][4], of[F32 ? NS * 4 : 1][4];
    constexpr int LPR = D / 4, RPP = 32 / LPR;  // fp32: lanes per row, rows per pass
    const int li = lane % LPR, half = lane / LPR;
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
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[kk][h][e] = 0.f;
    } else {
#pragma unroll
      for (int h = 0; h < NS * 4; ++h) {
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h < G) w = reinterpret_cast<const float4*>(static_cast<const T*>(a.q) + qrow + h * D)[li];
        qf[h][0] = w.x, qf[h][1] = w.y, qf[h][2] = w.z, qf[h][3] = w.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) of[h][e] = 0.f;
      }
    }

    for (; x < pe; x += kWarps) {
      // ---- the next tile's copies go out, this one's rows have landed
      __syncwarp();
      issue();
      if constexpr (LD == kCpAsync) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 1) : "memory");
        __syncwarp();
      } else {
        const bool ok = warp_pipe_wait(smem_addr(&sh.full[warp][cs]), phase, &sh.abort, geo.status, a.wait_cycles);
        if (!ok) {
          // no copy of this warp may be in flight when the CTA exits: the
          // stage's rows land before the warp goes on (without them)
          mbar_wait(smem_addr(&sh.full[warp][cs]), phase);
          __syncwarp();
          if (++cs == C::STAGES) cs = 0, phase ^= 1;
          continue;
        }
      }
      const uint32_t ks = ring + cs * 2 * C::HALF, vs = ks + C::HALF;
      const int left = n - int(x - u.begin) * TR;  // rows of the tile that count

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
        uint32_t ph[NT][2], pl[NT][2];
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
          const uint32_t h0 = pack_bf16x2(p0, p1), h1 = pack_bf16x2(p2, p3);
          const uint32_t l0 = pack_bf16x2(p0 - __uint_as_float(h0 << 16), p1 - __uint_as_float(h0 & 0xffff0000u));
          const uint32_t l1 = pack_bf16x2(p2 - __uint_as_float(h1 << 16), p3 - __uint_as_float(h1 & 0xffff0000u));
          ph[h][0] = movmatrix_trans(h0), ph[h][1] = movmatrix_trans(h1);
          pl[h][0] = movmatrix_trans(l0), pl[h][1] = movmatrix_trans(l1);
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
            mma_bf16_16816(o[kk][h], v0, v1, v2, v3, ph[h][0], ph[h][1]);
            mma_bf16_16816(o[kk][h], v0, v1, v2, v3, pl[h][0], pl[h][1]);
          }
        }
      } else {
        constexpr int PASS = TR / RPP;
#pragma unroll
        for (int h = 0; h < NS; ++h) {
          if (h * 4 >= G) break;
          float v[PASS * 4];
#pragma unroll
          for (int i = 0; i < PASS; ++i) {
            const uint4 w = lds128(ks + (i * RPP + half) * C::ROW + li * 16);
            const float k0 = __uint_as_float(w.x), k1 = __uint_as_float(w.y), k2 = __uint_as_float(w.z),
                        k3 = __uint_as_float(w.w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[i * 4 + e] = k0 * qf[h * 4 + e][0] + k1 * qf[h * 4 + e][1] + k2 * qf[h * 4 + e][2] + k3 * qf[h * 4 + e][3];
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
#pragma unroll
              for (int y = 0; y < 4; ++y) of[h * 4 + e][y] *= fe;
            }
          }
          const float p = ex2(fmaf(s, c, -(m[h][0] == -INFINITY ? 0.f : m[h][0] * c)));
          l[h][0] += p;
#pragma unroll
          for (int i = 0; i < PASS; ++i) {
            uint4 w = lds128(vs + (i * RPP + half) * C::ROW + li * 16);
            if (i * RPP + half >= left) w = make_uint4(0, 0, 0, 0);  // 0 * NaN is not 0
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float pe_ = __shfl_sync(kFull, p, half * LPR + i * 4 + e);
              of[h * 4 + e][0] = fmaf(pe_, __uint_as_float(w.x), of[h * 4 + e][0]);
              of[h * 4 + e][1] = fmaf(pe_, __uint_as_float(w.y), of[h * 4 + e][1]);
              of[h * 4 + e][2] = fmaf(pe_, __uint_as_float(w.z), of[h * 4 + e][2]);
              of[h * 4 + e][3] = fmaf(pe_, __uint_as_float(w.w), of[h * 4 + e][3]);
            }
          }
        }
      }
      if (++cs == C::STAGES) cs = 0, phase ^= 1;
    }

    // ---- merge the warps' states, MH heads at a time
    // the unit's pieces: parts of the CTAs that hold its first to its last tile
    const long long c0 = ((u.begin + 1) * parts - 1) / total, c1 = (u.end * parts - 1) / total;
    const int pieces = int(c1 - c0) + 1;
    const int uid = u.b * H_kv + u.g;
    float* const slot0 = a.partials + (c0 + uid) * int64_t(G) * (D + 2);
    float* const slot = slot0 + (blockIdx.x - c0) * int64_t(G) * (D + 2);
#pragma unroll
    for (int h0 = 0; h0 < C::HEADS; h0 += C::MH) {
      if (h0 >= G) break;
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
            if (RPP == 2) of[h * 4 + e][y] += __shfl_xor_sync(kFull, of[h * 4 + e][y], 16);
            if (half == 0) mine[e * C::MROW + li * 4 + y] = of[h * 4 + e][y];
          }
        }
      }
      __syncthreads();
      for (int i = tid; i < min(C::MH, G - h0) * D; i += kThreads) {
        const int h = i / D, d = i - h * D;
        const float* const row = merge + h * C::MROW;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, row[w * C::MH * C::MROW + D]);
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* const rw = row + w * C::MH * C::MROW;
          if (rw[D] == -INFINITY && rw[D + 1] == 0.f) continue;  // saw nothing
          const float f = ex2((rw[D] - M) * c);
          L += f * rw[D + 1];
          O += f * rw[d];
        }
        if (pieces == 1) {
          a.out[qrow + (h0 + h) * D + d] = L == 0.f ? 0.f : O / L;
          if (d == 0 && a.lse) a.lse[qrow / D + h0 + h] = (M * c + log2f(L)) * 0.6931471805599453f;
        } else {
          float* const p = slot + (h0 + h) * (D + 2);
          p[d] = O;
          if (d == 0) p[D] = M, p[D + 1] = L;
        }
      }
      __syncthreads();
    }
    if (pieces > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int seen = atomicAdd(a.counters + uid, 1);
        sh.last = seen == pieces - 1;
        if (sh.last) a.counters[uid] = 0;
      }
      __syncthreads();
      if (sh.last) {
        __threadfence();
        const int64_t step = int64_t(G) * (D + 2);
        for (int i = tid; i < G * D; i += kThreads) {
          const int h = i / D, d = i - h * D;
          const float* const p = slot0 + h * (D + 2);
          float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll 8
          for (int w = 0; w < pieces; ++w) M = fmaxf(M, __ldcg(p + w * step + D));
#pragma unroll 8
          for (int w = 0; w < pieces; ++w) {
            const float mw = __ldcg(p + w * step + D), lw = __ldcg(p + w * step + D + 1), ow = __ldcg(p + w * step + d);
            const bool none = mw == -INFINITY && lw == 0.f;
            const float f = ex2((mw - M) * c);
            L += none ? 0.f : f * lw;
            O += none ? 0.f : f * ow;
          }
          a.out[qrow + h * D + d] = L == 0.f ? 0.f : O / L;
          if (d == 0 && a.lse) a.lse[qrow / D + h] = (M * c + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
  }
}

template <typename T, int D, int NT, Load LD>
cudaError_t launch_t(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<T, D, NT>;
  auto* const kernel = paged_attn_kernel<T, D, NT, LD>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, C::SMEM, st>>>(a);
  return cudaGetLastError();
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

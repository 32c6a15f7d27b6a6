// Attention of one new token over a paged KV cache in 8 bits: the split over the
// length, the copying warps, pieces and joins are those of paged_attn.cu; a tile is 32
// positions of one (sequence, KV head), 32 d bytes of K and of V and their scales.
//
//   S_i = sk_i (q . ck_i) / sqrt(d),  out = sum_i p_i sv_i cv_i / sum_i p_i,  p_i = 2^(log2(e) S_i - m)
//
// Bound by HBM: 2 (d + 4) bytes a position, half of bf16's, so the work on the codes has
// half the time.  Codes become fp16 in registers, which holds all of them exactly (int8
// by a byte permutation into 1024 + code + 128 and one packed subtraction, e4m3 by the
// conversion instruction), and the products are m16n8k16 MMAs with the positions
// (S^T = K Q^T) or the dimensions (O^T += V^T P^T) as M and the group's heads as N.
// Scales stay out of the products: sk multiplies the finished fp32 score, sv goes into p.
//
// K: which 16 dimensions a k step takes is free as long as q takes the same, so a lane
// reads the codes that it needs as whole 16-byte pieces of its row.  V: ldmatrix.trans
// moves pairs of bytes, so a register holds two dimensions of two positions; the even ones
// are rows 0 to 7 of the MMA, the odd ones rows 8 to 15.
//
// fp16 operands: q is scaled by a power of two for each head so that its largest element
// lies in [2^14, 2^15) (bf16: exact down to 2^-32 of that; fp32: two terms, 22 bits); p sv
// by one for each tile and head in the same way, and it is split into two terms: 22 bits, and what
// is dropped below is under 2^-39 of the tile's largest p sv.  (Scaled by the tile's largest sv
// alone, a row of large values that the softmax leaves out would cost the others their bits.)  Each tile's product starts
// from zero and is added to o in fp32 (the tensor cores truncate where they add).
//
// Measured, 32 / 8 heads of 128 in bf16: 8 x 32768 positions in int8, pages of 64 (0.55 GB), in
// 92 us, 6.05 TB/s, where a copy reaches 6.78 (pages of 16: 96); 32 sequences of 4096 to 65536 in
// e4m3 (1.23 GB) in 197 us, 6.2 TB/s, with pages of 16 and 191 with pages of 64: a tile of two pages
// takes eight copies and not four.  (A copying lane that works its tile's addresses out while it
// issues the copies: 213.  Scales copied 4 bytes a lane: 220, and 98 for the other.)  One
// sequence of 700 10.5 us, the two launches.  8 x 32768 with fp32 queries: 93.  128 heads (16 a
// group): 125, with fp32 queries 147: the issue slots.  64 sequences of 1 to 32 with one KV head: 25, since a
// share is eight tiles and these lie in eight units, one after another.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "paged.h"
#include "paged_line.cuh"
#include "pdl.cuh"

namespace sfi {
namespace {

constexpr int kTile = 32;          // positions of a tile
constexpr int kRing = 196608;      // bytes of codes in flight
constexpr float kGrow = 4.0f;      // growth of the maximum (log2) that moves m

template <int D, int NT>
struct Q8 {
  static constexpr int HALF = kTile * D;                  // K part of a stage, then V's
  static constexpr int STAGES = kRing / kWarps / (2 * HALF);  // a warp's: 3 of 8 KB, 6 of 4 KB
  static constexpr int SLOTS = kWarps * STAGES;
  static constexpr int SCALES = 2 * kTile * 4;            // K's scales of a stage, then V's
  static constexpr int HEADS = NT * 8;
  static constexpr int MH = 4;                            // heads merged at a time
  static constexpr int MROW = D + 4;
  static constexpr int SMEM = 1024 + kRing + SLOTS * SCALES + kWarps * MH * MROW * 4;
};

struct SharedQ8 {
  Line ln;
  uint64_t full[48], empty[48];
  volatile int abort;
  uint64_t merge_free;
};

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Four codes as fp16 pairs: bytes (0, 1) and (2, 3).
template <bool E4M3>
__device__ __forceinline__ void codes_near(uint32_t w, uint32_t& x, uint32_t& y) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(w));
  } else {
    w ^= 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
  }
}
// The same, bytes (0, 2) and (1, 3).
template <bool E4M3>
__device__ __forceinline__ void codes_far(uint32_t w, uint32_t& x, uint32_t& y) {
  if constexpr (E4M3) {
    codes_near<true>(__byte_perm(w, 0, 0x3120), x, y);
  } else {
    w ^= 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(__byte_perm(w, 0x64646464u, 0x4240)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(__byte_perm(w, 0x64646464u, 0x4341)), "r"(0x64806480u));
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w >> 16))); }

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// 4 bytes, of which `bytes` (0 or 4) are read and the rest are zero.
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Where 16-byte chunk c of row r lies in a tile (the swizzle of the maps).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4);
}

// The copying warps: warp `p` takes the tiles of the attending warps p and p + 4.
template <int D, int NT, bool TMA>
__device__ __forceinline__ void copy_q8(const PagedAttnArgs& a, SharedQ8& sh, long long from, long long to,
                                        uint32_t ring, uint32_t scales, int p) {
  using C = Q8<D, NT>;
  const PagedGeo& geo = a.geo;
  const int lane = threadIdx.x & 31, P = geo.P, H_kv = geo.H_kv, cap = geo.max_pages * P;
  const uint8_t* const kp = static_cast<const uint8_t*>(a.k);
  const uint8_t* const vp = static_cast<const uint8_t*>(a.v);
  bool ok = true;
  const long long first[2] = {first_of(from, p, kWarps), first_of(from, p + kProducers, kWarps)};
  for (long long x0 = first_of(from, p, kProducers); x0 < to && ok; x0 += kProducers * 32) {
    // 32 tiles: each lane finds the place of its own, and with maps the page of each box
    const long long x = x0 + kProducers * lane;
    const bool mine = x < to;
    Unit u{0, 0, 0, 0};
    int t = 0, n = 0, page[2] = {0, 0}, row[2] = {0, 0}, boxes = 0;
    int64_t at[2] = {0, 0};  // bytes to the boxes' scales
    if (mine) {
      u = unit_at(x, sh.ln, geo.B, H_kv);
      t = int(x - u.begin);
      n = min(geo.len[u.b], cap);
    }
    if (TMA) {
      const int32_t* const urow = geo.table + int64_t(u.b) * geo.max_pages;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pos = t * kTile + i * a.box;
        if (!mine || pos >= n || i * a.box >= kTile) continue;
        page[i] = urow[pos / P];
        row[i] = u.g * P + pos % P;
        if (page[i] < 0 || page[i] >= geo.n_pages) bad = true, page[i] = 0;
        boxes = i + 1;
        at[i] = page[i] * geo.page_stride + a.scale_at + row[i] * 4LL;
      }
      if (bad) set_status(geo.status, SFI_DEV_BAD_INDEX);
    }
    const int count = int(min(32LL, (to - x0 + kProducers - 1) / kProducers));
    // without maps: this lane's row of the i-th tile: its page, and where in it, -1 for no
    // row.  A tile's pages are read while the one before it is copied.
    int pg = 0, in = -1;
    auto row_of = [&](int i) {
      const int ut = __shfl_sync(kFull, t, i), ug = __shfl_sync(kFull, u.g, i), un = __shfl_sync(kFull, n, i);
      const int32_t* const urow = geo.table + int64_t(__shfl_sync(kFull, u.b, i)) * geo.max_pages;
      const int pos = ut * kTile + lane;
      pg = pos < un ? urow[pos / P] : 0;
      in = pos < un ? ug * P + pos % P : -1;
    };
    if (!TMA) row_of(0);
    for (int i = 0; i < count && ok; ++i) {
      const long long xi = x0 + kProducers * i;
      const int w = int(xi >> 2) & 1;  // which of the two warps
      const uint32_t y = uint32_t(xi - first[w]) / kWarps;
      const int slot = (p + w * kProducers) * C::STAGES + int(y % C::STAGES);
      const uint32_t use = y / C::STAGES;
      if (use > 0) ok = warp_ctrl_wait(smem_addr(&sh.empty[slot]), (use - 1) & 1, &sh.abort, geo.status);
      if (!ok) break;
      const uint32_t dst = ring + slot * 2 * C::HALF, sdst = scales + slot * C::SCALES, bar = smem_addr(&sh.full[slot]);
      if constexpr (TMA) {
        if (lane == i) {
          mbar_arrive_expect_tx(bar, uint32_t(boxes * a.box) * 2 * (D + 4));
#pragma unroll
          for (int y2 = 0; y2 < 2; ++y2) {
            if (y2 >= boxes) break;
            tma_load_3d(dst + y2 * a.box * D, &a.tmk, 0, row[y2], page[y2], bar);
            bulk_load(sdst + y2 * a.box * 4, kp + at[y2], a.box * 4, bar);
            tma_load_3d(dst + C::HALF + y2 * a.box * D, &a.tmv, 0, row[y2], page[y2], bar);
            bulk_load(sdst + kTile * 4 + y2 * a.box * 4, vp + at[y2], a.box * 4, bar);
          }
        }
      } else {
        constexpr int CH = D / 16;  // chunks of a row
        if (pg < 0 || pg >= geo.n_pages) {
          set_status(geo.status, SFI_DEV_BAD_INDEX);
          pg = 0;
        }
        const int64_t base = pg * geo.page_stride;
        const int64_t at = in < 0 ? -1 : base + int64_t(in) * D, sat = in < 0 ? 0 : base + a.scale_at + in * 4LL;
        const uint32_t some4 = in < 0 ? 0 : 4;
        if (i + 1 < count) row_of(i + 1);
        cp_async4_zfill(sdst + lane * 4, kp + sat, some4);
        cp_async4_zfill(sdst + kTile * 4 + lane * 4, vp + sat, some4);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int r = (j * 32 + lane) / CH, ch = lane % CH;
          const int64_t from_row = __shfl_sync(kFull, at, r);
          const int64_t ra = max(from_row, int64_t(0)) + ch * 16;
          const uint32_t some = from_row >= 0 ? 16 : 0;
          const uint32_t dr = dst + chunk_at<D>(r, ch);
          cp_async16_zfill(dr, kp + ra, some);
          cp_async16_zfill(dr + C::HALF, vp + ra, some);
        }
        cp_async_arrive_noinc(bar);
      }
    }
    __syncwarp();
  }
  // (as in paged_attn.cu: no copy may be in flight when the CTA exits)
  if (!ok) sh.abort = 2;
  if (!TMA) asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int NT, bool E4M3, bool QF, bool TMA>
__global__ void __launch_bounds__(kAllThreads, 1) paged_attn_q8_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Q8<D, NT>;
  constexpr int NQ = QF ? 2 : 1;  // terms of q
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ SharedQ8 sh;
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, scales = ring + kRing;
  float* const merge = reinterpret_cast<float*>(smem_raw + (ring - smem_addr(smem_raw)) + kRing + C::SLOTS * C::SCALES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedGeo& geo = a.geo;
  const int B = geo.B, H_kv = geo.H_kv, G = a.G;
  const int cap = geo.max_pages * geo.P;

  if (tid < C::SLOTS) {
    mbar_init(smem_addr(&sh.full[tid]), TMA ? 1 : 32);
    mbar_init(smem_addr(&sh.empty[tid]), 1);
  } else if (tid == 96) {
    mbar_init(smem_addr(&sh.merge_free), kWarps);
    sh.abort = 0;
  }
  fence_mbar_init();
  pdl_launch();
  pdl_wait();
  scan_lengths<kTile>(geo, sh.ln, blockIdx.x == 0);
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
  const Cut cut(total, gridDim.x);
  const int share = blockIdx.x;
  const long long from = share < cut.shares ? cut.start(share) : total;
  const long long to = share < cut.shares ? cut.start(share + 1) : total;

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    copy_q8<D, NT, TMA>(a, sh, from, to, ring, scales, warp - kWarps);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAttendRegs));
    uint32_t y = 0;       // this warp's tiles so far
    uint32_t merges = 0;  // and rounds of merging
    const int r8 = lane >> 2, j4 = lane & 3;
    uint32_t qb[NT][NQ][KS][2];
    float fac[NT][2];  // what turns a head's products into scores in log2 units
    // The lane's part of a unit's queries: dimensions j4 d / 4 .. of head r8 (+ 8), and the
    // factors of its heads 2 j4 and 2 j4 + 1; the sequence's length.
    auto load_unit = [&](const Unit& u) {
      const int64_t qrow = (int64_t(u.b) * a.H_q + int64_t(u.g) * G) * D;
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const int head = h * 8 + r8;
        float x[D / 4];
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
        if (head < G) {
          if constexpr (QF) {
            const float4* const s = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + qrow + head * D + j4 * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const float4 v = s[i];
              x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
            }
          } else {
            const uint4* const s = reinterpret_cast<const uint4*>(static_cast<const bf16_t*>(a.q) + qrow + head * D + j4 * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              float v[8];
              Unpack<bf16_t>::run(s[i], v);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[8 * i + e] = v[e];
            }
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int ex = max(int(top >> 23), 20);  // (255: not finite)
        const float up = pow2(14 + 127 - ex);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x0 = x[4 * kk + 2 * e] * up, x1 = x[4 * kk + 2 * e + 1] * up;
            const uint32_t w = pack_f16x2(x0, x1);
            qb[h][0][kk][e] = w;
            if (QF) qb[h][NQ - 1][kk][e] = pack_f16x2(x0 - f16_lo(w), x1 - f16_hi(w));
          }
        const float down = pow2(ex - 127 - 14) * a.scale_log2;
        fac[h][0] = __shfl_sync(kFull, down, 8 * j4);
        fac[h][1] = __shfl_sync(kFull, down, 8 * j4 + 4);
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
        // state of head 2 j4 + e of column tile h, in every lane with the same j4
        float m[NT][2], l[NT][2], o[KS][NT][4];
#pragma unroll
        for (int h = 0; h < NT; ++h) {
#pragma unroll
          for (int e = 0; e < 2; ++e) m[h][e] = -INFINITY, l[h][e] = 0.f;
#pragma unroll
          for (int c = 0; c < KS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][h][e] = 0.f;
        }

        for (; x < pe; x += kWarps) {
          const int slot = warp * C::STAGES + int(y % C::STAGES);
          const uint32_t use = y / C::STAGES;
          ++y;
          const int left = n - int(x - u.begin) * kTile;  // rows of the tile that count
          const bool ok = warp_pipe_wait(smem_addr(&sh.full[slot]), use & 1, &sh.abort, geo.status, a.wait_cycles);
          if (!ok) {
            // the stage is given back once its rows have landed, without them
            if (sh.abort != 2) mbar_wait(smem_addr(&sh.full[slot]), use & 1);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.empty[slot]));
            continue;
          }
          const uint32_t ks = ring + slot * 2 * C::HALF, vs = ks + C::HALF, sc = scales + slot * C::SCALES;

          // ---- scores of 2 x 16 positions
          float s[2][NT][4];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
            for (int h = 0; h < NT; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][h][e] = 0.f;
            const int ra = mt * 16 + r8;
            uint32_t w0[KS], w1[KS];
#pragma unroll
            for (int i = 0; i < KS / 4; ++i) {
              const uint4 v0 = lds128(ks + chunk_at<D>(ra, j4 * (D / 64) + i)), v1 = lds128(ks + chunk_at<D>(ra + 8, j4 * (D / 64) + i));
              w0[4 * i] = v0.x, w0[4 * i + 1] = v0.y, w0[4 * i + 2] = v0.z, w0[4 * i + 3] = v0.w;
              w1[4 * i] = v1.x, w1[4 * i + 1] = v1.y, w1[4 * i + 2] = v1.z, w1[4 * i + 3] = v1.w;
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              uint32_t a0, a1, a2, a3;
              codes_near<E4M3>(w0[kk], a0, a2);
              codes_near<E4M3>(w1[kk], a1, a3);
#pragma unroll
              for (int h = 0; h < NT; ++h)
#pragma unroll
                for (int q = NQ - 1; q >= 0; --q) mma_f16_16816(s[mt][h], a0, a1, a2, a3, qb[h][q][kk][0], qb[h][q][kk][1]);
            }
          }
          // ---- scales: those of the rows r8 + 8 i
          float kscale[4], vscale[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = r8 + 8 * i;
            kscale[i] = lds32(sc + row * 4);
            vscale[i] = row < left ? lds32(sc + kTile * 4 + row * 4) : 0.f;
          }
          uint32_t pw[NT][2][2][2];  // P^T: [term][positions / 16][half]
          float down[NT][2];         // what turns the products with V back
#pragma unroll
          for (int h = 0; h < NT; ++h) {
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float& z = s[i >> 1][h][(i & 1) * 2 + e];
                z = r8 + 8 * i < left ? z * (kscale[i] * fac[h][e]) : -INFINITY;  // (large times small first)
              }
              top[e] = fmaxf(fmaxf(s[0][h][e], s[0][h][2 + e]), fmaxf(s[1][h][e], s[1][h][2 + e]));
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], w));
            }
            const bool g0 = top[0] - m[h][0] > kGrow, g1 = top[1] - m[h][1] > kGrow;
            if (__any_sync(kFull, g0 || g1)) {
              const float f0 = g0 ? ex2(m[h][0] - top[0]) : 1.f, f1 = g1 ? ex2(m[h][1] - top[1]) : 1.f;
              if (g0) m[h][0] = top[0];
              if (g1) m[h][1] = top[1];
              l[h][0] *= f0;
              l[h][1] *= f1;
#pragma unroll
              for (int c = 0; c < KS; ++c) {
                o[c][h][0] *= f0, o[c][h][1] *= f1;
                o[c][h][2] *= f0, o[c][h][3] *= f1;
              }
            }
            const float b0 = m[h][0] == -INFINITY ? 0.f : m[h][0], b1 = m[h][1] == -INFINITY ? 0.f : m[h][1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float &z0 = s[i >> 1][h][(i & 1) * 2], &z1 = s[i >> 1][h][(i & 1) * 2 + 1];
              const float p0 = ex2(z0 - b0), p1 = ex2(z1 - b1);
              l[h][0] += p0;
              l[h][1] += p1;
              z0 = p0 * vscale[i], z1 = p1 * vscale[i];
            }
            // the exponents of both heads' largest p sv, as the upper halves of the numbers
            uint32_t zt = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              zt = __vmaxu2(zt, __byte_perm(__float_as_uint(s[i >> 1][h][(i & 1) * 2]), __float_as_uint(s[i >> 1][h][(i & 1) * 2 + 1]), 0x7632) & 0x7fff7fffu);
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) zt = __vmaxu2(zt, __shfl_xor_sync(kFull, zt, w));
            const int ex0 = max(int(zt >> 7 & 0xff), 20), ex1 = max(int(zt >> 23), 20);
            const float up0 = pow2(14 + 127 - ex0), up1 = pow2(14 + 127 - ex1);
            down[h][0] = pow2(ex0 - 127 - 14), down[h][1] = pow2(ex1 - 127 - 14);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z0 = s[i >> 1][h][(i & 1) * 2] * up0, z1 = s[i >> 1][h][(i & 1) * 2 + 1] * up1;
              const uint32_t w = pack_f16x2(z0, z1);
              pw[h][0][i >> 1][i & 1] = movmatrix_trans(w);
              pw[h][1][i >> 1][i & 1] = movmatrix_trans(pack_f16x2(z0 - f16_lo(w), z1 - f16_hi(w)));
            }
          }
          // ---- O += P V
          const int vr = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll
          for (int c2 = 0; c2 < KS / 2; ++c2) {  // 32 dimensions
            uint32_t v[2][2][4];  // [positions / 16][dimensions / 16]: an MMA's A
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t x0, x1, x2, x3;
              ldsm_x4_trans(vs + chunk_at<D>(mt * 16 + vr, c2 * 2 + (lane >> 4)), x0, x1, x2, x3);
              if (E4M3 && left < kTile) {
                // rows behind the sequence's end may hold NaN: 0 * NaN is not 0
                const int row = mt * 16 + 2 * j4;
                const uint32_t m0 = (row < left ? 0xffffu : 0u) | (row + 1 < left ? 0xffff0000u : 0u);
                const uint32_t m1 = (row + 8 < left ? 0xffffu : 0u) | (row + 9 < left ? 0xffff0000u : 0u);
                x0 &= m0, x1 &= m1, x2 &= m0, x3 &= m1;
              }
              codes_far<E4M3>(x0, v[mt][0][0], v[mt][0][1]);
              codes_far<E4M3>(x1, v[mt][0][2], v[mt][0][3]);
              codes_far<E4M3>(x2, v[mt][1][0], v[mt][1][1]);
              codes_far<E4M3>(x3, v[mt][1][2], v[mt][1][3]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 1; t >= 0; --t)  // small terms first
#pragma unroll
                  for (int mt = 0; mt < 2; ++mt)
                    mma_f16_16816(d, v[mt][c][0], v[mt][c][1], v[mt][c][2], v[mt][c][3], pw[h][t][mt][0], pw[h][t][mt][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c2 * 2 + c][h][e] = fmaf(d[e], down[h][e & 1], o[c2 * 2 + c][h][e]);
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

        // ---- the piece: the warps' states merged, MH heads at a time, as in paged_attn.cu
        const bool alone = u.begin >= from && u.end <= to;  // the unit's only piece
        float* const slot = a.partials + (share + b * H_kv + g) * int64_t(G) * (D + 2);
#pragma unroll
        for (int h0 = 0; h0 < C::HEADS; h0 += C::MH) {
          if (h0 >= G) break;
          if (merges > 0) warp_ctrl_wait(smem_addr(&sh.merge_free), (merges - 1) & 1, &sh.abort, geo.status);
          ++merges;
          float* const mine = merge + warp * C::MH * C::MROW;
          const int h = h0 / 8;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = l[h][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(kFull, t, w);
            const int at = h * 8 + 2 * j4 + e - h0;  // this lane's head
            if (at < 0 || at >= C::MH) continue;
            float* const row = mine + at * C::MROW;
            if (lane < 4) row[D] = m[h][e], row[D + 1] = t;
#pragma unroll
            for (int c = 0; c < KS; ++c)
              *reinterpret_cast<float2*>(row + c * 16 + 2 * r8) = make_float2(o[c][h][e], o[c][h][2 + e]);
          }
          attend_sync();
          for (int i = tid; i < min(C::MH, G - h0) * D; i += kThreads) {
            const int hh = i / D, d = i - hh * D;
            float2 ml[kWarps];
            float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              ml[w] = *reinterpret_cast<const float2*>(merge + (w * C::MH + hh) * C::MROW + D);
              M = fmaxf(M, ml[w].x);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              // (a warp that saw nothing, or only scores of -infinity, adds nothing)
              const bool none = ml[w].x == -INFINITY && ml[w].y == 0.f;
              const float f = ex2(ml[w].x - M);
              L += none ? 0.f : f * ml[w].y;
              O += none ? 0.f : f * merge[(w * C::MH + hh) * C::MROW + d];
            }
            if (alone) {
              a.out[qrow + (h0 + hh) * D + d] = L == 0.f ? 0.f : O / L;
              if (d == 0 && a.lse) a.lse[qrow / D + h0 + hh] = (M + log2f(L)) * 0.6931471805599453f;
            } else {
              float* const p = slot + (h0 + hh) * (D + 2);
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

template <int D, int NT, bool E4M3, bool QF, bool TMA>
cudaError_t launch_q8(const PagedAttnArgs& a, int grid, cudaStream_t st) {
  auto* const kernel = paged_attn_q8_kernel<D, NT, E4M3, QF, TMA>;
  static std::atomic<uint64_t> allowed{0};  // the devices on which the kernel may use its shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Q8<D, NT>::SMEM, allowed);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_pdl(kernel, dim3(grid), kAllThreads, Q8<D, NT>::SMEM, st, a);
  if (e2 != cudaSuccess) return e2;
  PagedAttnArgs j = a;
  j.scale_log2 = 1.f;  // (the pieces' maxima are in log2 units)
  return launch_join<kTile, D>(j, grid, st);
}

template <int D, int NT, bool E4M3>
cudaError_t launch_q8_n(const PagedAttnArgs& a, bool q_f32, bool use_tma, int grid, cudaStream_t st) {
  if (q_f32) return use_tma ? launch_q8<D, NT, E4M3, true, true>(a, grid, st) : launch_q8<D, NT, E4M3, true, false>(a, grid, st);
  return use_tma ? launch_q8<D, NT, E4M3, false, true>(a, grid, st) : launch_q8<D, NT, E4M3, false, false>(a, grid, st);
}

}  // namespace

template <bool E4M3>
cudaError_t launch_q8_of(const PagedAttnArgs& a, int D, bool q_f32, bool use_tma, int grid, cudaStream_t st) {
  if (D == 64)
    return a.G <= 8 ? launch_q8_n<64, 1, E4M3>(a, q_f32, use_tma, grid, st) : launch_q8_n<64, 2, E4M3>(a, q_f32, use_tma, grid, st);
  return a.G <= 8 ? launch_q8_n<128, 1, E4M3>(a, q_f32, use_tma, grid, st) : launch_q8_n<128, 2, E4M3>(a, q_f32, use_tma, grid, st);
}

}  // namespace sfi

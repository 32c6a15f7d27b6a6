// RMS norm of each query and key head and its rotation by the position, in one
// pass over the rows.
//
//   n = x / sqrt(mean(x^2) + eps) * w;   (y_i, y_j) = (n_i cos a - n_j sin a, n_i sin a + n_j cos a)
//
// with a = position * inv_freq_i for the pair (i, j).  fp32 throughout, rounded once
// to the rows' type.
//
// The angle in turns is an integer product: inv_freq / 2 pi as a 64-bit fraction of a
// turn, times the position, modulo 2^64.  Wrapping around drops whole turns exactly, so
// a position of 2^30 has the angle of a near one (2^-34 turns), where pos * inv_freq in
// fp32 would be wrong by radians; the top 32 bits go to sincospi.
//
// A lane holds 4 + 4 elements of a head, both sides of its four pairs, so that nothing is
// exchanged but the sum of squares (d / 8 lanes a head), and reads and writes the same
// places, so that a call may work in place.  A row's warp computes its four angles once
// for all heads, and once for its query and its key heads the products of weight and cosine
// or sine, so that a head costs a factor and a rotation: with the weights read and applied head by
// head the instructions took longer than HBM, 67 us for 16384 rows of 32 + 8 heads of 128.
//
// Bound by HBM, 2 e d bytes a head.  Measured: those 16384 rows in bf16 (336 MB) in 58 us,
// 5.8 TB/s, call behind call, where a copy reaches 6.78; 5001 rows of 12 + 4 heads of 64 in fp32, half of them
// rotated (41 MB, which L2 holds), 9.7; 64 rows of 32 + 8 heads of 128 4.4, a launch and one dependent read.
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "pdl.cuh"
#include "rope.h"

namespace sfi {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // steps that a lane reads ahead

// Four elements as they lie in memory.
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  float4 v;
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ __forceinline__ void set(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Quad<bf16_t> {
  uint2 v;
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float (&x)[4]) { v = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }
};

// A lane's two quads as the first and the second elements of its four pairs, two pairs to a
// register, and back.
template <bool NEXT>
__device__ __forceinline__ void to_pairs(const float (&x)[4], const float (&y)[4], uint64_t (&u)[2], uint64_t (&v)[2]) {
  u[0] = NEXT ? pair(x[0], x[2]) : pair(x[0], x[1]), u[1] = NEXT ? pair(y[0], y[2]) : pair(x[2], x[3]);
  v[0] = NEXT ? pair(x[1], x[3]) : pair(y[0], y[1]), v[1] = NEXT ? pair(y[1], y[3]) : pair(y[2], y[3]);
}
template <bool NEXT>
__device__ __forceinline__ void from_pairs(const uint64_t (&u)[2], const uint64_t (&v)[2], float (&x)[4], float (&y)[4]) {
  if (NEXT) {
    x[0] = lo(u[0]), x[2] = hi(u[0]), y[0] = lo(u[1]), y[2] = hi(u[1]);
    x[1] = lo(v[0]), x[3] = hi(v[0]), y[1] = lo(v[1]), y[3] = hi(v[1]);
  } else {
    x[0] = lo(u[0]), x[1] = hi(u[0]), x[2] = lo(u[1]), x[3] = hi(u[1]);
    y[0] = lo(v[0]), y[1] = hi(v[0]), y[2] = lo(v[1]), y[3] = hi(v[1]);
  }
}

// The mean of a head's squares, over its d / 8 lanes.
template <int D>
__device__ __forceinline__ float mean_squares(const uint64_t (&xu)[2], const uint64_t (&xv)[2]) {
  const uint64_t q = fma2(xu[0], xu[0], fma2(xu[1], xu[1], fma2(xv[0], xv[0], mul2(xv[1], xv[1]))));
  float sum = lo(q) + hi(q);
#pragma unroll
  for (int w = 1; w < D / 8; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
  return sum * (1.f / D);
}

// Mean square + eps between which squares are safe: no element is above 2^54, and what its square
// loses below 2^-126 is less than 2^-26 of the sum.  Beyond, a warp squares its heads times a power of two
// again; a head's factor r then goes with elements that are scaled too, so that r itself stays
// a normal number: x / sqrt(v) = (x f) (r).  The heads beside keep their bits (f = 1).
constexpr float kLeast = 0x1p-100f, kMost = 0x1p100f;
template <int D>
__device__ __forceinline__ float far_norm(uint64_t (&xu)[2], uint64_t (&xv)[2], float v, float eps) {
  const bool large = !(v <= kMost);  // (NaN too)
  const float up = large ? 0x1p-96f : v < kLeast ? 0x1p96f : 1.f;
  const uint64_t uu = pair(up, up);
  const uint64_t su[2] = {mul2(xu[0], uu), mul2(xu[1], uu)}, sv[2] = {mul2(xv[0], uu), mul2(xv[1], uu)};
  const float z = mean_squares<D>(su, sv) + eps * up * up;
  const float r = z == 0.f ? 0.f : rsqrtf(z);  // (a head of zeros without eps stays one)
  const float f = large ? 0x1p-8f : up;
  const uint64_t ff = pair(f, f);
#pragma unroll
  for (int e = 0; e < 2; ++e) xu[e] = mul2(xu[e], ff), xv[e] = mul2(xv[e], ff);
  return large ? r * 0x1p-88f : r;
}

// FULL: all d dimensions are rotated.  CTAS: on an SM at least.
template <typename T, int D, bool NEXT, bool FULL, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPH = D / 8;        // lanes of a head
  constexpr int HPW = 32 / LPH;     // heads of a warp at a time
  __shared__ uint64_t freq[64];
  const int tid = threadIdx.x, lane = tid & 31, u = lane % LPH;
  if (tid < a.rot / 2) freq[tid] = a.freq[tid];
  pdl_launch();
  pdl_wait();
  __syncthreads();
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (tid >> 5);
  if (item >= (long long)a.total * a.parts) return;
  // (several parts only where there are few items)
  const int row = a.parts == 1 ? int(item) : int(uint32_t(item) / uint32_t(a.parts)), part = a.parts == 1 ? 0 : int(item) - row * a.parts;
  // the lane's elements: at and at + 4 .., or both sides of pairs that lie rot / 2 apart
  const bool turns = FULL || u < a.rot / 8;
  const int at0 = turns && !NEXT ? 4 * u : 8 * u, at1 = turns && !NEXT ? (FULL ? D / 2 : a.rot / 2) + 4 * u : 8 * u + 4;
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns) {
    const int64_t pos = int64_t(a.pos[row]) + a.pos_offset;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int32_t turn = int32_t((uint64_t(pos) * freq[4 * u + e]) >> 32);
      sincospif(float(turn) * 0x1p-31f, &s[e], &c[e]);
    }
  }
  // steps of HPW heads: those of q, then those of k
  const int q_steps = (a.H_q + HPW - 1) / HPW, steps = q_steps + (a.H_kv + HPW - 1) / HPW;
  const int from = steps * part / a.parts, to = steps * (part + 1) / a.parts;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int begin = max(from - (which ? q_steps : 0), 0), end = min(to, which ? steps : q_steps) - (which ? q_steps : 0);
    if (begin >= end) continue;
    const int heads = which ? a.H_kv : a.H_q;
    const T* const src = static_cast<const T*>(which ? a.k : a.q) + int64_t(row) * (which ? a.k_stride : a.q_stride);
    T* const dst = static_cast<T*>(which ? a.k_out : a.q_out) + int64_t(row) * (which ? a.k_out_stride : a.q_out_stride);
    // first = x wc - y ws', second = x ws + y wc' for a pair (x, y) of weights (w, w')
    uint64_t wc[2], ws[2], vc[2], vs[2];
    {
      float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
      const T* const w = static_cast<const T*>(which ? a.wk : a.wq);
      if (w) {
        reinterpret_cast<const Quad<T>*>(w + at0)->get(w0);
        reinterpret_cast<const Quad<T>*>(w + at1)->get(w1);
      }
      uint64_t wu[2], wv[2];
      to_pairs<NEXT>(w0, w1, wu, wv);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t ce = pair(c[2 * e], c[2 * e + 1]), se = pair(s[2 * e], s[2 * e + 1]);
        wc[e] = mul2(wu[e], ce), ws[e] = mul2(wu[e], se);
        vc[e] = mul2(wv[e], ce), vs[e] = mul2(wv[e], pair(-s[2 * e], -s[2 * e + 1]));
      }
    }
    const int head0 = lane / LPH;
#pragma unroll 1
    for (int i0 = begin; i0 < end; i0 += kAhead) {
      Quad<T> x0[kAhead], x1[kAhead];
      const int first = i0 * HPW + head0, n = min(end - i0, kAhead);
      const T* const x = src + first * D;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (j < n && first + j * HPW < heads) {
          x0[j] = *reinterpret_cast<const Quad<T>*>(x + j * HPW * D + at0);
          x1[j] = *reinterpret_cast<const Quad<T>*>(x + j * HPW * D + at1);
        }
      T* const y = dst + first * D;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j >= n) break;
        float p[4], o[4];
        x0[j].get(p), x1[j].get(o);
        uint64_t xu[2], xv[2], yu[2], yv[2];
        to_pairs<NEXT>(p, o, xu, xv);
        if (a.norm) {
          const float v = mean_squares<D>(xu, xv) + a.eps;
          float r = rsqrtf(v);
          if (__any_sync(kFull, !(v >= kLeast && v <= kMost))) r = far_norm<D>(xu, xv, v, a.eps);
          // (before the weights: their product with an element may be more than fp32 holds)
          const uint64_t rr = pair(r, r);
#pragma unroll
          for (int e = 0; e < 2; ++e) xu[e] = mul2(xu[e], rr), xv[e] = mul2(xv[e], rr);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          yu[e] = fma2(xu[e], wc[e], mul2(xv[e], vs[e]));
          yv[e] = fma2(xu[e], ws[e], mul2(xv[e], vc[e]));
          // (what is not rotated stays as it is, infinities among it)
          if (!FULL && !turns) yu[e] = mul2(xu[e], wc[e]), yv[e] = mul2(xv[e], vc[e]);
        }
        if (first + j * HPW >= heads) continue;
        from_pairs<NEXT>(yu, yv, p, o);
        Quad<T> v0, v1;
        v0.set(p), v1.set(o);
        *reinterpret_cast<Quad<T>*>(y + j * HPW * D + at0) = v0;
        *reinterpret_cast<Quad<T>*>(y + j * HPW * D + at1) = v1;
      }
    }
  }
}

template <typename T, int D, bool NEXT>
cudaError_t launch_t(RopeArgs a, cudaStream_t st) {
  // rows in abundance: a warp for each, which computes the angles once; few: their
  // heads over several warps
  constexpr int HPW = 256 / D;
  const int steps = (a.H_q + HPW - 1) / HPW + (a.H_kv + HPW - 1) / HPW;
  const long long want = 16LL * device_sm_count();
  a.parts = int(want / a.total < 1 ? 1 : want / a.total < steps ? want / a.total : steps);
  const long long items = (long long)a.total * a.parts;
  const dim3 grid(unsigned((items + kThreads / 32 - 1) / (kThreads / 32)));
  // bf16 rows are half as long, so more of them have to be on their way: in 64 registers 16384 rows
  // take 58 us and not 70, call behind call; fp32 rows 109 and not 102, and few rows 3.2 and not 2.8
  if (sizeof(T) == 2 && a.parts == 1)
    return a.rot == D ? launch_pdl(rope_kernel<T, D, NEXT, true, sizeof(T) == 2 ? 4 : 1>, grid, kThreads, 0, st, a)
                      : launch_pdl(rope_kernel<T, D, NEXT, false, sizeof(T) == 2 ? 4 : 1>, grid, kThreads, 0, st, a);
  return a.rot == D ? launch_pdl(rope_kernel<T, D, NEXT, true, 1>, grid, kThreads, 0, st, a)
                    : launch_pdl(rope_kernel<T, D, NEXT, false, 1>, grid, kThreads, 0, st, a);
}

template <typename T>
cudaError_t launch_d(const RopeArgs& a, int D, bool next, cudaStream_t st) {
  if (D == 64) return next ? launch_t<T, 64, true>(a, st) : launch_t<T, 64, false>(a, st);
  return next ? launch_t<T, 128, true>(a, st) : launch_t<T, 128, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int D, bool f32, bool next, cudaStream_t st) {
  return f32 ? launch_d<float>(a, D, next, st) : launch_d<bf16_t>(a, D, next, st);
}

}  // namespace sfi

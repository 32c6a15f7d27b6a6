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
// for all heads.  Bound by HBM: every row is read and written once.
#include <cuda_runtime.h>

#include "common.cuh"
#include "pdl.cuh"
#include "rope.h"

namespace sfi {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // heads that a lane reads ahead

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

template <typename T, int D, bool NEXT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
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
  const bool turns = u < a.rot / 8;
  const int at0 = turns && !NEXT ? 4 * u : 8 * u, at1 = turns && !NEXT ? a.rot / 2 + 4 * u : 8 * u + 4;
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns) {
    const int64_t pos = int64_t(a.pos[row]) + a.pos_offset;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int32_t turn = int32_t((uint64_t(pos) * freq[4 * u + e]) >> 32);
      sincospif(float(turn) * 0x1p-31f, &s[e], &c[e]);
    }
  }
  const int heads = a.H_q + a.H_kv;
  const int steps = (heads + HPW - 1) / HPW, from = steps * part / a.parts, to = steps * (part + 1) / a.parts;
  const T* const q = static_cast<const T*>(a.q) + int64_t(row) * a.q_stride;
  const T* const k = static_cast<const T*>(a.k) + int64_t(row) * a.k_stride;
  T* const qo = static_cast<T*>(a.q_out) + int64_t(row) * a.q_out_stride;
  T* const ko = static_cast<T*>(a.k_out) + int64_t(row) * a.k_out_stride;
  for (int i0 = from; i0 < to; i0 += kAhead) {
    Quad<T> x0[kAhead], x1[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = (i0 + j) * HPW + lane / LPH;
      if (i0 + j >= to || h >= heads) continue;
      const T* const x = h < a.H_q ? q + h * D : k + (h - a.H_q) * D;
      x0[j] = *reinterpret_cast<const Quad<T>*>(x + at0);
      x1[j] = *reinterpret_cast<const Quad<T>*>(x + at1);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = (i0 + j) * HPW + lane / LPH;
      if (i0 + j >= to) break;
      const bool there = h < heads, is_q = h < a.H_q;
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
      if (there) x0[j].get(x), x1[j].get(y);
      if (a.norm) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
        for (int w = 1; w < LPH; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
        const float r = rsqrtf(sum * (1.f / D) + a.eps);
        const T* const w = static_cast<const T*>(is_q ? a.wq : a.wk);
        float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
        if (w) {
          reinterpret_cast<const Quad<T>*>(w + at0)->get(w0);
          reinterpret_cast<const Quad<T>*>(w + at1)->get(w1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= r * w0[e], y[e] *= r * w1[e];
      }
      float p[4], o[4];
      if (NEXT) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[2 * e] = x[2 * e] * c[e] - x[2 * e + 1] * s[e];
          p[2 * e + 1] = x[2 * e] * s[e] + x[2 * e + 1] * c[e];
          o[2 * e] = y[2 * e] * c[2 + e] - y[2 * e + 1] * s[2 + e];
          o[2 * e + 1] = y[2 * e] * s[2 + e] + y[2 * e + 1] * c[2 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = x[e] * c[e] - y[e] * s[e];
          o[e] = x[e] * s[e] + y[e] * c[e];
        }
      }
      // (what is not rotated stays as it is, infinities among it)
      if (!turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = x[e], o[e] = y[e];
      }
      if (!there) continue;
      T* const to_ = is_q ? qo + h * D : ko + (h - a.H_q) * D;
      Quad<T> v0, v1;
      v0.set(p), v1.set(o);
      *reinterpret_cast<Quad<T>*>(to_ + at0) = v0;
      *reinterpret_cast<Quad<T>*>(to_ + at1) = v1;
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(RopeArgs a, bool next, cudaStream_t st) {
  // rows in abundance: a warp for each, which computes the angles once; few: their
  // heads over several warps
  const int steps = (a.H_q + a.H_kv + 256 / D - 1) / (256 / D);
  const long long want = 16LL * device_sm_count();
  a.parts = int(want / a.total < 1 ? 1 : want / a.total < steps ? want / a.total : steps);
  const long long items = (long long)a.total * a.parts;
  const dim3 grid(unsigned((items + kThreads / 32 - 1) / (kThreads / 32)));
  return next ? launch_pdl(rope_kernel<T, D, true>, grid, kThreads, 0, st, a)
              : launch_pdl(rope_kernel<T, D, false>, grid, kThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int D, bool f32, bool next, cudaStream_t st) {
  if (D == 64) return f32 ? launch_t<float, 64>(a, next, st) : launch_t<bf16_t, 64>(a, next, st);
  return f32 ? launch_t<float, 128>(a, next, st) : launch_t<bf16_t, 128>(a, next, st);
}

}  // namespace sfi

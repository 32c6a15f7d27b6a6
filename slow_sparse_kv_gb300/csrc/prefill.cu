// Causal attention over packed prompts (bf16, grouped heads) on the
// fifth-generation tensor cores.
//
// One CTA takes 2 x 128 query rows of one (sequence, KV head); a row is one
// (token, query head of the group), so a tile holds 128 / G tokens times the G
// heads that share the KV head, and K and V are read once for all of them.
// For each block of 128 keys: S = Q K^T (tcgen05.mma from shared memory into
// tensor memory), softmax statistics with one thread per row, P in bf16 over
// S's columns in tensor memory, O += P V (P from tensor memory).  The two
// tiles alternate: while one's softmax runs, the tensor cores work on the
// other's products.  Tensor memory: S0/P0, S1/P1, O0, O1 (4 x 128 columns).
//
// Bound by the tensor cores (4 d flops per row and visible key) as long as the
// exponentials keep up: 2 x 128 x 128 of them per 2 x 2 x 128 x 128 x d MACs.
//
// Online softmax: out = sum_j 2^(c (s_j - m)) v_j / sum_j 2^(c (s_j - m)) with
// c = log2(e) / sqrt(d) holds for any m, so m only follows the row maximum when
// that has grown by more than 8 in the exponent (P then stays below 2^8, fp32
// sums far from overflow, bf16's relative rounding the same); O is rescaled in
// tensor memory only then.
#include <cuda_runtime.h>

#include "prefill.h"
#include "tc5.cuh"

namespace sfi {
namespace {

constexpr int kThreads = 384;  // 2 softmax warpgroups; a load warp, an MMA warp and two idle ones
// Registers a thread: launched with 168 (64512 in all); the softmax threads
// hold a whole row of scores, the third warpgroup gives up what they take
// (128 * (2 * 208 + 88) = 64512).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kRows = 128;     // query rows per tile
constexpr int kKeys = 128;     // keys per block
constexpr float kGrow = 8.0f;  // growth of the maximum (log2) that moves m

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t TILE = kRows * 128 * HALVES;  // bytes of a 128-row tile
  static constexpr int STAGES = D == 128 ? 4 : 6;         // K and V blocks in flight
  static constexpr uint32_t SMEM = 1024 + (2 + STAGES) * TILE;
};

struct Shared {
  uint64_t q_full[2], s_full[2], p_ready[2][2], kv_full[6], kv_empty[6], v_clean, drained;
  uint32_t tmem;
  volatile int abort;
  int b, tile;
  int span[kMaxBatch];  // CTAs (tile pairs) of each sequence
  int lvl[kMaxBatch];   // its first one's level
};

// Bounded wait; false (and the CTA's abort flag and the status bit set) after
// `limit` clocks, false at once when another thread gave up.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Shared& sh, uint32_t* status,
                                     long long limit) {
  if (mbar_test_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (sh.abort) return false;
    if (clock64() - t0 > limit) {
      sh.abort = 1;
      set_status(status, SFI_DEV_WAIT_TIMEOUT);
      return false;
    }
    if (mbar_try_wait(bar, parity)) return true;
  }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float lo(uint64_t p) { return __uint_as_float(uint32_t(p)); }
__device__ __forceinline__ float hi(uint64_t p) { return __uint_as_float(uint32_t(p >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}

// Keeps uses of registers that a tcgen05.ld fills behind its wait.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Tiles of a level tau or above, over all sequences (one warp): sequence b has
// its tiles at levels lvl[b] .. lvl[b] + span[b] - 1.
__device__ __forceinline__ int tiles_from(const Shared& sh, int B, int tau) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < B; b += 32)
    n += min(max(sh.lvl[b] + sh.span[b] - tau, 0), sh.span[b]);
  return __reduce_add_sync(kFull, n);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.H_kv;
  const int rank = blockIdx.x / a.H_kv;

  // Which tile: levels stand for the keys that a tile sees (in units of its
  // tokens); the CTAs take them from the highest down, so that the long ones
  // start first.
  const int span_tok = 2 * a.tok;
  for (int b = tid; b < a.B; b += kThreads) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    const bool ok = q0 >= 0 && q0 <= q1 && q1 <= a.total_q && k0 >= 0 && k0 <= k1 && k1 <= a.total_k;
    if (!ok && blockIdx.x == 0) set_status(a.status, SFI_DEV_LEN_OVER_CAP);
    sh.span[b] = ok ? (q1 - q0 + span_tok - 1) / span_tok : 0;
    sh.lvl[b] = ok ? max(0, (k1 - k0) - (q1 - q0)) / span_tok : 0;
  }
  if (tid == 0) {
    sh.abort = 0;
    sh.b = -1;
  }
  __syncthreads();
  if (warp == 0) {
    int top = 0;
    for (int b = lane; b < a.B; b += 32) top = max(top, sh.span[b] > 0 ? sh.lvl[b] + sh.span[b] : 0);
    top = __reduce_max_sync(kFull, top);
    if (rank < tiles_from(sh, a.B, 0)) {
      // the level with tiles_from(tau + 1) <= rank < tiles_from(tau)
      int lo = 0, hi = top;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_from(sh, a.B, mid) > rank) lo = mid;
        else hi = mid;
      }
      int left = rank - tiles_from(sh, a.B, lo + 1);
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        const bool in = b < a.B && sh.lvl[b] <= lo && lo < sh.lvl[b] + sh.span[b];
        const uint32_t m = __ballot_sync(kFull, in);
        if (left < __popc(m)) {
          if (in && __popc(m & ((1u << lane) - 1)) == left) {
            sh.b = b;
            sh.tile = lo - sh.lvl[b];
          }
          break;
        }
        left -= __popc(m);
      }
    }
  } else if (warp == 9) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_addr(&sh.q_full[i]), 1);
        mbar_init(smem_addr(&sh.s_full[i]), 1);
        for (int h = 0; h < 2; ++h) mbar_init(smem_addr(&sh.p_ready[i][h]), 128);
      }
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(smem_addr(&sh.kv_full[i]), 1);
        mbar_init(smem_addr(&sh.kv_empty[i]), 1);
      }
      mbar_init(smem_addr(&sh.v_clean), 1);
      mbar_init(smem_addr(&sh.drained), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tc5::alloc(smem_addr(&sh.tmem), 512);
    tc5::fence_before();
  }
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = sh.tmem;

  if (sh.b >= 0) {
    const int b = sh.b;
    const int q0 = a.cu_q[b], nq = a.cu_q[b + 1] - q0;
    const int k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0;
    const int off = nk - nq;
    const int t0 = sh.tile * span_tok;
    int n_it[2];  // key blocks of each tile
    for (int i = 0; i < 2; ++i) {
      const int first = t0 + i * a.tok, last = min(first + a.tok, nq);
      n_it[i] = first < nq ? (max(0, min(off + last, nk)) + kKeys - 1) / kKeys : 0;
    }
    const int n = max(n_it[0], n_it[1]);
    const uint32_t q_sm = base, kv_sm = base + 2 * C::TILE;
    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == 8) {
        // ---- loads: Q once, then K_0, V_0, K_1, V_1, ... through the ring
        int issued = 0;
        bool ok = true;
        if (lane == 0) {
          for (int i = 0; i < 2; ++i) {
            if (n_it[i] == 0) continue;
            const uint32_t bar = smem_addr(&sh.q_full[i]);
            mbar_arrive_expect_tx(bar, uint32_t(a.tok * a.G) * 128 * C::HALVES);
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_3d(q_sm + i * C::TILE + h * (kRows * 128), &a.tmq, h * 64, g * a.G,
                          q0 + t0 + i * a.tok, bar);
          }
          for (; issued < 2 * n; ++issued) {
            const int st = issued % C::STAGES, use = issued / C::STAGES;
            if (use > 0) ok = wait(smem_addr(&sh.kv_empty[st]), (use - 1) & 1, sh, a.status, a.wait_cycles);
            if (!ok) break;
            const uint32_t bar = smem_addr(&sh.kv_full[st]);
            mbar_arrive_expect_tx(bar, C::TILE);
            const void* map = (issued & 1) ? &a.tmv : &a.tmk;
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_3d(kv_sm + st * C::TILE + h * (kKeys * 128), map, h * 64, g,
                          k0 + (issued >> 1) * kKeys, bar);
          }
        }
        issued = __shfl_sync(kFull, issued, 0);
        // no copy may be in flight when the CTA exits (after a wait that gave
        // up, some may never have been waited for)
        bool landed = true;
        for (int i = 0; i < 2; ++i)
          if (n_it[i] > 0) landed = mbar_wait(smem_addr(&sh.q_full[i]), 0) && landed;
        for (int x = max(0, issued - C::STAGES); x < issued; ++x)
          landed = mbar_wait(smem_addr(&sh.kv_full[x % C::STAGES]), (x / C::STAGES) & 1) && landed;
        if (issued == 2 * n && n * kKeys > nk && __all_sync(kFull, landed)) {
          // the rows of the last V block behind the sequence belong to nobody or
          // to the next one: P is zero there, but 0 * NaN is not
          const uint32_t v_sm = kv_sm + (2 * n - 1) % C::STAGES * C::TILE;
          for (int y = (nk - (n - 1) * kKeys) * 8 + lane; y < kKeys * 8; y += 32)
            for (int h = 0; h < C::HALVES; ++h)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_sm + h * (kKeys * 128) + y * 16), "r"(0)
                           : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.v_clean));
        }
      } else if (warp == 9) {
        // ---- products, all of them from one lane: a warp-wide vote or
        // __syncwarp between MMAs costs more than their issue
        if (tc5::elect()) {
          constexpr uint32_t kIdS = tc5::idesc_bf16(kRows, kKeys, false);
          constexpr uint32_t kIdO = tc5::idesc_bf16(kRows, D, true);
          auto full = [&](int x) {  // block x of the ring (K_j: 2j, V_j: 2j + 1) has landed
            return wait(smem_addr(&sh.kv_full[x % C::STAGES]), (x / C::STAGES) & 1, sh, a.status, a.wait_cycles);
          };
          auto release = [&](int x) { tc5::commit(smem_addr(&sh.kv_empty[x % C::STAGES])); };
          auto scores = [&](int i, int x) {  // S_i = Q_i K^T
            const uint64_t qd = tc5::desc_sw128(q_sm + i * C::TILE, 16, 1024);
            const uint64_t kd = tc5::desc_sw128(kv_sm + (x % C::STAGES) * C::TILE, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t at = ((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4;
              tc5::mma_ss(tmem + i * 128, qd + at, kd + at, kIdS, kk > 0);
            }
            tc5::commit(smem_addr(&sh.s_full[i]));
          };
          bool ok = n == 0 || full(0);
          for (int i = 0; i < 2 && ok; ++i) {
            if (n_it[i] == 0) continue;
            ok = wait(smem_addr(&sh.q_full[i]), 0, sh, a.status, a.wait_cycles);
            if (ok) scores(i, 0);
          }
          if (ok && n > 0) release(0);
          for (int j = 0; j < n && ok; ++j) {
            ok = (j + 1) * kKeys > nk ? wait(smem_addr(&sh.v_clean), 0, sh, a.status, a.wait_cycles) : full(2 * j + 1);
            if (!ok) break;
            const uint64_t vd = tc5::desc_sw128(kv_sm + ((2 * j + 1) % C::STAGES) * C::TILE, kKeys * 128, 1024);
            for (int i = 0; i < 2 && ok; ++i) {
              if (j >= n_it[i]) continue;
              for (int h = 0; h < 2; ++h) {  // O_i += P_i V, the halves of P as they come
                ok = wait(smem_addr(&sh.p_ready[i][h]), j & 1, sh, a.status, a.wait_cycles);
                if (!ok) break;
                tc5::fence_after();
#pragma unroll
                for (int kk = 0; kk < kKeys / 32; ++kk) {
                  const int k16 = h * (kKeys / 32) + kk;
                  tc5::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k16 * 8, vd + k16 * (2048 >> 4), kIdO, j > 0 || k16 > 0);
                }
              }
              if (!ok) break;
              if (j + 1 < n_it[i]) {
                ok = full(2 * j + 2);
                if (ok) scores(i, 2 * j + 2);
              } else {
                tc5::commit(smem_addr(&sh.s_full[i]));  // O_i is complete
              }
            }
            if (!ok) break;
            release(2 * j + 1);
            if (j + 1 < n) release(2 * j + 2);
          }
          // the products in flight end before tensor memory is freed, whether or
          // not a softmax warp still waits for them
          tc5::commit(smem_addr(&sh.drained));
          mbar_wait(smem_addr(&sh.drained), 0);
        }
        __syncwarp();
      }
    } else {
      // ---- softmax and output of tile i: one thread per row
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
      const int i = warp >> 2;
      const int r = tid & 127;
      const int tt = r / a.G;
      const int t = t0 + i * a.tok + tt;
      const bool valid = tt < a.tok && t < nq;
      const int limit = valid ? max(0, min(off + t + 1, nk)) : 0;  // keys this row sees
      const int open = max(0, min(off + t0 + i * a.tok + 1, nk));  // keys every valid row sees
      const uint32_t lanes = uint32_t(warp & 3) << 21;             // 32 * (warp % 4) in the lane field
      const uint32_t s_tm = tmem + i * 128 + lanes, o_tm = tmem + 256 + i * 128 + lanes;
      const uint32_t s_bar = smem_addr(&sh.s_full[i]), p_bar = smem_addr(&sh.p_ready[i][0]);
      const float c = a.scale_log2;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < n_it[i]; ++j) {
        ok = __all_sync(kFull, wait(s_bar, j & 1, sh, a.status, a.wait_cycles));
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
            const float f = grow ? ex2((m - top) * c) : 1.f;
            if (grow) m = top;
            l *= f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              uint32_t o[32];
              tc5::ld32(o_tm + 32 * x, o);
              tc5::wait_ld();
              pin(o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc5::st32(o_tm + 32 * x, o);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : -m * c;
        const uint64_t cc = pair(c, c), mm = pair(mc, mc);
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int x = 32 * h; x < 32 * h + 32; ++x) {
            uint64_t y = pair(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]));
            y = fma2(y, cc, mm);
            const float p0 = ex2(lo(y)), p1 = ex2(hi(y));
            sum[x & 3] = add2(sum[x & 3], pair(p0, p1));
            s[x] = pack_bf16x2(p0, p1);
          }
          tc5::st32(s_tm + 32 * h, s + 32 * h);
          tc5::wait_st();
          tc5::fence_before();
          mbar_arrive(p_bar + 8 * h);
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += lo(sum[0]) + hi(sum[0]);
      }
      if (ok && n_it[i] > 0)
        ok = __all_sync(kFull, wait(s_bar, n_it[i] & 1, sh, a.status, a.wait_cycles));
      if (ok) {
        tc5::fence_after();
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
        const int h = g * a.G + r - tt * a.G;
        const int64_t row = int64_t(q0) + t;
        uint8_t* dst = static_cast<uint8_t*>(a.out) + 2 * (row * a.out_stride + int64_t(h) * D);
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          uint32_t o[32];
          if (n_it[i] > 0) {
            tc5::ld32(o_tm + 32 * x, o);
            tc5::wait_ld();
            pin(o);
          } else {
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = 0;
          }
          if (valid) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              uint4 w;
              w.x = pack_bf16x2(__uint_as_float(o[y]) * inv, __uint_as_float(o[y + 1]) * inv);
              w.y = pack_bf16x2(__uint_as_float(o[y + 2]) * inv, __uint_as_float(o[y + 3]) * inv);
              w.z = pack_bf16x2(__uint_as_float(o[y + 4]) * inv, __uint_as_float(o[y + 5]) * inv);
              w.w = pack_bf16x2(__uint_as_float(o[y + 6]) * inv, __uint_as_float(o[y + 7]) * inv);
              if (limit == 0) w = make_uint4(0, 0, 0, 0);  // no key: O was never written for it alone
              *reinterpret_cast<uint4*>(dst + 2 * (32 * x + y)) = w;
            }
          }
        }
        if (valid && a.lse)
          a.lse[row * a.H_q + h] = limit == 0 ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
      }
      tc5::fence_before();
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc5::fence_after();
    tc5::dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(Cfg<D>::SMEM));
  if (e != cudaSuccess) return e;
  // sum_b ceil(n_b / span) <= total / span + B
  const long long tiles = (long long)a.total_q / (2 * a.tok) + a.B;
  prefill_kernel<D><<<unsigned(tiles * a.H_kv), kThreads, Cfg<D>::SMEM, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, int D, cudaStream_t st) {
  return D == 64 ? launch_t<64>(a, st) : launch_t<128>(a, st);
}

}  // namespace sfi

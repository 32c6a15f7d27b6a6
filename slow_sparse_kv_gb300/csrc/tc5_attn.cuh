// What the attentions on the fifth-generation tensor cores have in common: bounded
// waits, loads by maps, and the softmax threads' dealings with tensor memory.
#pragma once

#include "common.cuh"
#include "tc5.cuh"

namespace sfi {
namespace {

// Bounded wait; false (and the CTA's abort flag and the status bit set) after
// `limit` clocks, false at once when another thread gave up.
template <typename Shared>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Shared& sh, uint32_t* status, long long limit) {
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

// Store a part of P and tell the MMA lane.
template <typename Store>
__device__ __forceinline__ void hand_over(uint32_t bar, Store store) {
  store();
  tc5::wait_st();
  tc5::fence_before();
  mbar_arrive(bar);
}

// Keeps uses of registers that a tcgen05.ld fills behind its wait.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

}  // namespace
}  // namespace sfi

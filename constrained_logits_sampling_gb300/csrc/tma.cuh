// What the attention kernels need of TMA tensor copies and of mbarriers beyond bulk_copy.cuh.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "bulk_copy.cuh"

namespace clsample {

// One look at a phase, without the pause that a poll may make.
__device__ __forceinline__ bool mbar_test_wait(unsigned long long* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// One box of a tensor map of rank 3 to shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int head, int token,
                                          unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(token), "r"(smem_addr(bar))
      : "memory");
}

// One box of a tensor map of rank 4 to shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int slot, int head, int page,
                                          unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
      : "memory");
}

// What the bounded waits of a CTA share: the cycles that one may take, and whether one has run
// out, after which the others end too.
struct WaitLimit {
  long long cycles;
  volatile int dead;
};
constexpr long long kWaitCycles = 4000000000ll;  // about two seconds

// Bounded wait for a phase: false if it ran out.  (A later wait of the same thread for the next
// phase of that barrier would seem to succeed at once, so nothing may rest on one.)
__device__ __forceinline__ bool bounded_wait(unsigned long long* bar, uint32_t parity, WaitLimit* limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (limit->dead || clock64() - start > limit->cycles) break;
  }
  limit->dead = 1;
  return false;
}
// The same by a whole warp, whose lanes go on together and agree.
__device__ __forceinline__ bool warp_wait(unsigned long long* bar, uint32_t parity, WaitLimit* limit) {
  return __all_sync(~0u, bounded_wait(bar, parity, limit));
}

}  // namespace clsample

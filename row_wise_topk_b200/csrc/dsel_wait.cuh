// mbarriers in shared memory, and a bounded wait of a whole warp for one.
#pragma once

#include <cstdint>

#include "dsel_ops.cuh"

namespace dsel {

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// A whole warp's wait for the phase `parity` of a barrier: false, with DSEL_ERR_DEVICE_TIMEOUT in *status, after
// limit_ns.  What follows a wait are instructions of the whole warp (votes, shuffles, tensor memory reads), which lanes
// that disagree would never finish.  So the lanes vote on both answers and leave together: complete when each
// has seen the phase end (it lasts until this warp goes on), given up when any is late and not all have.
static __device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, uint64_t limit_ns, int* status) {
  const uint64_t t0 = now_ns();
  while (!__all_sync(0xFFFFFFFFu, bar_try(bar, parity))) {
    if (__any_sync(0xFFFFFFFFu, now_ns() - t0 > limit_ns)) {
      atomicExch(status, DSEL_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, int* status) {
  return __all_sync(0xFFFFFFFFu, bar_try(bar, parity)) || warp_wait_slow(bar, parity, limit_ns, status);
}

}  // namespace dsel

// Test build of the bounded wait: one block of two warps.  Warp 0 waits for a barrier, lane i
// with a limit of limit_ns + i * skew_ns of its own; warp 1 arrives after delay_ns (0: never).
// out[0], out[1]: which lanes of warp 0 saw the phase end in two waits for it, out[2]: the status word.
#include <cstdint>

#include <cuda_runtime.h>

#include "dsel_wait.cuh"

namespace {

__global__ void probe(uint64_t delay_ns, uint64_t limit_ns, uint64_t skew_ns, uint32_t* out, int* status) {
  __shared__ __align__(8) uint64_t word;
  const uint32_t bar = dsel::shared_addr(&word);
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  if (threadIdx.x == 0) dsel::bar_init(bar, 1);
  __syncthreads();
  if (warp == 0) {
    const uint64_t limit = limit_ns + uint64_t(lane) * skew_ns;
    const bool first = dsel::warp_wait(bar, 0, limit, status);
    const uint32_t a = __ballot_sync(0xFFFFFFFFu, first);
    const bool second = dsel::warp_wait(bar, 0, limit, status);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, second);
    if (lane == 0) {
      out[0] = a;
      out[1] = b;
    }
  } else if (delay_ns > 0 && lane == 0) {
    const uint64_t t0 = dsel::now_ns();
    for (int i = 0; i < 100000 && dsel::now_ns() - t0 < delay_ns; ++i) __nanosleep(1000);
    dsel::bar_arrive(bar);
  }
  __syncthreads();   // (the barrier's memory outlives both warps' use)
  if (threadIdx.x == 0) out[2] = uint32_t(*reinterpret_cast<volatile int*>(status));
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int wait_probe(uint64_t delay_ns, uint64_t limit_ns, uint64_t skew_ns,
                                                               uint32_t* host_out) {
  uint32_t* d = nullptr;
  if (cudaMalloc(&d, 16) != cudaSuccess || cudaMemset(d, 0, 16) != cudaSuccess) return 1;
  probe<<<1, 64>>>(delay_ns, limit_ns, skew_ns, d, reinterpret_cast<int*>(d + 3));
  const bool ok = cudaMemcpy(host_out, d, 12, cudaMemcpyDeviceToHost) == cudaSuccess;
  cudaFree(d);
  return ok ? 0 : 2;
}

// Shared by the operators around the TopK (logits processing, indexer scores,
// sparse attention): launch helpers and thin PTX wrappers.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "dsel_plan.h"   // the C ABI (include/dsel.h) and the shape limits

namespace dsel {

// ---- host ----

// The current device, an sm_100 GPU, and its SM count (asked of the runtime once per device).
inline int current_device(int* device, int* sms) {
  static std::atomic<int> known[64];   // SM count, 0: not asked yet; every thread stores the same value
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSEL_ERR_CUDA;
  if (dev < 0 || dev >= 64) return DSEL_ERR_DEVICE;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return DSEL_ERR_CUDA;
    if (major != 10 || minor != 0) return DSEL_ERR_DEVICE;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *device = dev;
  *sms = n;
  return DSEL_OK;
}

// Lets a kernel use `bytes` of dynamic shared memory on device `dev`; `done` is the kernel's
// own flag word (one bit per device), so that the runtime is asked once.
inline cudaError_t allow_smem(const void* kern, int bytes, int dev, std::atomic<uint64_t>* done) {
  const uint64_t bit = uint64_t(1) << dev;
  if ((done->load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch in clusters of `cluster` CTAs that may begin while the launch before it
// still runs: the kernel calls grid_wait() before it touches global memory.
template <typename Kern, typename Params>
cudaError_t launch_dependent(Kern kern, unsigned grid, int threads, int cluster, uint32_t smem, cudaStream_t st,
                             const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Whether [a, a + na * ea) and [b, b + nb * eb) share a byte.
inline bool ranges_meet(const void* a, int64_t na, int ea, const void* b, int64_t nb, int eb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + uintptr_t(nb) * uintptr_t(eb) && pb < pa + uintptr_t(na) * uintptr_t(ea);
}

// Reads and clears the status word of the score kernel's bounded waits (asynchronous on `st`).
int score_status(int* out, cudaStream_t st);

// ---- device ----

// The launches before this one in the stream are complete and visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next launch may start its set-up.
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared, asynchronous; zeros where !live (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread are complete.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace dsel

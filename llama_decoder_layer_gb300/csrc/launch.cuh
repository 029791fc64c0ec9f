// Host-side kernel launch with an optional programmatic dependency on the
// kernel before it on the stream (see pdl_wait / pdl_trigger in common.cuh).
// The first kernel of a public call is launched without it, so it starts only
// after everything the caller queued earlier has completed (but for the calls
// whose first kernel touches nothing before its pdl_wait); the kernels after
// it in the same call overlap their prologues (barrier setup, tensor-memory
// allocation, weight prefetch) with the tail of their predecessor.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>
#include <utility>

namespace llama {

// Kernels this process has launched through the library (every device);
// read by llama_launch_count().
extern std::atomic<unsigned long long> g_launch_count;

inline cudaError_t counted(cudaError_t e) {
  if (e == cudaSuccess) g_launch_count.fetch_add(1, std::memory_order_relaxed);
  return e;
}

// A kernel and the dynamic shared memory it is launched with.
struct SmemNeed {
  const void* kernel;
  size_t bytes;
};
template <typename... KArgs>
SmemNeed smem_need(void (*kernel)(KArgs...), size_t bytes) {
  return {reinterpret_cast<const void*>(kernel), bytes};
}

// Raises the dynamic shared-memory limit of a set of kernels, once on every
// device: the limit is the current device's, so a flag for the whole process
// would leave the others without it.  An error is not kept: the next call tries
// again.  (Two threads may both do it; the limits are the same.)
class SmemLimits {
 public:
  cudaError_t raise(std::initializer_list<SmemNeed> needs) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevs;
    if (known && done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    for (const SmemNeed& n : needs) {
      e = cudaFuncSetAttribute(n.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(n.bytes));
      if (e != cudaSuccess) return e;
    }
    if (known) done_[dev].store(true, std::memory_order_release);
    return cudaSuccess;
  }

 private:
  static constexpr int kDevs = 64;
  std::atomic<bool> done_[kDevs] = {};
};

template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool pdl,
                          Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return counted(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

// The same, for a kernel launched in thread-block clusters of cluster_x CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                  bool pdl, int cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster_x);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

}  // namespace llama

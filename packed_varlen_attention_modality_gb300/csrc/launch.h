// Kernel launch helpers shared by the kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <utility>

namespace h3 {

// Launch with programmatic stream serialization: the kernel may be scheduled while the previous
// kernel in the stream finishes (it calls grid_dependency_wait() before reading that kernel's
// results), which hides the launch latency between the plan, attention and merge kernels.
template <typename... Params, typename... Args>
inline cudaError_t launch_programmatic(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline int num_sms_of_current_device() {
  static std::atomic<int> cached[64];  // 0 until looked up; racing lookups store the same value
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Opt a kernel in to kBytes of dynamic shared memory, once per device (a racing second call is
// harmless).
template <int kBytes, typename K>
inline cudaError_t allow_shared_memory(K* kernel) {
  static std::atomic<K*> done[64][2];  // kernels of one type (one per head_dim) at most
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  for (auto& d : done[dev])
    if (d.load(std::memory_order_acquire) == kernel) return cudaSuccess;
  const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (s != cudaSuccess) return s;
  for (auto& d : done[dev]) {
    K* none = nullptr;
    if (d.compare_exchange_strong(none, kernel, std::memory_order_acq_rel) || none == kernel) break;
  }
  return cudaSuccess;
}

}  // namespace h3

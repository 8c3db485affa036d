// kv_launch.h -- launches of the key/value cache's kernels.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace qmm {

// One launch that may begin while the kernel before it ends (each kernel waits for it before its first access).
template <class P>
inline cudaError_t launch_after(void (*kern)(P), int64_t grid, int threads, size_t smem, cudaStream_t s, const P &p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The same for a kernel with more than 48 KB of dynamic shared memory, always as much.  `set_for` (one a kernel) has the
// device, plus 1, that its limit was raised on.
template <class P>
inline cudaError_t launch_large(void (*kern)(P), int64_t grid, int threads, size_t smem, cudaStream_t s, const P &p,
                                std::atomic<int> &set_for) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool set = set_for.load(std::memory_order_relaxed) == dev + 1;
  for (int pass = 0;; pass++) {
    if (!set || pass > 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      set_for.store(dev + 1, std::memory_order_relaxed);
    }
    e = launch_after(kern, grid, threads, smem, s, p);
    // the limit may have been lost with the context (a device reset): once more, with it raised again
    if (!(e == cudaErrorInvalidValue && set && pass == 0)) return e;
    (void)cudaGetLastError();
  }
}

}  // namespace qmm

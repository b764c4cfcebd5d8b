// Launches of a kernel that follows another of the same call on the same stream: its blocks may be brought up
// while the last blocks of the one before still run, and await_previous() is where they wait for its results.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <utility>

#include "ttl_internal.h"

namespace ttl {

// Every thread of the following kernel calls this before it reads what the kernel before wrote, and before it
// writes anything that kernel may still read.
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the following kernel's blocks be brought up from here on, where there is room for them; what they read still waits
// for await_previous().
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch that begins when all before it is done: for the first kernel of a call, which knows nothing of the caller's.
template <typename... Params, typename... Args>
cudaError_t launch_first(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                         Args&&... args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(block);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  return cudaLaunchKernelEx(&config, kernel, std::forward<Args>(args)...);
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                         Args&&... args) {
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(block);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &overlap;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, std::forward<Args>(args)...);
}

// Raises a kernel's dynamic shared-memory limit to `bytes`, once per device (thread-safe).
template <auto Kernel>
int allow_smem(size_t bytes, const char* what) {
  static std::mutex mu;
  static size_t done[64] = {};
  int dev = 0;
  int rc = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc || bytes <= 40 * 1024) return rc;   // (the limit of 48 KiB counts the static arrays too)
  if (dev < 0 || dev >= 64) return set_error(TTL_ERR_CUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev] >= bytes) return TTL_OK;
  rc = cuda_check(cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes)),
                  what);
  if (!rc) done[dev] = bytes;
  return rc;
}

}  // namespace ttl

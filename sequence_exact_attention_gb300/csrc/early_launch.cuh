// Programmatic dependent launch: a grid that may start while the one before it
// on the stream is still running.
#pragma once

#include <utility>

#include <cuda_runtime.h>

namespace ra {

// The next grid on the stream, if it was launched early, may start once every
// CTA of this one has said so or has left.
__device__ __forceinline__ void let_dependents_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Waits until the grid before this one has ended and its writes are visible.
// An early grid calls it before it reads what that one wrote, or, where it
// reads nothing of it, before it ends, so that its own end means both.
__device__ __forceinline__ void wait_for_prior_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a grid early; false on error.
template <class... Params, class... Args>
bool launch_early(void (*kernel)(Params...), long long grid, int block, int smem,
                  cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, Params(std::forward<Args>(args))...) == cudaSuccess)
    return true;
  cudaGetLastError();
  return false;
}

}  // namespace ra

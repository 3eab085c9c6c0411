// Kernels that are set up while the kernel in front of them on the stream still runs.
#pragma once

#include <cuda_runtime.h>

namespace sparge {

// ------------------------------------------------------------------------------------------
// Programmatic dependent launch.  A kernel launched with launch_dependent may be set up while the kernel in
// front of it on the stream still runs; wait_for_earlier() then holds every thread until that one has
// completed and its writes are visible.  Every thread of the kernel calls it before it reads or
// writes global memory, and none returns without it, so the order along the stream is whole.
// let_dependents_start() allows the same to the kernel behind this one.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                                    const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sparge

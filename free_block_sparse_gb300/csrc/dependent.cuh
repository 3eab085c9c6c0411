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
// What the kernel in front may have written is read with ordinary loads: the non-coherent ones (__ldg, ld.global.nc) want data
// that nothing writes while the kernel lives, and it lives from before that write.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 16 bytes that are read once: past the L1 cache
__device__ __forceinline__ uint4 ld_once_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

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

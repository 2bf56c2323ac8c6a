// ra_launch.cuh -- kernels of one call that follow each other by programmatic
// dependent launch.
#pragma once
#include <cuda_runtime.h>

namespace ra {

// The kernels of one call follow each other without waiting for the last CTA
// of the one before to leave (programmatic dependent launch): the next grid's
// CTAs take the SMs that become free, prepare, and wait here for the results.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... Params, class... Args>
cudaError_t launch_after(bool overlap, void (*kern)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                         Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace ra

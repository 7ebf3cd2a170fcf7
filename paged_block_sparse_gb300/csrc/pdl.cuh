// Two launches of one call, the second's CTAs resident before the first has ended (programmatic dependent
// launch): saves the second's launch latency (2-4 us). The first kernel calls pdl_release() when it starts,
// the second pdl_wait() before it touches anything the first writes (plain loads: not the read-only path).
#pragma once

#include <cuda_runtime.h>

namespace pbs {

__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kernel(args...) behind the launch before it on the stream.
template <typename... Params, typename... Args>
cudaError_t launch_second(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                          Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pbs

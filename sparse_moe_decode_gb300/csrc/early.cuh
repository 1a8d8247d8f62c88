// early.cuh -- launches that overlap the end of the kernel before them on the
// stream: their blocks take the places that it leaves and then wait, before
// they touch any memory, until it is complete.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// At the top of a kernel launched with launch_early, before its first access
// to global memory: everything launched before on the stream is complete
// after this, and the kernel launched next may begin to take free places.
__device__ __forceinline__ void early_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t s, const A &...args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace moe

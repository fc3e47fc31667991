// pdl.cuh -- programmatic dependent launch: the kernels of one call after its first
// are launched so that their blocks may come up while the kernel before still runs;
// each waits for that kernel's end, and for its writes, before it touches memory.
#pragma once

#include <cuda_runtime.h>

namespace mf {

// Waits until the kernel before in the stream has ended and its writes are visible
// (at once in a kernel that was launched the ordinary way).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel's blocks come up from here on. They wait for this kernel's
// end all the same, so it can stand anywhere.
__device__ __forceinline__ void pdl_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// kernel<<<grid, block, smem, st>>>(args...) as a dependent launch; the kernel calls
// pdl_wait() before its first access to memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace mf

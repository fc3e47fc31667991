// pdl.cuh -- programmatic dependent launch: a kernel's blocks may come up while the
// kernel before it in the stream still runs; each waits for that kernel's end, and for
// its writes, before it touches memory. What it hides is the launch and the prologue
// (barriers, tensor memory, tensor maps), which is most of a small call. Behind a
// kernel that does not release its successors early the launch is an ordinary one.
#pragma once

#include <cuda_runtime.h>

namespace mf {

// Waits until the kernel before in the stream has ended and its writes are visible
// (at once in a kernel that was launched the ordinary way).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel's blocks come up once every block of this one is here. They
// wait for this kernel's end all the same. It stands behind pdl_wait and behind a
// kernel's tensor-memory allocation: a block of the next kernel that holds tensor
// memory must not keep a block of this one from starting.
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

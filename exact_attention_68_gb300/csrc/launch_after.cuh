// launch_after.cuh — kernels that follow one another in a call: the next one set up
// while the last one ends.
#pragma once

#include <cuda_runtime.h>

namespace ea {

// Programmatic dependent launch: the next kernel of the stream may be set up
// once every CTA has said so or ended; its wait ends when this grid has.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch that may be set up before the stream's previous kernel has ended;
// the kernel calls wait_for_previous before it uses that one's results or ends.
template <class Params>
cudaError_t launch_after(void (*kern)(Params), dim3 grid, int threads, cudaStream_t stream, const Params& p,
                         size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace ea

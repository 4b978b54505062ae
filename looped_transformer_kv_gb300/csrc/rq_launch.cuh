// Kernels of one call in a row: each one's CTAs are launched while the kernel before still runs, as
// its own finish, and wait in grid_wait() until it is complete: before they touch what a kernel of the
// call writes, or write what one reads, and in any case before they end, so that "complete" carries
// through the row.  (In most kernels it is the first statement.)  Two or three kernels in a row: 2 to 5 us less (3 tokens after
// 256: 21 -> 18.6 us; one step with weights 96 -> 91).
#pragma once
#include <cuda_runtime.h>

namespace rq {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Once every CTA has begun (and called this), the next kernel's may be launched.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// after: the stream's last operation is a kernel of the same call.
template <typename... Params, typename... Args>
cudaError_t launch_after(bool after, void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace rq

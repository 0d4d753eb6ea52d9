// launch.cuh -- launches that overlap the kernel before them in the stream: the
// grid may be set up, and its blocks may run up to previous_done(), while the
// last blocks of that kernel finish.  A kernel launched this way calls
// previous_done() before it touches any memory that another one may write or
// read; it returns when all kernels before it have completed and their writes
// can be seen.  That holds for ordinary loads.  Such a kernel lives while its
// inputs are still being written, so it does not promise that they are constant
// for its lifetime: no __restrict__ on its pointers, no loads by the read-only
// path.  What the compiler would have batched under that promise is batched in
// the code.  (Back to back, 64 x 6144 x 12288 in 8 bits: 22.3 -> 21.3 us a
// product; one row of 6144 to 8 bits: 2.8 -> 2.55 us, and back 1.67 -> 1.3.)
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace srm {

__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel be set up before this one ends (without it, as this
// one's blocks end).  Worth it where a block holds an SM to itself (the 8-bit
// products: 32.8 -> 32.0 us at 1 x 24576 x 6144); kernels of many small blocks
// lose (64 tokens to the experts 4.5 -> 5.5 us), the next one's taking their
// places.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kern)(Params...), unsigned grid, unsigned threads, size_t smem,
                              cudaStream_t stream, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace srm

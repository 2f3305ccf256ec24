// Kernels that are set up while the stream's previous kernel still runs.
#pragma once

#include <cuda_runtime.h>

namespace ra {

// The cache's kernels, the rotation and batched attention with changed scores are launched so that their blocks may
// be set up while the stream's previous kernel still runs (programmatic dependent launch): every kernel
// calls after_previous_kernel before it touches memory, which waits until that
// kernel has ended and its writes are visible, and only then allows the same to
// the next one, so no more than two kernels overlap.  Global memory is read by
// plain loads, which stay behind the wait (loads through the read-only path need
// not).  Saves about 2 us a launch for single tokens and short sequences (257 capped tokens of 4 heads: 11.1 us,
// 13.4 without).
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}
// A plain load, whatever the compiler knows of the pointer.
template <class T>
__device__ __forceinline__ T load_now(const T* p) {
  return *const_cast<const volatile T*>(p);
}

}  // namespace ra

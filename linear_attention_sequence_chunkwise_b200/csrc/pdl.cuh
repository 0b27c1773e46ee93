// pdl.cuh -- programmatic dependent launch: a kernel may start while the one before it in the stream
// drains, and waits (pdl_wait) before it reads or writes global memory (tc_output_kernel touches some
// sooner, and says why it may).  Every kernel launched so waits, so that each still runs behind all that
// came before it; one that says pdl_go lets the next start sooner.  No pointer of such a kernel is
// __restrict__: a load that is taken for invariant may move above the wait.  Launches overlap so in a
// stream of calls: one token for 37 rows of 4 x 100 x 130 states 8.2 -> 5.5 us, a fork of four 512 KB slots
// 5.1 -> 3.7, 157 packed tokens 18.4 -> 16.2.
#pragma once

#include <cuda_runtime.h>

namespace retnet {

__device__ __forceinline__ void pdl_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace retnet

// Programmatic dependent launch for the chained decode-step kernels.
#pragma once
#include <cuda_runtime.h>

namespace kk {

// A kernel launched with programmatic stream serialisation may start while
// the kernel before it in the stream is still running; it waits here, before
// its first access to global memory, until that kernel has finished and its
// writes are visible (no wait when there is no such kernel). Signalling early
// lets the next kernel of the stream be launched in the meantime, so the
// launch latency of a chain of small kernels overlaps their execution.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel so that it may start while the one before it in the stream
// ends: it calls pdl_wait() before it reads or writes anything.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*k)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace kk

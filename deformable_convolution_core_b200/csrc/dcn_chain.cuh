// Kernels of one call that follow one another on its stream.  A follower is launched
// with programmatic stream serialization: its CTAs may start, set up their barriers and
// tensor memory and fetch their descriptors while the kernel before is ending.  It
// touches no global memory before chain_wait, which returns when the kernel before has
// completed and its writes are visible; as every kernel of a chain waits, so have all
// the ones before that.  The next call's first kernel is launched the ordinary way.
#pragma once

#include <cuda_runtime.h>

#include "dcn_core.h"

namespace dcn {

// Waits for the kernel before, if this one was launched as its follower.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The follower may be launched once every CTA of this kernel has said so.
__device__ __forceinline__ void chain_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
dcn_status launch_kernel(void (*kernel)(Params...), bool follows, dim3 grid, int threads,
                         size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute serial;
  serial.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  serial.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &serial;
  cfg.numAttrs = follows ? 1 : 0;
  const cudaError_t launched = cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
  return launched == cudaSuccess && cudaGetLastError() == cudaSuccess ? DCN_OK : DCN_ERR_CUDA;
}

}  // namespace dcn

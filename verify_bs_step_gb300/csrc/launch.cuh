// Dependent launches (sm_103a).
#pragma once

#include <cuda_runtime.h>

#include "vbs.h"

namespace vbs {

// A launch that may be set up while its predecessor in the stream finishes; the kernel waits for it
// (griddepcontrol.wait) before its first access to memory.
template <typename... KArgs, typename... Args>
int launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...) == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

}  // namespace vbs

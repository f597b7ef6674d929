// What the per-head and block-scaled operators' host code shares: a kernel launch with the
// process's choice of programmatic dependent launch.  (Every such kernel waits for the
// kernels ahead of it, griddepcontrol.wait, before it reads or writes global memory; the
// product's small kernel only has lines of wt brought into L2 earlier.  No kernel reads
// through the read-only path, ld.global.nc: what the kernel ahead writes is not read-only.)
#pragma once

#include <cuda_runtime.h>

#include "far.h"

namespace far {

template <typename... A>
cudaError_t launch_k(void (*k)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = far_get_programmatic_launch() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace far

// What the per-head, block-scaled, int8 and feed-forward operators' host code shares: a kernel launch with the
// process's choice of programmatic dependent launch.  (Every such kernel waits for the
// kernels ahead of it, griddepcontrol.wait, before it reads or writes global memory, but for
// two things: the kernels of few rows have lines of a weight brought into L2 earlier, and
// gemm_int8's kernel of many rows reads wt while the kernel ahead, its own, widens x; that one
// lets it start only behind its own wait.  No kernel reads through the read-only path,
// ld.global.nc: what the kernel ahead writes is not read-only.)
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

// CTAs (1 to 8, a cluster) that share out the `depth` steps of each of `tiles` tiles, for kernels whose CTAs keep
// `fixed` steps' time of their own and of which an SM holds `per_sm`.  A cluster lies in one part of the GPU, so that
// fewer of the larger ones fit at once: of one CTA an SM, on 152 SMs, as many as kClusters says
// (cudaOccupancyMaxActiveClusters; 16 x 5120 x 5120 of gemm_int8, 40 tiles, in clusters of 6, which all
// fit, 9.6 us, of 7 15.2).  At least two steps a CTA.
struct ClusterPlan {
  int split;
  int64_t waves;  // of clusters
};
inline ClusterPlan plan_clusters(int64_t tiles, int64_t depth, int per_sm, int64_t fixed) {
  constexpr int kClusters[8] = {152, 76, 46, 36, 28, 23, 15, 15};
  ClusterPlan best{1, 0};
  int64_t least = 0;
  for (int split = 1; split <= 8 && (split == 1 || depth >= 2 * split); ++split) {
    const int64_t room = (int64_t)per_sm * kClusters[split - 1], waves = (tiles + room - 1) / room;
    const int64_t cost = waves * (fixed + (depth + split - 1) / split);
    if (split == 1 || cost < least) {
      least = cost;
      best = ClusterPlan{split, waves};
    }
  }
  return best;
}

}  // namespace far

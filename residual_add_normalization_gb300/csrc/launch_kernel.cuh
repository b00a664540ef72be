// launch_kernel.cuh -- launches with programmatic dependent launch allowed, in
// clusters or not.
#pragma once

#include "launch.h"

namespace b200norm {

template <class Fn, class... A>
cudaError_t launch_clusters(Fn fn, dim3 grid, int block, int csize, size_t smem,
                            cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (csize > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    n = 1;
  }
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = add_pdl_attr(attr, n);
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <class Fn, class... A>
cudaError_t launch_pdl(Fn fn, dim3 grid, int block, cudaStream_t stream, const A&... args) {
  return launch_clusters(fn, grid, block, 1, 0, stream, args...);
}

}  // namespace b200norm

// How the decode kernels are launched.
#pragma once

#include <cuda_runtime.h>

namespace stem {

// A launch that may be set up while the stream's previous kernel still runs: the kernel waits for it
// itself (cudaGridDependencySynchronize) before it touches memory. Such a launch also costs the host
// 2.4 us where a plain one costs 2.9 (200 in a row of a kernel with 256 bytes of arguments). cluster: CTAs
// of a cluster along x; 1 launches without clusters.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                         cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace stem

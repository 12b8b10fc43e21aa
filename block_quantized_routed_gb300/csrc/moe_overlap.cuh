// Launches that overlap the end of the kernel before them in the stream.
//
// A kernel launched so may start while the one before it still runs, if that one
// lets it (let_next_start), else when it ends.  It touches no global memory
// before wait_for_previous, which returns when everything before it in the stream
// is done and visible; what it does until then (barriers, tensor memory, the
// arithmetic of its indexes) no longer adds to the step.  A kernel before or
// after it that knows nothing of this is ordered as ever.
#pragma once

#include <utility>

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// clusters: CTAs of a cluster along x (1: none)
template <typename... P, typename... A>
cudaError_t launch_overlapping(void (*kern)(P...), dim3 grid, int threads, int smem, int clusters, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)clusters;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = clusters > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

}  // namespace moe

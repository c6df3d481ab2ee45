// pdl.cuh -- launches that may begin before the kernel ahead of them in the stream has
// ended (programmatic dependent launch), for runs of short kernels.
//
// A kernel launched by launch_early() calls early_start() before it touches global
// memory: it waits until every kernel ahead of it has completed and its writes are
// visible.  What a kernel does before that (shared memory barriers, tensor memory, its
// place in the grid) overlaps the end of the one ahead.  Where its grid is small, it lets
// the kernel behind it start at once: for 64 tokens' combine, 2.57 against 2.72 us; blocks
// that wait beside a large grid or a product on tensor cores (which calls
// wait_for_kernels_ahead()) only cost it (gradients of 4096 tokens: 80.0 against 78.5 us;
// the 8-bit experts of 64 tokens: 145.5 against 141).  Kernels launched in the ordinary
// way keep the ordinary order.
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace moe {

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_kernels_ahead() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void early_start() {
  constexpr unsigned kSmallGrid = 8 * 148;
  if (gridDim.x * gridDim.y <= kSmallGrid)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_kernels_ahead();
}
#endif

// cluster: CTAs of a cluster (0: as the kernel is compiled).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                         cudaStream_t s, int cluster, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace moe

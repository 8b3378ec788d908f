// Launches whose set-up overlaps the end of the kernel before them on the stream (programmatic
// dependent launch): a kernel starts with pdl_start(), which lets the next one's blocks in as soon
// as its own leave room, and calls pdl_wait() before it first touches global memory, which returns
// when the kernel before has finished and its writes are visible. What it reads is then written
// during its own lifetime, which rules out loads through the read-only path: no __ldg and no
// const __restrict__ pointers in these kernels. In a row of launches one token's
// 2048 x 7680 projection takes 9.3 us, 12.3 without.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ void pdl_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs of a cluster (1: none).
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace moe

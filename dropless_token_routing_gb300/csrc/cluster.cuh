// Thread-block clusters: ranks, the cluster-wide barrier in its two halves, and reads of a peer's
// shared memory (the peer has to stay until they are done: it waits at a barrier that the reader
// arrives at afterwards).
#pragma once

#include <stdint.h>

namespace moe {

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The word at shared address `a` of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_address(uint32_t a, uint32_t rank) {
  uint32_t p;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(rank));
  return p;
}
__device__ __forceinline__ long long peer_ld64(uint32_t a, uint32_t rank) {
  long long v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(peer_address(a, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float peer_ldf(uint32_t a, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_address(a, rank)) : "memory");
  return v;
}

}  // namespace moe

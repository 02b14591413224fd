// Blocks of a cluster: their barrier and one another's shared memory; asynchronous copies of 16 bytes into a block's own.
#pragma once

#include <stdint.h>

namespace qmv {
namespace cluster {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Both halves of the barrier are ones that a warp executes as a whole, so its lanes meet first: they may come out of loops and
// branches that they took one by one.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of p, of this block's shared memory, in that of block `rank`.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}

// Sixteen bytes from memory to shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint32_t to, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }   // all of this thread's

}  // namespace cluster
}  // namespace qmv

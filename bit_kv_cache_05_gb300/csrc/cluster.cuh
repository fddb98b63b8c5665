// Thread-block clusters: rank, barrier, the other CTAs' shared memory, and a
// launch with a cluster size.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "bulk_pipe.cuh"

namespace vqk {

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_ctas() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// all threads of all CTAs of the cluster; what they wrote before is seen behind
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Another CTA's shared memory may be touched once that CTA is known to run:
// every thread arrives where its kernel begins, and waits before the first peer
// access, or where it leaves without one.
__device__ __forceinline__ void cluster_began() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_runs() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of `p`, a place in this CTA's shared memory, in CTA `rank`'s
__device__ __forceinline__ uint32_t peer_addr(const void *p, unsigned rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_load(const uint32_t *p, unsigned rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint64_t *p, unsigned rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_addr(p, rank)), "l"(v) : "memory");
}

template <typename... P, typename... A>
inline cudaError_t launch_cluster(void (*fn)(P...), dim3 grid, dim3 block, int cluster,
                                  size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace vqk

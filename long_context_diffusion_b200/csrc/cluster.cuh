// Thread-block clusters: rank, barrier, and reads of another CTA's shared
// memory.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "launch.cuh"

namespace dl {

__device__ __forceinline__ int cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// Barrier of all threads of the cluster; shared memory written before it is
// visible to the cluster after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ unsigned peer_address(const void* p, int rank) {
  unsigned there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(static_cast<unsigned>(__cvta_generic_to_shared(p))), "r"(rank));
  return there;
}
__device__ __forceinline__ int peer_int(const int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_address(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_float2(const float2* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(peer_address(p, rank))
               : "memory");
  return v;
}

// Launch configuration attributes of a cluster of `size` CTAs along x.
inline cudaLaunchAttribute cluster_of(int size) {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = size;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  return a;
}

// Clusters of `size` CTAs (2, 4 or 8) of a kernel that are resident at once: fewer
// than its CTAs make, because a cluster lies in one GPC (148 CTAs, one per SM: 15
// clusters of eight, 33 of four).  Asked of the runtime once per device.
template <auto Kernel>
int resident_clusters(int size, int threads, int smem) {
  static std::atomic<int> known[64][3];  // count + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>* slot = dev < 64 ? &known[dev][size == 2 ? 0 : size == 4 ? 1 : 2] : nullptr;
  if (slot && slot->load(std::memory_order_relaxed)) return slot->load(std::memory_order_relaxed) - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1] = {cluster_of(size)};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_smem<Kernel>(smem) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (slot) slot->store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace dl

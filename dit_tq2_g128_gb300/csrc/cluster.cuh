// What kernels of thread-block clusters share: barriers, and the other CTAs' shared memory.
#pragma once

#include <cstdint>

namespace tq2 {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A barrier of all threads of the cluster, in two halves: what comes before a thread's arrival is seen after the others' wait.
// The first one of a kernel also says that every CTA has begun: before it no other CTA's shared memory may be touched.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The same place in CTA `rank`'s shared memory, as a generic pointer.
template <typename P>
__device__ __forceinline__ P *at_cta(P *p, uint32_t rank) {
    uint64_t r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<P *>(r);
}

}  // namespace tq2

// Thread-block clusters: rank, size, barrier and reads of a peer's shared memory.
#pragma once

#include <stdint.h>

namespace usm {

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(n));
    return n;
}
// Every thread of the cluster; shared-memory writes before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at this CTA's shared address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ float load_cluster(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

}  // namespace usm

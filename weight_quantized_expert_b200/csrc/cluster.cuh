// Thread-block clusters: rank, barrier and stores into another CTA's shared memory.
#pragma once

#include "common.cuh"

namespace focr {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// writes the same variable in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ void st_cluster(float* p, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(p, rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(double* p, uint32_t rank, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa_shared(p, rank)), "d"(v) : "memory");
}

}  // namespace focr

// mxq_cluster.cuh -- thread-block clusters: their barrier, and reads of another CTA's
// shared memory (sm_100a).
#pragma once

#include "mxq_device.cuh"

namespace mxq {

// All threads of the cluster; shared memory written before is seen behind it.
__device__ __forceinline__ void cluster_sync_all()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes of the shared memory of CTA `rank` of the cluster, at this CTA's address `p`.
__device__ __forceinline__ float4 peer_f4(const float4 *p, uint32_t rank)
{
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// The same of one word.
__device__ __forceinline__ float peer_f(const float *p, uint32_t rank)
{
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

} // namespace mxq

// What a cluster of blocks that selects the largest of many keys shares: the
// keys, barriers, reads and sums across its shared memory, a prefix sum.
#pragma once

#include "common.cuh"

namespace mla {

// Larger weight <=> larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
    w = w != w ? __int_as_float(0xff800000) : w + 0.f;
    const uint32_t u = __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr uint32_t kKeyZero = 0x80000000u, kKeyLowest = ~0xff800000u;     // no key is below kKeyLowest

__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// All running blocks of the cluster, their shared-memory writes before it
// visible after it.  Both halves are for whole warps: lanes that took a
// branch before them meet first.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// What is at `p`'s place in the shared memory of block `rank`.
__device__ __forceinline__ uint32_t remote(const uint32_t *p, uint32_t rank) {
    uint32_t addr, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// A thread's bins.
template <int N>
struct Bins {
    static_assert(N == 2 || N % 4 == 0, "whole vectors");
    uint32_t n[N];
};
template <int N>
__device__ __forceinline__ Bins<N> local_bins(const uint32_t *p) {
    Bins<N> b;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + i);
            b.n[i] = v.x, b.n[i + 1] = v.y, b.n[i + 2] = v.z, b.n[i + 3] = v.w;
        }
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        b.n[0] = v.x, b.n[1] = v.y;
    }
    return b;
}
template <int N>
__device__ __forceinline__ Bins<N> remote_bins(const uint32_t *p, uint32_t rank) {
    static_assert(N <= 4, "one vector");
    uint32_t addr;
    Bins<N> b;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    if constexpr (N == 4)
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b.n[0]), "=r"(b.n[1]), "=r"(b.n[2]), "=r"(b.n[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(b.n[0]), "=r"(b.n[1]) : "r"(addr) : "memory");
    return b;
}

// Adds v at `p`'s place in the shared memory of block `rank`.
__device__ __forceinline__ void remote_add(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tred.relaxed.cluster.shared::cluster.add.u32 [a], %2;\n\t}" ::"r"(
            smem_u32(p)),
        "r"(rank), "r"(v)
        : "memory");
}

// Exclusive prefix sum of v over the block's threads.
template <int WARPS>
__device__ uint32_t block_scan(uint32_t v, uint32_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    const uint32_t w = lane < WARPS ? red[lane] : 0;
    uint32_t s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    return x - v + __shfl_sync(0xffffffffu, s - w, warp);
}

}  // namespace mla

// Thread-block clusters for sm_103a: rank and size, the cluster barrier and
// stores into another CTA's shared memory as inline PTX, and their launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "bulk.cuh"

namespace sv {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The two halves of the cluster barrier: every thread of every CTA arrives,
// and what was written before an arrival is visible after the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Stores into another CTA whose bytes count on an mbarrier there: what the
// mbarrier has counted is visible to who waits for its phase with
// cluster_mbar_wait.  Nothing else that this thread wrote is waited for, which
// a cluster barrier's release would.  addr and bar of the same CTA.
__device__ __forceinline__ void cluster_send(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_int(v)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_send(uint32_t addr, float2 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
                 "r"(__float_as_int(v.x)), "r"(__float_as_int(v.y)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_send(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     addr),
                 "r"(__float_as_int(v.x)), "r"(__float_as_int(v.y)), "r"(__float_as_int(v.z)),
                 "r"(__float_as_int(v.w)), "r"(bar)
                 : "memory");
}
// As mbar_wait, for a phase that other CTAs complete.
__device__ __forceinline__ bool cluster_mbar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_ns) return false;
    }
}

// Clusters of S CTAs of this shape that run at the same time on the current
// device (a GPC holds whole clusters only, so this is less than its CTAs over
// S).  The first call per (device, kernel, S, shared memory) asks, later ones
// read the table.
inline bool clusters_at_once(const void* kernel, int S, int block, size_t dyn_smem, int* out) {
    struct Entry {
        const void* fn;
        int dev, S, block;
        size_t dyn;
        int n;
    };
    constexpr int kEntries = 128;
    static std::mutex mu;
    static Entry table[kEntries];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].fn == kernel && table[i].dev == dev && table[i].S == S && table[i].block == block &&
            table[i].dyn == dyn_smem) {
            *out = table[i].n;
            return true;
        }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = dyn_smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return false;
    if (used < kEntries) table[used++] = Entry{kernel, dev, S, block, dyn_smem, n};
    *out = n;
    return true;
}

// A launch of n clusters of S CTAs (S = 1: of n CTAs), dependent (as
// launch_dependent) or ordinary.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), long long n, int S, int block, size_t dyn_smem,
                                   bool dependent, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * S));
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = dyn_smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int used = 0;
    if (dependent) {
        attr[used].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[used++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (S > 1) {
        attr[used].id = cudaLaunchAttributeClusterDimension;
        attr[used].val.clusterDim.x = S;
        attr[used].val.clusterDim.y = 1;
        attr[used++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = used;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace sv

// kda_gdn_ptx.cuh -- inline PTX of the gated delta rule's and the RMS norm's kernels, beside kda_ptx.cuh.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kda_ptx.cuh"

namespace kda {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// mbar_wait_pipe without its second wait, for a caller whose end of its own work is all that follows an expired wait while
// another thread waits for the operation.
__device__ __forceinline__ bool mbar_wait_or_stop(uint64_t* bar, uint32_t parity) {
    if constexpr (kWaitLimit == 0) return mbar_test(bar, parity);
    return mbar_wait(bar, parity, kWaitLimit);
}

// D[tmem] (+)= A[tmem] * B[smem desc]: A's 16-bit pairs along K in consecutive columns, a row a lane.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 8 32-bit columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Programmatic dependent launches: a kernel lets the next one's blocks start (on what the SMs have left) once
// all its own have begun, and the next one waits for its end and its writes before it reads them.
__device__ __forceinline__ void grid_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Blocks in clusters of `cluster` (1: none).
template <typename K, typename... A>
inline cudaError_t launch_dependent_clusters(int cluster, K kernel, int64_t blocks, int threads, uint32_t smem,
                                             cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename K, typename... A>
inline cudaError_t launch_dependent(K kernel, int64_t blocks, int threads, uint32_t smem, cudaStream_t stream,
                                    const A&... args) {
    return launch_dependent_clusters(1, kernel, blocks, threads, smem, stream, args...);
}

// -------------------------------------------------------------- clusters ----
// Every thread of every block of the cluster; writes before it are seen behind it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory address in block `rank` of the cluster, and a load from one.
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

}  // namespace kda

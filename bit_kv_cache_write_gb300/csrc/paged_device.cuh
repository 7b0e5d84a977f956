// Device helpers shared by the BF16 paged-cache kernels, and their launch with programmatic dependence.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "layout.cuh"
#include "paged_internal.h"

namespace oscar {
namespace {

// Waits for the grids before this one in the stream (everything they wrote is visible afterwards).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next grid's CTAs start where there is room; they wait in grid_wait().
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// 32 bytes of a 32-byte aligned address: four lanes cover a cache line, half the requests of 16-byte loads.
__device__ __forceinline__ void ldg_stream32(uint4& a, uint4& b, const void* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(p));
}

// Sequence length as the kernels use it: within [0, max_len]; anything else is recorded.
__device__ __forceinline__ int checked_len(int len, int max_len, int debug, DebugWord* dbg) {
    if (len < 0 || len > max_len) {
        if (debug) record_error(&dbg->kind, &dbg->index, 3, len);
        len = len < 0 ? 0 : max_len;
    }
    return len;
}

// Lets kernel Kern run in clusters of more than 8 CTAs on the current device; set once for each (see smem_opt_in).
template <auto Kern>
cudaError_t allow_large_clusters() {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
}  // namespace oscar

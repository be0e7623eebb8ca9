// Launches that need an attribute: clusters (with their barrier and rank), and kernels that begin
// while the one before them on the stream ends.
#pragma once
#include <cuda_runtime.h>

namespace kda {

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory"); }
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// In a kernel launched by launch_after: what the kernels before it wrote is there from here on (at
// once in other launches).  Every kernel of such a row waits, so that the whole row is over.
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// The next kernel's CTAs may take the room that this one leaves, and wait there.
__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// <<<grid, block, smem, s>>> of a kernel that calls previous_done() before it touches memory; `early`:
// it may begin before the one before it on the stream has ended (of the gated delta rule's few
// kernels in a row: 9 packed prompts 66 -> 61 us, 5 packed samples backwards 70 -> 65)
template <typename... Params, typename... Args>
cudaError_t launch_after(bool early, void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = early;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// <<<grid, block, smem, s>>> with clusters of `size` CTAs
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, unsigned size,
                            cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {size, 1, 1};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace kda

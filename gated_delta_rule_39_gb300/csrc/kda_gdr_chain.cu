// Outputs and final state of the gated delta rule: one CTA per (sequence, value head).
#include "kda_gdr_chain.cuh"

namespace kda {
namespace {

using namespace gdr;

__global__ void __launch_bounds__(chain::kChainThreads, 1) gdr_chain_kernel(GdrChunked P, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char raw[];
    previous_done();
    if (P.in.cu && !*P.in.valid) return;
    chain::run<false>(P, vmap, aligned_smem<chain::ChainSmem>(raw), sequence_of(P.chunks, blockIdx.x / P.in.Hv),
                      blockIdx.x % P.in.Hv);
}

}  // namespace

cudaError_t launch_gdr_chain(const GdrChunked& P, bool early, cudaStream_t s) {
    const long long units = (long long)P.in.N * P.in.Hv;
    if (units == 0) return cudaSuccess;
    constexpr size_t smem = sizeof(chain::ChainSmem) + 1024;
    CUtensorMap vmap{};
    cudaError_t e = allow_smem<gdr_chain_kernel>(smem);
    if (e == cudaSuccess) e = chain::values_map(P, &vmap);
    if (e != cudaSuccess) return e;
    return launch_after(early, gdr_chain_kernel, dim3((unsigned)units), chain::kChainThreads, smem, s, P, vmap);
}

}  // namespace kda

// The gated delta rule with one decay per value head (sm_103a): what its kernels share.
//
//   S' = e^g S,  d = beta (v - S'^T k),  S = S' + k d^T,  o = scale S^T q
//
// per (sequence, value head), S a 128 x 128 matrix (row = key channel); value head h reads
// the queries and keys of head h / (Hv / Hk).  g is the log of the decay as given (at most 0
// in use, down to -inf), beta the write strength as given.
#pragma once
#include "kda_host.cuh"

namespace kda {

struct GdrInputs {
    const __nv_bfloat16 *q, *k, *v;          // rows of Hk or Hv heads
    long long q_stride, k_stride, v_stride;  // elements from one token to the next
    const void *g, *beta;                    // [tokens][Hv] of gate_dtype
    int gate_dtype;
    float scale;
    const int* cu;        // [N + 1] token offsets on the device, or nullptr: N sequences of T
    const int* valid;     // with cu: 1 where cu passed its checks
    int N, T, Hk, Hv;     // T: tokens of a sequence (cu: of all)
};

struct GdrStep {          // the token-by-token kernel (kda_gdr_step.cu)
    GdrInputs in;         // N sequences of T (no cu)
    __nv_bfloat16* out;   // [tokens][Hv][128] or nullptr
    const void* state_in; // [pool][Hv][128][128] or nullptr (zero)
    int in_dtype;
    void* state_out;      // or nullptr
    int out_dtype;
    const int* slots;     // [N] or nullptr (sequence n uses state n)
    const int* lengths;   // [N] or nullptr: tokens after which the state is written
    int pool;
    int* err;
};

__device__ __forceinline__ float load_gate(const void* p, int dtype, size_t i) {
    return dtype == KDA_F32 ? static_cast<const float*>(p)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Host-side checks of what the entry points have in common; no CUDA call.
int gdr_validate(const GdrInputs& in, int B, int K, int V, const void* s0, int s0_dtype, const void* s1,
                 int s1_dtype, long long pool);
// Bytes from the first element of `tokens` strided rows to the last.
size_t gdr_span(long long tokens, int heads, long long stride);

cudaError_t launch_gdr_step(const GdrStep& P, cudaStream_t s);

}  // namespace kda

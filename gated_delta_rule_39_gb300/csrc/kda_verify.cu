// Verification of drafted tokens against the target's probabilities, from random numbers
// that the caller draws.
//
//   draft i (a token x_i drawn with probability q_i(x_i)) is kept while u_i q_i(x_i) < p_i(x_i);
//   after the first one that is not, at place a, the next token is drawn from what the
//   draft left of the target, rest(v) = max(p_a(v) - q_a(v), 0); if all are kept, from
//   the target's last row, rest = p_a.  Drawing is an exponential race: with independent
//   e(v) ~ Exp(1), argmax_v rest(v) / e(v) is v with probability rest(v) / sum rest.
//   (Keep-or-redraw leaves the target's own distribution: min(p, q) + (p - q)^+ = p.)
//
// Only one row of p, one of q and one of e are read per sequence, so the work is bound by
// those bytes, or for few sequences by latency.  The division is IEEE's and rest is one
// subtraction, so the scores, and the winner, do not depend on how the row is split; ties go to
// the lowest index.
#include <cmath>

#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kVerThreads = 1024;

struct VerifyProblem {
    const void* target;       // [N][D + 1][V]
    const void* draft;        // [N][D][V], or nullptr (the drafts were certain)
    const int* tokens;        // [N][D]
    const float* uniform;     // [N][D]
    const float* noise;       // [N][V]
    const int* count;         // [N] or nullptr (D)
    int* accepted;            // [N]
    int* result;              // [N][D + 1]
    int N, D, V;
    int* err;
};

__device__ __forceinline__ float prob(const __nv_bfloat16* p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float prob(const float* p, size_t i) { return p[i]; }

// Larger score first, then lower index; 0 where the score is not positive (or not a
// number).  A positive float's bits rise with its value.
__device__ __forceinline__ unsigned long long race_key(float rest, float noise, int v) {
    if (!(rest > 0.0f)) return 0ull;
    const float score = __fdiv_rn(rest, noise);
    if (!(score > 0.0f)) return 0ull;
    return (unsigned long long)__float_as_uint(score) << 32 | (unsigned)~v;
}

__device__ __forceinline__ unsigned long long max_key(unsigned long long a, unsigned long long b) {
    return a > b ? a : b;
}

// Drafts kept of sequence n, by one warp; -1: a count or a token out of range.
template <typename T>
__device__ int drafts_kept(const VerifyProblem& P, int n, int lane, int& count) {
    count = P.count ? P.count[n] : P.D;
    if (count < 0 || count > P.D) return -1;
    for (int first = 0; first < count; first += 32) {
        const int i = first + lane;
        bool keep = true, bad = false;
        if (i < count) {
            const size_t at = (size_t)n * P.D + i;
            const int x = P.tokens[at];
            bad = x < 0 || x >= P.V;
            if (!bad) {
                const float p = prob(static_cast<const T*>(P.target), ((size_t)n * (P.D + 1) + i) * P.V + x);
                const float q = P.draft ? prob(static_cast<const T*>(P.draft), at * P.V + x) : 1.0f;
                keep = __fmul_rn(P.uniform[at], q) < p;
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad)) return -1;
        const unsigned lost = __ballot_sync(0xFFFFFFFFu, !keep);
        if (lost) return first + __ffs(lost) - 1;
    }
    return count;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(VerifyProblem P) {
    __shared__ int s_kept, s_count;
    __shared__ unsigned long long s_best[kVerThreads / 32];
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) {
        int count;
        const int kept = drafts_kept<T>(P, n, lane, count);
        if (lane == 0) {
            s_kept = kept;
            s_count = count;
        }
    }
    __syncthreads();
    const int a = s_kept;
    if (a < 0) {
        if (tid == 0) set_error(P.err, KDA_ERR_BAD_INDEX);
        return;
    }
    const bool redraw = a < s_count;
    const T* p = static_cast<const T*>(P.target) + ((size_t)n * (P.D + 1) + a) * P.V;
    const T* q = redraw && P.draft ? static_cast<const T*>(P.draft) + ((size_t)n * P.D + a) * P.V : nullptr;
    const int sure = redraw && !P.draft ? P.tokens[(size_t)n * P.D + a] : -1;   // certain draft: q = 1 there
    const float* e = P.noise + (size_t)n * P.V;
    unsigned long long best = 0;
    // a second round, on p itself, where the first finds nothing left (p nowhere above q)
    for (int round = 0; round < 2; ++round) {
        for (int v = tid; v < P.V; v += kVerThreads) {
            const float pv = prob(p, v);
            const float qv = round ? 0.0f : q ? prob(q, v) : v == sure ? 1.0f : 0.0f;
            best = max_key(best, race_key(pv - qv, e[v], v));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
        if (lane == 0) s_best[tid >> 5] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVerThreads / 32; ++i) best = max_key(best, s_best[i]);
        if (best || !redraw) break;
        __syncthreads();
    }
    if (tid == 0) P.accepted[n] = a;
    int* out = P.result + (size_t)n * (P.D + 1);
    for (int i = tid; i <= P.D; i += kVerThreads)
        out[i] = i < a ? P.tokens[(size_t)n * P.D + i] : i == a && best ? (int)~(unsigned)best : -1;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_verify_drafts(const void* target_probs, const void* draft_probs, int dtype,
                                 const int32_t* draft_tokens, const float* uniform, const float* noise,
                                 const int32_t* num_drafts, int32_t* accepted, int32_t* tokens, int N,
                                 int D, int V, void* stream) {
    if (N < 0 || D < 0 || V < 1 || D > 65536) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (N > 0 && (!target_probs || !noise || !accepted || !tokens)) return KDA_ERR_NULL;
    if (N > 0 && D > 0 && (!draft_tokens || !uniform)) return KDA_ERR_NULL;
    const size_t size = dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {target_probs, draft_probs})
        if (reinterpret_cast<uintptr_t>(p) % size) return KDA_ERR_ALIGN;
    const void* in_p[] = {target_probs, draft_probs, draft_tokens, uniform, noise, num_drafts};
    const size_t nd = (size_t)N * D;
    const size_t in_n[] = {(nd + N) * V * size, nd * V * size, nd * 4, nd * 4, (size_t)N * V * 4, (size_t)N * 4};
    for (int i = 2; i < 6; ++i)
        if (reinterpret_cast<uintptr_t>(in_p[i]) % 4) return KDA_ERR_ALIGN;
    const void* out_p[] = {accepted, tokens};
    const size_t out_n[] = {(size_t)N * 4, (nd + N) * 4};
    for (int o = 0; o < 2; ++o) {
        if (reinterpret_cast<uintptr_t>(out_p[o]) % 4) return KDA_ERR_ALIGN;
        for (int i = 0; i < 6; ++i)
            if (overlaps(out_p[o], out_n[o], in_p[i], in_n[i])) return KDA_ERR_ALIAS;
    }
    if (overlaps(accepted, out_n[0], tokens, out_n[1])) return KDA_ERR_ALIAS;
    int dev = 0;
    int* err = nullptr;
    const int rc = device_setup(&dev, &err);
    if (rc != KDA_OK) return rc;
    if (N == 0) return KDA_OK;
    VerifyProblem P{target_probs, draft_probs, draft_tokens, uniform, noise, num_drafts,
                    accepted, tokens, N, D, V, err};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = timed_launch(KDA_KERNEL_VERIFY, s, [&] {
        if (dtype == KDA_BF16) verify_kernel<__nv_bfloat16><<<N, kVerThreads, 0, s>>>(P);
        else verify_kernel<float><<<N, kVerThreads, 0, s>>>(P);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

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
// those bytes (128 fp32 rows of 131,072: 35 us, 5 TB/s), or for few sequences by latency (one row
// of 50,257: 6 us with its launch).  The division is IEEE's and rest is one
// subtraction, so the scores, and the winner, do not depend on how the row is split; ties go to
// the lowest index.
#include "kda_cluster.cuh"
#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kVerThreads = 512;
constexpr int kMaxSplit = 16;             // CTAs (a cluster) for a sequence's row
constexpr int kMinSlice = 2048;           // elements of a row that a CTA is started for, at least

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

template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) Unit {
    T v[VEC];
};

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

// Drafts kept of sequence n, by a warp; -1: a count or a token out of range.
template <typename T>
__device__ int drafts_kept(const VerifyProblem& P, int n, int lane, int& count) {
    count = P.count ? P.count[n] : P.D;
    for (int first = 0; first < P.D; first += 32) {
        const int i = first + lane;
        bool keep = true, bad = false;
        if (i < P.D) {                         // the loads need not wait for the count
            const size_t at = (size_t)n * P.D + i;
            const int x = P.tokens[at];
            const float u = P.uniform[at];
            const bool in = x >= 0 && x < P.V;
            bad = i < count && !in;
            if (in && i < count) {
                const float p = prob(static_cast<const T*>(P.target), ((size_t)n * (P.D + 1) + i) * P.V + x);
                const float q = P.draft ? prob(static_cast<const T*>(P.draft), at * P.V + x) : 1.0f;
                keep = __fmul_rn(u, q) < p;
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) || count < 0 || count > P.D) return -1;
        const unsigned lost = __ballot_sync(0xFFFFFFFFu, !keep);
        if (lost) return first + __ffs(lost) - 1;
        if (first + 32 >= count) break;
    }
    return count < 0 || count > P.D ? -1 : count;
}

// writes to the same variable of another CTA of the cluster
__device__ __forceinline__ void put(unsigned long long* p, unsigned rank, unsigned long long x) {
    const unsigned at = (unsigned)__cvta_generic_to_shared(p);
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.u64 [a], %2;\n}\n" ::"r"(at), "r"(rank), "l"(x) : "memory");
}

// One cluster per sequence; its CTAs take VEC elements per thread in turn and exchange their
// winners.  Every warp decides for itself which drafts are kept, with the first noise on its way.
template <typename T, int VEC>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(VerifyProblem P, int split) {
    constexpr int kUnits = VEC == 1 ? 8 : sizeof(T) == 2 ? 2 : 1;      // of a thread at a time
    __shared__ unsigned long long s_best[2][kVerThreads / 32], s_rank[2][kMaxSplit];
    const int n = blockIdx.x / split, tid = threadIdx.x, lane = tid & 31;
    const unsigned rank = cluster_rank();
    cluster_arrive();                          // all CTAs have begun before one writes to another
    // unsigned: a turn may end up to kUnits x step after the row's end, past 2^31 for the longest rows
    const unsigned units = P.V / VEC, step = split * kVerThreads, begin = rank * kVerThreads + tid;
    using Noise = Unit<float, VEC>;
    using Prob = Unit<T, VEC>;
    const Noise* e = reinterpret_cast<const Noise*>(P.noise + (size_t)n * P.V);
    Noise ev[kUnits];
    const auto noise = [&](unsigned base) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
            if (base + j * step < units) ev[j] = e[base + j * step];
    };
    noise(begin);
    int count;
    const int a = drafts_kept<T>(P, n, lane, count);
    cluster_wait();
    if (a < 0) {
        if (rank == 0 && tid == 0) set_error(P.err, KDA_ERR_BAD_INDEX);
        return;
    }
    const bool redraw = a < count;
    const Prob* p = reinterpret_cast<const Prob*>(static_cast<const T*>(P.target) + ((size_t)n * (P.D + 1) + a) * P.V);
    const Prob* q = redraw && P.draft ? reinterpret_cast<const Prob*>(static_cast<const T*>(P.draft) + ((size_t)n * P.D + a) * P.V) : nullptr;
    const int sure = redraw && !P.draft ? P.tokens[(size_t)n * P.D + a] : -1;   // certain draft: q = 1 there
    unsigned long long best = 0;
    float top = 0.0f;                          // best's score
    // a second round, on p itself, where the first finds nothing left (p nowhere above q)
    for (int round = 0; round < 2; ++round) {
        for (unsigned base = begin; base < units; base += kUnits * step) {
            Prob pv[kUnits], qv[kUnits];
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                const unsigned u = base + j * step;
                if (u < units) {
                    pv[j] = p[u];
                    if (q && !round) qv[j] = q[u];
                }
            }
            if (round || base != begin) noise(base);
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                if (base + j * step >= units) break;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int v = (int)((base + j * step) * VEC + i);
                    float rest = prob(pv[j].v, i);
                    if (!round) rest -= q ? prob(qv[j].v, i) : v == sure ? 1.0f : 0.0f;
                    // the division only where the score may be above the thread's best: the product
                    // is below best x noise by more than its roundings, and far from underflow
                    const float least = top * ev[j].v[i] * 0.999999f;
                    if (rest <= least && least > 1e-30f) continue;
                    const unsigned long long key = race_key(rest, ev[j].v[i], v);
                    if (key > best) {
                        best = key;
                        top = __uint_as_float((unsigned)(key >> 32));
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
        if (lane == 0) s_best[round][tid >> 5] = best;
        __syncthreads();
        if (tid < 32) {
            best = lane < kVerThreads / 32 ? s_best[round][lane] : 0ull;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
            if (lane < split) put(&s_rank[round][rank], lane, best);
        }
        cluster_arrive();
        cluster_wait();
        best = 0;
        for (int i = 0; i < split; ++i) best = max_key(best, s_rank[round][i]);
        if (best || !redraw) break;
    }
    if (rank) return;
    if (tid == 0) P.accepted[n] = a;
    int* out = P.result + (size_t)n * (P.D + 1);
    for (int i = tid; i <= P.D; i += kVerThreads)
        out[i] = i < a ? P.tokens[(size_t)n * P.D + i] : i == a && best ? (int)~(unsigned)best : -1;
}

template <typename T, int VEC>
cudaError_t launch(const VerifyProblem& P, int split, cudaStream_t s) {
    const cudaError_t e = allow_large_clusters<verify_kernel<T, VEC>>();
    if (e != cudaSuccess) return e;
    return launch_clusters(verify_kernel<T, VEC>, (unsigned)(P.N * split), kVerThreads, 0, (unsigned)split, s, P, split);
}

// CTAs per sequence, as a cluster: up to twice the SMs in all if the rows are long enough for that.
// (fp32, with one CTA per sequence instead: 1 row of 50,257 19 us for 6 with its launch, 8 of
// 131,072 33 for 10, 128 of them 60 for 42; four times the SMs: 43.)
int split_of(int N, int V, int sms) {
    int split = 1;
    while (split < kMaxSplit && (long long)N * split * 2 <= 2LL * sms && (long long)V >= (long long)split * 2 * kMinSlice) split *= 2;
    return split;
}

template <typename T>
cudaError_t launch(const VerifyProblem& P, int sms, cudaStream_t s) {
    const int split = split_of(P.N, P.V, sms);
    // eight elements at a time where every row begins on that boundary (128 rows of 131,072: fp32 35
    // us, 45 one at a time; bf16 37 and 43)
    const auto fits = [](const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    if (P.V % 8 == 0 && fits(P.noise, 32) && fits(P.target, 8 * sizeof(T)) && fits(P.draft, 8 * sizeof(T)))
        return launch<T, 8>(P, split, s);
    return launch<T, 1>(P, split, s);
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
    int dev = 0, sms = 0;
    int* err = nullptr;
    const int rc = device_setup(&dev, &err, &sms);
    if (rc != KDA_OK) return rc;
    if (N == 0) return KDA_OK;
    VerifyProblem P{target_probs, draft_probs, draft_tokens, uniform, noise, num_drafts,
                    accepted, tokens, N, D, V, err};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = timed_launch(KDA_KERNEL_VERIFY, s, [&] {
        return dtype == KDA_BF16 ? launch<__nv_bfloat16>(P, sms, s) : launch<float>(P, sms, s);
    });
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

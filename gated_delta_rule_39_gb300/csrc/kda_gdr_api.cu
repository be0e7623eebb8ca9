// The C entry points of the gated delta rule with one decay per value head: checks,
// scratch and launches (the operation and its kernels: kda_gdr.cuh).
#include <algorithm>
#include <cmath>
#include <memory>
#include <mutex>
#include <vector>

#include "kda_gdr_chunk.cuh"

namespace kda {

size_t gdr_span(long long tokens, int heads, long long stride) {
    return tokens ? ((size_t)(tokens - 1) * stride + (size_t)heads * kDim) * 2 : 0;
}

int gdr_validate(const GdrInputs& in, int B, int K, int V, const void* s0, int s0_dtype, const void* s1,
                 int s1_dtype, long long pool) {
    if (K != kDim || V != kDim) return KDA_ERR_UNSUPPORTED_DIM;
    if (B < 0 || in.T < 0 || in.Hk < 1 || in.Hk > 65535 || in.Hv < 1 || in.Hv % in.Hk) return KDA_ERR_SHAPE;
    const long long tok = (long long)B * in.T;
    if (tok >= (1LL << 31) || tok * in.Hv * kDim >= (1LL << 40)) return KDA_ERR_SHAPE;
    if (pool < 0 || pool * in.Hv >= (1LL << 31) / 2) return KDA_ERR_SHAPE;
    if (tok > 0 && (!in.q || !in.k || !in.v || !in.g || !in.beta)) return KDA_ERR_NULL;
    if (in.gate_dtype != KDA_BF16 && in.gate_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (s0 && s0_dtype != KDA_BF16 && s0_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (s1 && s1_dtype != KDA_BF16 && s1_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (!std::isfinite(in.scale)) return KDA_ERR_ARG;
    if (in.q_stride < (long long)in.Hk * kDim || in.k_stride < (long long)in.Hk * kDim ||
        in.v_stride < (long long)in.Hv * kDim)
        return KDA_ERR_SHAPE;
    if (in.q_stride % 8 || in.k_stride % 8 || in.v_stride % 8) return KDA_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(in.q), static_cast<const void*>(in.k),
                          static_cast<const void*>(in.v), s0, s1})
        if (!aligned16(p)) return KDA_ERR_ALIGN;
    const size_t gate = in.gate_dtype == KDA_F32 ? 4 : 2;
    for (const void* p : {in.g, in.beta})
        if (reinterpret_cast<uintptr_t>(p) % gate) return KDA_ERR_ALIGN;
    return KDA_OK;
}

namespace {

size_t state_bytes(long long count, int Hv, int dtype) {
    return (size_t)count * Hv * kDim * kDim * (dtype == KDA_F32 ? 4 : 2);
}

// Whether [p, p + n) overlaps an input of the rule.
bool hits_inputs(const GdrInputs& in, long long tok, const void* p, size_t n) {
    const size_t gates = (size_t)tok * in.Hv * (in.gate_dtype == KDA_F32 ? 4 : 2);
    return overlaps(p, n, in.q, gdr_span(tok, in.Hk, in.q_stride)) ||
           overlaps(p, n, in.k, gdr_span(tok, in.Hk, in.k_stride)) ||
           overlaps(p, n, in.v, gdr_span(tok, in.Hv, in.v_stride)) || overlaps(p, n, in.g, gates) ||
           overlaps(p, n, in.beta, gates);
}

bool states_clash(const void* s0, size_t n0, int d0, const void* s1, size_t n1, int d1) {
    return overlaps(s0, n0, s1, n1) && (s0 != s1 || d0 != d1);
}

// Where a call's chunks are; returns the bytes of the map of packed sequences (first chunk
// of each, whether the offsets are valid, and the sequences by length).
size_t plan_chunks(bool varlen, int B, int T, int N, gdr::Chunks* c) {
    c->per_seq = varlen ? 0 : (T + gdr::kC - 1) / gdr::kC;
    c->total = varlen ? T / gdr::kC + N : B * c->per_seq;
    return varlen ? align_up((2 * (size_t)N + 2) * sizeof(int)) : 0;
}

constexpr int kPartUnits = 1000;          // chunks x heads from which a backward pass is done in two parts

// Scratch of a backward pass (bytes from its start): the map of packed sequences, states
// between two parts, and per (chunk, value head) a block, T, S^T, X^T, dS^T and Y^T.
struct BwdLayout {
    gdr::Chunks chunks{};
    size_t carry, blocks, ts, states, xs, dstates, ys, total;
};
BwdLayout bwd_layout(bool varlen, int B, int T, int Hv, int N) {
    BwdLayout L{};
    L.carry = plan_chunks(varlen, B, T, N, &L.chunks);
    const size_t units = (size_t)L.chunks.total * Hv;
    L.blocks = L.carry + (N == 1 && (long long)L.chunks.total * Hv >= kPartUnits ? align_up(state_bytes(1, Hv, KDA_F32)) : 0);
    L.ts = L.blocks + units * gdr::kBlockBytes;
    L.states = L.ts + units * gdr::kTileBytes;
    L.xs = align_up(L.states + units * gdr::kStateTile);
    L.dstates = L.xs + units * gdr::kTokenTile;
    L.ys = L.dstates + units * gdr::kStateTile;
    L.total = L.ys + units * gdr::kTokenTile + kAlign;
    return L;
}

// More (sequence, head) units than SMs, of fixed length and no more tokens than this, go through the
// token-by-token kernel, where a short chunk's fixed costs (8 us a unit and SM) do not arise.  32 heads, fp32
// states in place: 8 sequences of 1 and 8 tokens 15 and 17 us (in chunks 21 and 21), 256 of them 158 and 326
// (451 and 473); with 12 tokens 22 for 21 and 448 for 507.  Fewer units (8: 15 for 21 us) stay with the
// chunks.  Its arithmetic is fp32 where the chunks' operands are fp16, so the last bits of a short call
// depend on which side of the rule its number of units is: one sequence's last piece has the bits that it has
// in the whole only where its heads are no more than the SMs.
constexpr int kFewTokens = 8;

// A second stream for the calls on `s`, of its priority: one for each of the caller's streams, so that
// calls on streams that do not depend on each other do not wait for each other there.  The streams
// used last are kept (making one takes longer than a launch); one that falls out ends with its work.
struct SideStream {
    int device = -1;
    unsigned long long of = 0;             // the caller's stream: an id that is never used again
    cudaStream_t stream = nullptr;
    SideStream() = default;
    SideStream(const SideStream&) = delete;
    SideStream& operator=(const SideStream&) = delete;
    ~SideStream() {
        if (stream) cudaStreamDestroy(stream);
    }
};
constexpr size_t kSideStreams = 32;

cudaError_t side_stream(cudaStream_t s, std::shared_ptr<SideStream>* out) {
    static std::mutex mu;
    // last used first; never destroyed, since the driver may be gone by the time that statics are
    static auto& kept = *new std::vector<std::shared_ptr<SideStream>>;
    int dev = 0, priority = 0;
    unsigned long long id = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaStreamGetId(s, &id);
    if (e == cudaSuccess) e = cudaStreamGetPriority(s, &priority);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    auto at = std::find_if(kept.begin(), kept.end(), [&](const auto& x) { return x->device == dev && x->of == id; });
    if (at == kept.end()) {
        auto made = std::make_shared<SideStream>();
        made->device = dev;
        made->of = id;
        e = cudaStreamCreateWithPriority(&made->stream, cudaStreamNonBlocking, priority);
        if (e != cudaSuccess) return e;
        if (kept.size() == kSideStreams) kept.pop_back();      // a call that still has it keeps it
        at = kept.insert(kept.end(), std::move(made));
    }
    std::rotate(kept.begin(), at, at + 1);
    *out = kept.front();
    return cudaSuccess;
}

// Whether a stream is being captured into a graph (or cannot say: then it is not forked either).
bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capture) == cudaSuccess) return capture != cudaStreamCaptureStatusNone;
    cudaGetLastError();                    // not a fault of the call
    return true;
}

// How many chunks of one long sequence to prepare before its chains begin; the rest are prepared
// beside them, on the SMs that the chains (one per value head) leave.  0: not worth it, or the stream is
// being captured.  A chain takes 1.7 us per chunk and the whole GPU 0.0122 us to prepare a chunk of a
// head, so while a chain walks a chunk the idle SMs prepare `rate` of them; of two parts the first is 1
// in 1 + rate.  (Times of this GPU: others would cost some overlap, no result.  8,192 tokens: 96 heads 373 -> 343
// us, 64 heads 321 -> 283, 32 heads 268 -> 245.)
int chunks_before(const GdrChunked& P, int sms, cudaStream_t s) {
    const int units = P.in.Hv, chunks = P.chunks.total;
    if (P.in.cu || P.in.N != 1 || chunks < 64 || (long long)chunks * units < 2500 || units >= sms - sms / 8) return 0;
    if (capturing(s)) return 0;
    const float rate = 1.7f / 0.0122f * (float)(sms - units) / ((float)units * (float)sms);
    return std::max(8, (int)std::ceil((float)chunks / (1.0f + rate)));
}

// The chunks [first, first + count) of a sequence as a problem of its own.
GdrChunked part_of(const GdrChunked& P, int first, int count) {
    GdrChunked Q = P;
    const long long t = (long long)first * gdr::kC;
    const size_t gate = P.in.gate_dtype == KDA_F32 ? 4 : 2;
    Q.in.q += t * P.in.q_stride;
    Q.in.k += t * P.in.k_stride;
    Q.in.v += t * P.in.v_stride;
    Q.in.g = static_cast<const char*>(P.in.g) + (size_t)t * P.in.Hv * gate;
    Q.in.beta = static_cast<const char*>(P.in.beta) + (size_t)t * P.in.Hv * gate;
    Q.in.T = (int)std::min<long long>(P.in.T - t, (long long)count * gdr::kC);
    Q.chunks.per_seq = Q.chunks.total = count;
    Q.blocks += (size_t)first * P.in.Hv * gdr::kBlockBytes;
    if (Q.out) Q.out += t * P.in.Hv * kDim;
    const size_t at = (size_t)first * P.in.Hv;
    if (Q.states) {                        // a backward pass
        Q.states += at * gdr::kStateTile;
        Q.xs += at * gdr::kTokenTile;
        Q.ts += at * gdr::kTileBytes;
    }
    return Q;
}

// Two streams' work between two events: the second one joins the caller's again whatever happens.
struct Fork {
    std::shared_ptr<SideStream> kept;
    cudaStream_t s, side = nullptr;
    cudaEvent_t begun = nullptr, over = nullptr;
    explicit Fork(cudaStream_t s_) : s(s_) {}
    cudaError_t make() {
        cudaError_t e = side_stream(s, &kept);
        if (e == cudaSuccess) side = kept->stream;
        if (e == cudaSuccess) e = cudaEventCreateWithFlags(&begun, cudaEventDisableTiming);
        if (e == cudaSuccess) e = cudaEventCreateWithFlags(&over, cudaEventDisableTiming);
        return e;
    }
    // what comes on `side` from here on follows what is on s up to now
    cudaError_t mark() { return cudaEventRecord(begun, s); }
    cudaError_t begin() { return cudaStreamWaitEvent(side, begun, 0); }
    cudaError_t join() {
        return cudaEventRecord(over, side) == cudaSuccess ? cudaStreamWaitEvent(s, over, 0) : cudaStreamSynchronize(side);
    }
    ~Fork() {
        if (begun) cudaEventDestroy(begun);
        if (over) cudaEventDestroy(over);
    }
};

// Prep and chain in two parts, the second's prep on a stream of its own beside the first's
// chain; `carry` holds the fp32 states between the parts.  (No kernel begins early here: the chains'
// CTAs would hold SMs that prep could use, 8,192 tokens x 96 heads 358 us for 334.)
cudaError_t run_in_parts(const GdrChunked& P, int first, float* carry, int sms, cudaStream_t s) {
    GdrChunked a = part_of(P, 0, first), b = part_of(P, first, P.chunks.total - first);
    a.final_state = carry;
    a.final_dtype = KDA_F32;
    b.init_state = carry;
    b.init_dtype = KDA_F32;
    const auto prep = [&](const GdrChunked& part, cudaStream_t on) {
        return timed_launch(KDA_KERNEL_GDR_PREP, on, [&] { return launch_gdr_prep(part, sms, false, on); });
    };
    const auto chain = [&](const GdrChunked& part) {
        return timed_launch(KDA_KERNEL_GDR_CHAIN, s, [&] { return launch_gdr_chain(part, false, s); });
    };
    Fork fork(s);
    cudaError_t e = fork.make();
    if (e == cudaSuccess) e = prep(a, s);
    if (e == cudaSuccess) e = fork.mark();
    if (e == cudaSuccess) e = chain(a);
    if (e == cudaSuccess) e = fork.begin();
    if (e == cudaSuccess) {
        e = prep(b, fork.side);
        const cudaError_t joined = fork.join();
        if (e == cudaSuccess) e = joined;
    }
    if (e == cudaSuccess) e = chain(b);
    return e;
}

// The same for a backward pass, after prep: whether one long sequence of few heads is worth two parts,
bool in_two_parts(const GdrInputs& in, int chunks, int sms) {
    return !in.cu && in.N == 1 && (long long)chunks * in.Hv >= kPartUnits && 4 * in.Hv <= sms;
}
// and how many chunks at its end to have the gradient's chain walk first, so that the chunk kernel
// can take them beside the rest of the chain, on the SMs that it leaves.  The gradient's chain takes 2.4
// us per chunk, the one for the states, which has to be over by then, 1.6, and the chunk kernel on the
// whole GPU 0.073 us per chunk and head (times of this GPU; the ones measured last, 2.45, 1.7 and 0.076, choose no
// better).  (4,096 tokens: 32 heads 354 -> 326 us, 16 heads 270 -> 240; 8,192 tokens, 8 heads: 410 -> 357.)
int chunks_first(const GdrBackward& B, int sms, cudaStream_t s) {
    const int units = B.fwd.in.Hv, chunks = B.fwd.chunks.total;
    if (!in_two_parts(B.fwd.in, chunks, sms)) return 0;
    if (capturing(s)) return 0;
    const float rate = 0.073f / 2.4f * (float)units * (float)sms / (float)(sms - units);
    return std::min(chunks - 1, (int)((float)chunks * std::max(1.6f / 2.4f, 1.0f / (1.0f + rate))));
}

GdrBackward part_of(const GdrBackward& B, int first, int count) {
    GdrBackward C = B;
    const GdrInputs& in = B.fwd.in;
    const size_t t = (size_t)first * gdr::kC, at = (size_t)first * in.Hv, gate = in.gate_dtype == KDA_F32 ? 4 : 2;
    C.fwd = part_of(B.fwd, first, count);
    C.in.dout += t * in.Hv * kDim;
    C.dstates += at * gdr::kStateTile;
    C.ys += at * gdr::kTokenTile;
    C.dq += t * in.Hk * kDim;
    C.dk += t * in.Hk * kDim;
    C.dv += t * in.Hv * kDim;
    C.dg = static_cast<char*>(B.dg) + t * in.Hv * gate;
    C.dbeta = static_cast<char*>(B.dbeta) + t * in.Hv * gate;
    return C;
}

// Chains and chunk kernel, in two parts if `last` (chunks at the end) is not 0; `carry` holds the fp32
// gradient of the states between them.
cudaError_t run_backward(const GdrBackward& B, int last, float* carry, int sms, cudaStream_t s) {
    const auto chain = [&](const GdrBackward& part, const GdrChunked* states_too) {
        return timed_launch(KDA_KERNEL_GDR_BWD_CHAIN, s, [&] { return launch_gdr_bwd_chain(part, states_too, s); });
    };
    const int split = gdr_bwd_chunk_split(B, sms);
    const auto chunk = [&](const GdrBackward& part, int on_sms, cudaStream_t on) {
        return timed_launch(KDA_KERNEL_GDR_BWD_CHUNK, on, [&] { return launch_gdr_bwd_chunk(part, split, on_sms, on); });
    };
    if (!last) {
        const cudaError_t e = chain(B, &B.fwd);
        return e == cudaSuccess ? chunk(B, sms, s) : e;
    }
    const int first = B.fwd.chunks.total - last;
    GdrBackward a = part_of(B, 0, first), b = part_of(B, first, last);
    a.in.dfinal = b.dinit = carry;
    a.in.dfinal_dtype = b.dinit_dtype = KDA_F32;
    if (!b.fwd.init_state) b.fwd.init_state = carry;       // (not read) its first chunk has a state before it
    Fork fork(s);
    cudaError_t e = fork.make();
    if (e == cudaSuccess) e = chain(b, &B.fwd);
    if (e == cudaSuccess) e = fork.mark();
    if (e == cudaSuccess) e = chain(a, nullptr);
    if (e == cudaSuccess) e = fork.begin();
    if (e == cudaSuccess) {
        e = chunk(b, sms - B.fwd.in.Hv, fork.side);
        if (e == cudaSuccess) e = chunk(a, sms, s);
        const cudaError_t joined = fork.join();
        if (e == cudaSuccess) e = joined;
    }
    return e;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_gdr_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
                 int gate_dtype, float scale, void* out, const void* state_in, int state_in_dtype,
                 void* state_out, int state_out_dtype, const int32_t* slots, int num_slots,
                 const int32_t* lengths, int N, int T, int Hk, int Hv, int K, int V,
                 long long q_stride, long long k_stride, long long v_stride, void* stream) {
    GdrStep P{};
    P.in = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
            static_cast<const __nv_bfloat16*>(v), q_stride, k_stride, v_stride, g, beta, gate_dtype,
            scale, nullptr, nullptr, N, T, Hk, Hv};
    const long long pool = slots ? num_slots : N;
    int rc = gdr_validate(P.in, N, K, V, state_in, state_in_dtype, state_out, state_out_dtype,
                          std::max<long long>(pool, N));
    if (rc != KDA_OK) return rc;
    if (slots && num_slots < 1) return KDA_ERR_SHAPE;
    if (!aligned16(out)) return KDA_ERR_ALIGN;
    for (const int32_t* p : {slots, lengths})
        if (reinterpret_cast<uintptr_t>(p) % 4) return KDA_ERR_ALIGN;
    const long long tok = (long long)N * T;
    const size_t n_out = (size_t)tok * Hv * kDim * 2, n_ids = (size_t)N * 4;
    const size_t n_in = state_bytes(pool, Hv, state_in_dtype), n_so = state_bytes(pool, Hv, state_out_dtype);
    if (hits_inputs(P.in, tok, out, n_out) || hits_inputs(P.in, tok, state_out, n_so) ||
        overlaps(out, n_out, state_in, n_in) || overlaps(out, n_out, state_out, n_so) ||
        states_clash(state_in, n_in, state_in_dtype, state_out, n_so, state_out_dtype))
        return KDA_ERR_ALIAS;
    for (const int32_t* p : {slots, lengths})
        if (overlaps(out, n_out, p, n_ids) || overlaps(state_out, n_so, p, n_ids)) return KDA_ERR_ALIAS;
    int dev = 0;
    int* err = nullptr;
    rc = device_setup(&dev, &err);
    if (rc != KDA_OK) return rc;
    P.out = static_cast<__nv_bfloat16*>(out);
    P.state_in = state_in;
    P.in_dtype = state_in_dtype;
    P.state_out = state_out;
    P.out_dtype = state_out_dtype;
    P.slots = slots;
    P.lengths = lengths;
    P.pool = (int)pool;
    P.err = err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = timed_launch(KDA_KERNEL_GDR_STEP, s, [&] { return launch_gdr_step(P, s); });
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

int kda_gdr_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                int gate_dtype, float scale, void* out, const void* initial_state,
                int initial_state_dtype, void* final_state, int final_state_dtype,
                const int32_t* cu_seqlens, int num_seqs, int B, int T, int Hk, int Hv, int K, int V,
                long long q_stride, long long k_stride, long long v_stride, void* stream) {
    const bool varlen = cu_seqlens != nullptr;
    const int N = varlen ? num_seqs : B;
    GdrChunked P{};
    P.in = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
            static_cast<const __nv_bfloat16*>(v), q_stride, k_stride, v_stride, g, beta, gate_dtype,
            scale, cu_seqlens, nullptr, N, T, Hk, Hv};
    if (B < 1 || (varlen && (B != 1 || num_seqs < 1))) return KDA_ERR_SHAPE;
    int rc = gdr_validate(P.in, B, K, V, initial_state, initial_state_dtype, final_state,
                          final_state_dtype, N);
    if (rc != KDA_OK) return rc;
    const long long tok = (long long)B * T;
    if (tok > 0 && !out) return KDA_ERR_NULL;
    if (!aligned16(out) || reinterpret_cast<uintptr_t>(cu_seqlens) % 4) return KDA_ERR_ALIGN;
    const size_t n_out = (size_t)tok * Hv * kDim * 2;
    const size_t n_in = state_bytes(N, Hv, initial_state_dtype), n_so = state_bytes(N, Hv, final_state_dtype);
    if (hits_inputs(P.in, tok, out, n_out) || hits_inputs(P.in, tok, final_state, n_so) ||
        overlaps(out, n_out, initial_state, n_in) || overlaps(out, n_out, final_state, n_so) ||
        states_clash(initial_state, n_in, initial_state_dtype, final_state, n_so, final_state_dtype) ||
        overlaps(out, n_out, cu_seqlens, ((size_t)N + 1) * 4) ||
        overlaps(final_state, n_so, cu_seqlens, ((size_t)N + 1) * 4))
        return KDA_ERR_ALIAS;
    int dev = 0, sms = 0;
    rc = device_setup(&dev, &P.err, &sms);
    if (rc != KDA_OK) return rc;
    P.out = static_cast<__nv_bfloat16*>(out);
    P.init_state = initial_state;
    P.init_dtype = initial_state_dtype;
    P.final_state = final_state;
    P.final_dtype = final_state_dtype;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!varlen && T <= kFewTokens && (long long)N * Hv > sms) {
        const GdrStep Q{P.in, P.out, initial_state, initial_state_dtype, final_state, final_state_dtype, nullptr, nullptr, N, P.err};
        const cudaError_t e = timed_launch(KDA_KERNEL_GDR_STEP, s, [&] { return launch_gdr_step(Q, s); });
        return e == cudaSuccess ? KDA_OK : cuda_fail(KDA_ERR_LAUNCH, e);
    }
    const size_t map_bytes = plan_chunks(varlen, B, T, N, &P.chunks);
    unsigned char* scratch = nullptr;
    const size_t block_bytes = align_up(map_bytes + (size_t)P.chunks.total * Hv * gdr::kBlockBytes);
    const int first_part = chunks_before(P, sms, s);
    cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&scratch),
                                    block_bytes + (first_part ? state_bytes(1, Hv, KDA_F32) : 0) + kAlign, s);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_ALLOC, e);
    P.blocks = scratch + map_bytes;
    if (varlen) {
        int* first = reinterpret_cast<int*>(scratch);
        P.chunks.first = first;
        P.in.valid = first + N + 1;
        P.chunks.order = first + N + 2;
        e = timed_launch(KDA_KERNEL_GDR_MAP, s,
                         [&] { return launch_gdr_map(P.in, first, first + N + 2, first + N + 1, P.err, s); });
    }
    if (first_part) {
        e = run_in_parts(P, first_part, reinterpret_cast<float*>(scratch + block_bytes), sms, s);
    } else {
        if (e == cudaSuccess) e = timed_launch(KDA_KERNEL_GDR_PREP, s, [&] { return launch_gdr_prep(P, sms, true, s); });
        if (e == cudaSuccess)
            e = timed_launch(KDA_KERNEL_GDR_CHAIN, s, [&] { return launch_gdr_chain(P, true, s); });
    }
    cudaFreeAsync(scratch, s);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

size_t kda_gdr_bwd_workspace_bytes(int B, int T, int Hk, int Hv, int num_seqs, int varlen) {
    if (B < 1 || T < 0 || Hk < 1 || Hv < 1 || (varlen && num_seqs < 1)) return 0;
    return bwd_layout(varlen != 0, B, T, Hv, varlen ? num_seqs : B).total;
}

int kda_gdr_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                int gate_dtype, float scale, const void* initial_state, int initial_state_dtype,
                const void* d_out, const void* d_final_state, int d_final_state_dtype, void* dq, void* dk,
                void* dv, void* dg, void* dbeta, void* d_initial_state, int d_initial_state_dtype,
                const int32_t* cu_seqlens, int num_seqs, int B, int T, int Hk, int Hv, int K, int V,
                long long q_stride, long long k_stride, long long v_stride, void* stream) {
    const bool varlen = cu_seqlens != nullptr;
    const int N = varlen ? num_seqs : B;
    GdrBackward P{};
    GdrInputs& in = P.fwd.in;
    in = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
          static_cast<const __nv_bfloat16*>(v), q_stride, k_stride, v_stride, g, beta, gate_dtype,
          scale, cu_seqlens, nullptr, N, T, Hk, Hv};
    if (B < 1 || (varlen && (B != 1 || num_seqs < 1))) return KDA_ERR_SHAPE;
    int rc = gdr_validate(in, B, K, V, initial_state, initial_state_dtype, d_final_state,
                          d_final_state_dtype, N);
    if (rc != KDA_OK) return rc;
    if (d_initial_state && d_initial_state_dtype != KDA_BF16 && d_initial_state_dtype != KDA_F32)
        return KDA_ERR_DTYPE;
    const long long tok = (long long)B * T;
    if (tok > 0 && (!d_out || !dq || !dk || !dv || !dg || !dbeta)) return KDA_ERR_NULL;
    for (const void* p : {d_out, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv), static_cast<const void*>(d_initial_state)})
        if (!aligned16(p)) return KDA_ERR_ALIGN;
    const size_t gate = gate_dtype == KDA_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(dg) % gate || reinterpret_cast<uintptr_t>(dbeta) % gate ||
        reinterpret_cast<uintptr_t>(cu_seqlens) % 4)
        return KDA_ERR_ALIGN;
    const size_t nk = (size_t)tok * Hk * kDim * 2, nv = (size_t)tok * Hv * kDim * 2, ng = (size_t)tok * Hv * gate;
    const void* out_p[] = {dq, dk, dv, dg, dbeta, d_initial_state};
    const size_t out_n[] = {nk, nk, nv, ng, ng, state_bytes(N, Hv, d_initial_state_dtype)};
    const void* in_p[] = {initial_state, d_out, d_final_state, cu_seqlens};
    const size_t in_n[] = {state_bytes(N, Hv, initial_state_dtype), nv, state_bytes(N, Hv, d_final_state_dtype),
                           ((size_t)N + 1) * 4};
    for (int o = 0; o < 6; ++o) {
        if (hits_inputs(in, tok, out_p[o], out_n[o])) return KDA_ERR_ALIAS;
        for (int i = 0; i < 4; ++i)
            if (overlaps(out_p[o], out_n[o], in_p[i], in_n[i])) return KDA_ERR_ALIAS;
        for (int o2 = o + 1; o2 < 6; ++o2)
            if (overlaps(out_p[o], out_n[o], out_p[o2], out_n[o2])) return KDA_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    rc = device_setup(&dev, &P.fwd.err, &sms);
    if (rc != KDA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const BwdLayout L = bwd_layout(varlen, B, T, Hv, N);
    unsigned char* scratch = nullptr;
    cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&scratch), L.total, s);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_ALLOC, e);
    P.fwd.chunks = L.chunks;
    P.fwd.blocks = scratch + L.blocks;
    P.fwd.ts = scratch + L.ts;
    P.fwd.init_state = initial_state;
    P.fwd.init_dtype = initial_state_dtype;
    P.fwd.states = scratch + L.states;
    P.fwd.xs = scratch + L.xs;
    P.in.dout = static_cast<const __nv_bfloat16*>(d_out);
    P.in.dfinal = d_final_state;
    P.in.dfinal_dtype = d_final_state_dtype;
    P.dstates = scratch + L.dstates;
    P.ys = scratch + L.ys;
    P.dq = static_cast<__nv_bfloat16*>(dq);
    P.dk = static_cast<__nv_bfloat16*>(dk);
    P.dv = static_cast<__nv_bfloat16*>(dv);
    P.dg = dg;
    P.dbeta = dbeta;
    P.dinit = d_initial_state;
    P.dinit_dtype = d_initial_state_dtype;
    if (varlen) {
        int* first = reinterpret_cast<int*>(scratch);
        P.fwd.chunks.first = first;
        in.valid = first + N + 1;
        P.fwd.chunks.order = first + N + 2;
        e = timed_launch(KDA_KERNEL_GDR_MAP, s,
                         [&] { return launch_gdr_map(in, first, first + N + 2, first + N + 1, P.fwd.err, s); });
    }
    if (e == cudaSuccess) e = timed_launch(KDA_KERNEL_GDR_PREP, s, [&] { return launch_gdr_prep(P, sms, s); });
    if (e == cudaSuccess)
        e = run_backward(P, chunks_first(P, sms, s), reinterpret_cast<float*>(scratch + L.carry), sms, s);
    cudaFreeAsync(scratch, s);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

}  // extern "C"

// The chunked form of the gated delta rule with one decay per value head: the layout of
// its scratch and the tensor-core helpers its kernels share.
//
// A chunk is 64 tokens.  With G the running sum of g inside it, M_ij = e^(G_i - G_j) for
// j <= i, A the strictly lower triangle of beta_i M_ij k_i.k_j, T = (I + A)^-1 and S the
// state before it,
//
//   R = V - e^G K S,  X = T beta R            (row j of X is the update d_j)
//   O = scale (e^G Q S + (M . Q K^T) X)
//   S <- e^(G_C) S + (e^(G_C - G) K)^T X
//
// T and P = M . Q K^T depend on queries, keys and gates alone: the prep kernel forms
// them for all chunks in parallel; the chain kernel then walks the chunks of a sequence.
//
// Numerics: G, the decays and every product's accumulator are fp32, and so is the state
// between chunks.  The operands of the tensor-core products are fp16: queries, keys (bf16
// data) times their decays, T beta, P, R, X and the rounded state.
// fp16's 11 bits keep states within 2^-10 of the exact ones on unit keys (3.3 to 5.2e-4 of their norm; gradients of
// the gates and of the initial state 3 to 12e-4), where bf16 operands gave 3e-3.  Its price is its range: values, states and gradients are scaled for it (below);
// queries, keys, q.k and the entries of T beta are not.  The inverse T is formed in fp32 with tf32 products
// between its blocks.
#pragma once
#include "kda_cluster.cuh"
#include "kda_gdr.cuh"

#ifndef KDA_WAIT_TRIES
#define KDA_WAIT_TRIES (1u << 20)    // of a wait inside a kernel (a fraction of a second to 20 s)
#endif

namespace kda {
namespace gdr {

constexpr int kC = 64;                        // tokens per chunk
// One (chunk, value head)'s block of scratch: T beta (columns scaled) and P as fp16 [64][64]
// tiles (128-byte rows whose 16-byte units are stored at unit ^ (row & 7)), then fp32 b, b e^G, e^G, e^(G_C - G)
// and G (in base 2) of its 64 tokens, and of the whole chunk e^(G_C), the biased exponent of the largest
// |scale dO| (of four parts of the rows, a byte each) and the scales (int) that the forward and the backward chain chose.
constexpr int kTileBytes = kC * kC * 2;
constexpr int kGateB = 0, kGateBe = kC, kGateE = 2 * kC, kGateEnd = 3 * kC, kGateG = 4 * kC, kGateAll = 5 * kC;
constexpr int kGateDo = kGateAll + 1, kGateScale = kGateAll + 2, kGateGradScale = kGateAll + 3;
static_assert(kGateScale % 2 == 0 && kGateGradScale == kGateScale + 1, "one access");
constexpr int kGateFloats = kGateAll + 4;
constexpr int kBlockUsed = 2 * kTileBytes + kGateFloats * 4;   // 17,680
constexpr int kBlockBytes = (kBlockUsed + 127) / 128 * 128;

struct Chunks {           // where the chunks of each sequence are
    const int* first;     // [N + 1] first chunk of each sequence (packed), or nullptr
    const int* order;     // [N] the sequences by falling length (packed), or nullptr
    int per_seq;          // fixed length: chunks of each sequence
    int total;            // chunks in all (packed: an upper bound)
};

struct Span {
    long long start;      // first token
    int len;              // tokens
    int chunk;            // first chunk
};
__device__ __forceinline__ Span span_of(const GdrInputs& I, const Chunks& C, int n) {
    if (I.cu) return {I.cu[n], I.cu[n + 1] - I.cu[n], C.first[n]};
    return {(long long)n * I.T, I.T, n * C.per_seq};
}

// The i-th sequence that a chain kernel takes.
__device__ __forceinline__ int sequence_of(const Chunks& C, int i) { return C.order ? C.order[i] : i; }

// Sequence and place of a chunk; false past the end of packed sequences (or for bad ones).
__device__ __forceinline__ bool find_chunk(const GdrInputs& I, const Chunks& C, int chunk, int& n, int& c) {
    if (!I.cu) {
        n = chunk / C.per_seq;
        c = chunk % C.per_seq;
        return true;
    }
    if (!*I.valid || chunk >= C.first[I.N]) return false;
    int lo = 0, hi = I.N;              // the last sequence whose first chunk is at most `chunk`
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (C.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    n = lo;
    c = chunk - C.first[n];
    return true;
}

// ---- mbarriers ----------------------------------------------------------------------
// Of a wait for what is on its way already (copies, MMAs, warps that are leaving): a role that
// gave up on something else still waits for these.
constexpr unsigned kDrainTries = 1u << 20;
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(b)) : "memory");
}
// Waits, as a whole warp, for a phase to end; after `tries` tries (each of which sleeps
// for up to 20 us, as the hardware sees fit) records a timeout and gives up.  Every lane gets
// the same answer.  Kept short: it is part of every role's loop.
__device__ __forceinline__ bool bar_wait(uint64_t* b, unsigned parity, int* err, unsigned tries = KDA_WAIT_TRIES) {
#pragma unroll 1
    for (unsigned n = 0; n < tries; ++n) {
        unsigned ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
        if (__all_sync(0xFFFFFFFFu, ok)) return true;
    }
    set_error(err, KDA_ERR_DEVICE_TIMEOUT);
    return false;
}

// ---- fragments --------------------------------------------------------------------------
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void stsm(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n"
                 ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n"
                 ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
// D += A(16x16 bf16, row) * B(16x8 bf16, col), fp32 accumulate
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// fp32 bits rounded to tf32 (nearest, ties away): the tensor core reads the top 19 bits
__device__ __forceinline__ uint32_t tf32_bits(float x) { return __float_as_uint(x) + 0x1000u; }

// Shared-memory tiles of 16-bit elements whose rows hold a power of two of 16-byte units:
// unit u of row r is at unit u ^ (r & 7), which spreads the 8 rows of an ldmatrix over the
// banks.  kRow = bytes per row.
template <int kRow>
__device__ __forceinline__ uint32_t unit_at(uint32_t base, int row, int unit) {
    return base + row * kRow + ((unit ^ (row & 7)) << 4);
}
// ldmatrix address of this lane for a 16 x 16 block as an A operand (or, stored transposed,
// as two B operands): rows r0 .. r0 + 15, units u0, u0 + 1; the matrices come in the order
// (rows 0-7, u0), (rows 8-15, u0), (rows 0-7, u0 + 1), (rows 8-15, u0 + 1)
template <int kRow>
__device__ __forceinline__ uint32_t a_addr(uint32_t base, int r0, int u0, int lane) {
    return unit_at<kRow>(base, r0 + (lane & 15), u0 + (lane >> 4));
}
// the same for two B operands whose n runs along the rows and k along the units: matrices
// (rows 0-7, u0), (rows 0-7, u0 + 1), (rows 8-15, u0), (rows 8-15, u0 + 1)
template <int kRow>
__device__ __forceinline__ uint32_t b_addr(uint32_t base, int r0, int u0, int lane) {
    return unit_at<kRow>(base, r0 + (lane & 7) + ((lane >> 4) << 3), u0 + ((lane >> 3) & 1));
}

// What the backward pass keeps of each (chunk, value head), in fp16: S^T before the chunk (128
// value channels x 128 key channels) and the gradient of the state after it (dS^T), X^T and
// Y^T (128 x 64 tokens), T.  Rows are value channels; the 16-byte unit u of row v is at
// (128 u + v) * 16, so that a warp whose lanes are rows writes 512 consecutive bytes, and 8
// rows of an ldmatrix are 128 consecutive ones.
__device__ __forceinline__ int row_unit(int v, int u) { return (128 * u + v) * 16; }
constexpr int kStateTile = kDim * kDim * 2;
constexpr int kTokenTile = kDim * kC * 2;

// ---- scales -------------------------------------------------------------------------------
// fp16 keeps its 11 bits between 2^-14 and 65,504.  All that a chain rounds to it is linear in V and
// the initial state (S, R, X), or in the gradients that come in (dO, dS, dX, Y).  So a chain works on
// them times a power of two, 2^scale, that it chooses again for every chunk from the exponent of
// the largest of what enters there, and results of any size keep their accuracy.  A scale stays while that
// exponent is in a window: forwards 2^-6 .. 2^6, so that ordinary values are taken as they are, and
// backwards 2^-1 .. 2^7, where rows of dX and Y may be far apart.  Above it 9 bits are left for what a chunk's 64 tokens
// and the two chunks that the choice does not know yet can add up to with queries and keys of length 1.
constexpr int kNothing = -1000;            // exponent of zero and of what is not finite
__device__ __forceinline__ int exponent_of(float x) {      // of a magnitude
    const int e = (int)(__float_as_uint(x) >> 23);
    return e == 0 || e == 255 ? kNothing : e - 127;
}
__device__ __forceinline__ int exponent_of_bytes(unsigned x) {       // the largest of four biased ones
    x = __vmaxu4(x, x >> 16);
    x = max(x & 0xFFu, x >> 8 & 0xFFu);
    return x == 0 || x == 255 ? kNothing : (int)x - 127;
}
// The scale of what is next, whose largest has exponent e.  Exponents of 120 and more in a scale would leave fp32.
__device__ __forceinline__ int next_scale(int scale, int e, int low, int high, int best) {
    if (e == kNothing || (e + scale >= low && e + scale <= high)) return scale;
    return max(-120, min(120, best - e));
}
__device__ __forceinline__ int forward_scale(int scale, int e) { return next_scale(scale, e, -6, 5, 2); }
__device__ __forceinline__ int gradient_scale(int scale, int e) { return next_scale(scale, e, -1, 6, 3); }
__device__ __forceinline__ float power_of_two(int e) {     // e <= 127; 0 below fp32's normal numbers
    return e < -126 ? 0.0f : __int_as_float((e + 127) << 23);
}
// x 2^e for |e| <= 252, without leaving fp32 on the way
__device__ __forceinline__ float times_power(float x, int e) { return x * power_of_two(e / 2) * power_of_two(e - e / 2); }

}  // namespace gdr

struct GdrChunked {       // a chunked forward pass
    GdrInputs in;
    gdr::Chunks chunks;
    unsigned char* blocks;            // [chunk][Hv] blocks of kBlockBytes
    __nv_bfloat16* out;
    const void* init_state;           // [N][Hv][128][128] or nullptr
    int init_dtype;
    void* final_state;                // or nullptr
    int final_dtype;
    int* err;
    // backward pass: the forward pass keeps states and X instead of writing outputs
    unsigned char* states = nullptr;  // [chunk][Hv] of kStateTile
    unsigned char* xs = nullptr;      // [chunk][Hv] of kTokenTile
    unsigned char* ts = nullptr;      // [chunk][Hv] of kTileBytes: T without beta
};

struct GdrGrads {         // the gradients that enter a backward pass
    const __nv_bfloat16* dout;        // [tokens][Hv][128]
    const void* dfinal;               // [N][Hv][128][128] or nullptr
    int dfinal_dtype;
};

struct GdrBackward {      // what the backward pass has besides
    GdrChunked fwd;
    GdrGrads in;
    unsigned char* dstates;           // [chunk][Hv] of kStateTile: gradient of the state after
    unsigned char* ys;                // [chunk][Hv] of kTokenTile: Y^T
    __nv_bfloat16 *dq, *dk, *dv;      // [tokens][heads][128]
    void *dg, *dbeta;                 // [tokens][Hv] of the gates' type
    void* dinit;                      // [N][Hv][128][128] of dinit_dtype or nullptr
    int dinit_dtype;
};

// the gradient's chain, and with it the one that computes the states of `states_too` again (or nullptr)
cudaError_t launch_gdr_bwd_chain(const GdrBackward& P, const GdrChunked* states_too, cudaStream_t s);
// on `sms` SMs, with `split` CTAs (a cluster) to a (chunk, key head) pair
cudaError_t launch_gdr_bwd_chunk(const GdrBackward& P, int split, int sms, cudaStream_t s);
// as many as the whole call has room for; its parts take the same, since the order in which a
// group's heads are added up depends on it
int gdr_bwd_chunk_split(const GdrBackward& P, int sms);
cudaError_t launch_gdr_map(const GdrInputs& in, int* first, int* order, int* valid, int* err, cudaStream_t s);
// `early`: may begin before the kernel before it has ended
cudaError_t launch_gdr_prep(const GdrChunked& P, int sms, bool early, cudaStream_t s);
cudaError_t launch_gdr_prep(const GdrBackward& P, int sms, cudaStream_t s);   // finds the largest |scale dO| too
cudaError_t launch_gdr_chain(const GdrChunked& P, bool early, cudaStream_t s);

}  // namespace kda

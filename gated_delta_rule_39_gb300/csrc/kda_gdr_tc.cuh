// What the two chain kernels of the gated delta rule (forwards and backwards) share: tiles in
// shared memory as tcgen05.mma reads them, products, and the hand-over between warps.
#pragma once
#include "kda_gdr_chunk.cuh"
#include "kda_tcgen05_warp.cuh"

namespace kda {
namespace gdr {

// ---- tiles ----------------------------------------------------------------------------------
// 64 tokens x 128 channels of 16-bit elements: two blocks of 64 channels, rows of 128 bytes (one
// token) with the 128-byte swizzle.  Read with the channels along k (K-major) or, with the
// tokens along k, as an operand whose M or N index (the channel) is contiguous (MN-major).
constexpr int kRowsTile = kC * kDim * 2;
constexpr int kHalfTile = kC * 128;
__device__ __forceinline__ int rows_tile_at(int token, int unit) {   // byte of a 16-byte unit
    return (unit >> 3) * kHalfTile + token * 128 + (((unit & 7) ^ (token & 7)) << 4);
}
constexpr int kTokenRows = 8;             // tokens of a row tile that a producer thread holds
constexpr int kProducers = 128;           // threads of a group: (token row0 + 8 i, unit)

// Descriptors: K-major tiles start at their k-step's 32 bytes, 4 steps a block
__device__ __forceinline__ uint64_t desc_k(uint32_t smem) { return tc::smem_desc(smem, 16, 1024, tc::kSwizzle128B); }
// MN-major: 64 indices per block, `block` bytes to the next ones
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem, uint32_t block) {
    return tc::smem_desc(smem, block, 1024, tc::kSwizzle128B);
}
__host__ __device__ constexpr int kstep_k(int k, int block) { return ((k >> 2) * block + (k & 3) * 32) >> 4; }
__host__ __device__ constexpr int kstep_mn(int k) { return (k * 16 * 128) >> 4; }      // 16 rows of k

constexpr uint32_t kId64 = tc::idesc_f16_f32(128, kC), kId128 = tc::idesc_f16_f32(128, kDim);

// D (+)= A B^T, A in tensor memory (16 kSteps deep); B a K-major tile.  Issued by the lane
// whose `on` is set; the whole warp comes by.
template <int kSteps>
__device__ __forceinline__ void product_k(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add, uint32_t on) {
    const uint64_t desc = desc_k(b);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) tc::mma_ts_on(d, a + 8 * k, desc + kstep_k(k, kHalfTile), id, add || k > 0, on);
}
// the same over 64 tokens with B an MN-major tile (blocks of 64 columns kHalfTile apart)
__device__ __forceinline__ void product_mn(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add, uint32_t on) {
    const uint64_t desc = desc_mn(b, kHalfTile);
#pragma unroll
    for (int k = 0; k < 4; ++k) tc::mma_ts_on(d, a + 8 * k, desc + kstep_mn(k), id | tc::kIdMnB, add || k > 0, on);
}
// the same in all lanes, and known to the compiler to be
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// the line of p into L2
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

// ---- copies by the tensor memory accelerator ---------------------------------------------------
// 64 rows x 64 channels, one block of a row tile
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap* map, int channel, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(channel), "r"(row), "r"(bar) : "memory");
}

// The rows of a chunk of one head on their way to a tile: fetched to registers a chunk ahead.
struct Rows {
    const __nv_bfloat16* src;                 // row row0 of the sequence, this thread's unit
    long long stride;
    int len, row0;
    uint4 x[kTokenRows];
    __device__ __forceinline__ Rows(const __nv_bfloat16* base, long long stride_, const Span& span, int channel, int p)
        : src(base + (span.start + (p >> 4)) * stride_ + channel + (p & 15) * 8), stride(stride_), len(span.len), row0(p >> 4) {}
    __device__ __forceinline__ void fetch(int c) {
        const int rows = len - c * kC - row0;
        const __nv_bfloat16* s = src + (long long)c * kC * stride;
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            x[i] = 8 * i < rows ? __ldg(reinterpret_cast<const uint4*>(s)) : make_uint4(0u, 0u, 0u, 0u);
            s += 8 * stride;
        }
    }
};
// into L2: the line that thread p has of a chunk's rows
__device__ __forceinline__ void prefetch_rows(const __nv_bfloat16* base, long long stride, const Span& span, int channel, int c, int p) {
    const int row = c * kC + (p >> 1);
    if (row >= 0 && row < span.len) prefetch_l2(base + (span.start + row) * stride + channel + 64 * (p & 1));
}

// ---- hand-over -----------------------------------------------------------------------------
constexpr int kStateWarps = 8;            // 128 lanes x two halves of the columns
// This warp's part of an operand is in tensor memory (and it has read what it comes from).
__device__ __forceinline__ void operand_ready(uint64_t* bar, int lane) {
    tc::wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
}
// pairs of fp32 registers as fp16
template <int kN>
__device__ __forceinline__ void to_half(const uint32_t (&x)[2 * kN], uint32_t (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = pack_half2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
}
template <typename T>
__device__ __forceinline__ T& aligned_smem(unsigned char* raw) {
    return *reinterpret_cast<T*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
}
// 32 fp16 values of row v of a tile kept in memory, from unit u on: the lanes of a warp are rows
// next to one another, so a store is 512 consecutive bytes
__device__ __forceinline__ void keep_units(unsigned char* tile, int v, int u, const uint32_t (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(tile + row_unit(v, u + i)) = make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
__device__ __forceinline__ void scale32(uint32_t (&x)[32], float d) {
    unsigned long long dd;
    asm("mov.b64 %0, {%1, %1};" : "=l"(dd) : "f"(d));
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        unsigned long long v;
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x[i]), "r"(x[i + 1]));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(dd));
        asm("mov.b64 {%0, %1}, %2;" : "=r"(x[i]), "=r"(x[i + 1]) : "l"(v));
    }
}
// ---- scales ----------------------------------------------------------------------------------
// One warp of a chain chooses the scales; the others find the factors that they need here.  Entry i % 4
// is chunk i's (as the chain walks); what is published before chunk i is at i % 4 too.
struct ScaleRing {
    int top[4][kStateWarps];                  // exponents of each state warp's largest
    float ratio[4];                           // of a chunk's scale to the one before
    float in[4], out[4];                      // backwards `scale` 2^scale, for dO; 2^-scale, for results
    int look[4];                              // forwards: whether the state's size is to be published in a chunk
};
// the largest exponent that the state warps published, in a scale, before chunk i
__device__ __forceinline__ int published(const ScaleRing& R, int i, int scale) {
    int e = kNothing;
#pragma unroll
    for (int w = 0; w < kStateWarps; ++w) e = max(e, R.top[i & 3][w]);
    return e == kNothing ? kNothing : e - scale;
}
// The exponents of the state warps' largest, each warp's at its place.  Of a state,
__device__ __forceinline__ void publish(int& top, float largest, int lane) {
    const int e = exponent_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(largest))));
    if (lane == 0) top = e;
}
__device__ __forceinline__ void publish(int& top, const uint32_t (&x)[2][32], int lane) {
    float m[4] = {};
#pragma unroll
    for (int i = 0; i < 64; ++i) m[i & 3] = fmaxf(m[i & 3], fabsf(__uint_as_float(x[i >> 5][i & 31])));
    publish(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), lane);
}
// and, a chunk on, of d times one whose fp16 pairs are in tensor memory, in the chunk's scale.  (Read again from
// there: kept in registers for this, they cost the backward pass 140 cycles a chunk, whether it looks or not.)
__device__ __forceinline__ void publish(int& top, uint32_t taddr, float d, int lane) {
    uint32_t f[32];
    tc::ld32(taddr, f);
    tc::wait_ld();
    __half2 m[2] = {__float2half2_rn(0.0f), __float2half2_rn(0.0f)};
#pragma unroll
    for (int i = 0; i < 32; ++i) m[i & 1] = __hmax2(m[i & 1], __habs2(*reinterpret_cast<const __half2*>(&f[i])));
    const float2 y = __half22float2(__hmax2(m[0], m[1]));
    publish(top, d * fmaxf(y.x, y.y), lane);
}
// A state warp's part of a state in tensor memory times `by`: through other registers than the ones that the chain
// keeps it in, whose moves around a branch would cost every chunk 330 cycles.
__device__ __forceinline__ void rescale(uint32_t taddr, float by) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        uint32_t y[32];
        tc::ld32(taddr + 32 * i, y);
        tc::wait_ld();
        scale32(y, by);
        tc::st32(taddr + 32 * i, y);
    }
    tc::wait_st();
}
// two bf16 values times `by`, as fp16
__device__ __forceinline__ uint32_t scaled_half2(uint32_t u, unsigned long long by) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(u << 16), "r"(u & 0xFFFF0000u));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(by));
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return pack_half2(lo, hi);
}
__device__ __forceinline__ uint4 scaled_half8(uint4 u, float by) {
    unsigned long long b;
    asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(by));
    return make_uint4(scaled_half2(u.x, b), scaled_half2(u.y, b), scaled_half2(u.z, b), scaled_half2(u.w, b));
}

// Accumulators (32 value channels of the warp x 64 tokens, at taddr) as bf16 rows in memory (`step`
// elements from one token to the next), times by(token, the one after): read as fragments and
// turned round in `stage` (32 tokens x 32 channels) by stmatrix.  read() is called once
// tensor memory has been read.
constexpr int kTurnTokens = 32;               // at a time
constexpr int kTurnBytes = kTurnTokens * 64;
__device__ __forceinline__ uint32_t turn_at(uint32_t stage, int token, int unit) {   // 8 rows: all banks
    return stage + token * 64 + ((unit ^ ((token >> 1) & 3)) << 4);
}
template <class F, class G>
__device__ __forceinline__ void store_tokens(__nv_bfloat16* out, size_t step, int rows, uint32_t taddr,
                                             unsigned char* stage, int lane, F&& by, G&& read) {
    const uint32_t st = smem_u32(stage);
    const int first = lane >> 2;
    out += first * step + (lane & 3) * 8;
#pragma unroll 1
    for (int half = 0; half < kC / kTurnTokens; ++half) {
        uint32_t o[2][16];                    // channels 16 i ..
        tc::ld_fragments(taddr + kTurnTokens * half, o[0]);
        tc::ld_fragments(taddr + (16u << 16) + kTurnTokens * half, o[1]);
        tc::wait_ld();
        if (half == kC / kTurnTokens - 1) {
            tc::fence_before_sync();
            read();
        }
        __syncwarp();                         // the last rows have been read
#pragma unroll
        for (int j = 0; j < kTurnTokens / 8; ++j) {
            const float2 f = by(half * kTurnTokens + 8 * j + 2 * (lane & 3));
            uint32_t r[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {     // channels 8 m ..
                const uint32_t* x = &o[m >> 1][4 * j + 2 * (m & 1)];
                r[m] = pack_bf16(f.x * __uint_as_float(x[0]), f.y * __uint_as_float(x[1]));
            }
            stsm_t(turn_at(st, 8 * j + (lane & 7), lane >> 3), r[0], r[1], r[2], r[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kTurnTokens; i += 8) {
            if (half * kTurnTokens + first + i < rows)
                *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(stage + (turn_at(0, first + i, lane & 3)));
            out += 8 * step;
        }
    }
}

// A state warp's part of a state in memory: 64 rows of its lane's column, from element `at` on.  (One
// branch on the type, so that all loads are on their way together; nullptr: zeros.)
__device__ __forceinline__ void load_state(uint32_t (&x)[2][32], const void* p, int dtype, size_t at) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i >> 5][i & 31] = 0u;
    } else if (dtype == KDA_F32) {
        const uint32_t* s = static_cast<const uint32_t*>(p) + at;
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i >> 5][i & 31] = s[i * kDim];
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + at;
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i >> 5][i & 31] = (uint32_t)s[i * kDim] << 16;
    }
}
// the same to memory, times `by`
__device__ __forceinline__ void store_state(const uint32_t (&x)[2][32], float by, void* p, int dtype, size_t at) {
    if (dtype == KDA_F32) {
        float* s = static_cast<float*>(p) + at;
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i * kDim] = by * __uint_as_float(x[i >> 5][i & 31]);
    } else {
        __nv_bfloat16* s = static_cast<__nv_bfloat16*>(p) + at;
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i * kDim] = __float2bfloat16_rn(by * __uint_as_float(x[i >> 5][i & 31]));
    }
}

}  // namespace gdr
}  // namespace kda

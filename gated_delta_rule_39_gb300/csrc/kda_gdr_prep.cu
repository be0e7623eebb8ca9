// Chunk-parallel part of the gated delta rule with one decay per value head: where the
// chunks of packed sequences are (map), and each chunk's T = (I + A)^-1 (times beta), P =
// M . Q K^T and decays (prep).
#include "kda_gdr_chunk.cuh"

namespace kda {
namespace {

using namespace gdr;

// ---- map: checks cu_seqlens, first[n] = chunks of the sequences before n, order = the sequences, long
// ones first (so that the chains, a CTA per sequence and head, end together: 9 prompts of 1 to 18
// chunks x 32 heads on 152 SMs take 11 us less) ----------------------------------------------
constexpr int kMapThreads = 1024;
constexpr int kBuckets = 128;             // of lengths: four to a factor of two

__device__ __forceinline__ int bucket_of(int chunks) {     // long sequences first
    if (chunks < 4) return kBuckets - 1 - chunks;
    const int e = 31 - __clz(chunks);
    return kBuckets - 1 - (4 * (e - 1) + ((chunks >> (e - 2)) & 3));
}

__global__ void __launch_bounds__(kMapThreads) gdr_map_kernel(GdrInputs I, int* first, int* order, int* valid, int* err) {
    __shared__ int sums[kMapThreads / 32];
    __shared__ int places[kBuckets];
    __shared__ int bad;
    next_may_begin();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0) bad = I.cu[0] != 0 || I.cu[I.N] != I.T;
    if (tid < kBuckets) places[tid] = 0;
    __syncthreads();
    for (int n = tid; n < I.N; n += kMapThreads)
        if (I.cu[n + 1] < I.cu[n]) bad = 1;
    __syncthreads();
    if (tid == 0) {
        *valid = !bad;
        if (bad) set_error(err, KDA_ERR_BAD_SEQLENS);
    }
    if (bad) return;
    int before = 0;
    for (int base = 0; base < I.N; base += kMapThreads) {
        const int n = base + tid;
        const int c = n < I.N ? (I.cu[n + 1] - I.cu[n] + kC - 1) / kC : 0;
        int x = c;                     // inclusive sums of the warp, then of the warps before
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();               // the last round's sums have been read
        if (lane == 31) sums[w] = x;
        __syncthreads();
        int all = 0;
        for (int i = 0; i < kMapThreads / 32; ++i) {
            if (i == w) x += all;
            all += sums[i];
        }
        if (n < I.N) {
            first[n] = before + x - c;
            atomicAdd(&places[bucket_of(c)], 1);
        }
        before += all;
    }
    if (tid == 0) first[I.N] = before;
    __syncthreads();
    if (w == 0) {                      // where each bucket begins
        int count[kBuckets / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kBuckets / 32; ++i) {
            count[i] = places[kBuckets / 32 * lane + i];
            sum += count[i];
        }
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        x -= sum;
#pragma unroll
        for (int i = 0; i < kBuckets / 32; ++i) {
            places[kBuckets / 32 * lane + i] = x;
            x += count[i];
        }
    }
    __syncthreads();
    // within a bucket as it comes: only which CTA takes what depends on it
    for (int n = tid; n < I.N; n += kMapThreads)
        order[atomicAdd(&places[bucket_of((I.cu[n + 1] - I.cu[n] + kC - 1) / kC)], 1)] = n;
}

// ---- prep -------------------------------------------------------------------------------
// One CTA of 4 warps per (chunk, query/key head), or `split` of them that share the value heads
// where all are on the GPU at once.  Warp w forms rows 16 w .. 16 w + 15 of
// K K^T and Q K^T with mma.sync (bf16 data, fp32 sums; kept in registers for all value
// heads of the group), and per value head: the gates' running sum, A and P, and
// T = (I + A)^-1: the four 16 x 16 diagonal blocks by forward substitution in fp32 (a lane
// owns a column), then T21 = -T22 A21 T11 for blocks of 16 and of 32 with tf32 products.  T
// takes A's place block by block.
//
// Five CTAs share an SM to cover each other's chains of small steps: A, T and P live where K and Q
// were.  Measured: 8,192 tokens x 96 heads 155 us, 4.0 TB/s (K and Q once, 17 KB out per chunk and
// head): 72 % of the cycles move shared memory, which the fp32 tile's small products read in 4-byte
// pieces, and the waits between them take most of the rest.
constexpr int kPrepThreads = 128, kPrepPerSm = 5;
constexpr int kLd = 68;               // row length of the fp32 tile: rows 4 banks apart

struct PrepSmem {
    union {
        struct {
            __align__(128) unsigned char k[kC * kDim * 2];
            __align__(128) unsigned char q[kC * kDim * 2];
        };
        struct {
            __align__(16) float a[kC][kLd];                // A (strictly lower), then T
            __align__(128) unsigned char p[kTileBytes];    // P as fp16
        };
    };
    float g[kC];                                           // running sum of g in base 2
    float b[kC];
};

// rows [0, 64) of one head, zeros from row `rows` on, into a tile of 256-byte rows
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, long long stride, int rows,
                                          int tid) {
#pragma unroll
    for (int i = 0; i < kC * 16 / kPrepThreads; ++i) {
        const int unit = tid & 15, row = (tid >> 4) + i * (kPrepThreads / 16);
        const int bytes = row < rows ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n"
                     ::"r"(unit_at<256>(dst, row, unit)), "l"(src + (row < rows ? row * stride : 0) + unit * 8),
                       "r"(bytes) : "memory");
    }
}

// F(16 x 8 kN) = M(rows ar .., cols ac ..) M(rows br .., cols bc ..), 8 kK deep
template <int kN, int kK>
__device__ __forceinline__ void tf32_product(float (&c)[kN][4], const float (*M)[kLd], int ar, int ac, int br, int bc,
                                             int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < kN; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        const uint32_t a[4] = {tf32_bits(M[ar + g][ac + 8 * k + t]), tf32_bits(M[ar + g + 8][ac + 8 * k + t]),
                               tf32_bits(M[ar + g][ac + 8 * k + t + 4]),
                               tf32_bits(M[ar + g + 8][ac + 8 * k + t + 4])};
#pragma unroll
        for (int n = 0; n < kN; ++n)
            mma_tf32(c[n], a, tf32_bits(M[br + 8 * k + t][bc + 8 * n + g]),
                     tf32_bits(M[br + 8 * k + t + 4][bc + 8 * n + g]));
    }
}
// c (16 x 8 kN) = F M(rows br .., cols bc ..): F (16 x 8 kK) from accumulators.  An accumulator
// holds columns 2 t and 2 t + 1 where an A operand wants t and t + 4: the depth is walked in
// that order on both sides.
template <int kN, int kK>
__device__ __forceinline__ void tf32_second(float (&c)[kN][4], const float (&f)[kK][4], const float (*M)[kLd], int br,
                                            int bc, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const uint32_t a[4] = {tf32_bits(f[k][0]), tf32_bits(f[k][2]), tf32_bits(f[k][1]), tf32_bits(f[k][3])};
            mma_tf32(c[n], a, tf32_bits(M[br + 8 * k + 2 * t][bc + 8 * n + g]),
                     tf32_bits(M[br + 8 * k + 2 * t + 1][bc + 8 * n + g]));
        }
    }
}
// M(16 x 8 kN at row, col) = -c
template <int kN>
__device__ __forceinline__ void put_negative(float (*M)[kLd], int row, int col, const float (&c)[kN][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        *reinterpret_cast<float2*>(&M[row + g][col + 8 * n + 2 * t]) = make_float2(-c[n][0], -c[n][1]);
        *reinterpret_cast<float2*>(&M[row + g + 8][col + 8 * n + 2 * t]) = make_float2(-c[n][2], -c[n][3]);
    }
}

// Backward: the biased exponent of the largest |scale dO| (not of NaN) in this warp's rows of a chunk and head
__device__ __forceinline__ unsigned size_of_rows(const __nv_bfloat16* src, long long stride, int rows, float scale, int tid) {
    uint4 u[kC * 16 / kPrepThreads];
    src += (tid & 15) * 8;
#pragma unroll
    for (int i = 0; i < kC * 16 / kPrepThreads; ++i)      // rows past the end repeat the last one
        u[i] = __ldg(reinterpret_cast<const uint4*>(src + min((tid >> 4) + i * (kPrepThreads / 16), rows - 1) * stride));
    __nv_bfloat162 top = __float2bfloat162_rn(0.0f);
#pragma unroll
    for (int i = 0; i < kC * 16 / kPrepThreads; ++i)
        for (const uint32_t x : {u[i].x, u[i].y, u[i].z, u[i].w}) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)));
    const float2 f = __bfloat1622float2(top);
    return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(scale) * fmaxf(f.x, f.y))) >> 23;
}

template <bool kGrads, bool kSplit>
__global__ void __launch_bounds__(kPrepThreads, kPrepPerSm) gdr_prep_kernel(GdrChunked P, GdrGrads B, int ways) {
    const int split = kSplit ? ways : 1;
    extern __shared__ __align__(128) unsigned char raw[];
    next_may_begin();
    previous_done();
    PrepSmem& S = *reinterpret_cast<PrepSmem*>(raw);
    const GdrInputs& I = P.in;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int chunk = blockIdx.x, hk = blockIdx.y / split, part = blockIdx.y % split;
    // rows of this warp; the last ones have four times the work of the first, so the warps of
    // one scheduler take different ones in different CTAs
    const int w = ((tid >> 5) + chunk) & 3;
    int n, c;
    if (!find_chunk(I, P.chunks, chunk, n, c)) return;
    const Span span = span_of(I, P.chunks, n);
    const long long tok = span.start + (long long)c * kC;
    const int rows = min(kC, span.len - c * kC);
    const uint32_t sk = smem_u32(S.k), sq = smem_u32(S.q), sp = smem_u32(S.p);
    load_tile(sk, I.k + tok * I.k_stride + hk * kDim, I.k_stride, rows, tid);
    load_tile(sq, I.q + tok * I.q_stride + hk * kDim, I.q_stride, rows, tid);
    cp_async_commit();
    // gates of two tokens per lane of warp 0, one value head ahead
    const int share = I.Hv / I.Hk;
    float g0 = 0.0f, g1 = 0.0f, b0 = 0.0f, b1 = 0.0f;
    const auto fetch_gates = [&](int h) {
        if (w != 0) return;
        const size_t at = (size_t)(tok + 2 * lane) * I.Hv + h;
        g0 = g1 = b0 = b1 = 0.0f;
        if (2 * lane < rows) {
            g0 = load_gate(I.g, I.gate_dtype, at);
            b0 = load_gate(I.beta, I.gate_dtype, at);
        }
        if (2 * lane + 1 < rows) {
            g1 = load_gate(I.g, I.gate_dtype, at + I.Hv);
            b1 = load_gate(I.beta, I.gate_dtype, at + I.Hv);
        }
    };
    fetch_gates(hk * share + part);
    if (kGrads)                        // for the scales of the gradient's chain, while the rows are on their way
        for (int h = hk * share + part; h < (hk + 1) * share; h += split) {
            const unsigned x = size_of_rows(B.dout + (tok * I.Hv + h) * kDim, (long long)I.Hv * kDim, rows, I.scale, tid);
            if (lane == 0) (P.blocks + ((size_t)chunk * I.Hv + h) * kBlockBytes + 2 * kTileBytes + 4 * kGateDo)[tid >> 5] = (unsigned char)x;
        }
    cp_async_wait<0>();
    __syncthreads();
    // rows 16 w ..  of K K^T and Q K^T, columns 0 .. 16 w + 15
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        uint32_t ak[4], aq[4];
        ldsm(ak, a_addr<256>(sk, 16 * w, 2 * ks, lane));
        ldsm(aq, a_addr<256>(sq, 16 * w, 2 * ks, lane));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > w) break;
            uint32_t b[4];
            ldsm(b, b_addr<256>(sk, 16 * np, 2 * ks, lane));
            mma_bf16(kk[2 * np], ak, b[0], b[1]);
            mma_bf16(kk[2 * np + 1], ak, b[2], b[3]);
            mma_bf16(qk[2 * np], aq, b[0], b[1]);
            mma_bf16(qk[2 * np + 1], aq, b[2], b[3]);
        }
    }
    for (int h = hk * share + part; h < (hk + 1) * share; h += split) {
        __syncthreads();               // K and Q, or the last head's tiles, have been read
        unsigned char* block = P.blocks + ((size_t)chunk * I.Hv + h) * kBlockBytes;
        if (w == 0) {
            g0 *= kLog2e;
            g1 *= kLog2e;
            // 2^-160 is 0 in fp32 already: lower logs (-inf) only would spoil the differences
            g0 = g0 < -160.0f ? -160.0f : g0;
            g1 = g1 < -160.0f ? -160.0f : g1;
            float x = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            const float last = __shfl_sync(0xFFFFFFFFu, x, 31);
            const float x0 = x - g1;
            S.g[2 * lane] = x0;
            S.g[2 * lane + 1] = x;
            S.b[2 * lane] = b0;
            S.b[2 * lane + 1] = b1;
            float* gates = reinterpret_cast<float*>(block + 2 * kTileBytes);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x);
            reinterpret_cast<float2*>(gates + kGateB)[lane] = make_float2(b0, b1);
            reinterpret_cast<float2*>(gates + kGateBe)[lane] = make_float2(b0 * e0, b1 * e1);
            reinterpret_cast<float2*>(gates + kGateE)[lane] = make_float2(e0, e1);
            reinterpret_cast<float2*>(gates + kGateEnd)[lane] = make_float2(ex2_approx(last - x0), ex2_approx(last - x));
            reinterpret_cast<float2*>(gates + kGateG)[lane] = make_float2(x0, x);
            if (lane == 0) gates[kGateAll] = ex2_approx(last);
            if (h + split < (hk + 1) * share) fetch_gates(h + split);
        }
        __syncthreads();
        // A in fp32 and P in fp16
        const float gi0 = S.g[16 * w + g], gi1 = S.g[16 * w + g + 8];
        const float bi0 = S.b[16 * w + g], bi1 = S.b[16 * w + g + 8];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t p[4] = {0u, 0u, 0u, 0u};
            if (np <= w) {
                float pv[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int nt = 2 * np + m, j = 8 * nt + 2 * t, i0 = 16 * w + g, i1 = i0 + 8;
                    const float gj0 = S.g[j], gj1 = S.g[j + 1];
                    const float m00 = j <= i0 ? ex2_approx(gi0 - gj0) : 0.0f;
                    const float m01 = j + 1 <= i0 ? ex2_approx(gi0 - gj1) : 0.0f;
                    const float m10 = j <= i1 ? ex2_approx(gi1 - gj0) : 0.0f;
                    const float m11 = j + 1 <= i1 ? ex2_approx(gi1 - gj1) : 0.0f;
                    *reinterpret_cast<float2*>(&S.a[i0][j]) =
                        make_float2(j < i0 ? bi0 * m00 * kk[nt][0] : 0.0f, j + 1 < i0 ? bi0 * m01 * kk[nt][1] : 0.0f);
                    *reinterpret_cast<float2*>(&S.a[i1][j]) =
                        make_float2(j < i1 ? bi1 * m10 * kk[nt][2] : 0.0f, j + 1 < i1 ? bi1 * m11 * kk[nt][3] : 0.0f);
                    pv[m][0] = j <= i0 ? m00 * qk[nt][0] : 0.0f;
                    pv[m][1] = j + 1 <= i0 ? m01 * qk[nt][1] : 0.0f;
                    pv[m][2] = j <= i1 ? m10 * qk[nt][2] : 0.0f;
                    pv[m][3] = j + 1 <= i1 ? m11 * qk[nt][3] : 0.0f;
                }
                p[0] = pack_half2(pv[0][0], pv[0][1]);
                p[1] = pack_half2(pv[0][2], pv[0][3]);
                p[2] = pack_half2(pv[1][0], pv[1][1]);
                p[3] = pack_half2(pv[1][2], pv[1][3]);
            }
            stsm(a_addr<128>(sp, 16 * w, 2 * np, lane), p[0], p[1], p[2], p[3]);
        }
        __syncwarp();
        // inverse of this warp's diagonal block, a column per lane (both halves of the warp alike)
        {
            const int d = 16 * w, col = lane & 15;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float even = r == col ? 1.0f : 0.0f, odd = 0.0f;
#pragma unroll
                for (int m = 0; m < r; m += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(&S.a[d + r][d + m]);
                    even = fmaf(-v.x, x[m], even);
                    if (m + 1 < r) odd = fmaf(-v.y, x[m + 1], odd);
                    if (m + 2 < r) even = fmaf(-v.z, x[m + 2], even);
                    if (m + 3 < r) odd = fmaf(-v.w, x[m + 3], odd);
                }
                x[r] = even + odd;
            }
            __syncwarp();
            if (lane < 16) {
#pragma unroll
                for (int r = 0; r < 16; ++r) S.a[d + r][d + col] = x[r];
            }
        }
        __syncthreads();
        {   // blocks of 16: T21 = -(T22 A21) T11, half of the columns per warp
            const int r0 = 32 * (w >> 1);
            float f[2][4], c16[1][4];
            tf32_product<2, 2>(f, S.a, r0 + 16, r0 + 16, r0 + 16, r0, lane);
            tf32_second<1, 2>(c16, f, S.a, r0, r0 + 8 * (w & 1), lane);
            __syncthreads();           // A21 has been read
            put_negative<1>(S.a, r0 + 16, r0 + 8 * (w & 1), c16, lane);
            // zeros above the diagonal blocks, which the next products read
            if (w & 1) {
#pragma unroll
                for (int i = lane; i < 16 * 16; i += 32) S.a[r0 + (i >> 4)][r0 + 16 + (i & 15)] = 0.0f;
            }
        }
        __syncthreads();
        {   // blocks of 32: 16 rows and 16 columns per warp
            const int r0 = 32 + 16 * (w >> 1);
            float f[4][4], c32[2][4];
            tf32_product<4, 4>(f, S.a, r0, 32, 32, 0, lane);
            tf32_second<2, 4>(c32, f, S.a, 0, 16 * (w & 1), lane);
            __syncthreads();
            put_negative<2>(S.a, r0, 16 * (w & 1), c32, lane);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kC * 8 / kPrepThreads; ++i) {
            const int unit = tid & 7, row = (tid >> 3) + i * (kPrepThreads / 8);
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (8 * unit <= row) {
                const float4 lo = *reinterpret_cast<const float4*>(&S.a[row][8 * unit]);
                const float4 hi = *reinterpret_cast<const float4*>(&S.a[row][8 * unit + 4]);
                float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int j = 1; j < 8; ++j)      // columns after the diagonal are not part of T
                    if (8 * unit + j > row) f[j] = 0.0f;
                const float* b = S.b + 8 * unit;
                x = make_uint4(pack_half2(f[0] * b[0], f[1] * b[1]), pack_half2(f[2] * b[2], f[3] * b[3]),
                               pack_half2(f[4] * b[4], f[5] * b[5]), pack_half2(f[6] * b[6], f[7] * b[7]));
                y = make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
            }
            const int at = row * 128 + ((unit ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(block + at) = x;
            if (kGrads)
                *reinterpret_cast<uint4*>(P.ts + ((size_t)chunk * I.Hv + h) * kTileBytes + at) = y;
            *reinterpret_cast<uint4*>(block + kTileBytes + at) = *reinterpret_cast<const uint4*>(S.p + at);
        }
    }
}

}  // namespace

cudaError_t launch_gdr_map(const GdrInputs& in, int* first, int* order, int* valid, int* err, cudaStream_t s) {
    gdr_map_kernel<<<1, kMapThreads, 0, s>>>(in, first, order, valid, err);
    return cudaGetLastError();
}

template <bool kGrads, bool kSplit>
static cudaError_t launch_prep(const GdrChunked& P, const GdrGrads& B, int split, bool early, cudaStream_t s) {
    const cudaError_t e = allow_smem<gdr_prep_kernel<kGrads, kSplit>>(sizeof(PrepSmem));
    if (e != cudaSuccess) return e;
    return launch_after(early, gdr_prep_kernel<kGrads, kSplit>, dim3(P.chunks.total, P.in.Hk * split), kPrepThreads, sizeof(PrepSmem), s, P, B, split);
}
template <bool kGrads>
static cudaError_t launch_prep(const GdrChunked& P, const GdrGrads& B, int sms, bool early, cudaStream_t s) {
    if (P.chunks.total == 0) return cudaSuccess;
    const int share = P.in.Hv / P.in.Hk;
    int split = 1;
    while (2 * split <= share && (long long)P.chunks.total * P.in.Hk * 2 * split <= (long long)kPrepPerSm * sms &&
           P.in.Hk * 2 * split <= 65535)
        split *= 2;
    return split > 1 ? launch_prep<kGrads, true>(P, B, split, early, s) : launch_prep<kGrads, false>(P, B, 1, early, s);
}

cudaError_t launch_gdr_prep(const GdrChunked& P, int sms, bool early, cudaStream_t s) { return launch_prep<false>(P, {}, sms, early, s); }
cudaError_t launch_gdr_prep(const GdrBackward& B, int sms, cudaStream_t s) { return launch_prep<true>(B.fwd, B.in, sms, true, s); }

}  // namespace kda

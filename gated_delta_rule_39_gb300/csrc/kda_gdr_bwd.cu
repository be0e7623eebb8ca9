// Backward pass of the gated delta rule with one decay per value head, in chunks of 64
// tokens (the forward's equations and their names: kda_gdr_chunk.cuh).
//
// With dS the gradient of the state after a chunk, the chunk's own are
//
//   dX = e^(GC-G) K dS + scale P^T dO          Y = T^T dX   (so dR = beta Y)
//   dS <- e^GC dS + scale Q^T (e^G dO) - K^T (beta e^G Y)
//
// which is the forward chain mirrored; a kernel of its own walks the chunks backwards and
// keeps dS and Y (kda_gdr_bwd_chain.cu).  What remains is parallel over chunks (here, from S
// and X of the forward pass):
//
//   dV = beta Y                                (written by the chain)
//   dQ = scale e^G (dO S^T) + dP K,             dP = scale M . (dO X^T)
//   dK = e^(GC-G) (X dS^T) - beta e^G (Y S^T) + dP^T Q + (dB + dB^T) K,
//                                              dB = -beta_i M . strictly lower (Y X^T)
//   dbeta = Y.V - e^G K.(Y S^T) - sum_j (M . Y X^T . K K^T)_ij
//   dG_i = q.dQ's first term - k.dK's first term + k.dK's second term
//          + row sums - column sums of (dP . Q K^T + dB . K K^T);
//   dG of the last token also gets sum k.dK's first term + e^GC <S, dS>
//   dg = suffix sums of dG inside the chunk.
//
// Operands are fp16, with the incoming gradients scaled by a power of two per (sequence,
// key head) (grad_scale) and scale folded into dO; sums and states are fp32.  Gradients of
// queries and keys that a group of value heads shares are summed in registers by one CTA, in a
// fixed order.
#include "kda_gdr_chunk.cuh"

namespace kda {
namespace {

using namespace gdr;

// ---- the largest incoming gradient of each (sequence, key head) ---------------------------
constexpr int kAmaxThreads = 256;

// one CTA per (chunk, key head): dO of the chunk's tokens; chunk 0 also takes the states'
__global__ void __launch_bounds__(kAmaxThreads) gdr_amax_kernel(GdrBackward B) {
    const GdrInputs& I = B.fwd.in;
    int n, c;
    if (!find_chunk(I, B.fwd.chunks, blockIdx.x, n, c)) return;
    const int hk = blockIdx.y, share = I.Hv / I.Hk, tid = threadIdx.x;
    const Span span = span_of(I, B.fwd.chunks, n);
    const int rows = min(kC, span.len - c * kC), units = share * 16;   // 16-byte units of a token
    const __nv_bfloat16* src = B.dout + ((span.start + (long long)c * kC) * I.Hv + hk * share) * kDim;
    unsigned top = 0;
    const auto take = [](unsigned u, unsigned& m) {   // two bf16 values; NaN compares above infinity
        m = max(m, max(u & 0x7FFF0000u, (u & 0x7FFFu) << 16));
    };
    for (int i = tid; i < rows * units; i += kAmaxThreads) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + (size_t)(i / units) * I.Hv * kDim + (i % units) * 8);
        take(u.x, top); take(u.y, top); take(u.z, top); take(u.w, top);
    }
    top = __float_as_uint(fabsf(I.scale) * __uint_as_float(top));
    unsigned dfinal_top = 0;
    if (c == 0 && B.dfinal) {
        const size_t base = ((size_t)n * I.Hv + hk * share) * kDim * kDim, count = (size_t)share * kDim * kDim;
        if (B.dfinal_dtype == KDA_F32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(B.dfinal) + base);
            for (size_t i = tid; i < count / 4; i += kAmaxThreads) {
                const uint4 u = p[i];
                dfinal_top = max(dfinal_top, max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu)));
            }
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(B.dfinal) + base);
            for (size_t i = tid; i < count / 8; i += kAmaxThreads) {
                const uint4 u = p[i];
                take(u.x, dfinal_top); take(u.y, dfinal_top); take(u.z, dfinal_top); take(u.w, dfinal_top);
            }
        }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, max(top, dfinal_top));
    // a maximum does not depend on the order of the atomics
    if ((tid & 31) == 0) atomicMax(&B.amax[(size_t)n * I.Hk + hk], top);
}

// ---- chunk by chunk ---------------------------------------------------------------------------
// One CTA of 8 warps per (chunk, key head), which walks the group's value heads.  Warp w
// forms rows (tokens) 16 (w & 3) .. of dQ and dK for the key channels 64 (w >> 2) .., and
// the columns 32 (w >> 2) .. of the token-by-token products.
constexpr int kChunkThreads = 256;

struct ChunkSmem {
    __align__(128) unsigned char k[kC * kDim * 2];   // fp16, 256-byte rows
    __align__(128) unsigned char q[kC * kDim * 2];
    __align__(128) unsigned char o[kC * kDim * 2];   // dO, fp16, scaled
    __align__(128) unsigned char s[kStateTile];      // S^T (rows in units, as kept in memory)
    __align__(128) unsigned char ds[kStateTile];     // dS^T
    __align__(128) unsigned char x[kTokenTile];      // X^T
    __align__(128) unsigned char y[kTokenTile];      // Y^T
    __align__(128) unsigned char block[kBlockBytes]; // T (then dP), P (then dB), gates
    float row[5][2][kC];      // sums over channels or columns, one slot per half
    float col[4][kC];         // column sums of dP . Q K^T + dB . K K^T, one slot per 16 rows
    float yv[2][kC];
    float dot[kChunkThreads / 32];
};

// ldmatrix addresses in a tile kept in units: 16 rows from r0, units u0 and u0 + 1, in the
// orders of a_addr and b_addr
__device__ __forceinline__ uint32_t row_a(uint32_t base, int r0, int u0, int lane) {
    return base + row_unit(r0 + (lane & 15), u0 + (lane >> 4));
}
__device__ __forceinline__ uint32_t row_b(uint32_t base, int r0, int u0, int lane) {
    return base + row_unit(r0 + (lane & 7) + ((lane >> 4) << 3), u0 + ((lane >> 3) & 1));
}
__device__ __forceinline__ float2 half2_at(const unsigned char* tile, int row, int ch) {   // 256-byte rows
    const __half2 h = *reinterpret_cast<const __half2*>(tile + row * 256 + (((ch >> 3) ^ (row & 7)) << 4) + (ch & 7) * 2);
    return __half22float2(h);
}
__device__ __forceinline__ float quad_sum(float x) {       // over the 4 lanes of a row
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
    return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}
__device__ __forceinline__ float rows_sum(float x) {       // over the 8 rows of a column
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
    return x + __shfl_xor_sync(0xFFFFFFFFu, x, 16);
}

// 64 rows of 128 bf16 channels (zeros from row `rows` on) as a tile of fp16, times `by`
__device__ __forceinline__ void load_half_tile(unsigned char* dst, const __nv_bfloat16* src, long long stride, int rows,
                                               float by, int tid) {
#pragma unroll
    for (int i = 0; i < kC * 16 / kChunkThreads; ++i) {
        const int unit = tid & 15, row = (tid >> 4) + i * (kChunkThreads / 16);
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) u = __ldg(reinterpret_cast<const uint4*>(src + row * stride + unit * 8));
        u.x = pack_half2(by * bf16_lo(u.x), by * bf16_hi(u.x));
        u.y = pack_half2(by * bf16_lo(u.y), by * bf16_hi(u.y));
        u.z = pack_half2(by * bf16_lo(u.z), by * bf16_hi(u.z));
        u.w = pack_half2(by * bf16_lo(u.w), by * bf16_hi(u.w));
        *reinterpret_cast<uint4*>(dst + row * 256 + ((unit ^ (row & 7)) << 4)) = u;
    }
}
__device__ __forceinline__ void copy_tile(unsigned char* dst, const unsigned char* src, int bytes, int tid) {
    for (int i = tid; i < bytes / 16; i += kChunkThreads) cp_async16(dst + 16 * i, src + 16 * i);
}

__device__ __forceinline__ void store_gate(void* p, int dtype, size_t i, float x) {
    if (dtype == KDA_F32) static_cast<float*>(p)[i] = x;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

__global__ void __launch_bounds__(kChunkThreads, 1) gdr_bwd_chunk_kernel(GdrBackward B) {
    extern __shared__ __align__(128) unsigned char raw[];
    ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(raw);
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int chunk = blockIdx.x, hk = blockIdx.y;
    int n, c;
    if (!find_chunk(I, P.chunks, chunk, n, c)) return;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rw = w & 3, half = w >> 2, share = I.Hv / I.Hk;
    const Span span = span_of(I, P.chunks, n);
    const long long tok = span.start + (long long)c * kC;
    const int rows = min(kC, span.len - c * kC);
    const float sigma = grad_scale(B.amax[(size_t)n * I.Hk + hk]), back = 1.0f / sigma;
    load_half_tile(S.k, I.k + tok * I.k_stride + hk * kDim, I.k_stride, rows, 1.0f, tid);
    load_half_tile(S.q, I.q + tok * I.q_stride + hk * kDim, I.q_stride, rows, 1.0f, tid);
    const uint32_t sk = smem_u32(S.k), sq = smem_u32(S.q), so = smem_u32(S.o), ss = smem_u32(S.s),
                   sds = smem_u32(S.ds), sx = smem_u32(S.x), sy = smem_u32(S.y), sT = smem_u32(S.block),
                   sP = sT + kTileBytes;
    const float* gate = reinterpret_cast<const float*>(S.block + 2 * kTileBytes);
    const int i0 = 16 * rw + g, i1 = i0 + 8;               // this lane's rows
    float dq[8][4], dk[8][4], kk[4][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[j][e] = dk[j][e] = 0.0f;
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        const size_t at = (size_t)chunk * I.Hv + h;
        copy_tile(S.s, P.states + at * kStateTile, kStateTile, tid);
        copy_tile(S.y, B.ys + at * kTokenTile, kTokenTile, tid);
        copy_tile(S.block, P.blocks + at * kBlockBytes, kBlockUsed, tid);
        copy_tile(S.ds, B.dstates + at * kStateTile, kStateTile, tid);
        copy_tile(S.x, P.xs + at * kTokenTile, kTokenTile, tid);
        cp_async_commit();
        load_half_tile(S.o, B.dout + (tok * I.Hv + h) * kDim, (long long)I.Hv * kDim, rows, I.scale * sigma, tid);
        cp_async_wait<0>();
        __syncthreads();
        if (h == hk * share) {         // K K^T, this warp's 16 rows and 32 columns
#pragma unroll
            for (int j = 0; j < 4; ++j) kk[j][0] = kk[j][1] = kk[j][2] = kk[j][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t a[4];
                ldsm(a, a_addr<256>(sk, 16 * rw, 2 * ks, lane));
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    uint32_t b[4];
                    ldsm(b, b_addr<256>(sk, 32 * half + 16 * np, 2 * ks, lane));
                    mma_f16(kk[2 * np], a, b[0], b[1]);
                    mma_f16(kk[2 * np + 1], a, b[2], b[3]);
                }
            }
        }
        const float e0 = gate[kGateE + i0], e1 = gate[kGateE + i1];
        const float be0 = gate[kGateBe + i0], be1 = gate[kGateBe + i1];
        const float b0 = gate[kGateB + i0], b1 = gate[kGateB + i1];
        // dO S^T and Y S^T: this warp's rows, 64 key channels, over 128 value channels
        {
            float a[8][4], z[8][4], yv0 = 0.0f, yv1 = 0.0f;
            const __nv_bfloat16* vp = I.v + (tok + i0) * I.v_stride + h * kDim + 2 * t;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) a[j][e] = z[j][e] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t fo[4], fy[4];
                ldsm(fo, a_addr<256>(so, 16 * rw, 2 * ks, lane));
                // Y as an A operand from Y^T: (tokens, v) blocks transposed; Y.V over half of the
                // value channels by this warp
                ldsm_t(fy, row_b(sy, 16 * ks, 2 * rw, lane));
                if ((ks >> 2) == half) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) {          // rows i0, i1; channels 16 ks + 2 t (+ 8)
                        if ((m & 1 ? i1 : i0) < rows) {
                            const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(vp + (m & 1 ? 8 * I.v_stride : 0) + 16 * ks + 8 * (m >> 1)));
                            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&fy[m]));
                            (m & 1 ? yv1 : yv0) += y.x * bf16_lo(v) + y.y * bf16_hi(v);
                        }
                    }
                }
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, row_a(ss, 16 * ks, 8 * half + 2 * np, lane));
                    mma_f16(a[2 * np], fo, b[0], b[1]);
                    mma_f16(a[2 * np + 1], fo, b[2], b[3]);
                    mma_f16(z[2 * np], fy, b[0], b[1]);
                    mma_f16(z[2 * np + 1], fy, b[2], b[3]);
                }
            }
            float qa0 = 0.0f, qa1 = 0.0f, kz0 = 0.0f, kz1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int ch = 64 * half + 8 * j + 2 * t;
                const float2 q0 = half2_at(S.q, i0, ch), q1 = half2_at(S.q, i1, ch);
                const float2 k0 = half2_at(S.k, i0, ch), k1 = half2_at(S.k, i1, ch);
                a[j][0] *= e0; a[j][1] *= e0; a[j][2] *= e1; a[j][3] *= e1;
                qa0 += q0.x * a[j][0] + q0.y * a[j][1];
                qa1 += q1.x * a[j][2] + q1.y * a[j][3];
                kz0 += k0.x * z[j][0] + k0.y * z[j][1];
                kz1 += k1.x * z[j][2] + k1.y * z[j][3];
                dq[j][0] += a[j][0]; dq[j][1] += a[j][1]; dq[j][2] += a[j][2]; dq[j][3] += a[j][3];
                dk[j][0] -= be0 * z[j][0]; dk[j][1] -= be0 * z[j][1];
                dk[j][2] -= be1 * z[j][2]; dk[j][3] -= be1 * z[j][3];
            }
            qa0 = quad_sum(qa0); qa1 = quad_sum(qa1); kz0 = quad_sum(kz0); kz1 = quad_sum(kz1);
            yv0 = quad_sum(yv0); yv1 = quad_sum(yv1);
            if (t == 0) {
                S.yv[half][i0] = yv0; S.yv[half][i1] = yv1;
                S.row[0][half][i0] = qa0; S.row[0][half][i1] = qa1;
                S.row[1][half][i0] = kz0; S.row[1][half][i1] = kz1;
            }
        }
        // X dS^T
        {
            float a[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j][0] = a[j][1] = a[j][2] = a[j][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t fx[4];
                ldsm_t(fx, row_b(sx, 16 * ks, 2 * rw, lane));
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, row_a(sds, 16 * ks, 8 * half + 2 * np, lane));
                    mma_f16(a[2 * np], fx, b[0], b[1]);
                    mma_f16(a[2 * np + 1], fx, b[2], b[3]);
                }
            }
            const float f0 = gate[kGateEnd + i0], f1 = gate[kGateEnd + i1];
            float ka0 = 0.0f, ka1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int ch = 64 * half + 8 * j + 2 * t;
                const float2 k0 = half2_at(S.k, i0, ch), k1 = half2_at(S.k, i1, ch);
                a[j][0] *= f0; a[j][1] *= f0; a[j][2] *= f1; a[j][3] *= f1;
                ka0 += k0.x * a[j][0] + k0.y * a[j][1];
                ka1 += k1.x * a[j][2] + k1.y * a[j][3];
                dk[j][0] += a[j][0]; dk[j][1] += a[j][1]; dk[j][2] += a[j][2]; dk[j][3] += a[j][3];
            }
            ka0 = quad_sum(ka0); ka1 = quad_sum(ka1);
            if (t == 0) {
                S.row[2][half][i0] = ka0; S.row[2][half][i1] = ka1;
            }
        }
        // <S, dS>
        {
            float d = 0.0f;
            for (int i = tid; i < kStateTile / 16; i += kChunkThreads) {
                const uint4 a = reinterpret_cast<const uint4*>(S.s)[i], b = reinterpret_cast<const uint4*>(S.ds)[i];
                const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&ua[j]));
                    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&ub[j]));
                    d += x.x * y.x + x.y * y.y;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
            if (lane == 0) S.dot[w] = d;
        }
        // dO X^T and Y X^T: this warp's 16 rows, 32 columns
        float dp[4][4], da[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) dp[j][e] = da[j][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t fo[4], fy[4];
            ldsm(fo, a_addr<256>(so, 16 * rw, 2 * ks, lane));
            ldsm_t(fy, row_b(sy, 16 * ks, 2 * rw, lane));
#pragma unroll
            for (int np = 0; np < 2; ++np) {
                if (2 * half + np > rw) break;             // columns past the rows
                uint32_t b[4];
                ldsm_t(b, row_a(sx, 16 * ks, 4 * half + 2 * np, lane));
                mma_f16(dp[2 * np], fo, b[0], b[1]);
                mma_f16(dp[2 * np + 1], fo, b[2], b[3]);
                mma_f16(da[2 * np], fy, b[0], b[1]);
                mma_f16(da[2 * np + 1], fy, b[2], b[3]);
            }
        }
        // dP, dB and the sums of dP . Q K^T + dB . K K^T (M . Q K^T is P)
        uint32_t fp[4][2], fb[4][2];
        float rs0 = 0.0f, rs1 = 0.0f, bs0 = 0.0f, bs1 = 0.0f;
        {
            const float g0 = gate[kGateG + i0], g1 = gate[kGateG + i1];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int j = 32 * half + 8 * nt + 2 * t;
                float cs[2] = {0.0f, 0.0f}, pv[4], bv[4];
                const float2 gj = *reinterpret_cast<const float2*>(gate + kGateG + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = e < 2 ? i0 : i1, jj = j + (e & 1);
                    const float m = jj <= i ? ex2_approx((e < 2 ? g0 : g1) - (e & 1 ? gj.y : gj.x)) : 0.0f;
                    const float pq = __half2float(*reinterpret_cast<const __half*>(
                        S.block + kTileBytes + i * 128 + (((jj >> 3) ^ (i & 7)) << 4) + (jj & 7) * 2));
                    const float mk = jj < i ? m * kk[nt][e] : 0.0f;
                    const float dpv = dp[nt][e], dav = -da[nt][e], bi = e < 2 ? b0 : b1;
                    pv[e] = jj <= i ? m * dpv : 0.0f;
                    bv[e] = jj < i ? bi * m * dav : 0.0f;
                    const float sum = (jj <= i ? dpv * pq : 0.0f) + bi * dav * mk;
                    cs[e & 1] += sum;
                    (e < 2 ? rs0 : rs1) += sum;
                    (e < 2 ? bs0 : bs1) += dav * mk;
                }
                fp[nt][0] = pack_half2(pv[0], pv[1]);
                fp[nt][1] = pack_half2(pv[2], pv[3]);
                fb[nt][0] = pack_half2(bv[0], bv[1]);
                fb[nt][1] = pack_half2(bv[2], bv[3]);
                cs[0] = rows_sum(cs[0]);
                cs[1] = rows_sum(cs[1]);
                if (g == 0) {
                    S.col[rw][j] = cs[0];
                    S.col[rw][j + 1] = cs[1];
                }
            }
            rs0 = quad_sum(rs0); rs1 = quad_sum(rs1); bs0 = quad_sum(bs0); bs1 = quad_sum(bs1);
            if (t == 0) {
                S.row[3][half][i0] = rs0; S.row[3][half][i1] = rs1;
                S.row[4][half][i0] = bs0; S.row[4][half][i1] = bs1;
            }
        }
        __syncthreads();               // P has been read
        // dP over T, dB over P (both lower triangles, zeros above)
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            stsm(a_addr<128>(sT, 16 * rw, 4 * half + 2 * np, lane), fp[2 * np][0], fp[2 * np][1], fp[2 * np + 1][0], fp[2 * np + 1][1]);
            stsm(a_addr<128>(sP, 16 * rw, 4 * half + 2 * np, lane), fb[2 * np][0], fb[2 * np][1], fb[2 * np + 1][0], fb[2 * np + 1][1]);
        }
        __syncthreads();
        // dQ += dP K, dK += dP^T Q + dB K + dB^T K
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t fpn[4], fbn[4], fpt[4], fbt[4];
            if (ks <= rw) {            // rows reach tokens up to their own
                ldsm(fpn, a_addr<128>(sT, 16 * rw, 2 * ks, lane));
                ldsm(fbn, a_addr<128>(sP, 16 * rw, 2 * ks, lane));
            }
            if (ks >= rw) {            // transposed: from their own on
                ldsm_t(fpt, b_addr<128>(sT, 16 * ks, 2 * rw, lane));
                ldsm_t(fbt, b_addr<128>(sP, 16 * ks, 2 * rw, lane));
            }
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t b[4];
                ldsm_t(b, a_addr<256>(sk, 16 * ks, 8 * half + 2 * np, lane));
                if (ks <= rw) {
                    mma_f16(dq[2 * np], fpn, b[0], b[1]);
                    mma_f16(dq[2 * np + 1], fpn, b[2], b[3]);
                    mma_f16(dk[2 * np], fbn, b[0], b[1]);
                    mma_f16(dk[2 * np + 1], fbn, b[2], b[3]);
                }
                if (ks >= rw) {
                    mma_f16(dk[2 * np], fbt, b[0], b[1]);
                    mma_f16(dk[2 * np + 1], fbt, b[2], b[3]);
                    ldsm_t(b, a_addr<256>(sq, 16 * ks, 8 * half + 2 * np, lane));
                    mma_f16(dk[2 * np], fpt, b[0], b[1]);
                    mma_f16(dk[2 * np + 1], fpt, b[2], b[3]);
                }
            }
        }
        // gates: two tokens per lane of one warp
        if (w == 0) {
            float dgv[2], ka[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int j = 2 * lane + m;
                const float qa = S.row[0][0][j] + S.row[0][1][j], kz = S.row[1][0][j] + S.row[1][1][j];
                ka[m] = S.row[2][0][j] + S.row[2][1][j];
                const float rs = S.row[3][0][j] + S.row[3][1][j], bs = S.row[4][0][j] + S.row[4][1][j];
                const float cs = S.col[0][j] + S.col[1][j] + S.col[2][j] + S.col[3][j];
                const float yv = S.yv[0][j] + S.yv[1][j];
                dgv[m] = qa - ka[m] - gate[kGateBe + j] * kz + rs - cs;
                if (j < rows)
                    store_gate(B.dbeta, I.gate_dtype, (size_t)(tok + j) * I.Hv + h,
                               back * (yv - gate[kGateE + j] * kz + bs));
            }
            float all = ka[0] + ka[1];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kChunkThreads / 32; ++i) dot += S.dot[i];
            if (lane == 31) dgv[1] += all + gate[kGateAll] * dot;
            float x = dgv[0] + dgv[1];         // sums from a token to the chunk's last
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_down_sync(0xFFFFFFFFu, x, o);
                if (lane + o < 32) x += y;
            }
            if (2 * lane < rows) store_gate(B.dg, I.gate_dtype, (size_t)(tok + 2 * lane) * I.Hv + h, back * x);
            if (2 * lane + 1 < rows)
                store_gate(B.dg, I.gate_dtype, (size_t)(tok + 2 * lane + 1) * I.Hv + h, back * (x - dgv[0]));
        }
        __syncthreads();               // the tiles are free for the next head
    }
    // dQ and dK as bf16 rows
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int ch = 64 * half + 8 * j + 2 * t;
        if (i0 < rows) {
            const size_t o = ((size_t)(tok + i0) * I.Hk + hk) * kDim + ch;
            *reinterpret_cast<uint32_t*>(B.dq + o) = pack_bf16(back * dq[j][0], back * dq[j][1]);
            *reinterpret_cast<uint32_t*>(B.dk + o) = pack_bf16(back * dk[j][0], back * dk[j][1]);
        }
        if (i1 < rows) {
            const size_t o = ((size_t)(tok + i1) * I.Hk + hk) * kDim + ch;
            *reinterpret_cast<uint32_t*>(B.dq + o) = pack_bf16(back * dq[j][2], back * dq[j][3]);
            *reinterpret_cast<uint32_t*>(B.dk + o) = pack_bf16(back * dk[j][2], back * dk[j][3]);
        }
    }
}

}  // namespace

cudaError_t launch_gdr_amax(const GdrBackward& B, cudaStream_t s) {
    if (B.fwd.chunks.total == 0) return cudaSuccess;
    gdr_amax_kernel<<<dim3(B.fwd.chunks.total, B.fwd.in.Hk), kAmaxThreads, 0, s>>>(B);
    return cudaGetLastError();
}

cudaError_t launch_gdr_bwd_chunk(const GdrBackward& B, cudaStream_t s) {
    if (B.fwd.chunks.total == 0) return cudaSuccess;
    const cudaError_t e = allow_smem<gdr_bwd_chunk_kernel>(sizeof(ChunkSmem));
    if (e != cudaSuccess) return e;
    gdr_bwd_chunk_kernel<<<dim3(B.fwd.chunks.total, B.fwd.in.Hk), kChunkThreads, sizeof(ChunkSmem), s>>>(B);
    return cudaGetLastError();
}

}  // namespace kda

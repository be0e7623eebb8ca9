// Backward pass of the gated delta rule with one decay per value head, in chunks of 64
// tokens (the forward's equations and their names: kda_gdr_chunk.cuh).
//
// With dS the gradient of the state after a chunk, the chunk's own are
//
//   dX = e^(GC-G) K dS + scale P^T dO          Y = T^T dX   (so dR = beta Y)
//   dS <- e^GC dS + scale Q^T (e^G dO) - K^T (beta e^G Y)
//
// which is the forward chain mirrored: the bwd-chain kernel walks the chunks backwards
// with the same split (a warp per 16 value channels, dS^T in its accumulators, 148 MMAs a
// chunk on the chain) and keeps dS and Y.  What remains is parallel over chunks (the
// bwd-chunk kernel, from S and X of the forward pass):
//
//   dV = beta Y
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
// key head) (grad_scale); sums and states are fp32.  Gradients of queries and keys that a
// group of value heads shares are summed in registers by one CTA, in a fixed order.
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
    const auto take = [&](unsigned u) {   // two bf16 values; NaN compares above infinity
        top = max(top, max(u & 0x7FFF0000u, (u & 0x7FFFu) << 16));
    };
    for (int i = tid; i < rows * units; i += kAmaxThreads) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + (size_t)(i / units) * I.Hv * kDim + (i % units) * 8);
        take(u.x); take(u.y); take(u.z); take(u.w);
    }
    if (c == 0 && B.dfinal) {
        const size_t base = ((size_t)n * I.Hv + hk * share) * kDim * kDim, count = (size_t)share * kDim * kDim;
        if (B.dfinal_dtype == KDA_F32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(B.dfinal) + base);
            for (size_t i = tid; i < count / 4; i += kAmaxThreads) {
                const uint4 u = p[i];
                top = max(top, max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu)));
            }
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(B.dfinal) + base);
            for (size_t i = tid; i < count / 8; i += kAmaxThreads) {
                const uint4 u = p[i];
                take(u.x); take(u.y); take(u.z); take(u.w);
            }
        }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    // a maximum does not depend on the order of the atomics
    if ((tid & 31) == 0) atomicMax(&B.amax[(size_t)n * I.Hk + hk], top);
}

// ---- the chain, backwards -------------------------------------------------------------------
constexpr int kProducers = 128;
constexpr int kStages = 2;

template <int NW>
struct BackSmem {
    struct Stage {
        unsigned char k[kC * kDim * 2];
        unsigned char q[kC * kDim * 2];
        unsigned char block[kBlockBytes];
        unsigned char o[NW][kC * 32];           // dO, each warp's 16 columns (fp16, scaled)
    };
    __align__(128) Stage stage[kStages];
    struct Keep {                               // from a state warp to its helper
        unsigned char s[16 * kDim * 2];         // dS^T after the chunk
        unsigned char y[16 * kC * 2];           // Y^T
    };
    __align__(128) Keep hand[NW][2];
    __align__(128) float4 u[NW][16][32];        // helper to state warp: scale (e^G dO)^T Q
    __align__(128) float4 p[NW][8][32];         //   and scale dO^T P, as accumulators
    uint64_t full[kStages], empty[kStages];
    uint64_t s_full[NW][2], y_full[NW][2], hand_empty[NW][2];
    uint64_t u_full[NW], u_empty[NW], p_full[NW], p_empty[NW];
};

// 16-byte units of [token][16 columns] tiles, flipped every 4 rows
__device__ __forceinline__ uint32_t v_at(uint32_t base, int row, int unit) {
    return base + row * 32 + ((unit ^ ((row >> 2) & 1)) << 4);
}

template <int NW>
__device__ void back_produce(const GdrBackward& B, BackSmem<NW>& S, const Span& span, int nch, int h, int part,
                             float sigma, int p) {
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk);
    const int unit = p & 15, row0 = p >> 4;
    const __nv_bfloat16* kp = I.k + (span.start + row0) * I.k_stride + hk * kDim + unit * 8;
    const __nv_bfloat16* qp = I.q + (span.start + row0) * I.q_stride + hk * kDim + unit * 8;
    const long long o_stride = (long long)I.Hv * kDim;
    const __nv_bfloat16* op = B.dout + span.start * o_stride + h * kDim + part * (16 * NW);
    const int dst = row0 * 256 + ((unit ^ (row0 & 7)) << 4);
    uint4 ka[8], qa[8], oa[NW];
    const auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = c * kC + 8 * i;
            ka[i] = qa[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row + row0 < span.len) {
                ka[i] = __ldg(reinterpret_cast<const uint4*>(kp + row * I.k_stride));
                qa[i] = __ldg(reinterpret_cast<const uint4*>(qp + row * I.q_stride));
            }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int at = p + i * kProducers, row = c * kC + at / (2 * NW);
            oa[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < span.len) oa[i] = __ldg(reinterpret_cast<const uint4*>(op + row * o_stride + at % (2 * NW) * 8));
        }
    };
    const auto half4 = [](uint4 u) {
        return make_uint4(bf16_to_half2(u.x), bf16_to_half2(u.y), bf16_to_half2(u.z), bf16_to_half2(u.w));
    };
    const auto scaled2 = [&](uint32_t u) { return pack_half2(sigma * bf16_lo(u), sigma * bf16_hi(u)); };
    fetch(nch - 1);
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i, st = i % kStages;
        auto& G = S.stage[st];
        if (i >= kStages && !bar_wait(&S.empty[st], (unsigned)((i / kStages - 1) & 1), P.err)) break;
        const unsigned char* block = P.blocks + ((size_t)(span.chunk + c) * I.Hv + h) * kBlockBytes;
        for (int j = p; j < kBlockUsed / 16; j += kProducers) cp_async16(G.block + 16 * j, block + 16 * j);
        bar_arrive_copies(&S.full[st]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<uint4*>(G.k + dst + 2048 * j) = half4(ka[j]);
            *reinterpret_cast<uint4*>(G.q + dst + 2048 * j) = half4(qa[j]);
        }
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int at = p + j * kProducers, token = at / (2 * NW), vu = at % (2 * NW);
            *reinterpret_cast<uint4*>(G.o[vu >> 1] + v_at(0, token, vu & 1)) =
                make_uint4(scaled2(oa[j].x), scaled2(oa[j].y), scaled2(oa[j].z), scaled2(oa[j].w));
        }
        bar_arrive(&S.full[st]);
        if (c > 0) fetch(c - 1);
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
}

template <int NW>
__device__ void back_chain(const GdrBackward& B, BackSmem<NW>& S, int nch, int w, int lane, size_t sbase, int v0,
                           float sigma) {
    const GdrChunked& P = B.fwd;
    const int g = lane >> 2, t = lane & 3;
    const float back = 1.0f / sigma;
    const auto at = [&](int nt, int e) {
        return sbase + (size_t)(8 * nt + 2 * t + (e & 1)) * kDim + v0 + g + (e >> 1) * 8;
    };
    float s[16][4];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = 0.0f;
            if (B.dfinal)
                x = B.dfinal_dtype == KDA_F32 ? static_cast<const float*>(B.dfinal)[at(nt, e)]
                                              : __bfloat162float(static_cast<const __nv_bfloat16*>(B.dfinal)[at(nt, e)]);
            s[nt][e] = sigma * x;
        }
    for (int i = 0; i < nch; ++i) {
        const int st = i % kStages, buf = i & 1;
        auto& G = S.stage[st];
        auto& H = S.hand[w][buf];
        const uint32_t sk = smem_u32(G.k), sT = smem_u32(G.block), so = smem_u32(G.o[w]);
        const float* gate = reinterpret_cast<const float*>(G.block + 2 * kTileBytes);
        uint32_t sf[8][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            sf[ks][0] = pack_half2(s[2 * ks][0], s[2 * ks][1]);
            sf[ks][1] = pack_half2(s[2 * ks][2], s[2 * ks][3]);
            sf[ks][2] = pack_half2(s[2 * ks + 1][0], s[2 * ks + 1][1]);
            sf[ks][3] = pack_half2(s[2 * ks + 1][2], s[2 * ks + 1][3]);
        }
        if (i >= 2 && !bar_wait(&S.hand_empty[w][buf], (unsigned)((i / 2 - 1) & 1), P.err)) return;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            stsm(a_addr<256>(smem_u32(H.s), 0, 2 * ks, lane), sf[ks][0], sf[ks][1], sf[ks][2], sf[ks][3]);
        __syncwarp();
        if (lane == 0) bar_arrive(&S.s_full[w][buf]);
        if (!bar_wait(&S.full[st], (unsigned)((i / kStages) & 1), P.err)) return;
        float y[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t b[4];
                ldsm(b, b_addr<256>(sk, 16 * np, 2 * ks, lane));
                mma_f16(y[2 * np], sf[ks], b[0], b[1]);
                mma_f16(y[2 * np + 1], sf[ks], b[2], b[3]);
            }
        // dX^T = e^(GC-G) (K dS)^T + scale (P^T dO)^T
        if (!bar_wait(&S.p_full[w], (unsigned)(i & 1), P.err)) return;
        uint32_t xf[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int nt = 2 * ks + m;
                const float2 ed = *reinterpret_cast<const float2*>(gate + kGateEnd + 8 * nt + 2 * t);
                const float4 p = S.p[w][nt][lane];
                xf[ks][2 * m] = pack_half2(fmaf(ed.x, y[nt][0], p.x), fmaf(ed.y, y[nt][1], p.y));
                xf[ks][2 * m + 1] = pack_half2(fmaf(ed.x, y[nt][2], p.z), fmaf(ed.y, y[nt][3], p.w));
            }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.p_empty[w]);
        // Y^T = dX^T T: column j of T starts at row j
#pragma unroll
        for (int np = 0; np < 4; ++np) {
#pragma unroll
            for (int m = 0; m < 2; ++m) y[2 * np + m][0] = y[2 * np + m][1] = y[2 * np + m][2] = y[2 * np + m][3] = 0.0f;
#pragma unroll
            for (int ks = np; ks < 4; ++ks) {
                uint32_t b[4];
                ldsm_t(b, a_addr<128>(sT, 16 * ks, 2 * np, lane));
                mma_f16(y[2 * np], xf[ks], b[0], b[1]);
                mma_f16(y[2 * np + 1], xf[ks], b[2], b[3]);
            }
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                xf[ks][2 * m] = pack_half2(y[2 * ks + m][0], y[2 * ks + m][1]);
                xf[ks][2 * m + 1] = pack_half2(y[2 * ks + m][2], y[2 * ks + m][3]);
            }
            stsm(a_addr<128>(smem_u32(H.y), 0, 2 * ks, lane), xf[ks][0], xf[ks][1], xf[ks][2], xf[ks][3]);
            // dV = beta Y from the fp32 sums, as rows of 16 channels per token, over the warp's
            // dO tile (the helper read it before it raised p_full)
            uint32_t r[4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 bt = *reinterpret_cast<const float2*>(gate + kGateB + 16 * ks + 8 * m + 2 * t);
                const float f0 = back * bt.x, f1 = back * bt.y;
                r[2 * m] = pack_bf16(f0 * y[2 * ks + m][0], f1 * y[2 * ks + m][1]);
                r[2 * m + 1] = pack_bf16(f0 * y[2 * ks + m][2], f1 * y[2 * ks + m][3]);
            }
            stsm_t(v_at(so, 16 * ks + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1), r[0], r[1], r[2], r[3]);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.y_full[w][buf]);
        // dS^T = e^GC dS^T + scale (e^G dO)^T Q - (beta e^G Y)^T K
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 be = *reinterpret_cast<const float2*>(gate + kGateBe + 16 * ks + 8 * m + 2 * t);
                xf[ks][2 * m] = pack_half2(-be.x * y[2 * ks + m][0], -be.y * y[2 * ks + m][1]);
                xf[ks][2 * m + 1] = pack_half2(-be.x * y[2 * ks + m][2], -be.y * y[2 * ks + m][3]);
            }
        const float d = gate[kGateAll];
        if (!bar_wait(&S.u_full[w], (unsigned)(i & 1), P.err)) return;
#pragma unroll
        for (int nt = 0; nt < 16; ++nt) {
            const float4 u = S.u[w][nt][lane];
            s[nt][0] = fmaf(d, s[nt][0], u.x); s[nt][1] = fmaf(d, s[nt][1], u.y);
            s[nt][2] = fmaf(d, s[nt][2], u.z); s[nt][3] = fmaf(d, s[nt][3], u.w);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.u_empty[w]);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int np = 0; np < 8; ++np) {
                uint32_t b[4];
                ldsm_t(b, a_addr<256>(sk, 16 * ks, 2 * np, lane));
                mma_f16(s[2 * np], xf[ks], b[0], b[1]);
                mma_f16(s[2 * np + 1], xf[ks], b[2], b[3]);
            }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.empty[st]);
    }
    if (B.dinit) {
#pragma unroll
        for (int nt = 0; nt < 16; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = back * s[nt][e];
                if (B.dinit_dtype == KDA_F32) static_cast<float*>(B.dinit)[at(nt, e)] = x;
                else static_cast<__nv_bfloat16*>(B.dinit)[at(nt, e)] = __float2bfloat16_rn(x);
            }
    }
}

// The helper of a state warp: scale dO^T P and scale (e^G dO)^T Q of the coming chunk, then the
// copies of dS^T, Y^T and dV of the chunk that the state warp is at to memory.
template <int NW>
__device__ void back_help(const GdrBackward& B, BackSmem<NW>& S, const Span& span, int nch, int w, int lane, int h,
                          int v0) {
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int t = lane & 3;
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i, st = i % kStages, buf = i & 1;
        auto& G = S.stage[st];
        auto& H = S.hand[w][buf];
        const uint32_t sq = smem_u32(G.q), sP = smem_u32(G.block) + kTileBytes, so = smem_u32(G.o[w]);
        const float* gate = reinterpret_cast<const float*>(G.block + 2 * kTileBytes);
        if (!bar_wait(&S.full[st], (unsigned)((i / kStages) & 1), P.err)) return;
        uint32_t of[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            ldsm_t(of[ks], v_at(so, 16 * ks + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1));
        {
            float y[8][4];
#pragma unroll
            for (int np = 0; np < 4; ++np) {
#pragma unroll
                for (int m = 0; m < 2; ++m) y[2 * np + m][0] = y[2 * np + m][1] = y[2 * np + m][2] = y[2 * np + m][3] = 0.0f;
#pragma unroll
                for (int ks = np; ks < 4; ++ks) {
                    uint32_t b[4];
                    ldsm_t(b, a_addr<128>(sP, 16 * ks, 2 * np, lane));
                    mma_f16(y[2 * np], of[ks], b[0], b[1]);
                    mma_f16(y[2 * np + 1], of[ks], b[2], b[3]);
                }
            }
            if (i >= 1 && !bar_wait(&S.p_empty[w], (unsigned)((i - 1) & 1), P.err)) return;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
                S.p[w][nt][lane] = make_float4(I.scale * y[nt][0], I.scale * y[nt][1], I.scale * y[nt][2], I.scale * y[nt][3]);
            __syncwarp();
            if (lane == 0) bar_arrive(&S.p_full[w]);
        }
        {
            float u[16][4];
#pragma unroll
            for (int nt = 0; nt < 16; ++nt) u[nt][0] = u[nt][1] = u[nt][2] = u[nt][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t a[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {     // registers 0, 1: tokens 2 t of the first 8; 2, 3: of the next
                    const float2 e = *reinterpret_cast<const float2*>(gate + kGateE + 16 * ks + 8 * (m >> 1) + 2 * t);
                    const __half2 o = *reinterpret_cast<const __half2*>(&of[ks][m]);
                    a[m] = pack_half2(e.x * __low2float(o), e.y * __high2float(o));
                }
#pragma unroll
                for (int np = 0; np < 8; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, a_addr<256>(sq, 16 * ks, 2 * np, lane));
                    mma_f16(u[2 * np], a, b[0], b[1]);
                    mma_f16(u[2 * np + 1], a, b[2], b[3]);
                }
            }
            if (i >= 1 && !bar_wait(&S.u_empty[w], (unsigned)((i - 1) & 1), P.err)) return;
#pragma unroll
            for (int nt = 0; nt < 16; ++nt)
                S.u[w][nt][lane] = make_float4(I.scale * u[nt][0], I.scale * u[nt][1], I.scale * u[nt][2], I.scale * u[nt][3]);
            __syncwarp();
            if (lane == 0) bar_arrive(&S.u_full[w]);
        }
        const size_t at = (size_t)(span.chunk + c) * I.Hv + h;
        if (!bar_wait(&S.s_full[w][buf], (unsigned)((i / 2) & 1), P.err)) return;
        uint4* ds = reinterpret_cast<uint4*>(B.dstates + at * kStateTile + v0 * kDim * 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) ds[j * 32 + lane] = reinterpret_cast<const uint4*>(H.s)[j * 32 + lane];
        if (!bar_wait(&S.y_full[w][buf], (unsigned)((i / 2) & 1), P.err)) return;
        uint4* dy = reinterpret_cast<uint4*>(B.ys + at * kTokenTile + v0 * kC * 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) dy[j * 32 + lane] = reinterpret_cast<const uint4*>(H.y)[j * 32 + lane];
        __syncwarp();
        if (lane == 0) bar_arrive(&S.hand_empty[w][buf]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int token = 16 * j + (lane >> 1), row = c * kC + token;
            if (row < span.len)
                *reinterpret_cast<uint4*>(B.dv + ((span.start + row) * I.Hv + h) * kDim + v0 + 8 * (lane & 1)) =
                    *reinterpret_cast<const uint4*>(G.o[w] + v_at(0, token, lane & 1));
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.empty[st]);
    }
}

template <int NW>
__global__ void __launch_bounds__(64 * NW + kProducers, 1) gdr_bwd_chain_kernel(GdrBackward B) {
    extern __shared__ __align__(128) unsigned char raw[];
    BackSmem<NW>& S = *reinterpret_cast<BackSmem<NW>*>(raw);
    const GdrInputs& I = B.fwd.in;
    if (I.cu && !*I.valid) return;
    constexpr int kParts = kDim / (16 * NW);
    const int part = blockIdx.x % kParts, unit = blockIdx.x / kParts;
    const int h = unit % I.Hv, n = unit / I.Hv;
    const Span span = span_of(I, B.fwd.chunks, n);
    const int nch = (span.len + kC - 1) / kC;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const float sigma = grad_scale(B.amax[(size_t)n * I.Hk + h / (I.Hv / I.Hk)]);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&S.full[i], 2 * kProducers);
            bar_init(&S.empty[i], 2 * NW);
        }
        for (int i = 0; i < NW; ++i) {
            for (int j = 0; j < 2; ++j) {
                bar_init(&S.s_full[i][j], 1);
                bar_init(&S.y_full[i][j], 1);
                bar_init(&S.hand_empty[i][j], 1);
            }
            bar_init(&S.u_full[i], 1);
            bar_init(&S.u_empty[i], 1);
            bar_init(&S.p_full[i], 1);
            bar_init(&S.p_empty[i], 1);
        }
    }
    __syncthreads();
    const size_t sbase = ((size_t)n * I.Hv + h) * kDim * kDim;
    if (w < NW) {
        back_chain<NW>(B, S, nch, w, lane, sbase, part * 16 * NW + 16 * w, sigma);
    } else if (w < 2 * NW) {
        back_help<NW>(B, S, span, nch, w - NW, lane, h, part * 16 * NW + 16 * (w - NW));
    } else if (nch > 0) {
        back_produce<NW>(B, S, span, nch, h, part, sigma, tid - 64 * NW);
    }
}

template <int NW>
cudaError_t launch_chain(const GdrBackward& B, cudaStream_t s) {
    const cudaError_t e = allow_smem<gdr_bwd_chain_kernel<NW>>(sizeof(BackSmem<NW>));
    if (e != cudaSuccess) return e;
    const long long ctas = (long long)B.fwd.in.N * B.fwd.in.Hv * (kDim / (16 * NW));
    gdr_bwd_chain_kernel<NW><<<(unsigned)ctas, 64 * NW + kProducers, sizeof(BackSmem<NW>), s>>>(B);
    return cudaGetLastError();
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
    __align__(128) unsigned char s[kStateTile];      // S^T, then dS^T
    __align__(128) unsigned char ds[kStateTile];
    __align__(128) unsigned char x[kTokenTile];      // X^T
    __align__(128) unsigned char y[kTokenTile];      // Y^T
    __align__(128) unsigned char block[kBlockBytes]; // T (then dP), P (then dB + dB^T), gates
    float row[5][2][kC];      // sums over channels or columns, one slot per half
    float col[4][kC];         // column sums of dP . Q K^T + dB . K K^T, one slot per 16 rows
    float yv[4][kC];
    float dot[kChunkThreads / 32];
};

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
        load_half_tile(S.o, B.dout + (tok * I.Hv + h) * kDim, (long long)I.Hv * kDim, rows, sigma, tid);
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
            float a[8][4], z[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) a[j][e] = z[j][e] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t fo[4], fy[4];
                ldsm(fo, a_addr<256>(so, 16 * rw, 2 * ks, lane));
                // Y as an A operand from Y^T: (tokens, v) blocks transposed
                ldsm_t(fy, b_addr<128>(sy, 16 * ks, 2 * rw, lane));
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, a_addr<256>(ss, 16 * ks, 8 * half + 2 * np, lane));
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
                const float f0 = I.scale * e0, f1 = I.scale * e1;
                a[j][0] *= f0; a[j][1] *= f0; a[j][2] *= f1; a[j][3] *= f1;
                qa0 += q0.x * a[j][0] + q0.y * a[j][1];
                qa1 += q1.x * a[j][2] + q1.y * a[j][3];
                kz0 += k0.x * z[j][0] + k0.y * z[j][1];
                kz1 += k1.x * z[j][2] + k1.y * z[j][3];
                dq[j][0] += a[j][0]; dq[j][1] += a[j][1]; dq[j][2] += a[j][2]; dq[j][3] += a[j][3];
                dk[j][0] -= be0 * z[j][0]; dk[j][1] -= be0 * z[j][1];
                dk[j][2] -= be1 * z[j][2]; dk[j][3] -= be1 * z[j][3];
            }
            qa0 = quad_sum(qa0); qa1 = quad_sum(qa1); kz0 = quad_sum(kz0); kz1 = quad_sum(kz1);
            if (t == 0) {
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
                ldsm_t(fx, b_addr<128>(sx, 16 * ks, 2 * rw, lane));
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, a_addr<256>(sds, 16 * ks, 8 * half + 2 * np, lane));
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
        // <S, dS>, and Y.V
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
            const int j = tid & 63, v0 = (tid >> 6) * 32;
            float yv = 0.0f;
            if (j < rows) {
                const __nv_bfloat16* vp = I.v + (tok + j) * I.v_stride + h * kDim + v0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(vp + 8 * i));
                    const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int v = v0 + 8 * i + m;
                        const __half y = *reinterpret_cast<const __half*>(S.y + v * 128 + (((j >> 3) ^ (v & 7)) << 4) + (j & 7) * 2);
                        yv += __half2float(y) * (m & 1 ? bf16_hi(uu[m >> 1]) : bf16_lo(uu[m >> 1]));
                    }
                }
            }
            S.yv[tid >> 6][j] = yv;
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
            ldsm_t(fy, b_addr<128>(sy, 16 * ks, 2 * rw, lane));
#pragma unroll
            for (int np = 0; np < 2; ++np) {
                if (2 * half + np > rw) break;             // columns past the rows
                uint32_t b[4];
                ldsm_t(b, a_addr<128>(sx, 16 * ks, 4 * half + 2 * np, lane));
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
                    const float dpv = I.scale * dp[nt][e], dav = -da[nt][e], bi = e < 2 ? b0 : b1;
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
                const float yv = S.yv[0][j] + S.yv[1][j] + S.yv[2][j] + S.yv[3][j];
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

cudaError_t launch_gdr_bwd_chain(const GdrBackward& B, int sms, cudaStream_t s) {
    const long long units = (long long)B.fwd.in.N * B.fwd.in.Hv;
    if (units == 0) return cudaSuccess;
    return units * 2 <= sms ? launch_chain<2>(B, s) : launch_chain<4>(B, s);
}

cudaError_t launch_gdr_bwd_chunk(const GdrBackward& B, cudaStream_t s) {
    if (B.fwd.chunks.total == 0) return cudaSuccess;
    const cudaError_t e = allow_smem<gdr_bwd_chunk_kernel>(sizeof(ChunkSmem));
    if (e != cudaSuccess) return e;
    gdr_bwd_chunk_kernel<<<dim3(B.fwd.chunks.total, B.fwd.in.Hk), kChunkThreads, sizeof(ChunkSmem), s>>>(B);
    return cudaGetLastError();
}

}  // namespace kda

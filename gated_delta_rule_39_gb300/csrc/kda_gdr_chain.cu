// The chunks of a sequence one after another: the sequential part of the gated delta rule
// with one decay per value head (the chunked form's equations: kda_gdr_chunk.cuh).
//
// The columns of S (value channels) never meet, so a warp owns 16 of them with all 128 key
// channels and runs the whole recurrence without waiting for another warp of the head:
// it holds S^T (16 x 128, fp32) as tensor-core accumulators, and every product has its
// left operand in the layout that the last one left in registers:
//
//   (K S)^T = S^T K^T        A = S^T rounded to fp16
//   X^T = R^T T^T            A = R^T = (beta (V - e^G K S))^T
//   S^T = e^GC S^T + (e^(GC-G) X)^T K
//
// mma.sync and not tcgen05: its operands and results stay in registers, where a tcgen05
// chain pays a trip through tensor memory and two barriers per product; and it can
// spread a head over 8 warps on as many as 4 SMs, so that few heads still use the GPU.
// What a chunk costs a state warp is its 148 MMAs at 8.16 cycles (measured per
// sub-partition, m16n8k16).  The outputs' 84 MMAs (S^T Q^T, then X^T P^T) are done by a
// second warp, which gets S^T and X^T through shared memory: they are not on the chain.
// Four more warps bring in the next chunks: keys and queries are converted to fp16 on
// the way from global to shared memory, the rest is copied with cp.async.
#include "kda_gdr_chunk.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int kProducers = 128;
constexpr int kStages = 3;            // chunks in shared memory

template <int NW>
struct ChainSmem {
    struct Stage {
        unsigned char k[kC * kDim * 2];         // fp16, rows of 256 bytes
        unsigned char q[kC * kDim * 2];
        unsigned char block[kBlockBytes];       // T, P, gates
        unsigned char v[NW][kC * 32];           // each warp's 16 columns, rows of 32 bytes
    };
    __align__(128) Stage stage[kStages];
    struct Hand {                               // from a state warp to its output warp
        unsigned char s[16 * kDim * 2];         // S^T before the chunk, fp16
        unsigned char x[16 * kC * 2];           // X^T, fp16
    };
    __align__(128) Hand hand[NW][2];
    uint64_t full[kStages], empty[kStages];
    uint64_t s_full[NW][2], x_full[NW][2], hand_empty[NW][2];
};

// V tiles: rows of two 16-byte units, the unit's index flipped every 4 rows (8 rows of an
// ldmatrix then cover all banks)
__device__ __forceinline__ uint32_t v_at(uint32_t base, int row, int unit) {
    return base + row * 32 + ((unit ^ ((row >> 2) & 1)) << 4);
}

__device__ __forceinline__ float load_state(const void* p, int dtype, size_t i) {
    return dtype == KDA_F32 ? static_cast<const float*>(p)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_state(void* p, int dtype, size_t i, float x) {
    if (dtype == KDA_F32) static_cast<float*>(p)[i] = x;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// ---- producers ----------------------------------------------------------------------------
template <int NW, bool kSave>
__device__ void produce(const GdrChunked& P, ChainSmem<NW>& S, const Span& span, int nch, int h, int part,
                        int p) {
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk);
    const int unit = p & 15, row0 = p >> 4;
    const __nv_bfloat16* kp = I.k + (span.start + row0) * I.k_stride + hk * kDim + unit * 8;
    const __nv_bfloat16* qp = I.q + (span.start + row0) * I.q_stride + hk * kDim + unit * 8;
    const __nv_bfloat16* vp = I.v + span.start * I.v_stride + h * kDim + part * (16 * NW);
    const int dst = row0 * 256 + ((unit ^ (row0 & 7)) << 4);      // rows row0 + 8 i: 2,048 bytes apart
    uint4 ka[2][8], qa[2][8];
    const auto fetch = [&](int c, uint4 (&kr)[8], uint4 (&qr)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = c * kC + 8 * i;
            kr[i] = qr[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row + row0 < span.len) {
                kr[i] = __ldg(reinterpret_cast<const uint4*>(kp + row * I.k_stride));
                if (!kSave) qr[i] = __ldg(reinterpret_cast<const uint4*>(qp + row * I.q_stride));
            }
        }
    };
    const auto half4 = [](uint4 u) {
        return make_uint4(bf16_to_half2(u.x), bf16_to_half2(u.y), bf16_to_half2(u.z), bf16_to_half2(u.w));
    };
    const auto put = [&](int c, const uint4 (&kr)[8], const uint4 (&qr)[8]) {
        const int st = c % kStages;
        auto& G = S.stage[st];
        if (c >= kStages && !bar_wait(&S.empty[st], (unsigned)((c / kStages - 1) & 1), P.err)) return false;
        const unsigned char* block = P.blocks + ((size_t)(span.chunk + c) * I.Hv + h) * kBlockBytes;
        for (int i = p; i < kBlockUsed / 16; i += kProducers) cp_async16(G.block + 16 * i, block + 16 * i);
#pragma unroll
        for (int i = 0; i < kC * 2 * NW / kProducers; ++i) {
            const int at = p + i * kProducers, token = at / (2 * NW), vu = at % (2 * NW);
            const int row = c * kC + token, bytes = row < span.len ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n"
                         ::"r"(v_at(smem_u32(G.v[vu >> 1]), token, vu & 1)),
                           "l"(vp + (bytes ? row * I.v_stride : 0) + vu * 8), "r"(bytes) : "memory");
        }
        bar_arrive_copies(&S.full[st]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            *reinterpret_cast<uint4*>(G.k + dst + 2048 * i) = half4(kr[i]);
            if (!kSave) *reinterpret_cast<uint4*>(G.q + dst + 2048 * i) = half4(qr[i]);
        }
        bar_arrive(&S.full[st]);
        return true;
    };
    // two chunks' rows in flight in registers, kStages in shared memory
    fetch(0, ka[0], qa[0]);
    if (nch > 1) fetch(1, ka[1], qa[1]);
    for (int c = 0; c < nch; c += 2) {
        if (!put(c, ka[0], qa[0])) break;
        if (c + 2 < nch) fetch(c + 2, ka[0], qa[0]);
        if (c + 1 >= nch || !put(c + 1, ka[1], qa[1])) break;
        if (c + 3 < nch) fetch(c + 3, ka[1], qa[1]);
    }
    cp_async_wait<0>();                // nothing lands after the CTA has gone
    asm volatile("cp.async.wait_all;\n" ::: "memory");
}

// ---- a state warp ---------------------------------------------------------------------------
template <int NW>
__device__ void chain(const GdrChunked& P, ChainSmem<NW>& S, int nch, int w, int lane, size_t sbase, int v0) {
    const int g = lane >> 2, t = lane & 3;
    // element (v, ch) of S^T is state[ch * 128 + v]
    const auto at = [&](int nt, int e) {
        return sbase + (size_t)(8 * nt + 2 * t + (e & 1)) * kDim + v0 + g + (e >> 1) * 8;
    };
    float s[16][4];
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = P.init_state ? load_state(P.init_state, P.init_dtype, at(nt, e)) : 0.0f;
    for (int c = 0; c < nch; ++c) {
        const int st = c % kStages, buf = c & 1;
        auto& G = S.stage[st];
        auto& H = S.hand[w][buf];
        const uint32_t sk = smem_u32(G.k), sT = smem_u32(G.block), sv = smem_u32(G.v[w]);
        const float* gate = reinterpret_cast<const float*>(G.block + 2 * kTileBytes);
        // S^T as A operands: accumulators of neighbouring n-tiles side by side
        uint32_t sf[8][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            sf[ks][0] = pack_half2(s[2 * ks][0], s[2 * ks][1]);
            sf[ks][1] = pack_half2(s[2 * ks][2], s[2 * ks][3]);
            sf[ks][2] = pack_half2(s[2 * ks + 1][0], s[2 * ks + 1][1]);
            sf[ks][3] = pack_half2(s[2 * ks + 1][2], s[2 * ks + 1][3]);
        }
        if (c >= 2 && !bar_wait(&S.hand_empty[w][buf], (unsigned)((c / 2 - 1) & 1), P.err)) return;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            stsm(a_addr<256>(smem_u32(H.s), 0, 2 * ks, lane), sf[ks][0], sf[ks][1], sf[ks][2], sf[ks][3]);
        __syncwarp();
        if (lane == 0) bar_arrive(&S.s_full[w][buf]);
        if (!bar_wait(&S.full[st], (unsigned)((c / kStages) & 1), P.err)) return;
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
        // R^T = b V^T - (b e^G) (K S)^T, tokens along the columns
        uint32_t rf[4][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t vr[4];
            ldsm_t(vr, v_at(sv, 16 * np + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int nt = 2 * np + m;
                const float2 b = *reinterpret_cast<const float2*>(gate + kGateB + 8 * nt + 2 * t);
                const float2 be = *reinterpret_cast<const float2*>(gate + kGateBe + 8 * nt + 2 * t);
                rf[np][2 * m] = pack_half2(b.x * bf16_lo(vr[2 * m]) - be.x * y[nt][0],
                                           b.y * bf16_hi(vr[2 * m]) - be.y * y[nt][1]);
                rf[np][2 * m + 1] = pack_half2(b.x * bf16_lo(vr[2 * m + 1]) - be.x * y[nt][2],
                                               b.y * bf16_hi(vr[2 * m + 1]) - be.y * y[nt][3]);
            }
        }
        // X^T = R^T T^T; row i of T ends at column i
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.0f;
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                if (2 * kp > nt / 2) break;
                uint32_t b[4];
                ldsm(b, unit_at<128>(sT, 8 * nt + (lane & 7), 4 * kp + (lane >> 3)));
                mma_f16(y[nt], rf[2 * kp], b[0], b[1]);
                if (2 * kp + 1 <= nt / 2) mma_f16(y[nt], rf[2 * kp + 1], b[2], b[3]);
            }
        }
        uint32_t xf[4][4];             // X^T, then (e^(GC-G) X)^T
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                xf[ks][2 * m] = pack_half2(y[2 * ks + m][0], y[2 * ks + m][1]);
                xf[ks][2 * m + 1] = pack_half2(y[2 * ks + m][2], y[2 * ks + m][3]);
            }
            stsm(a_addr<128>(smem_u32(H.x), 0, 2 * ks, lane), xf[ks][0], xf[ks][1], xf[ks][2], xf[ks][3]);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.x_full[w][buf]);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 ed = *reinterpret_cast<const float2*>(gate + kGateEnd + 16 * ks + 8 * m + 2 * t);
                xf[ks][2 * m] = pack_half2(ed.x * y[2 * ks + m][0], ed.y * y[2 * ks + m][1]);
                xf[ks][2 * m + 1] = pack_half2(ed.x * y[2 * ks + m][2], ed.y * y[2 * ks + m][3]);
            }
        const float d = gate[kGateAll];
#pragma unroll
        for (int nt = 0; nt < 16; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] *= d;
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
    if (P.final_state)
#pragma unroll
        for (int nt = 0; nt < 16; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) store_state(P.final_state, P.final_dtype, at(nt, e), s[nt][e]);
}

// ---- an output warp: O^T = scale (e^G (S^T Q^T) + X^T P^T) ------------------------------------
template <int NW>
__device__ void outputs(const GdrChunked& P, ChainSmem<NW>& S, const Span& span, int nch, int w, int lane,
                        int h, int v0) {
    const GdrInputs& I = P.in;
    const int t = lane & 3;
    for (int c = 0; c < nch; ++c) {
        const int st = c % kStages, buf = c & 1;
        auto& G = S.stage[st];
        auto& H = S.hand[w][buf];
        const uint32_t sq = smem_u32(G.q), sP = smem_u32(G.block) + kTileBytes, sv = smem_u32(G.v[w]);
        const float* gate = reinterpret_cast<const float*>(G.block + 2 * kTileBytes);
        if (!bar_wait(&S.full[st], (unsigned)((c / kStages) & 1), P.err)) return;
        if (!bar_wait(&S.s_full[w][buf], (unsigned)((c / 2) & 1), P.err)) return;
        float y[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t a[4];
            ldsm(a, a_addr<256>(smem_u32(H.s), 0, 2 * ks, lane));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t b[4];
                ldsm(b, b_addr<256>(sq, 16 * np, 2 * ks, lane));
                mma_f16(y[2 * np], a, b[0], b[1]);
                mma_f16(y[2 * np + 1], a, b[2], b[3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const float2 e = *reinterpret_cast<const float2*>(gate + kGateE + 8 * nt + 2 * t);
            y[nt][0] *= e.x; y[nt][1] *= e.y; y[nt][2] *= e.x; y[nt][3] *= e.y;
        }
        if (!bar_wait(&S.x_full[w][buf], (unsigned)((c / 2) & 1), P.err)) return;
        uint32_t xf[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) ldsm(xf[ks], a_addr<128>(smem_u32(H.x), 0, 2 * ks, lane));
        __syncwarp();
        if (lane == 0) bar_arrive(&S.hand_empty[w][buf]);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                if (2 * kp > nt / 2) break;
                uint32_t b[4];
                ldsm(b, unit_at<128>(sP, 8 * nt + (lane & 7), 4 * kp + (lane >> 3)));
                mma_f16(y[nt], xf[2 * kp], b[0], b[1]);
                if (2 * kp + 1 <= nt / 2) mma_f16(y[nt], xf[2 * kp + 1], b[2], b[3]);
            }
        // [v][token] -> rows of 16 channels per token, through the warp's V tile (its state
        // warp has read V before it raised x_full), then 16-byte stores
#pragma unroll
        for (int np = 0; np < 4; ++np)
            stsm_t(v_at(sv, 16 * np + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1),
                   pack_bf16(I.scale * y[2 * np][0], I.scale * y[2 * np][1]),
                   pack_bf16(I.scale * y[2 * np][2], I.scale * y[2 * np][3]),
                   pack_bf16(I.scale * y[2 * np + 1][0], I.scale * y[2 * np + 1][1]),
                   pack_bf16(I.scale * y[2 * np + 1][2], I.scale * y[2 * np + 1][3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int token = 16 * i + (lane >> 1), row = c * kC + token;
            if (row < span.len)
                *reinterpret_cast<uint4*>(P.out + ((span.start + row) * I.Hv + h) * kDim + v0 + 8 * (lane & 1)) =
                    *reinterpret_cast<const uint4*>(G.v[w] + (v_at(0, token, lane & 1)));
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.empty[st]);
    }
}

// For the backward pass: the output warps copy S^T and X^T of every chunk to memory instead.
template <int NW>
__device__ void keep(const GdrChunked& P, ChainSmem<NW>& S, const Span& span, int nch, int w, int lane, int h,
                     int v0) {
    for (int c = 0; c < nch; ++c) {
        const int st = c % kStages, buf = c & 1;
        auto& H = S.hand[w][buf];
        const size_t at = (size_t)(span.chunk + c) * P.in.Hv + h;
        if (!bar_wait(&S.s_full[w][buf], (unsigned)((c / 2) & 1), P.err)) return;
        uint4* ds = reinterpret_cast<uint4*>(P.states + at * kStateTile + v0 * kDim * 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) ds[i * 32 + lane] = reinterpret_cast<const uint4*>(H.s)[i * 32 + lane];
        if (!bar_wait(&S.x_full[w][buf], (unsigned)((c / 2) & 1), P.err)) return;
        uint4* dx = reinterpret_cast<uint4*>(P.xs + at * kTokenTile + v0 * kC * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) dx[i * 32 + lane] = reinterpret_cast<const uint4*>(H.x)[i * 32 + lane];
        __syncwarp();
        if (lane == 0) {
            bar_arrive(&S.hand_empty[w][buf]);
            bar_arrive(&S.empty[st]);
        }
    }
}

// One CTA per 16 NW value channels of a (sequence, value head): NW state warps, NW output
// warps, 4 producer warps.
template <int NW, bool kSave>
__global__ void __launch_bounds__(64 * NW + kProducers, 1) gdr_chain_kernel(GdrChunked P) {
    extern __shared__ __align__(128) unsigned char raw[];
    ChainSmem<NW>& S = *reinterpret_cast<ChainSmem<NW>*>(raw);
    const GdrInputs& I = P.in;
    if (I.cu && !*I.valid) return;
    constexpr int kParts = kDim / (16 * NW);
    const int part = blockIdx.x % kParts, unit = blockIdx.x / kParts;
    const int h = unit % I.Hv, n = unit / I.Hv;
    const Span span = span_of(I, P.chunks, n);
    const int nch = (span.len + kC - 1) / kC;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&S.full[i], 2 * kProducers);
            bar_init(&S.empty[i], 2 * NW);
        }
        for (int i = 0; i < NW; ++i)
            for (int j = 0; j < 2; ++j) {
                bar_init(&S.s_full[i][j], 1);
                bar_init(&S.x_full[i][j], 1);
                bar_init(&S.hand_empty[i][j], 1);
            }
    }
    __syncthreads();
    const size_t sbase = ((size_t)n * I.Hv + h) * kDim * kDim;
    if (w < NW) {
        chain<NW>(P, S, nch, w, lane, sbase, part * 16 * NW + 16 * w);
    } else if (w < 2 * NW) {
        const int v0 = part * 16 * NW + 16 * (w - NW);
        if (kSave) keep<NW>(P, S, span, nch, w - NW, lane, h, v0);
        else outputs<NW>(P, S, span, nch, w - NW, lane, h, v0);
    } else if (nch > 0) {
        produce<NW, kSave>(P, S, span, nch, h, part, tid - 64 * NW);
    }
}

template <int NW, bool kSave>
cudaError_t launch(const GdrChunked& P, cudaStream_t s) {
    const cudaError_t e = allow_smem<gdr_chain_kernel<NW, kSave>>(sizeof(ChainSmem<NW>));
    if (e != cudaSuccess) return e;
    const long long ctas = (long long)P.in.N * P.in.Hv * (kDim / (16 * NW));
    gdr_chain_kernel<NW, kSave><<<(unsigned)ctas, 64 * NW + kProducers, sizeof(ChainSmem<NW>), s>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_chain(const GdrChunked& P, int sms, cudaStream_t s) {
    const long long units = (long long)P.in.N * P.in.Hv;
    if (units == 0) return cudaSuccess;
    if (P.states) return units * 2 <= sms ? launch<2, true>(P, s) : launch<4, true>(P, s);
    return units * 2 <= sms ? launch<2, false>(P, s) : launch<4, false>(P, s);
}

}  // namespace kda

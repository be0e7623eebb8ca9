// The chunks of a sequence backwards: the sequential part of the backward pass of the gated
// delta rule with one decay per value head (equations: kda_gdr_bwd.cu).
//
// The mirror image of the forward chain (kda_gdr_chain.cuh), with the same roles and the same
// hand-over between them; the gradient dS^T of the state (lane = value channel) is an fp32
// accumulator in tensor memory, and
//
//   dX^T = dO^T P + DS16 (e^(GC-G) K)^T        N = 64     DS16 = fp16(dS^T)
//   Y^T  = DX16 T                              N = 64     DX16 = fp16(dX^T)
//   dS^T = e^GC dS^T + dO^T (e^G Q) + Y16 (-beta e^G K)   N = 128
//
// with dO = fp16(scale dO), all of it times 2^scale (kda_gdr_chunk.cuh).  The warps that bring in dO are up to two
// chunks ahead of the chain, so chunk i's scale (counted as the chain walks) comes from e^GC dS as chunk i - 2 began and
// dO of the three, with the decay in between.  Products with dO as the left operand read it from shared
// memory (channels contiguous: MN-major) and are off the chain.  The state warps also write
// DS16 and Y16 of every chunk to memory; four warps write dV = beta Y.
//
// Measured: 2.4 us per chunk (4,096 tokens x 32 heads: 157 us, 153 with scales left out); without those 48 KB to
// memory it would be 2.0, without dV 2.1: the stores share the load/store unit with the conversions.
#include "kda_gdr_chain.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int kStages = 2;
constexpr int kOutWarps = 4;
constexpr int kFirstKeys = kStateWarps + kOutWarps, kFirstQueries = kFirstKeys + kProducers / 32,
              kMmaWarp = kFirstQueries + kProducers / 32;
constexpr int kScaleWarp = kMmaWarp + 1;
constexpr int kBackThreads = 32 * (kMmaWarp + 4);
// registers of a thread: 80 at launch, then by role (2 x 112 + 64 + 72 + 88 + 32 = 6 x 80)
constexpr int kStateRegs = 112, kOutRegs = 64, kKeyRegs = 72, kQueryRegs = 88, kMmaRegs = 32;
// tensor memory columns; the accumulators of dX and Y alternate between two buffers
constexpr uint32_t kTmS = 0, kTmS16 = 128, kTmX16 = 192, kTmY16 = 224, kTmAcc = 256, kTmCols = 512;

struct BackSmem {
    struct Stage {
        unsigned char kd[kRowsTile];          // e^(GC-G) K, fp16
        unsigned char kb[kRowsTile];          // -beta e^G K, fp16
        unsigned char q[kRowsTile];           // e^G Q, fp16
        unsigned char o[kRowsTile];           // dO, fp16
        unsigned char t[kTileBytes], p[kTileBytes];
    } stage[kStages];
    unsigned char turn[kOutWarps][kTurnBytes];
    uint64_t full[kStages], copied[kStages], empty[kStages];
    uint64_t s16, x16, y16;                   // operands written by the state warps
    uint64_t acc, y, s_done;                  // products done
    uint64_t y_free, done, drain;
    uint64_t begun, ready;                    // the last state's gradient's exponents, the first two scales are there
    ScaleRing scales;                         // published: of that gradient, then of e^GC dS of the chunk before
    uint32_t tmem;
};

static_assert(sizeof(BackSmem::Stage) % 1024 == 0, "the 128-byte swizzle wants 1,024-byte alignment");

// ---- producers ----------------------------------------------------------------------------
// one group for keys, T and P
__device__ void back_keys(const GdrBackward& B, BackSmem& S, const Span& span, int nch, int h, int p) {
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk), unit = p & 15, row0 = p >> 4, lane = p & 31;
    const int dst = rows_tile_at(row0, unit);
    const size_t at = (size_t)span.chunk * I.Hv + h, step = (size_t)I.Hv * kBlockBytes;
    const unsigned char* block = P.blocks + at * kBlockBytes;
    const unsigned char* ts = P.ts + at * kTileBytes;
    // a thread's gate: beta e^G (unit < 8) or e^(GC-G) of row row0 + 8 (unit % 8)
    const float* gate = reinterpret_cast<const float*>(block + 2 * kTileBytes) + row0 + 8 * (unit & 7) +
                        (unit < 8 ? kGateBe : kGateEnd);
    Rows k(I.k, I.k_stride, span, hk * kDim, p);
    const auto ahead = [&](int c) {           // what will be fetched two chunks on, into L2
        if (c < 0) return;
        prefetch_rows(I.k, I.k_stride, span, hk * kDim, c, p);
        if (p < 64) prefetch_l2(block + c * step + kTileBytes + 128 * p);
        else prefetch_l2(ts + (size_t)c * I.Hv * kTileBytes + 128 * (p - 64));
        if (p < 8) prefetch_l2(block + c * step + 2 * kTileBytes + 128 * p);
    };
    k.fetch(nch - 1);
    float ga = gate[(nch - 1) * (step / 4)];
    ahead(nch - 2);
    ahead(nch - 3);
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i, st = i % kStages;
        const unsigned phase = (unsigned)((i / kStages) & 1);
        auto& G = S.stage[st];
        if (i >= kStages && !bar_wait(&S.empty[st], phase ^ 1u, P.err)) return;
        if (p == 0) {
            const uint32_t bar = smem_u32(&S.copied[st]);
            tc::mbar_arrive_expect_tx(bar, 2 * kTileBytes);
            tc::bulk_g2s(smem_u32(G.t), ts + (size_t)c * I.Hv * kTileBytes, kTileBytes, bar);
            tc::bulk_g2s(smem_u32(G.p), block + c * step + kTileBytes, kTileBytes, bar);
        }
#pragma unroll
        for (int j = 0; j < kTokenRows; ++j) {
            const float be = __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + j), ed = __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + 8 + j);
            *reinterpret_cast<uint4*>(G.kd + dst + 1024 * j) = scaled_half8(k.x[j], ed);
            *reinterpret_cast<uint4*>(G.kb + dst + 1024 * j) = scaled_half8(k.x[j], -be);
        }
        tc::fence_proxy_async_smem();         // the MMAs read what was stored here
        // `full` means the copies too, and no copy is on its way when the warp that started it leaves
        if (p < 32) bar_wait(&S.copied[st], phase, P.err, kDrainTries);
        bar_arrive(&S.full[st]);
        if (c > 0) {
            k.fetch(c - 1);
            ga = gate[(c - 1) * (step / 4)];
        }
        ahead(c - 3);
    }
}

// one for queries and the outputs' gradients
__device__ void back_queries(const GdrBackward& B, BackSmem& S, const Span& span, int nch, int h, int p) {
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk), unit = p & 15, row0 = p >> 4, lane = p & 31;
    const int dst = rows_tile_at(row0, unit);
    const float* gate = reinterpret_cast<const float*>(P.blocks + ((size_t)span.chunk * I.Hv + h) * kBlockBytes + 2 * kTileBytes) +
                        kGateE + row0 + 8 * (unit & 7);
    const size_t step = (size_t)I.Hv * (kBlockBytes / 4);
    const long long o_stride = (long long)I.Hv * kDim;
    Rows q(I.q, I.q_stride, span, hk * kDim, p), o(B.in.dout, o_stride, span, h * kDim, p);
    const auto ahead = [&](int c) {
        prefetch_rows(I.q, I.q_stride, span, hk * kDim, c, p);
        prefetch_rows(B.in.dout, o_stride, span, h * kDim, c, p);
    };
    q.fetch(nch - 1);
    o.fetch(nch - 1);
    float ga = gate[(nch - 1) * step];
    ahead(nch - 2);
    ahead(nch - 3);
    if (!bar_wait(&S.ready, 0u, P.err)) return;
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i, st = i % kStages;
        auto& G = S.stage[st];
        if (i >= kStages && !bar_wait(&S.empty[st], (unsigned)(((i / kStages) & 1) ^ 1), P.err)) return;
        const float by = S.scales.in[i & 3];
#pragma unroll
        for (int j = 0; j < kTokenRows; ++j) {
            *reinterpret_cast<uint4*>(G.q + dst + 1024 * j) = scaled_half8(q.x[j], __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + j));
            *reinterpret_cast<uint4*>(G.o + dst + 1024 * j) = scaled_half8(o.x[j], by);
        }
        tc::fence_proxy_async_smem();
        bar_arrive(&S.full[st]);
        if (c > 0) {
            q.fetch(c - 1);
            o.fetch(c - 1);
            ga = gate[(c - 1) * step];
        }
        ahead(c - 3);
    }
}

// ---- the MMAs (one warp) ------------------------------------------------------------------------
__device__ void back_issue(const GdrBackward& B, BackSmem& S, int nch, uint32_t tmem) {
    int* err = B.fwd.err;
    const auto stage_of = [&](int i) { return uniform(smem_u32(&S.stage[i % kStages])); };
    const auto wait = [&](uint64_t& b, unsigned parity) {
        const bool ok = bar_wait(&b, parity, err);
        tc::fence_after_sync();
        return ok;
    };
    const auto there = [&](int i) { return wait(S.full[i % kStages], (unsigned)((i / kStages) & 1)); };
    // D (+)= dO^T B: dO and B (N columns) with the tokens along k
    const auto from_o = [&](uint32_t d, uint32_t stage, uint32_t b, uint32_t id, bool add) {
        const uint32_t on = tc::elect();
        const uint64_t d_o = desc_mn(stage + offsetof(BackSmem::Stage, o), kHalfTile), d_b = desc_mn(stage + b, kHalfTile);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            tc::mma_ss_on(d, d_o + kstep_mn(k), d_b + kstep_mn(k), id | tc::kIdMnA | tc::kIdMnB, add || k > 0, on);
    };
    // dX^T's part that does not need the state: dO^T P
    const auto begin = [&](int i) {
        from_o(tmem + kTmAcc + 64 * uniform(i & 1), stage_of(i), offsetof(BackSmem::Stage, p), kId64, false);
    };
    if (!there(0)) return;
    begin(0);
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        const unsigned turn = (unsigned)(i & 1);
        const uint32_t stage = stage_of(i), acc = tmem + kTmAcc + 64 * uniform(turn), on = tc::elect();
        if (!wait(S.s16, turn)) return;
        product_k<8>(acc, tmem + kTmS16, stage + offsetof(BackSmem::Stage, kd), kId64, true, on);
        tc::commit_on(smem_u32(&S.acc), on);
        if (i > 0 && !wait(S.y_free, turn ^ 1u)) return;     // Y of chunk i - 1 has been read
        if (!wait(S.x16, turn)) return;
        product_mn(acc, tmem + kTmX16, stage + offsetof(BackSmem::Stage, t), kId64, false, on);
        tc::commit_on(smem_u32(&S.y), on);
        tc::arrive_on(smem_u32(&S.y), on);   // hands on the scales, too
        from_o(tmem + kTmS, stage, offsetof(BackSmem::Stage, q), kId128, true);
        if (i + 1 < nch && !there(i + 1)) return;
        if (!wait(S.y16, turn)) return;
        product_mn(tmem + kTmS, tmem + kTmY16, stage + offsetof(BackSmem::Stage, kb), kId128, true, on);
        tc::commit_on(smem_u32(&S.s_done), on);
        tc::arrive_on(smem_u32(&S.s_done), on);
        tc::commit_on(smem_u32(&S.empty[i % kStages]), on);
        tc::arrive_on(smem_u32(&S.empty[i % kStages]), on);
        if (i + 1 < nch) begin(i + 1);
    }
}

// ---- state warps ----------------------------------------------------------------------------
__device__ void back_states(const GdrBackward& B, BackSmem& S, const Span& span, int nch, int w, int lane, size_t sbase,
                            int h, uint32_t tmem) {
    const GdrChunked& P = B.fwd;
    const int half = w >> 2, v = 32 * (w & 3) + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (w & 3)) << 16);
    const size_t at = sbase + (size_t)(64 * half) * kDim + v;
    const float* dp = reinterpret_cast<const float*>(P.blocks + ((size_t)span.chunk * P.in.Hv + h) * kBlockBytes +
                                                     2 * kTileBytes) + kGateAll;
    const size_t d_step = (size_t)P.in.Hv * (kBlockBytes / 4);
    float d = nch > 0 ? dp[(nch - 1) * d_step] : 0.0f;
    uint32_t x[2][32];
    load_state(x, B.in.dfinal, B.in.dfinal_dtype, at);
    if (nch > 0) {
        if (B.in.dfinal) {
            publish(S.scales.top[0][w], x, lane);
            if (lane == 0) bar_arrive(&S.begun);
        }
        if (!bar_wait(&S.ready, 0u, P.err)) return;
        scale32(x[0], S.scales.ratio[0]);
        scale32(x[1], S.scales.ratio[0]);
    }
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i;
        const unsigned turn = (unsigned)(i & 1);
        const float next_d = c > 0 ? dp[(c - 1) * d_step] : 0.0f;
        uint32_t f[2][16];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            to_half<16>(x[j], f[j]);
            tc::st16(tl + kTmS16 + 32 * half + 16 * j, f[j]);
            scale32(x[j], d);
            tc::st32(tl + kTmS + 64 * half + 32 * j, x[j]);
        }
        operand_ready(&S.s16, lane);
        const size_t unit = (size_t)(span.chunk + c) * P.in.Hv + h;
        keep_units(B.dstates + unit * kStateTile, v, 8 * half, f[0]);
        keep_units(B.dstates + unit * kStateTile, v, 8 * half + 4, f[1]);
        publish(S.scales.top[(i + 1) & 3][w], tl + kTmS16 + 32 * half, d, lane);
        uint32_t y[32];
        if (!bar_wait(&S.acc, turn, P.err)) return;
        tc::fence_after_sync();
        tc::ld32(tl + kTmAcc + 64 * turn + 32 * half, y);
        tc::wait_ld();
        to_half<16>(y, f[0]);
        tc::st16(tl + kTmX16 + 16 * half, f[0]);
        operand_ready(&S.x16, lane);
        if (!bar_wait(&S.y, turn, P.err)) return;
        tc::fence_after_sync();
        tc::ld32(tl + kTmAcc + 64 * turn + 32 * half, y);
        tc::wait_ld();
        to_half<16>(y, f[0]);
        tc::st16(tl + kTmY16 + 16 * half, f[0]);
        operand_ready(&S.y16, lane);
        keep_units(B.ys + unit * kTokenTile, v, 4 * half, f[0]);
        d = next_d;
        if (!bar_wait(&S.s_done, turn, P.err)) return;
        tc::fence_after_sync();
        const float ratio = S.scales.ratio[(i + 1) & 3];
        if (__builtin_expect(c > 0 && ratio != 1.0f, 0)) rescale(tl + kTmS + 64 * half, ratio);
        tc::ld32(tl + kTmS + 64 * half, x[0]);
        tc::ld32(tl + kTmS + 64 * half + 32, x[1]);
        tc::wait_ld();
    }
    if (B.dinit) store_state(x, nch > 0 ? S.scales.out[(nch - 1) & 3] : 1.0f, B.dinit, B.dinit_dtype, at);
}

// ---- scales (one warp) ------------------------------------------------------------------------
// Chunk i + 2's once the state warps have published e^GC dS of chunk i (with dX16); Y16's barrier hands the choice
// to the issuing warp and its arrivals to everyone else.
__device__ void back_scales(const GdrBackward& B, BackSmem& S, const Span& span, int nch, int h, int lane) {
    const GdrChunked& P = B.fwd;
    const size_t step = (size_t)P.in.Hv * (kBlockBytes / 4);
    float* gates = reinterpret_cast<float*>(P.blocks + ((size_t)(span.chunk + nch - 1) * P.in.Hv + h) * kBlockBytes + 2 * kTileBytes);
    const auto d_o = [&](int i) { return i < nch ? *reinterpret_cast<const unsigned*>(gates - i * step + kGateDo) : 0u; };
    const auto decay = [&](int i) { return i < nch ? gates[kGateAll - (ptrdiff_t)(i * step)] : 0.0f; };
    int scale = 0, one = kNothing, two = kNothing;    // exponents of dO one and two chunks back
    const auto next = [&](int i, int before, unsigned bytes) {
        const int now = exponent_of_bytes(bytes), last = scale;
        scale = gradient_scale(scale, max(before, max(one, now)));
        two = one;
        one = now;
        if (lane != 0 || i >= nch) return;
        S.scales.ratio[i & 3] = power_of_two(min(scale - last, 127));
        S.scales.in[i & 3] = P.in.scale * power_of_two(scale);
        S.scales.out[i & 3] = power_of_two(-scale);
        reinterpret_cast<int*>(gates - i * step)[kGateGradScale] = scale;
    };
    const auto product = [](int a, int b) { return max(a + b, kNothing); };      // of exponents
    unsigned ahead = d_o(2);
    float fade = decay(1);
    const unsigned first = d_o(0), second = d_o(1);
    const int fade0 = exponent_of(decay(0));
    if (B.in.dfinal && !bar_wait(&S.begun, 0u, P.err)) return;
    const int begun = published(S.scales, 0, 0);
    next(0, begun, first);
    int held = scale;                         // chunk i's scale, in which e^GC dS is published
    next(1, product(begun, fade0), second);
    __syncwarp();
    if (lane == 0) bar_arrive(&S.ready);
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        if (!bar_wait(&S.x16, (unsigned)(i & 1), P.err)) return;
        if (i + 2 < nch) {
            const int now = exponent_of(fade);
            const unsigned bytes = ahead;
            ahead = d_o(i + 3);
            fade = decay(i + 2);
            const int before = product(max(published(S.scales, i + 1, held), two), now);
            held = scale;
            next(i + 2, before, bytes);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.y16);
    }
}

// ---- output warps: dV = beta Y ---------------------------------------------------------------
__device__ void back_outputs(const GdrBackward& B, BackSmem& S, const Span& span, int nch, int w, int lane, int h,
                             uint32_t tmem) {
    const GdrChunked& P = B.fwd;
    const uint32_t tl = tmem + ((uint32_t)(32 * (w & 3)) << 16);
    const size_t step = (size_t)P.in.Hv * kDim;
#pragma unroll 1
    for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i;
        const unsigned turn = (unsigned)(i & 1);
        // beta / 2^scale of tokens 2 lane and 2 lane + 1
        float2 b = reinterpret_cast<const float2*>(P.blocks + ((size_t)(span.chunk + c) * P.in.Hv + h) * kBlockBytes +
                                                   2 * kTileBytes + 4 * kGateB)[lane];
        if (!bar_wait(&S.y, turn, P.err)) return;
        tc::fence_after_sync();
        const float back = S.scales.out[i & 3];
        b.x *= back;
        b.y *= back;
        store_tokens(B.dv + (span.start + (long long)c * kC) * step + h * kDim + 32 * (w & 3), step,
                     min(kC, span.len - c * kC), tl + kTmAcc + 64 * turn, S.turn[w & 3], lane,
                     [&](int t) {
                         return make_float2(__shfl_sync(0xFFFFFFFFu, b.x, t >> 1), __shfl_sync(0xFFFFFFFFu, b.y, t >> 1));
                     },
                     [&] {
                         __syncwarp();
                         if (lane == 0) bar_arrive(&S.y_free);
                     });
    }
}

__device__ __forceinline__ void back_run(const GdrBackward& B, BackSmem& S, int n, int h) {
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const Span span = span_of(I, P.chunks, n);
    const int nch = (int)uniform((span.len + kC - 1) / kC);
    const int tid = threadIdx.x, lane = tid & 31, w = (int)uniform(tid >> 5);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&S.full[i], 2 * kProducers);
            bar_init(&S.copied[i], 1);
            bar_init(&S.empty[i], 2);
        }
        for (uint64_t* b : {&S.acc, &S.drain, &S.ready}) bar_init(b, 1);
        for (uint64_t* b : {&S.y, &S.s_done}) bar_init(b, 2);
        for (uint64_t* b : {&S.s16, &S.x16, &S.begun}) bar_init(b, kStateWarps);
        bar_init(&S.y16, kStateWarps + 1);
        bar_init(&S.y_free, kOutWarps);
        bar_init(&S.done, kStateWarps + kOutWarps);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < kStateWarps) S.scales.top[0][tid] = kNothing;
    tc::fence_proxy_async_smem();
    if (w == kMmaWarp) {
        tc::tmem_alloc(smem_u32(&S.tmem), kTmCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(S.tmem);
    const size_t sbase = ((size_t)n * I.Hv + h) * kDim * kDim;
    if (w < kStateWarps) {
        tc::registers_up<kStateRegs>();
        back_states(B, S, span, nch, w, lane, sbase, h, tmem);
    } else if (w < kFirstKeys) {
        tc::registers_down<kOutRegs>();
        back_outputs(B, S, span, nch, w, lane, h, tmem);
    } else if (w < kFirstQueries) {
        tc::registers_down<kKeyRegs>();
        if (nch > 0) back_keys(B, S, span, nch, h, tid - 32 * kFirstKeys);
        return;
    } else if (w < kMmaWarp) {
        tc::registers_up<kQueryRegs>();
        if (nch > 0) back_queries(B, S, span, nch, h, tid - 32 * kFirstQueries);
        return;
    } else {
        tc::registers_down<kMmaRegs>();
        if (w > kMmaWarp) {
            if (w == kScaleWarp && nch > 0) back_scales(B, S, span, nch, h, lane);
            return;
        }
        if (nch > 0) back_issue(B, S, nch, tmem);
        // every MMA and every arrival of this warp is over, and all other warps have left tensor
        // memory, before it is freed
        tc::commit_on(smem_u32(&S.drain), tc::elect());
        bar_wait(&S.drain, 0u, P.err, kDrainTries);
        bar_wait(&S.done, 0u, P.err, kDrainTries);
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmCols);
        return;
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) bar_arrive(&S.done);
}

static_assert(kBackThreads == chain::kChainThreads, "one launch for both chains");

// Both chains of a (sequence, value head), a CTA each: the gradient's and the one that computes the
// states again (where `states_too`) do not need each other, and with both in one launch a
// sequence's time is the longer one's, not the sum.  The longer ones, the gradient's, come first.
__global__ void __launch_bounds__(kBackThreads, 1) gdr_bwd_chain_kernel(GdrBackward B, GdrChunked F, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char raw[];
    previous_done();
    const GdrInputs& I = B.fwd.in;
    if (I.cu && !*I.valid) return;
    const int units = I.N * I.Hv, unit = blockIdx.x % units, n = sequence_of(B.fwd.chunks, unit / I.Hv), h = unit % I.Hv;
    if (blockIdx.x < units) back_run(B, aligned_smem<BackSmem>(raw), n, h);
    else chain::run<true>(F, vmap, aligned_smem<chain::ChainSmem>(raw), n, h);
}

}  // namespace

cudaError_t launch_gdr_bwd_chain(const GdrBackward& B, const GdrChunked* states_too, cudaStream_t s) {
    const long long units = (long long)B.fwd.in.N * B.fwd.in.Hv;
    if (units == 0) return cudaSuccess;
    constexpr size_t smem = (sizeof(BackSmem) > sizeof(chain::ChainSmem) ? sizeof(BackSmem) : sizeof(chain::ChainSmem)) + 1024;
    CUtensorMap vmap{};
    cudaError_t e = allow_smem<gdr_bwd_chain_kernel>(smem);
    if (e == cudaSuccess && states_too) e = chain::values_map(*states_too, &vmap);
    if (e != cudaSuccess) return e;
    return launch_after(true, gdr_bwd_chain_kernel, dim3((unsigned)(states_too ? 2 * units : units)), kBackThreads, smem, s, B,
                        states_too ? *states_too : B.fwd, vmap);
}

}  // namespace kda

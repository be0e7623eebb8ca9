// The chunks of a sequence one after another: the sequential part of the gated delta rule
// with one decay per value head (the chunked form's equations: kda_gdr_chunk.cuh).
//
// One CTA per (sequence, value head) walks the chunks with the state S^T (lane = value
// channel, column = key channel) as an fp32 accumulator in tensor memory.  All products
// are tcgen05.mma with M = 128 value channels:
//
//   R^T = V^T I - S16 (e^G K)^T       N = 64 tokens     S16 = fp16(S^T)
//   X^T = R16 (T beta)^T              N = 64            R16 = fp16(R^T)
//   S^T = e^GC S^T + X16 (e^(GC-G) K) N = 128           X16 = fp16(X^T)
//   O^T = S16 (e^G Q)^T + X16 P^T     N = 64, off the chain
//
// The left operands are fp16 in tensor memory; decays and signs are folded into the keys and
// queries on their way to shared memory, and V enters R as a product with the identity (bf16,
// exact), so that between two products the state warps only round an accumulator.  V, R, X and S stand for
// 2^scale times themselves (kda_gdr_chunk.cuh): the identity's ones are 2^scale, the state is multiplied
// when the scale changes, and the outputs are multiplied back.  Chunk c's scale comes from e^GC S as chunk c - 1
// began, and the values of both, so that it is known before chunk c's first product.  S is looked at every kLookEvery
// chunks, and wherever what remains of it after the decays may be far above the values; else its size is
// taken to follow both.
//
// Warps: 8 state warps (lane quarter w % 4, half of the columns each) do that rounding; one
// warp issues the MMAs, those that the chain does not need behind the state's update;
// 4 warps bring in keys, values, T and P of the next chunks, 4 the queries, 4 write the
// outputs, one chooses the scales and two find out how large the values are.  Every role's loop is
// kept small: with the MMAs issued from a state warp, the others' jumps over that code cost 200 cycles
// each (instruction cache misses).
// Measured: 1.65 us per chunk of 64 tokens (8,192 tokens x 96 heads on 96 SMs: 213 us, 204 with scales left out; the
// same chain with mma.sync and a warp per 16 channels took 645).  Of some 3,100 cycles the tensor core runs
// 1,200; the rest are the three roundings (100 to 350 cycles each), the hand-overs (130 to 190
// cycles from a warp's arrival to the MMA, as many back) and their contention
// with the other roles (0.49 of the issue slots are taken).
// All waits are bounded: a role whose wait gives up returns, and so do those that wait for it.
#pragma once

#include <cstddef>

#include "kda_gdr_tc.cuh"

namespace kda {
namespace gdr {
namespace chain {

constexpr int kStages = 3;                    // chunks in shared memory
// A look at the state takes issue slots where the chain waits for them: with one in every chunk 20,000 tokens x 8 heads take
// 484 us, in every 4th 476, in every 8th 473.
constexpr int kLookEvery = 4, kFarAbove = 8;  // (2^8)
constexpr int kOutWarps = 4;
constexpr int kFirstKeys = kStateWarps + kOutWarps, kFirstQueries = kFirstKeys + kProducers / 32,
              kMmaWarp = kFirstQueries + kProducers / 32;
constexpr int kScaleWarp = kMmaWarp + 1;
constexpr int kChainThreads = 32 * (kMmaWarp + 4);   // whole warpgroups
// registers of a thread: 80 at launch, then by role (2 x 112 + 64 + 72 + 80 + 40 = 6 x 80)
constexpr int kStateRegs = 112, kOutRegs = 64, kKeyRegs = 72, kMmaRegs = 40;
// tensor memory columns; S16 and O alternate between two buffers
constexpr uint32_t kTmS = 0, kTmS16 = 128, kTmAcc = 256, kTmR16 = 320, kTmX16 = 352, kTmO = 384, kTmCols = 512;

struct ChainSmem {
    struct Stage {
        unsigned char kn[kRowsTile];          // -e^G K, fp16
        unsigned char kd[kRowsTile];          // e^(GC-G) K, fp16
        unsigned char v[kRowsTile];           // V, bf16
        unsigned char tp[2 * kTileBytes];     // T beta, P
    } stage[kStages];
    unsigned char q[kRowsTile];               // e^G Q, fp16
    unsigned char eye[kTileBytes];            // identity, bf16 [64][64]
    unsigned char turn[kOutWarps][kTurnBytes];
    uint64_t full[kStages], copied[kStages], empty[kStages];
    uint64_t s16, r16, x16;                   // operands written by the state warps
    uint64_t acc, x, s_done;                  // products done
    uint64_t q_full, o_done[2], o_free[2];
    uint64_t done, drain;
    uint64_t begun, tops, ready;              // the initial state's exponents, a chunk's, chunk 0's scale are there
    uint64_t sized[kStages];
    float largest[kStages][2];                // |V| of the halves of a stage's values
    ScaleRing scales;                         // published: of the initial state, then of e^GC S of the chunk before
    uint32_t tmem;
};
static_assert(sizeof(ChainSmem::Stage) % 1024 == 0, "the 128-byte swizzle wants 1,024-byte alignment");

// ---- producers ----------------------------------------------------------------------------
__device__ inline void keys(const GdrChunked& P, const CUtensorMap& vmap, ChainSmem& S, const Span& span, int nch, int h, int p) {
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk), unit = p & 15, row0 = p >> 4, lane = p & 31;
    const int dst = rows_tile_at(row0, unit);                 // rows 8 apart: 1,024 bytes
    const size_t step = (size_t)I.Hv * kBlockBytes;
    const unsigned char* block = P.blocks + ((size_t)span.chunk * I.Hv + h) * kBlockBytes;
    // a thread's gate: e^G (unit < 8) or e^(GC-G) of row row0 + 8 (unit % 8)
    const float* gate = reinterpret_cast<const float*>(block + 2 * kTileBytes) + row0 + 8 * (unit & 7) +
                        (unit < 8 ? kGateE : kGateEnd);
    Rows k(I.k, I.k_stride, span, hk * kDim, p);
    const auto ahead = [&](int c) {           // what will be fetched two chunks on, into L2
        if (c >= nch) return;
        prefetch_rows(I.k, I.k_stride, span, hk * kDim, c, p);
        prefetch_rows(I.v, I.v_stride, span, h * kDim, c, p);
        prefetch_l2(block + c * step + 128 * p);                               // T beta and P
        if (p < 8) prefetch_l2(block + c * step + 2 * kTileBytes + 128 * p);   // gates
    };
    // no copy is on its way when the warp that started it leaves
    const auto leave = [&](int begun) {
        if (p < 32)
            for (int c = max(0, begun - kStages); c < begun; ++c) bar_wait(&S.copied[c % kStages], (unsigned)((c / kStages) & 1), P.err, kDrainTries);
    };
    k.fetch(0);
    float ga = gate[0];
    ahead(1);
    ahead(2);
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        const int st = c % kStages, rows = min(kC, span.len - c * kC);
        auto& G = S.stage[st];
        if (c >= kStages && !bar_wait(&S.empty[st], (unsigned)((c / kStages) & 1) ^ 1u, P.err)) return leave(c);
        if (p == 0) {
            const uint32_t bar = smem_u32(&S.copied[st]);
            tc::mbar_arrive_expect_tx(bar, 2 * kTileBytes + (rows == kC ? kRowsTile : 0));
            tc::bulk_g2s(smem_u32(G.tp), block + c * step, 2 * kTileBytes, bar);
            if (rows == kC) {
                const int row = (int)(span.start + (long long)c * kC);
                tma_block(smem_u32(G.v), &vmap, h * kDim, row, bar);
                tma_block(smem_u32(G.v) + kHalfTile, &vmap, h * kDim + 64, row, bar);
            }
        }
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i) {
            const float eg = __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + i), ed = __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + 8 + i);
            *reinterpret_cast<uint4*>(G.kn + dst + 1024 * i) = scaled_half8(k.x[i], -eg);
            *reinterpret_cast<uint4*>(G.kd + dst + 1024 * i) = scaled_half8(k.x[i], ed);
        }
        if (rows < kC) {                      // the last values: zeros after the sequence's end
            const __nv_bfloat16* v = I.v + (span.start + (long long)c * kC + row0) * I.v_stride + h * kDim + unit * 8;
#pragma unroll 1
            for (int i = 0; i < kTokenRows; ++i)
                *reinterpret_cast<uint4*>(G.v + dst + 1024 * i) =
                    row0 + 8 * i < rows ? __ldg(reinterpret_cast<const uint4*>(v + 8 * i * I.v_stride)) : make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_proxy_async_smem();         // the MMAs read what was stored here
        bar_arrive(&S.full[st]);
        if (c + 1 < nch) {
            k.fetch(c + 1);
            ga = gate[(c + 1) * (step / 4)];
        }
        ahead(c + 3);
    }
    leave(nch);
}

__device__ inline void queries(const GdrChunked& P, ChainSmem& S, const Span& span, int nch, int h, int p) {
    const GdrInputs& I = P.in;
    const int hk = h / (I.Hv / I.Hk), unit = p & 15, row0 = p >> 4, lane = p & 31;
    const int dst = rows_tile_at(row0, unit);
    const float* gate = reinterpret_cast<const float*>(P.blocks + ((size_t)span.chunk * I.Hv + h) * kBlockBytes + 2 * kTileBytes) +
                        kGateE + row0 + 8 * (unit & 7);
    Rows q(I.q, I.q_stride, span, hk * kDim, p);
    q.fetch(0);
    float ga = gate[0];
    prefetch_rows(I.q, I.q_stride, span, hk * kDim, 1, p);
    prefetch_rows(I.q, I.q_stride, span, hk * kDim, 2, p);
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        if (c > 0 && !bar_wait(&S.o_done[(c - 1) & 1], (unsigned)(((c - 1) >> 1) & 1), P.err)) return;   // the last ones have been used
#pragma unroll
        for (int i = 0; i < kTokenRows; ++i)
            *reinterpret_cast<uint4*>(S.q + dst + 1024 * i) = scaled_half8(q.x[i], __shfl_sync(0xFFFFFFFFu, ga, (lane & 16) + i));
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&S.q_full);
        if (c + 1 < nch) {
            q.fetch(c + 1);
            ga = gate[(size_t)(c + 1) * I.Hv * (kBlockBytes / 4)];
        }
        prefetch_rows(I.q, I.q_stride, span, hk * kDim, c + 3, p);
    }
}

// ---- the MMAs (one warp) ------------------------------------------------------------------------
template <bool kSave>
__device__ void issue(const GdrChunked& P, ChainSmem& S, int nch, uint32_t tmem) {
    const auto stage_of = [&](int c) { return uniform(smem_u32(&S.stage[c % kStages])); };
    const auto wait = [&](uint64_t& b, unsigned parity) {
        const bool ok = bar_wait(&b, parity, P.err);
        tc::fence_after_sync();
        return ok;
    };
    const auto there = [&](int c) {
        const unsigned phase = (unsigned)((c / kStages) & 1);
        return wait(S.copied[c % kStages], phase) && wait(S.full[c % kStages], phase);
    };
    // R^T's part that does not need the state: V^T I, the identity's ones being 2^scale
    const auto begin = [&](int c) {
        const uint32_t on = tc::elect();
        const uint64_t dv = desc_mn(stage_of(c) + offsetof(ChainSmem::Stage, v), kHalfTile), de = desc_k(smem_u32(S.eye));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            tc::mma_ss_on(tmem + kTmAcc, dv + kstep_mn(k), de + kstep_k(k, 0), kId64 | tc::kIdBf16 | tc::kIdMnA, k > 0, on);
    };
    if (!wait(S.ready, 0u) || !there(0)) return;
    begin(0);
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        const unsigned turn = (unsigned)(c & 1), phase = (unsigned)((c >> 1) & 1);
        const uint32_t stage = stage_of(c), s16 = tmem + kTmS16 + 64 * uniform(turn), on = tc::elect();
        if (!wait(S.s16, turn)) return;
        product_k<8>(tmem + kTmAcc, s16, stage + offsetof(ChainSmem::Stage, kn), kId64, true, on);
        tc::commit_on(smem_u32(&S.acc), on);
        // a wait takes 200 cycles even if it is over: each is where nothing waits for this warp
        if (c + 1 < nch && !there(c + 1)) return;
        if (!kSave && c >= 2 && !wait(S.o_free[turn], phase ^ 1u)) return;   // the outputs of chunk c - 2 have been read
        if (!wait(S.r16, turn)) return;
        product_k<4>(tmem + kTmAcc, tmem + kTmR16, stage + offsetof(ChainSmem::Stage, tp), kId64, false, on);
        tc::commit_on(smem_u32(&S.x), on);
        if (!kSave && !wait(S.q_full, turn)) return;
        if (!wait(S.x16, turn)) return;
        product_mn(tmem + kTmS, tmem + kTmX16, stage + offsetof(ChainSmem::Stage, kd), kId128, true, on);
        tc::commit_on(smem_u32(&S.s_done), on);
        if (!kSave) {                         // outputs
            const uint32_t o = tmem + kTmO + 64 * uniform(turn);
            product_k<8>(o, s16, smem_u32(S.q), kId64, false, on);
            product_k<4>(o, tmem + kTmX16, stage + offsetof(ChainSmem::Stage, tp) + kTileBytes, kId64, true, on);
            tc::commit_on(smem_u32(&S.o_done[turn]), on);
            tc::arrive_on(smem_u32(&S.o_done[turn]), on);    // hands on the scale, too
        }
        if (c + 1 < nch) begin(c + 1);
        tc::commit_on(smem_u32(&S.empty[c % kStages]), on);
    }
}

// ---- state warps ----------------------------------------------------------------------------
template <bool kSave>
__device__ void states(const GdrChunked& P, ChainSmem& S, const Span& span, int nch, int w, int lane, size_t sbase,
                       int h, uint32_t tmem) {
    const int half = w >> 2, v = 32 * (w & 3) + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (w & 3)) << 16);
    const size_t at = sbase + (size_t)(64 * half) * kDim + v;     // channel 64 half of row v of S^T
    const float* dp = reinterpret_cast<const float*>(P.blocks + ((size_t)span.chunk * P.in.Hv + h) * kBlockBytes +
                                                     2 * kTileBytes) + kGateAll;
    const size_t d_step = (size_t)P.in.Hv * (kBlockBytes / 4);
    float d = nch > 0 ? *dp : 0.0f;
    uint32_t x[2][32];
    load_state(x, P.init_state, P.init_dtype, at);
    if (nch > 0) {
        if (P.init_state) {
            publish(S.scales.top[0][w], x, lane);
            if (lane == 0) bar_arrive(&S.begun);
        }
        if (!bar_wait(&S.ready, 0u, P.err)) return;
        scale32(x[0], S.scales.ratio[0]);
        scale32(x[1], S.scales.ratio[0]);
    }
    int look = 0;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        const unsigned turn = (unsigned)(c & 1);
        const float next_d = c + 1 < nch ? dp[(c + 1) * d_step] : 0.0f;
        // S16, and e^GC S^T for the update to add to (now: once the products run, stores to tensor
        // memory wait for them)
        uint32_t f[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            to_half<16>(x[i], f[i]);
            tc::st16(tl + kTmS16 + 64 * turn + 32 * half + 16 * i, f[i]);
            scale32(x[i], d);
            tc::st32(tl + kTmS + 64 * half + 32 * i, x[i]);
        }
        operand_ready(&S.s16, lane);
        const size_t unit = (size_t)(span.chunk + c) * P.in.Hv + h;
        if (kSave) {                          // for the backward pass
            keep_units(P.states + unit * kStateTile, v, 8 * half, f[0]);
            keep_units(P.states + unit * kStateTile, v, 8 * half + 4, f[1]);
        }
        if (look) {
            publish(S.scales.top[(c + 1) & 3][w], tl + kTmS16 + 64 * turn + 32 * half, d, lane);
            if (lane == 0) bar_arrive(&S.tops);
        }
        uint32_t y[32];
        if (!bar_wait(&S.acc, turn, P.err)) return;
        tc::fence_after_sync();
        tc::ld32(tl + kTmAcc + 32 * half, y);
        tc::wait_ld();
        to_half<16>(y, f[0]);
        tc::st16(tl + kTmR16 + 16 * half, f[0]);
        operand_ready(&S.r16, lane);
        if (!bar_wait(&S.x, turn, P.err)) return;
        tc::fence_after_sync();
        tc::ld32(tl + kTmAcc + 32 * half, y);
        tc::wait_ld();
        to_half<16>(y, f[0]);
        tc::st16(tl + kTmX16 + 16 * half, f[0]);
        operand_ready(&S.x16, lane);
        if (kSave) keep_units(P.xs + unit * kTokenTile, v, 4 * half, f[0]);
        d = next_d;
        const float ratio = c + 1 < nch ? S.scales.ratio[(c + 1) & 3] : 1.0f;     // there since X is
        look = S.scales.look[(c + 1) & 3];
        if (!bar_wait(&S.s_done, turn, P.err)) return;
        tc::fence_after_sync();
        if (__builtin_expect(ratio != 1.0f, 0)) rescale(tl + kTmS + 64 * half, ratio);
        tc::ld32(tl + kTmS + 64 * half, x[0]);
        tc::ld32(tl + kTmS + 64 * half + 32, x[1]);
        tc::wait_ld();
    }
    if (P.final_state) store_state(x, nch > 0 ? S.scales.out[(nch - 1) & 3] : 1.0f, P.final_state, P.final_dtype, at);
}

// ---- sizes of the values (two warps, half a tile each) -------------------------------------------
// They run ahead of the scales, but a stage is not given back before the scale warp's arrival for its chunk (with X),
// which comes after theirs: so neither the values nor a stage's barrier change while someone still needs them.
__device__ inline void sizes(const GdrChunked& P, ChainSmem& S, const Span& span, int nch, int half, int lane) {
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        const int st = c % kStages;
        const unsigned char* tile = S.stage[st].v + half * kHalfTile + 16 * lane;
        const unsigned phase = (unsigned)((c / kStages) & 1);
        // whole tiles are copied, the last one's rows stored by the warps that bring in the keys
        if (!bar_wait(span.len - c * kC >= kC ? &S.copied[st] : &S.full[st], phase, P.err)) return;
        __nv_bfloat162 top[4] = {};
#pragma unroll 4
        for (int i = 0; i < kHalfTile; i += 16 * 32) {
            const uint4 u = *reinterpret_cast<const uint4*>(tile + i);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top[j] = __hmax2(top[j], __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[j])));
        }
        const float2 m = __bfloat1622float2(__hmax2(__hmax2(top[0], top[1]), __hmax2(top[2], top[3])));
        const unsigned all = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(m.x, m.y)));
        if (lane == 0) {
            S.largest[st][half] = __uint_as_float(all);
            bar_arrive(&S.sized[st]);
        }
    }
}

// ---- scales (one warp) ------------------------------------------------------------------------
// Chunk c + 1's while chunk c's R and X are formed; X's barrier hands the choice to the state warps (and X16's on to the
// issuing warp, with the identity as the next chunk wants it).
template <bool kSave>
__device__ void scales(const GdrChunked& P, ChainSmem& S, const Span& span, int nch, int h, int lane) {
    float* gates = reinterpret_cast<float*>(P.blocks + ((size_t)span.chunk * P.in.Hv + h) * kBlockBytes + 2 * kTileBytes);
    const size_t step = (size_t)P.in.Hv * (kBlockBytes / 4);
    // the exponent of a chunk's largest value; false: the wait gave up
    const auto values = [&](int c, int& e) {
        const int st = c % kStages;
        if (!bar_wait(&S.sized[st], (unsigned)((c / kStages) & 1), P.err)) return false;
        e = exponent_of(fmaxf(S.largest[st][0], S.largest[st][1]));
        return true;
    };
    const auto set = [&](int c, int scale, int before) {
        if (lane != 0) return;
        S.scales.ratio[c & 3] = power_of_two(min(scale - before, 127));
        S.scales.out[c & 3] = power_of_two(-scale);
        if (kSave) reinterpret_cast<int*>(gates + c * step)[kGateScale] = scale;
    };
    const auto identity = [&](int scale) {    // ones of 2^scale at (i, i)
        for (int row = lane; row < kC; row += 32)
            *reinterpret_cast<uint16_t*>(S.eye + row * 128 + (((row >> 3) ^ (row & 7)) << 4) + (row & 7) * 2) = (uint16_t)((scale + 127) << 7);
        tc::fence_proxy_async_smem();
    };
    int v, next_v = kNothing;
    if (!values(0, v) || (P.init_state && !bar_wait(&S.begun, 0u, P.err))) return;
    int size = published(S.scales, 0, 0);     // exponent of the state as a chunk begins
    int scale = forward_scale(0, max(size, v)), look = 0;
    unsigned looks = 0;
    float d = gates[kGateAll];
    if (scale) identity(scale);
    set(0, scale, 0);
    __syncwarp();
    if (lane == 0) bar_arrive(&S.ready);
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        if (c + 1 < nch && !values(c + 1, next_v)) return;
        const float next_d = c + 1 < nch ? gates[(c + 1) * step + kGateAll] : 0.0f;
        size = max(size + exponent_of(d), kNothing);
        d = next_d;
        if (look) {
            if (!bar_wait(&S.tops, looks++ & 1, P.err)) return;
            size = published(S.scales, c + 1, scale);
        }
        size = max(size, v);
        if (c + 1 < nch) {
            const int next = forward_scale(scale, max(size, next_v));
            look = (c + 1) % kLookEvery == 0 || size > next_v + kFarAbove;
            if (lane == 0) S.scales.look[(c + 1) & 3] = look;
            v = next_v;
            if (next != scale) {
                if (!bar_wait(&S.acc, (unsigned)(c & 1), P.err)) return;      // the last product with the identity is over
                identity(next);
            }
            set(c + 1, next, scale);
            scale = next;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&S.x);
        // no further than X: one arrival a phase, and what is written for chunk c + 2 takes the place of chunk c - 2's, whose
        // outputs the issuing warp has seen read before X
        if (!bar_wait(&S.x, (unsigned)(c & 1), P.err)) return;
    }
}

// ---- output warps -----------------------------------------------------------------------------
__device__ inline void outputs(const GdrChunked& P, ChainSmem& S, const Span& span, int nch, int w, int lane, int h,
                        uint32_t tmem) {
    const GdrInputs& I = P.in;
    const uint32_t tl = tmem + ((uint32_t)(32 * (w & 3)) << 16);
    const size_t step = (size_t)I.Hv * kDim;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        const int buf = c & 1;
        if (!bar_wait(&S.o_done[buf], (unsigned)((c >> 1) & 1), P.err)) return;
        tc::fence_after_sync();
        const float by = I.scale * S.scales.out[c & 3];
        store_tokens(P.out + (span.start + (long long)c * kC) * step + h * kDim + 32 * (w & 3), step,
                     min(kC, span.len - c * kC), tl + kTmO + 64 * buf, S.turn[w & 3], lane,
                     [&](int) { return make_float2(by, by); },
                     [&] {
                         __syncwarp();
                         if (lane == 0) bar_arrive(&S.o_free[buf]);
                     });
    }
}

// a CTA's work: value head h of sequence n.  kSave: keeps S16 and X16 of every chunk for the
// backward pass instead of writing outputs
template <bool kSave>
__device__ __forceinline__ void run(const GdrChunked& P, const CUtensorMap& vmap, ChainSmem& S, int n, int h) {
    const GdrInputs& I = P.in;
    const Span span = span_of(I, P.chunks, n);
    const int nch = (int)uniform((span.len + kC - 1) / kC);
    const int tid = threadIdx.x, lane = tid & 31, w = (int)uniform(tid >> 5);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&S.full[i], kProducers);
            bar_init(&S.copied[i], 1);
            bar_init(&S.empty[i], 1);
            bar_init(&S.sized[i], 2);
        }
        for (uint64_t* b : {&S.acc, &S.s_done, &S.drain, &S.ready}) bar_init(b, 1);
        bar_init(&S.x, 2);                    // the product and the next scale
        for (uint64_t* b : {&S.s16, &S.r16, &S.x16, &S.begun, &S.tops}) bar_init(b, kStateWarps);
        for (int i = 0; i < 2; ++i) bar_init(&S.o_done[i], 2);
        bar_init(&S.q_full, kProducers / 32);
        for (int i = 0; i < 2; ++i) bar_init(&S.o_free[i], kOutWarps);
        bar_init(&S.done, kStateWarps + kOutWarps);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < kStateWarps) S.scales.top[0][tid] = kNothing;
    // the identity: 1 at (i, i)
    for (int i = tid; i < kTileBytes / 16; i += kChainThreads) {
        const int row = i >> 3, at = row & 7, hit = (i & 7) == (row >> 3);
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = hit && at / 2 == j ? (at & 1 ? 0x3F800000u : 0x3F80u) : 0u;
        *reinterpret_cast<uint4*>(S.eye + row * 128 + (((i & 7) ^ (row & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
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
        states<kSave>(P, S, span, nch, w, lane, sbase, h, tmem);
    } else if (w < kFirstKeys) {
        tc::registers_down<kOutRegs>();
        if (!kSave) outputs(P, S, span, nch, w, lane, h, tmem);
    } else if (w < kFirstQueries) {
        tc::registers_down<kKeyRegs>();
        if (nch > 0) keys(P, vmap, S, span, nch, h, tid - 32 * kFirstKeys);
        return;
    } else if (w < kMmaWarp) {
        if (!kSave && nch > 0) queries(P, S, span, nch, h, tid - 32 * kFirstQueries);
        return;
    } else {
        tc::registers_down<kMmaRegs>();
        if (w > kMmaWarp) {
            if (w == kScaleWarp) {
                if (nch > 0) scales<kSave>(P, S, span, nch, h, lane);
            } else {
                sizes(P, S, span, nch, w - kScaleWarp - 1, lane);
            }
            return;
        }
        if (nch > 0) issue<kSave>(P, S, nch, tmem);
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

// the tensor map of the values
inline cudaError_t values_map(const GdrChunked& P, CUtensorMap* map) {
    const long long rows = P.in.cu ? P.in.T : (long long)P.in.N * P.in.T;
    return rows > 0 ? encode_rows_map(map, P.in.v, (long long)P.in.Hv * kDim, rows, P.in.v_stride, kC) : cudaSuccess;
}

}  // namespace chain
}  // namespace gdr
}  // namespace kda

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
// Operands are fp16: S and X times 2^scale of the forward chain, dO (with `scale` folded in), dS and Y times 2^scale of the
// backward one (kda_gdr_chunk.cuh), a chunk and value head's sums times the product of both; sums are fp32.  dP and dB
// are products of two such operands, and are rounded to fp16 times a power of two of each 16 x 16 block's own where their size asks
// for one.  Gradients of queries and keys that a group of value heads shares are summed in registers by one CTA, in a
// fixed order, times the smallest 2^scale of the group's so far.
#include <algorithm>

#include "kda_gdr_chunk.cuh"

namespace kda {
namespace {

using namespace gdr;

// ---- chunk by chunk ---------------------------------------------------------------------------
// One CTA of 16 warps per (chunk, key head), which walks the group's value heads.  Warp w
// forms rows (tokens) 16 (w & 3) .. of dQ and dK for the key channels 32 (w >> 2) .., and
// the columns 16 (w >> 2) .. of the token-by-token products.  The CTAs, one per SM, walk the
// (chunk, key head) pairs with a stride; a head's tiles are fetched while the one before is worked on, each
// as soon as its place is free (without that, waiting for them took 40 % of the time).  With
// fewer pairs than SMs (kSplit), a cluster shares a pair's value heads and adds dQ and dK up,
// in the order of its CTAs (512 tokens x 8 heads on 4 key heads: 15 us, 25 without).
//
// Measured: 4,096 tokens x 32 heads 155 us, 11.5 us per head and SM; 60 % of the cycles move shared
// memory (operands of mma.sync, read again by every warp that needs them) and 0.40 of the issue
// slots are taken.
constexpr int kChunkThreads = 512, kParts = kChunkThreads / 128;

constexpr int kPairBytes = kBlockUsed - kTileBytes;   // of a block, from P on

struct ChunkSmem {
    __align__(128) unsigned char k[2][kC * kDim * 2];   // fp16, 256-byte rows; this pair's and the next one's
    __align__(128) unsigned char q[2][kC * kDim * 2];
    __align__(128) unsigned char o[kC * kDim * 2];   // dO, fp16, scaled
    __align__(128) unsigned char s[kStateTile];      // S^T (rows in units, as kept in memory)
    __align__(128) unsigned char ds[kStateTile];     // dS^T
    __align__(128) unsigned char x[kTokenTile];      // X^T
    __align__(128) unsigned char y[kTokenTile];      // Y^T
    __align__(128) unsigned char pg[2][(kPairBytes + 127) / 128 * 128];   // P, gates; this head's and the next one's
    __align__(128) unsigned char dp[kTileBytes], db[kTileBytes];
    float row[5][kParts][kC]; // sums over channels or columns, one slot per part
    float col[4][kC];         // column sums of dP . Q K^T + dB . K K^T, one slot per 16 rows
    float yv[kParts][kC];
    float dot[kChunkThreads / 32];
    int block[kChunkThreads / 32];   // exponents that blocks of dP and dB are held with, kEmpty without one
};
constexpr int kEmpty = 1000;

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

// 64 rows of 128 bf16 channels (zeros from row `rows` on) on their way to a tile, which the threads
// that fetched them then turn into fp16 in place, times `by`
__device__ __forceinline__ void fetch_rows(unsigned char* dst, const __nv_bfloat16* src, long long stride, int rows, int tid) {
#pragma unroll
    for (int i = 0; i < kC * 16 / kChunkThreads; ++i) {
        const int unit = tid & 15, row = (tid >> 4) + i * (kChunkThreads / 16);
        const bool there = row < rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n"
                     ::"r"(smem_u32(dst + row * 256 + ((unit ^ (row & 7)) << 4))), "l"(src + (there ? row * stride : 0) + unit * 8),
                       "r"(there ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ void rows_to_half(unsigned char* tile, float by, int tid) {
#pragma unroll
    for (int i = 0; i < kC * 16 / kChunkThreads; ++i) {
        const int unit = tid & 15, row = (tid >> 4) + i * (kChunkThreads / 16);
        uint4& u = *reinterpret_cast<uint4*>(tile + row * 256 + ((unit ^ (row & 7)) << 4));
        u = make_uint4(pack_half2(by * bf16_lo(u.x), by * bf16_hi(u.x)), pack_half2(by * bf16_lo(u.y), by * bf16_hi(u.y)),
                       pack_half2(by * bf16_lo(u.z), by * bf16_hi(u.z)), pack_half2(by * bf16_lo(u.w), by * bf16_hi(u.w)));
    }
}
__device__ __forceinline__ void copy_tile(unsigned char* dst, const unsigned char* src, int bytes, int tid) {
    for (int i = tid; i < bytes / 16; i += kChunkThreads) cp_async16(dst + 16 * i, src + 16 * i);
}

// `bytes` (a multiple of 16) from p on into L2
__device__ __forceinline__ void bulk_prefetch(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(p), "r"(bytes) : "memory");
}

// A (chunk, key head) pair of the grid's walk
struct Place {
    int chunk, hk, rows, n;
    long long tok;            // the chunk's first token
    bool from_zero;           // its state before is zero: a sequence's first chunk, without an initial state
};
__device__ __forceinline__ bool place(const GdrChunked& P, int pair, Place& p) {
    const GdrInputs& I = P.in;
    if (pair >= P.chunks.total * I.Hk) return false;
    int c;
    p.chunk = pair / I.Hk;
    p.hk = pair % I.Hk;
    if (!find_chunk(I, P.chunks, p.chunk, p.n, c)) return false;     // nor are there any after it
    const Span span = span_of(I, P.chunks, p.n);
    p.tok = span.start + (long long)c * kC;
    p.rows = min(kC, span.len - c * kC);
    p.from_zero = c == 0 && !P.init_state;
    return true;
}

// four floats of another CTA of the cluster, at the same place
__device__ __forceinline__ float4 peer_float4(const float* p, int rank) {
    float4 x;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(smem_u32(p)), "r"(rank) : "memory");
    return x;
}

// an operand's fragment times `by` (a power of two)
__device__ __forceinline__ void times(uint32_t (&f)[4], __half2 by) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&f[i]), by);
        f[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
}

__device__ __forceinline__ void store_gate(void* p, int dtype, size_t i, float x) {
    if (dtype == KDA_F32) static_cast<float*>(p)[i] = x;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

template <bool kSplit>
__global__ void __launch_bounds__(kChunkThreads, 1) gdr_bwd_chunk_kernel(GdrBackward B, int split) {
    extern __shared__ __align__(128) unsigned char raw[];
    previous_done();
    ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(raw);
    const GdrChunked& P = B.fwd;
    const GdrInputs& I = P.in;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rw = w & 3, part = w >> 2, share = I.Hv / I.Hk;
    const uint32_t so = smem_u32(S.o), ss = smem_u32(S.s), sds = smem_u32(S.ds), sx = smem_u32(S.x), sy = smem_u32(S.y),
                   sdp = smem_u32(S.dp), sdb = smem_u32(S.db);
    const int i0 = 16 * rw + g, i1 = i0 + 8;               // this lane's rows
    // what the head's parts need, in the order in which their places become free
    const auto fetch_pair = [&](const Place& p, int to) {
        fetch_rows(S.k[to], I.k + p.tok * I.k_stride + p.hk * kDim, I.k_stride, p.rows, tid);
        fetch_rows(S.q[to], I.q + p.tok * I.q_stride + p.hk * kDim, I.q_stride, p.rows, tid);
    };
    const auto fetch_gates = [&](const Place& p, int h, int to) {
        copy_tile(S.pg[to], P.blocks + ((size_t)p.chunk * I.Hv + h) * kBlockBytes + kTileBytes, kPairBytes, tid);
    };
    const auto fetch_first = [&](const Place& p, int h) {
        const size_t at = (size_t)p.chunk * I.Hv + h;
        copy_tile(S.s, P.states + at * kStateTile, kStateTile, tid);
        copy_tile(S.y, B.ys + at * kTokenTile, kTokenTile, tid);
        fetch_rows(S.o, B.in.dout + (p.tok * I.Hv + h) * kDim, (long long)I.Hv * kDim, p.rows, tid);
    };
    const auto fetch_second = [&](const Place& p, int h) {
        const size_t at = (size_t)p.chunk * I.Hv + h;
        copy_tile(S.ds, B.dstates + at * kStateTile, kStateTile, tid);
        copy_tile(S.x, P.xs + at * kTokenTile, kTokenTile, tid);
    };
    // into L2, what is fetched later in this step
    const auto prefetch = [&](const Place& p, int h) {
        const size_t at = (size_t)p.chunk * I.Hv + h;
        if (tid < 128) {                       // dO and V: lines of 64 channels
            const int row = tid >> 1, ch = 64 * (tid & 1);
            if (row < p.rows) {
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(B.in.dout + ((p.tok + row) * I.Hv + h) * kDim + ch));
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(I.v + (p.tok + row) * I.v_stride + h * kDim + ch));
            }
        } else if (tid == 128) {
            bulk_prefetch(P.states + at * kStateTile, kStateTile);
            bulk_prefetch(B.ys + at * kTokenTile, kTokenTile);
            bulk_prefetch(B.dstates + at * kStateTile, kStateTile);
            bulk_prefetch(P.xs + at * kTokenTile, kTokenTile);
        }
    };
    Place now, next;
    const int rank = kSplit ? (int)cluster_rank() : 0;
    int pair = kSplit ? blockIdx.x / split : blockIdx.x, turn = 0, kq = 0;
    if (!place(P, pair, now)) return;
    fetch_pair(now, 0);
    fetch_gates(now, now.hk * share + rank, 0);
    fetch_first(now, now.hk * share + rank);
    fetch_second(now, now.hk * share + rank);
    // the exponents of S and X, and of dO, dS and Y: fetched a head ahead
    const auto scales_of = [&](const Place& p, int h) {
        return *reinterpret_cast<const int2*>(P.blocks + ((size_t)p.chunk * I.Hv + h) * kBlockBytes + 2 * kTileBytes + 4 * kGateScale);
    };
    int2 scales = scales_of(now, now.hk * share + rank);
    float dq[4][4], dk[4][4], kk[2][4];
    for (bool more = true; more; now = next, kq ^= 1) {
        pair += gridDim.x;
        more = !kSplit && place(P, pair, next);
        const int hk = now.hk, rows = now.rows;
        // blocks of 16 tokens that the chunk has; the warps of the others only keep their sums at zero
        const int blocks = (rows + 15) / 16;
        const bool mine = rw < blocks;
        const long long tok = now.tok;
        const uint32_t sk = smem_u32(S.k[kq]), sq = smem_u32(S.q[kq]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[j][e] = dk[j][e] = 0.0f;
        const int h0 = hk * share + rank, step = kSplit ? split : 1;
        int unit = 0;                          // dq and dk are held times 2^unit
        const auto lower_unit = [&](int to) {
            const float by = power_of_two(to - unit);
            unit = to;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dq[j][e] *= by;
                    dk[j][e] *= by;
                }
        };
        for (int h = h0; h < (hk + 1) * share; h += step, turn ^= 1) {
            const bool last = h + step >= (hk + 1) * share;
            const Place& then = last ? next : now;             // where the head after this one is
            const int then_h = last ? next.hk * share : h + step;
            const bool follows = !last || more;
            const unsigned char* pg = S.pg[turn];
            const float* gate = reinterpret_cast<const float*>(pg + kTileBytes);
            // values for Y.V: rows i0 and i1, a quarter of the channels
            uint32_t v[2][4];
            const __nv_bfloat16* vp = I.v + (tok + i0) * I.v_stride + h * kDim + 32 * part + 2 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    v[i][m] = (m & 1 ? i1 : i0) < rows ? __ldg(reinterpret_cast<const uint32_t*>(vp + (m & 1 ? 8 * I.v_stride : 0) + 16 * i + 8 * (m >> 1))) : 0u;
            const int held = scales.x + scales.y;
            const float by = I.scale * power_of_two(scales.y);
            if (h == h0) unit = held;
            else if (held < unit) lower_unit(held);
            const float f = power_of_two(unit - held);
            asm volatile("cp.async.wait_all;\n" ::: "memory");
            rows_to_half(S.o, by, tid);
            if (h == h0) {
                rows_to_half(S.k[kq], 1.0f, tid);
                rows_to_half(S.q[kq], 1.0f, tid);
            }
            __syncthreads();
            if (follows) {
                scales = scales_of(then, then_h);
                prefetch(then, then_h);
                fetch_gates(then, then_h, turn ^ 1);
                if (last) fetch_pair(next, kq ^ 1);
            }
            if (h == h0 && mine) { // K K^T, this warp's 16 rows and 16 columns
#pragma unroll
                for (int j = 0; j < 2; ++j) kk[j][0] = kk[j][1] = kk[j][2] = kk[j][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t a[4], b[4];
                    ldsm(a, a_addr<256>(sk, 16 * rw, 2 * ks, lane));
                    ldsm(b, b_addr<256>(sk, 16 * part, 2 * ks, lane));
                    mma_f16(kk[0], a, b[0], b[1]);
                    mma_f16(kk[1], a, b[2], b[3]);
                }
            }
            const float e0 = gate[kGateE + i0], e1 = gate[kGateE + i1];
            const float be0 = gate[kGateBe + i0], be1 = gate[kGateBe + i1];
            const float b0 = gate[kGateB + i0], b1 = gate[kGateB + i1];
            if (mine) {
                float yv0 = 0.0f, yv1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t fy[4];
                    ldsm_t(fy, row_b(sy, 32 * part + 16 * i, 2 * rw, lane));
#pragma unroll
                    for (int m = 0; m < 4; ++m) {              // rows i0, i1; channels 2 t (+ 8)
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&fy[m]));
                        (m & 1 ? yv1 : yv0) += y.x * bf16_lo(v[i][m]) + y.y * bf16_hi(v[i][m]);
                    }
                }
                yv0 = quad_sum(yv0);
                yv1 = quad_sum(yv1);
                if (t == 0) {
                    S.yv[part][i0] = yv0; S.yv[part][i1] = yv1;
                }
            } else {
                if (t == 0)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S.row[r][part][i0] = S.row[r][part][i1] = 0.0f;
                if (lane < 16) S.col[rw][16 * part + lane] = 0.0f;
                if (lane == 0) S.block[w] = kEmpty;
            }
            // <S, dS>: the diagonal of S^T dS, rows 16 (w / 2) .. over half of the key channels
            {
                float d[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t a[4], b[4];
                    ldsm(a, row_a(ss, 16 * (w >> 1), 8 * (w & 1) + 2 * ks, lane));
                    ldsm(b, row_b(sds, 16 * (w >> 1), 8 * (w & 1) + 2 * ks, lane));
                    mma_f16(d[0], a, b[0], b[1]);
                    mma_f16(d[1], a, b[2], b[3]);
                }
                // rows g (and g + 8), columns 2 t, 2 t + 1 (and the same + 8)
                float x = g == 2 * t ? d[0][0] + d[1][2] : g == 2 * t + 1 ? d[0][1] + d[1][3] : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                if (lane == 0) S.dot[w] = x;
            }
            if (mine) {
                // dO X^T and Y X^T: this warp's 16 rows, 16 columns
                float dp[2][4], da[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dp[j][e] = da[j][e] = 0.0f;
                if (part <= rw) {              // else columns past the rows
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        uint32_t fo[4], fy[4], b[4];
                        ldsm(fo, a_addr<256>(so, 16 * rw, 2 * ks, lane));
                        ldsm_t(fy, row_b(sy, 16 * ks, 2 * rw, lane));
                        ldsm_t(b, row_a(sx, 16 * ks, 2 * part, lane));
                        mma_f16(dp[0], fo, b[0], b[1]);
                        mma_f16(dp[1], fo, b[2], b[3]);
                        mma_f16(da[0], fy, b[0], b[1]);
                        mma_f16(da[1], fy, b[2], b[3]);
                    }
                }
                // dP, dB and the sums of dP . Q K^T + dB . K K^T (M . Q K^T is P)
                float pv[2][4], bv[2][4], top = 0.0f;
                float rs0 = 0.0f, rs1 = 0.0f, bs0 = 0.0f, bs1 = 0.0f;
                {
                    const float g0 = gate[kGateG + i0], g1 = gate[kGateG + i1];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int j = 16 * part + 8 * nt + 2 * t;
                        float cs[2] = {0.0f, 0.0f};
                        const float2 gj = *reinterpret_cast<const float2*>(gate + kGateG + j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = e < 2 ? i0 : i1, jj = j + (e & 1);
                            const float m = jj <= i ? ex2_approx((e < 2 ? g0 : g1) - (e & 1 ? gj.y : gj.x)) : 0.0f;
                            const float pq = __half2float(*reinterpret_cast<const __half*>(
                                pg + i * 128 + (((jj >> 3) ^ (i & 7)) << 4) + (jj & 7) * 2));
                            const float mk = jj < i ? m * kk[nt][e] : 0.0f;
                            const float dpv = dp[nt][e], dav = -da[nt][e], bi = e < 2 ? b0 : b1;
                            pv[nt][e] = jj <= i ? m * dpv : 0.0f;
                            bv[nt][e] = jj < i ? bi * m * dav : 0.0f;
                            top = fmaxf(top, fmaxf(fabsf(pv[nt][e]), fabsf(bv[nt][e])));
                            const float sum = (jj <= i ? dpv * pq : 0.0f) + bi * dav * mk;
                            cs[e & 1] += sum;
                            (e < 2 ? rs0 : rs1) += sum;
                            (e < 2 ? bs0 : bs1) += dav * mk;
                        }
                        cs[0] = rows_sum(cs[0]);
                        cs[1] = rows_sum(cs[1]);
                        if (g == 0) {
                            S.col[rw][j] = cs[0];
                            S.col[rw][j + 1] = cs[1];
                        }
                    }
                    rs0 = quad_sum(rs0); rs1 = quad_sum(rs1); bs0 = quad_sum(bs0); bs1 = quad_sum(bs1);
                    if (t == 0) {
                        S.row[3][part][i0] = rs0; S.row[3][part][i1] = rs1;
                        S.row[4][part][i0] = bs0; S.row[4][part][i1] = bs1;
                    }
                }
                const int e = exponent_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top))));
                const int own = next_scale(0, e, -8, 14, 8);
                if (lane == 0) S.block[w] = e == kNothing ? kEmpty : own;
                if (own) {
                    const float up = power_of_two(own);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        pv[j >> 2][j & 3] *= up;
                        bv[j >> 2][j & 3] *= up;
                    }
                }
                stsm(a_addr<128>(sdp, 16 * rw, 2 * part, lane), pack_half2(pv[0][0], pv[0][1]), pack_half2(pv[0][2], pv[0][3]),
                     pack_half2(pv[1][0], pv[1][1]), pack_half2(pv[1][2], pv[1][3]));
                stsm(a_addr<128>(sdb, 16 * rw, 2 * part, lane), pack_half2(bv[0][0], bv[0][1]), pack_half2(bv[0][2], bv[0][3]),
                     pack_half2(bv[1][0], bv[1][1]), pack_half2(bv[1][2], bv[1][3]));
            }
            // dO S^T and Y S^T: this warp's rows, 32 key channels, over 128 value channels
            if (mine) {
                float a[4][4], z[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[j][e] = z[j][e] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t fo[4], fy[4];
                    ldsm(fo, a_addr<256>(so, 16 * rw, 2 * ks, lane));
                    ldsm_t(fy, row_b(sy, 16 * ks, 2 * rw, lane));   // Y as an A operand from Y^T
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t b[4];
                        ldsm_t(b, row_a(ss, 16 * ks, 4 * part + 2 * np, lane));
                        mma_f16(a[2 * np], fo, b[0], b[1]);
                        mma_f16(a[2 * np + 1], fo, b[2], b[3]);
                        mma_f16(z[2 * np], fy, b[0], b[1]);
                        mma_f16(z[2 * np + 1], fy, b[2], b[3]);
                    }
                }
                const float fb0 = f * be0, fb1 = f * be1;
                float qa0 = 0.0f, qa1 = 0.0f, kz0 = 0.0f, kz1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ch = 32 * part + 8 * j + 2 * t;
                    const float2 q0 = half2_at(S.q[kq], i0, ch), q1 = half2_at(S.q[kq], i1, ch);
                    const float2 k0 = half2_at(S.k[kq], i0, ch), k1 = half2_at(S.k[kq], i1, ch);
                    a[j][0] *= e0; a[j][1] *= e0; a[j][2] *= e1; a[j][3] *= e1;
                    qa0 += q0.x * a[j][0] + q0.y * a[j][1];
                    qa1 += q1.x * a[j][2] + q1.y * a[j][3];
                    kz0 += k0.x * z[j][0] + k0.y * z[j][1];
                    kz1 += k1.x * z[j][2] + k1.y * z[j][3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dq[j][e] = fmaf(f, a[j][e], dq[j][e]);
                        dk[j][e] = fmaf(-(e < 2 ? fb0 : fb1), z[j][e], dk[j][e]);
                    }
                }
                qa0 = quad_sum(qa0); qa1 = quad_sum(qa1); kz0 = quad_sum(kz0); kz1 = quad_sum(kz1);
                if (t == 0) {
                    S.row[0][part][i0] = qa0; S.row[0][part][i1] = qa1;
                    S.row[1][part][i0] = kz0; S.row[1][part][i1] = kz1;
                }
            }
            __syncthreads();               // dP and dB are there; S, Y and dO have been read
            if (follows) fetch_first(then, then_h);
            // X dS^T
            if (mine) {
                float a[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j][0] = a[j][1] = a[j][2] = a[j][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t fx[4];
                    ldsm_t(fx, row_b(sx, 16 * ks, 2 * rw, lane));
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t b[4];
                        ldsm_t(b, row_a(sds, 16 * ks, 4 * part + 2 * np, lane));
                        mma_f16(a[2 * np], fx, b[0], b[1]);
                        mma_f16(a[2 * np + 1], fx, b[2], b[3]);
                    }
                }
                const float f0 = gate[kGateEnd + i0], f1 = gate[kGateEnd + i1];
                float ka0 = 0.0f, ka1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ch = 32 * part + 8 * j + 2 * t;
                    const float2 k0 = half2_at(S.k[kq], i0, ch), k1 = half2_at(S.k[kq], i1, ch);
                    a[j][0] *= f0; a[j][1] *= f0; a[j][2] *= f1; a[j][3] *= f1;
                    ka0 += k0.x * a[j][0] + k0.y * a[j][1];
                    ka1 += k1.x * a[j][2] + k1.y * a[j][3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) dk[j][e] = fmaf(f, a[j][e], dk[j][e]);
                }
                ka0 = quad_sum(ka0); ka1 = quad_sum(ka1);
                if (t == 0) {
                    S.row[2][part][i0] = ka0; S.row[2][part][i1] = ka1;
                }
            }
            __syncthreads();               // dS and X have been read, all sums are there
            if (follows) fetch_second(then, then_h);
            // dQ += dP K, dK += dP^T Q + dB K + dB^T K, with all blocks brought to the sums' exponent
            const int block = lane < kChunkThreads / 32 ? S.block[lane] : kEmpty;
            const int least = __reduce_min_sync(0xFFFFFFFFu, block);
            if (least != kEmpty && held + least < unit) lower_unit(held + least);
            const int move = block == kEmpty ? 0 : max(unit - held - block, -40);      // at most 0
            const bool moves = __any_sync(0xFFFFFFFFu, move != 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (!mine || ks >= blocks) break;
                uint32_t fpn[4], fbn[4], fpt[4], fbt[4];
                if (ks <= rw) {            // rows reach tokens up to their own
                    ldsm(fpn, a_addr<128>(sdp, 16 * rw, 2 * ks, lane));
                    ldsm(fbn, a_addr<128>(sdb, 16 * rw, 2 * ks, lane));
                }
                if (ks >= rw) {            // transposed: from their own on
                    ldsm_t(fpt, b_addr<128>(sdp, 16 * ks, 2 * rw, lane));
                    ldsm_t(fbt, b_addr<128>(sdb, 16 * ks, 2 * rw, lane));
                }
                if (moves) {
                    const __half2 n = __float2half2_rn(power_of_two(__shfl_sync(0xFFFFFFFFu, move, rw + 4 * ks)));
                    const __half2 r = __float2half2_rn(power_of_two(__shfl_sync(0xFFFFFFFFu, move, ks + 4 * rw)));
                    if (ks <= rw) {
                        times(fpn, n);
                        times(fbn, n);
                    }
                    if (ks >= rw) {
                        times(fpt, r);
                        times(fbt, r);
                    }
                }
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    uint32_t b[4];
                    ldsm_t(b, a_addr<256>(sk, 16 * ks, 4 * part + 2 * np, lane));
                    if (ks <= rw) {
                        mma_f16(dq[2 * np], fpn, b[0], b[1]);
                        mma_f16(dq[2 * np + 1], fpn, b[2], b[3]);
                        mma_f16(dk[2 * np], fbn, b[0], b[1]);
                        mma_f16(dk[2 * np + 1], fbn, b[2], b[3]);
                    }
                    if (ks >= rw) {
                        mma_f16(dk[2 * np], fbt, b[0], b[1]);
                        mma_f16(dk[2 * np + 1], fbt, b[2], b[3]);
                        ldsm_t(b, a_addr<256>(sq, 16 * ks, 4 * part + 2 * np, lane));
                        mma_f16(dk[2 * np], fpt, b[0], b[1]);
                        mma_f16(dk[2 * np + 1], fpt, b[2], b[3]);
                    }
                }
            }
            // gates: two tokens per lane of one warp
            if (w == 0) {
                const int es = reinterpret_cast<const int*>(gate)[kGateScale], eg = reinterpret_cast<const int*>(gate)[kGateGradScale];
                float dgv[2], ka[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int j = 2 * lane + m;
                    const auto parts = [&](const float (&x)[kParts][kC]) { return (x[0][j] + x[1][j]) + (x[2][j] + x[3][j]); };
                    const float qa = parts(S.row[0]), kz = parts(S.row[1]), rs = parts(S.row[3]), bs = parts(S.row[4]), yv = parts(S.yv);
                    ka[m] = parts(S.row[2]);
                    const float cs = S.col[0][j] + S.col[1][j] + S.col[2][j] + S.col[3][j];
                    dgv[m] = qa - ka[m] - gate[kGateBe + j] * kz + rs - cs;
                    if (j < rows)
                        store_gate(B.dbeta, I.gate_dtype, (size_t)(tok + j) * I.Hv + h,
                                   power_of_two(-eg) * (yv + power_of_two(-es) * (bs - gate[kGateE + j] * kz)));
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
                if (now.from_zero && lane == 0) x = 0.0f;      // the first token has nothing to forget: else sums that cancel
                if (2 * lane < rows) store_gate(B.dg, I.gate_dtype, (size_t)(tok + 2 * lane) * I.Hv + h, times_power(x, -held));
                if (2 * lane + 1 < rows)
                    store_gate(B.dg, I.gate_dtype, (size_t)(tok + 2 * lane + 1) * I.Hv + h, times_power(x - dgv[0], -held));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dq[j][e] = times_power(dq[j][e], -unit);
                dk[j][e] = times_power(dk[j][e], -unit);
            }
        if constexpr (kSplit) {            // in place of S and dS: fp32 rows, 8-channel groups turned by the row
            float* mine[2] = {reinterpret_cast<float*>(S.s), reinterpret_cast<float*>(S.ds)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int ch = 32 * part + 8 * j + 2 * t;
                const int at0 = i0 * kDim + (ch ^ (8 * (i0 & 7))), at1 = i1 * kDim + (ch ^ (8 * (i1 & 7)));
                *reinterpret_cast<float2*>(mine[0] + at0) = make_float2(dq[j][0], dq[j][1]);
                *reinterpret_cast<float2*>(mine[0] + at1) = make_float2(dq[j][2], dq[j][3]);
                *reinterpret_cast<float2*>(mine[1] + at0) = make_float2(dk[j][0], dk[j][1]);
                *reinterpret_cast<float2*>(mine[1] + at1) = make_float2(dk[j][2], dk[j][3]);
            }
            cluster_arrive();
            cluster_wait();
            // four channels of a row at a time, the rows between the CTAs
            for (int i = rank * kChunkThreads + tid; i < 2 * kC * (kDim / 4); i += split * kChunkThreads) {
                const int side = i / (kC * (kDim / 4)), row = i / (kDim / 4) % kC, ch = i % (kDim / 4) * 4;
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int r = 0; r < split; ++r) {
                    const float4 x = peer_float4(mine[side] + row * kDim + (ch ^ (8 * (row & 7))), r);
                    sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
                }
                if (row < rows)
                    *reinterpret_cast<uint2*>((side ? B.dk : B.dq) + ((size_t)(tok + row) * I.Hk + hk) * kDim + ch) =
                        make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
            }
            cluster_arrive();                  // until then the others read this CTA's part
            cluster_wait();
        } else {                               // dQ and dK as bf16 rows
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int ch = 32 * part + 8 * j + 2 * t;
                if (i0 < rows) {
                    const size_t o = ((size_t)(tok + i0) * I.Hk + hk) * kDim + ch;
                    *reinterpret_cast<uint32_t*>(B.dq + o) = pack_bf16(dq[j][0], dq[j][1]);
                    *reinterpret_cast<uint32_t*>(B.dk + o) = pack_bf16(dk[j][0], dk[j][1]);
                }
                if (i1 < rows) {
                    const size_t o = ((size_t)(tok + i1) * I.Hk + hk) * kDim + ch;
                    *reinterpret_cast<uint32_t*>(B.dq + o) = pack_bf16(dq[j][2], dq[j][3]);
                    *reinterpret_cast<uint32_t*>(B.dk + o) = pack_bf16(dk[j][2], dk[j][3]);
                }
            }
        }
    }
}

}  // namespace

int gdr_bwd_chunk_split(const GdrBackward& B, int sms) {
    const long long pairs = (long long)B.fwd.chunks.total * B.fwd.in.Hk;
    const int share = B.fwd.in.Hv / B.fwd.in.Hk;
    int split = 1;                         // at most 8 CTAs, as many as there are heads and SMs for
    while (split < 8 && 2 * split <= share && pairs * 2 * split <= sms) split *= 2;
    return split;
}

cudaError_t launch_gdr_bwd_chunk(const GdrBackward& B, int split, int sms, cudaStream_t s) {
    if (B.fwd.chunks.total == 0) return cudaSuccess;
    const long long pairs = (long long)B.fwd.chunks.total * B.fwd.in.Hk;
    if (split > 1) {
        const cudaError_t e = allow_smem<gdr_bwd_chunk_kernel<true>>(sizeof(ChunkSmem));
        if (e != cudaSuccess) return e;
        return launch_clusters(gdr_bwd_chunk_kernel<true>, (unsigned)(pairs * split), kChunkThreads, sizeof(ChunkSmem),
                               (unsigned)split, s, B, split);
    }
    const cudaError_t e = allow_smem<gdr_bwd_chunk_kernel<false>>(sizeof(ChunkSmem));
    if (e != cudaSuccess) return e;
    return launch_after(true, gdr_bwd_chunk_kernel<false>, dim3((unsigned)std::min<long long>(pairs, sms)), kChunkThreads, sizeof(ChunkSmem), s, B, 1);
}

}  // namespace kda

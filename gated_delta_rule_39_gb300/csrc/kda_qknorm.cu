// Norms of queries and keys for each head, with the position rotation in the same pass,
// and their backward pass.
//
//   forward   r = 1 / sqrt(c sum_i x_i^2 + eps),  c = 1 (l2) or 1 / D (rms)
//             y = w x r,  z = y with the pairs of its first rotary_dim channels turned by
//             the token's angles:  z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin
//   backward  dy = dz turned back,  du = w dy,
//             dx = r (du - x c r^2 sum_i x_i du_i),  dw = sum over rows of dy x r
//
// Both are bound by memory: a row is read once (twice in the backward pass: x and dz) and
// written once, and everything in between stays in registers.  A row of D channels is
// held by a group of lanes; a lane owns "slots" of two times VEC channels arranged so that
// both members of every rotation pair are its own: with halves as pairs, VEC channels
// from the first half and their partners from the second (two 16-byte accesses); with
// neighbours as pairs, 2 VEC consecutive channels.  So the rotation needs no exchange
// between lanes and the sums over a row are a butterfly over its group.  Sums, the norm,
// the rotation and the products are fp32; the result is rounded once, on the store.
#include <algorithm>
#include <cmath>

#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxDim = 512;

struct NormSide {             // the queries' part of a call, or the keys'
    const void* x;
    const void* dz;           // backward: dL/dz, contiguous rows
    void* y;                  // z, or dL/dx (contiguous rows)
    const float* w;           // [D] or nullptr
    float* dw_part;           // backward: [blocks][D] partial sums, or nullptr
    long long stride;         // elements from one token of x to the next
    int heads;
};

struct NormProblem {
    NormSide side[2];
    const float* cos;         // [rows][half], nullptr: no rotation
    const float* sin;
    const int* pos;           // [T] or nullptr (token t uses row t)
    int T, D, half, inter, rows, lanes;   // lanes: group of lanes per row (a power of two)
    float c, eps;
    int* err;
};

// VEC elements at p as floats
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(p[i]);
    }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 u = *reinterpret_cast<const float4*>(p + 4 * i);
            v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = p[i];
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = __float2bfloat16_rn(v[i]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            *reinterpret_cast<float4*>(p + 4 * i) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = v[i];
    }
}

// First channels of a slot's two units of VEC channels.
template <int VEC>
__device__ __forceinline__ void slot_channels(int slot, int half, int inter, int& u0, int& u1) {
    const int first = slot * VEC;
    if (!inter && first < half) {          // a unit of the first half and its partners
        u0 = first;
        u1 = half + first;
    } else {                               // 2 VEC consecutive channels
        u0 = 2 * first;
        u1 = 2 * first + VEC;
    }
}
// A slot's channels in a row: pair i is (a[i], b[i]) when the slot is rotated.
template <int VEC, typename T>
__device__ __forceinline__ void load_slot(const T* row, int slot, int half, int inter,
                                          float (&a)[VEC], float (&b)[VEC]) {
    int u0, u1;
    slot_channels<VEC>(slot, half, inter, u0, u1);
    float e0[VEC], e1[VEC];
    load_vec<VEC>(row + u0, e0);
    load_vec<VEC>(row + u1, e1);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (VEC > 1 && inter) {
            a[i] = 2 * i < VEC ? e0[(2 * i) % VEC] : e1[(2 * i) % VEC];
            b[i] = 2 * i + 1 < VEC ? e0[(2 * i + 1) % VEC] : e1[(2 * i + 1) % VEC];
        } else {
            a[i] = e0[i];
            b[i] = e1[i];
        }
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_slot(T* row, int slot, int half, int inter,
                                           const float (&a)[VEC], const float (&b)[VEC]) {
    int u0, u1;
    slot_channels<VEC>(slot, half, inter, u0, u1);
    float e0[VEC], e1[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (VEC > 1 && inter) {
            e0[i] = i % 2 ? b[i / 2] : a[i / 2];
            e1[i] = i % 2 ? b[(VEC + i) / 2] : a[(VEC + i) / 2];
        } else {
            e0[i] = a[i];
            e1[i] = b[i];
        }
    }
    store_vec<VEC>(row + u0, e0);
    store_vec<VEC>(row + u1, e1);
}

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// The angles of a slot at a token (1, 0 where it is not rotated); false: bad position.
template <int VEC>
__device__ __forceinline__ bool load_angles(const NormProblem& P, int t, int slot, float (&cs)[VEC],
                                            float (&sn)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
    }
    if (!P.cos) return true;
    const int p = P.pos ? P.pos[t] : t;
    if (p < 0 || p >= P.rows) return false;
    if (slot * VEC < P.half) {
        const size_t at = (size_t)p * P.half + slot * VEC;
        load_vec<VEC>(P.cos + at, cs);
        load_vec<VEC>(P.sin + at, sn);
    }
    return true;
}

// One group of P.lanes lanes per row (token, head); NS slots per lane.  The rows of the
// queries come first, then the keys'.
template <typename T, int VEC, int NS>
__global__ void __launch_bounds__(kNormThreads) qk_norm_kernel(NormProblem P) {
    const int per_warp = 32 / P.lanes;
    const int lane = threadIdx.x & 31, li = lane % P.lanes;
    const long long warp = (long long)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
    long long row = warp * per_warp + lane / P.lanes;
    const long long nq = (long long)P.T * P.side[0].heads;
    const long long total = nq + (long long)P.T * P.side[1].heads;
    const bool there = row < total;
    if (!there) row = total - 1;           // keeps the lane in the butterflies
    const int w = row >= nq;
    const NormSide& S = P.side[w];
    if (w) row -= nq;
    const int t = (int)(row / S.heads), h = (int)(row % S.heads);
    const T* x = static_cast<const T*>(S.x) + t * S.stride + (long long)h * P.D;
    const int slots = P.D / (2 * VEC);
    float a[NS][VEC], b[NS][VEC], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int slot = li + j * P.lanes;
        if (slot < slots) {
            load_slot<VEC>(x, slot, P.half, P.inter, a[j], b[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum += a[j][i] * a[j][i] + b[j][i] * b[j][i];
        }
    }
    const float r = 1.0f / sqrtf(P.c * group_sum(sum, P.lanes) + P.eps);
    T* z = static_cast<T*>(S.y) + row * P.D;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int slot = li + j * P.lanes;
        if (slot >= slots || !there) continue;
        float cs[VEC], sn[VEC], wa[VEC], wb[VEC];
        if (!load_angles<VEC>(P, t, slot, cs, sn)) {
            set_error(P.err, KDA_ERR_BAD_INDEX);
            continue;
        }
        if (S.w) load_slot<VEC>(S.w, slot, P.half, P.inter, wa, wb);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float ya = a[j][i] * r * (S.w ? wa[i] : 1.0f), yb = b[j][i] * r * (S.w ? wb[i] : 1.0f);
            a[j][i] = ya * cs[i] - yb * sn[i];
            b[j][i] = yb * cs[i] + ya * sn[i];
        }
        store_slot<VEC>(z, slot, P.half, P.inter, a[j], b[j]);
    }
}

// Backward: blockIdx.y picks the queries or the keys, whose rows the grid's groups walk
// with a stride; each lane sums its channels of dw over its rows, and the block writes one
// partial row of D sums (in a fixed order: results do not depend on scheduling).
template <typename T, int VEC, int NS>
__global__ void __launch_bounds__(kNormThreads) qk_norm_bwd_kernel(NormProblem P) {
    __shared__ __align__(16) float part[kNormThreads / 32][kNormMaxDim];
    const NormSide& S = P.side[blockIdx.y];
    const int per_warp = 32 / P.lanes;
    const int lane = threadIdx.x & 31, li = lane % P.lanes, wid = threadIdx.x >> 5;
    const long long groups = (long long)gridDim.x * (kNormThreads / 32) * per_warp;
    const long long rows = (long long)P.T * S.heads;
    const int slots = P.D / (2 * VEC);
    float wa[NS][VEC], wb[NS][VEC], ga[NS][VEC], gb[NS][VEC];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            wa[j][i] = wb[j][i] = 1.0f;
            ga[j][i] = gb[j][i] = 0.0f;
        }
        const int slot = li + j * P.lanes;
        if (S.w && slot < slots) load_slot<VEC>(S.w, slot, P.half, P.inter, wa[j], wb[j]);
    }
    // whole warps leave the loop together: a warp's first row decides
    for (long long first = ((long long)blockIdx.x * (kNormThreads / 32) + wid) * per_warp; first < rows;
         first += groups) {
        long long row = first + lane / P.lanes;
        const bool there = row < rows;
        if (!there) row = rows - 1;
        const int t = (int)(row / S.heads), h = (int)(row % S.heads);
        const T* x = static_cast<const T*>(S.x) + t * S.stride + (long long)h * P.D;
        const T* dz = static_cast<const T*>(S.dz) + row * P.D;
        float a[NS][VEC], b[NS][VEC], da[NS][VEC], db[NS][VEC], sum = 0.0f, dot = 0.0f;
        bool good = there;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int slot = li + j * P.lanes;
            if (slot >= slots) continue;
            load_slot<VEC>(x, slot, P.half, P.inter, a[j], b[j]);
            load_slot<VEC>(dz, slot, P.half, P.inter, da[j], db[j]);
            float cs[VEC], sn[VEC];
            if (!load_angles<VEC>(P, t, slot, cs, sn)) {
                if (there) set_error(P.err, KDA_ERR_BAD_INDEX);
                good = false;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float ya = da[j][i] * cs[i] + db[j][i] * sn[i];
                db[j][i] = db[j][i] * cs[i] - da[j][i] * sn[i];
                da[j][i] = ya;
                sum += a[j][i] * a[j][i] + b[j][i] * b[j][i];
                dot += a[j][i] * (wa[j][i] * da[j][i]) + b[j][i] * (wb[j][i] * db[j][i]);
            }
        }
        const float r = 1.0f / sqrtf(P.c * group_sum(sum, P.lanes) + P.eps);
        const float m = P.c * r * r * group_sum(dot, P.lanes);
        if (!good) continue;
        T* dx = static_cast<T*>(S.y) + row * P.D;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int slot = li + j * P.lanes;
            if (slot >= slots) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ga[j][i] += da[j][i] * (a[j][i] * r);
                gb[j][i] += db[j][i] * (b[j][i] * r);
                a[j][i] = r * (wa[j][i] * da[j][i] - a[j][i] * m);
                b[j][i] = r * (wb[j][i] * db[j][i] - b[j][i] * m);
            }
            store_slot<VEC>(dx, slot, P.half, P.inter, a[j], b[j]);
        }
    }
    if (!S.dw_part) return;
    // groups of a warp, then the block's warps
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            for (int o = P.lanes; o < 32; o <<= 1) {
                ga[j][i] += __shfl_xor_sync(0xFFFFFFFFu, ga[j][i], o);
                gb[j][i] += __shfl_xor_sync(0xFFFFFFFFu, gb[j][i], o);
            }
    if (lane < P.lanes) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int slot = li + j * P.lanes;
            if (slot < slots) store_slot<VEC>(part[wid], slot, P.half, P.inter, ga[j], gb[j]);
        }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < P.D; ch += kNormThreads) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kNormThreads / 32; ++i) s += part[i][ch];
        S.dw_part[(size_t)blockIdx.x * P.D + ch] = s;
    }
}

// dw[ch] = sum over blocks of part[block][ch]; one block of 8 warps per 32 channels
__global__ void __launch_bounds__(256) qk_norm_dw_kernel(const float* part0, const float* part1, float* dw0,
                                                         float* dw1, int blocks, int D) {
    __shared__ float s[8][33];
    const float* part = blockIdx.y ? part1 : part0;
    float* dw = blockIdx.y ? dw1 : dw0;
    if (!dw) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, ch = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (ch < D)
        for (int i = w; i < blocks; i += 8) sum += part[(size_t)i * D + ch];
    s[w][lane] = sum;
    __syncthreads();
    if (w == 0 && ch < D) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += s[i][lane];
        dw[ch] = sum;
    }
}

// Calls f<T, VEC, NS>() for the widest access that the problem's sizes, strides and
// addresses allow: 16 bytes, or single elements.
template <class F>
cudaError_t with_width(const NormProblem& P, int dtype, bool wide, F&& f) {
    const int vec = !wide ? 1 : dtype == KDA_BF16 ? 8 : 4;
    const int slots = P.D / (2 * vec);
    if (dtype == KDA_BF16) {
        if (wide) return f.template operator()<__nv_bfloat16, 8, 1>(slots);
        return f.template operator()<__nv_bfloat16, 1, 8>(slots);
    }
    if (wide) return f.template operator()<float, 4, 2>(slots);
    return f.template operator()<float, 1, 8>(slots);
}

bool wide_ok(const NormProblem& P, int dtype) {
    const int vec = dtype == KDA_BF16 ? 8 : 4;
    if (P.D % (2 * vec) || P.half % vec) return false;
    for (const NormSide& S : P.side) {
        if (!S.heads) continue;
        if (S.stride % vec) return false;
        for (const void* p : {S.x, S.dz, static_cast<const void*>(S.y), static_cast<const void*>(S.w)})
            if (!aligned16(p)) return false;
    }
    return aligned16(P.cos) && aligned16(P.sin);
}

int group_lanes(int slots) {
    int lanes = 1;
    while (lanes < slots && lanes < 32) lanes *= 2;
    return lanes;
}

struct LaunchFwd {
    NormProblem P;
    cudaStream_t s;
    template <typename T, int VEC, int NS>
    cudaError_t operator()(int slots) {
        P.lanes = group_lanes(slots);
        const long long rows = (long long)P.T * (P.side[0].heads + P.side[1].heads);
        const long long per_block = (long long)kNormThreads / P.lanes;
        qk_norm_kernel<T, VEC, NS><<<(unsigned)((rows + per_block - 1) / per_block), kNormThreads, 0, s>>>(P);
        return cudaGetLastError();
    }
};
struct LaunchBwd {
    NormProblem P;
    int blocks;
    cudaStream_t s;
    template <typename T, int VEC, int NS>
    cudaError_t operator()(int slots) {
        P.lanes = group_lanes(slots);
        const dim3 grid(blocks, P.side[1].heads ? 2 : 1);
        qk_norm_bwd_kernel<T, VEC, NS><<<grid, kNormThreads, 0, s>>>(P);
        return cudaGetLastError();
    }
};

// Host-side checks of both passes; no CUDA call.
int validate_norm(const void* q, const void* k, const void* yq, const void* yk, int dtype, int norm,
                  float eps, const float* qw, const float* kw, const float* cos, const float* sin,
                  const int32_t* pos, int table_rows, int rotary_dim, int T, int Hq, int Hk, int D,
                  long long q_stride, long long k_stride) {
    if (D < 2 || D > kNormMaxDim || D % 2) return KDA_ERR_UNSUPPORTED_DIM;
    if (T < 0 || Hq < 1 || Hk < 0 || Hq > 65536 || Hk > 65536) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (norm != KDA_NORM_L2 && norm != KDA_NORM_RMS) return KDA_ERR_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return KDA_ERR_ARG;
    if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 2) return KDA_ERR_ARG;
    if (T > 0 && (!q || !yq || (Hk && (!k || !yk)))) return KDA_ERR_NULL;
    if (rotary_dim) {
        if (T > 0 && (!cos || !sin)) return KDA_ERR_NULL;
        if (table_rows < 0 || (!pos && table_rows < T)) return KDA_ERR_SHAPE;
    }
    if (q_stride < (long long)Hq * D || (Hk && k_stride < (long long)Hk * D)) return KDA_ERR_SHAPE;
    if ((long long)T * (Hq + Hk) >= (1LL << 32)) return KDA_ERR_SHAPE;
    const size_t size = dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {q, k, yq, yk})
        if (reinterpret_cast<uintptr_t>(p) % size) return KDA_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(qw), static_cast<const void*>(kw),
                          static_cast<const void*>(cos), static_cast<const void*>(sin),
                          static_cast<const void*>(pos)})
        if (reinterpret_cast<uintptr_t>(p) % 4) return KDA_ERR_ALIGN;
    return KDA_OK;
}

// bytes from the first element of strided rows to the last
size_t span_bytes(int T, int H, int D, long long stride, size_t size) {
    return T ? ((size_t)(T - 1) * stride + (size_t)H * D) * size : 0;
}

NormProblem problem(const void* q, const void* k, int norm, float eps, const float* qw, const float* kw,
                    const float* cos, const float* sin, const int32_t* pos, int table_rows,
                    int rotary_dim, int interleaved, int T, int Hq, int Hk, int D, long long q_stride,
                    long long k_stride, int* err) {
    NormProblem P{};
    P.side[0].x = q;
    P.side[0].w = qw;
    P.side[0].stride = q_stride;
    P.side[0].heads = Hq;
    P.side[1].x = k;
    P.side[1].w = kw;
    P.side[1].stride = k_stride;
    P.side[1].heads = Hk;
    P.cos = rotary_dim ? cos : nullptr;
    P.sin = rotary_dim ? sin : nullptr;
    P.pos = pos;
    P.T = T;
    P.D = D;
    P.half = rotary_dim / 2;
    P.inter = interleaved != 0;
    P.rows = table_rows;
    P.c = norm == KDA_NORM_RMS ? 1.0f / (float)D : 1.0f;
    P.eps = eps;
    P.err = err;
    return P;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_qk_norm(const void* q, const void* k, void* q_out, void* k_out, int dtype, int norm, float eps,
                const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                const int32_t* positions, int table_rows, int rotary_dim, int interleaved, int T,
                int Hq, int Hk, int D, long long q_stride, long long k_stride, void* stream) {
    int rc = validate_norm(q, k, q_out, k_out, dtype, norm, eps, q_weight, k_weight, cos, sin, positions,
                           table_rows, rotary_dim, T, Hq, Hk, D, q_stride, k_stride);
    if (rc != KDA_OK) return rc;
    const size_t size = dtype == KDA_BF16 ? 2 : 4;
    const void* in_p[] = {q, k, q_weight, k_weight, cos, sin, positions};
    const size_t table = rotary_dim ? (size_t)table_rows * (rotary_dim / 2) * 4 : 0;
    const size_t in_n[] = {span_bytes(T, Hq, D, q_stride, size), span_bytes(T, Hk, D, k_stride, size),
                           (size_t)D * 4, (size_t)D * 4, table, table, (size_t)T * 4};
    const void* out_p[] = {q_out, k_out};
    const size_t out_n[] = {(size_t)T * Hq * D * size, (size_t)T * Hk * D * size};
    const long long strides[] = {q_stride, k_stride};
    const int heads[] = {Hq, Hk};
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 7; ++i) {
            // each row is read whole before it is written: in place on contiguous rows is fine
            if (i == o && out_p[o] == in_p[i] && strides[o] == (long long)heads[o] * D) continue;
            if (overlaps(out_p[o], out_n[o], in_p[i], in_n[i])) return KDA_ERR_ALIAS;
        }
    }
    if (overlaps(q_out, out_n[0], k_out, out_n[1])) return KDA_ERR_ALIAS;
    int dev = 0, sms = 0;
    int* err = nullptr;
    rc = device_setup(&dev, &err, &sms);
    if (rc != KDA_OK) return rc;
    if (T == 0) return KDA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchFwd L{problem(q, k, norm, eps, q_weight, k_weight, cos, sin, positions, table_rows, rotary_dim,
                        interleaved, T, Hq, Hk, D, q_stride, k_stride, err), s};
    L.P.side[0].y = q_out;
    L.P.side[1].y = k_out;
    const cudaError_t e = timed_launch(KDA_KERNEL_QK_NORM, s,
                                       [&] { return with_width(L.P, dtype, wide_ok(L.P, dtype), L); });
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

int kda_qk_norm_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq,
                    void* dk, int dtype, int norm, float eps, const float* q_weight,
                    const float* k_weight, float* dq_weight, float* dk_weight, const float* cos,
                    const float* sin, const int32_t* positions, int table_rows, int rotary_dim,
                    int interleaved, int T, int Hq, int Hk, int D, long long q_stride,
                    long long k_stride, void* stream) {
    int rc = validate_norm(q, k, dq, dk, dtype, norm, eps, q_weight, k_weight, cos, sin, positions,
                           table_rows, rotary_dim, T, Hq, Hk, D, q_stride, k_stride);
    if (rc != KDA_OK) return rc;
    if (T > 0 && (!dq_out || (Hk && !dk_out))) return KDA_ERR_NULL;
    if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
        return KDA_ERR_NULL;
    if (!Hk && dk_weight) return KDA_ERR_SHAPE;
    const size_t size = dtype == KDA_BF16 ? 2 : 4;
    for (const void* p : {dq_out, dk_out})
        if (reinterpret_cast<uintptr_t>(p) % size) return KDA_ERR_ALIGN;
    for (const float* p : {dq_weight, dk_weight})
        if (reinterpret_cast<uintptr_t>(p) % 4) return KDA_ERR_ALIGN;
    const size_t nq = (size_t)T * Hq * D * size, nk = (size_t)T * Hk * D * size;
    const size_t table = rotary_dim ? (size_t)table_rows * (rotary_dim / 2) * 4 : 0;
    const void* in_p[] = {q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions};
    const size_t in_n[] = {span_bytes(T, Hq, D, q_stride, size), span_bytes(T, Hk, D, k_stride, size),
                           nq, nk, (size_t)D * 4, (size_t)D * 4, table, table, (size_t)T * 4};
    const void* out_p[] = {dq, dk, dq_weight, dk_weight};
    const size_t out_n[] = {nq, nk, (size_t)D * 4, (size_t)D * 4};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 9; ++i)
            if (overlaps(out_p[o], out_n[o], in_p[i], in_n[i])) return KDA_ERR_ALIAS;
        for (int o2 = o + 1; o2 < 4; ++o2)
            if (overlaps(out_p[o], out_n[o], out_p[o2], out_n[o2])) return KDA_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    int* err = nullptr;
    rc = device_setup(&dev, &err, &sms);
    if (rc != KDA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (T == 0) {   // no rows: the weights' gradients are zero
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, (size_t)D * 4, s);
        if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, (size_t)D * 4, s);
        return e == cudaSuccess ? KDA_OK : cuda_fail(KDA_ERR_CUDA, e);
    }
    const long long per_block = kNormThreads / 16;   // rows of a block's first pass, or more
    const int blocks = (int)std::min<long long>(4LL * sms, ((long long)T * std::max(Hq, Hk) + per_block - 1) / per_block);
    LaunchBwd L{problem(q, k, norm, eps, q_weight, k_weight, cos, sin, positions, table_rows, rotary_dim,
                        interleaved, T, Hq, Hk, D, q_stride, k_stride, err), blocks, s};
    L.P.side[0].dz = dq_out;
    L.P.side[1].dz = dk_out;
    L.P.side[0].y = dq;
    L.P.side[1].y = dk;
    float* part = nullptr;
    if (dq_weight || dk_weight) {
        const cudaError_t ea = cudaMallocAsync(reinterpret_cast<void**>(&part), (size_t)2 * blocks * D * 4, s);
        if (ea != cudaSuccess) return cuda_fail(KDA_ERR_ALLOC, ea);
        if (dq_weight) L.P.side[0].dw_part = part;
        if (dk_weight) L.P.side[1].dw_part = part + (size_t)blocks * D;
    }
    e = timed_launch(KDA_KERNEL_QK_NORM_BWD, s,
                     [&] { return with_width(L.P, dtype, wide_ok(L.P, dtype), L); });
    if (part && e == cudaSuccess)
        e = timed_launch(KDA_KERNEL_QK_NORM_DW, s, [&] {
            qk_norm_dw_kernel<<<dim3((D + 31) / 32, 2), 256, 0, s>>>(part, part + (size_t)blocks * D,
                                                                     dq_weight, dk_weight, blocks, D);
            return cudaGetLastError();
        });
    if (part) cudaFreeAsync(part, s);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

}  // extern "C"

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
//
// Measured (GB300, copy bandwidth 6.78 TB/s): 8,192 tokens x 72 heads x 128 bf16 with weights
// and rotation 57 us, 5.3 TB/s, where issue slots (0.62 per cycle) begin to matter beside
// memory; the same backwards 100 us, 76 without either (6.0 TB/s); 16,384 x 64 heads backwards without
// either 121 us, 6.6 TB/s.  fp32, 8,192 x 72 x 128: 100 us, backwards 169 (142 without weights).
#include <algorithm>
#include <cmath>

#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kNormThreads = 256;
// Heads that a group of the forward pass holds at a time: as many as 128 registers have room for.
__host__ __device__ constexpr int rows_at_once(int vec) { return vec > 1 ? 2 : 1; }
constexpr int kManyHeads = 8;             // of a token, at most, for a group that reads its angles once
// Blocks per SM, by the registers that a lane's part takes (vec x ns channels of each half of a row;
// angles, weights and the weights' gradients add as many each).  Forwards:
__host__ __device__ constexpr int fwd_per_sm(int vec, int ns) { return vec * ns <= 2 ? 3 : 2; }
// Backwards, three where 80 registers are enough (bf16, 16,384 x 64 heads without angles and weights 123
// us, with two blocks 141).  Even the 128 of two blocks are not enough where the weights' sums are largest: bf16 with
// weights and angles on 16-byte accesses spills 48 bytes, fp32 with weights and two slots 60 (with angles 190), single
// elements with eight slots 44 to 184 (8 with angles alone).
__host__ __device__ constexpr int bwd_per_sm(int vec, int ns, bool rot, bool w) {
    return vec * ns <= 2 || (vec * ns <= 4 && !w) || (vec == 8 && !rot && !w) ? 3 : 2;
}
constexpr int kNormMaxDim = 512;

struct NormSide {             // the queries' part of a call, or the keys'
    const void* x;
    const void* dz;           // backward: dL/dz, contiguous rows
    void* y;                  // z, or dL/dx (contiguous rows)
    const float* w;           // [D] or nullptr
    float* dw_part;           // backward: [blocks][D] partial sums, or nullptr
    float* dw;                // and their sums [D]
    long long stride;         // elements from one token of x to the next
    int heads;
    int blocks;               // backward: blocks that walk this side's rows
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
// A slot's channels as they are in memory: two units, read 16 bytes at a time at most (which is what
// wide_ok asks of every address: a unit of 8 fp32 weights begins on 16 bytes, not on 32).
template <typename T, int VEC>
struct __align__(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Unit {
    T v[VEC];
};
static_assert(alignof(Unit<float, 8>) == 16 && alignof(Unit<__nv_bfloat16, 8>) == 16 && alignof(Unit<float, 4>) == 16 &&
                  alignof(Unit<float, 1>) == 4 && alignof(Unit<__nv_bfloat16, 1>) == 2,
              "no access wider than the alignment that calls are checked for");
template <typename T, int VEC>
struct Raw {
    Unit<T, VEC> e0, e1;
};
template <int VEC, typename T>
__device__ __forceinline__ Raw<T, VEC> fetch_slot(const T* row, int slot, int half, int inter) {
    int u0, u1;
    slot_channels<VEC>(slot, half, inter, u0, u1);
    return {*reinterpret_cast<const Unit<T, VEC>*>(row + u0), *reinterpret_cast<const Unit<T, VEC>*>(row + u1)};
}
// A slot's channels: pair i is (a[i], b[i]) when the slot is rotated.
template <int VEC, typename T>
__device__ __forceinline__ void spread(const Raw<T, VEC>& r, int inter, float (&a)[VEC], float (&b)[VEC]) {
    float e0[VEC], e1[VEC];
    load_vec<VEC>(r.e0.v, e0);
    load_vec<VEC>(r.e1.v, e1);
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
__device__ __forceinline__ void load_slot(const T* row, int slot, int half, int inter, float (&a)[VEC], float (&b)[VEC]) {
    spread<VEC>(fetch_slot<VEC>(row, slot, half, inter), inter, a, b);
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

// An item is up to `hb` heads of a token, the work of one group of P.lanes lanes with NS slots per
// lane, so that angles and weights, in fp32 twice a bf16 row's bytes each, are read once for all
// of them.  The queries' items come first, then the keys'; groups walk them with a stride,
// R heads at a time with the next ones' rows on their way.
__host__ __device__ inline unsigned head_blocks(int heads, int hb) { return ((unsigned)heads + hb - 1) / hb; }

template <typename T, int VEC, int NS>
__global__ void __launch_bounds__(kNormThreads, fwd_per_sm(VEC, NS)) qk_norm_kernel(NormProblem P, int hb) {
    constexpr int R = rows_at_once(VEC);
    const unsigned per_warp = 32 / P.lanes;
    const int lane = threadIdx.x & 31, li = lane % P.lanes, slots = P.D / (2 * VEC);
    const unsigned nq = P.T * head_blocks(P.side[0].heads, hb), total = nq + P.T * head_blocks(P.side[1].heads, hb);
    const unsigned stride = gridDim.x * (kNormThreads / 32) * per_warp;
    struct Place {
        int w, t, h, left;                 // side, token, first head, heads
    };
    const auto place = [&](unsigned item) {
        if (item >= total) return Place{0, 0, 0, 0};
        const int w = item >= nq;
        if (w) item -= nq;
        const int heads = P.side[w].heads;
        const unsigned blocks = head_blocks(heads, hb);
        const int h = (int)(item % blocks) * hb;
        return Place{w, (int)(item / blocks), h, min(hb, heads - h)};
    };
    Raw<T, VEC> raw[R][NS] = {};
    const auto fetch = [&](const Place& p, int j) {
        const NormSide& S = P.side[p.w];
        const T* x = static_cast<const T*>(S.x) + p.t * S.stride + (long long)(p.h + j) * P.D;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (j + r < p.left && li + m * P.lanes < slots)
                    raw[r][m] = fetch_slot<VEC>(x + r * P.D, li + m * P.lanes, P.half, P.inter);
    };
    unsigned first = (blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5)) * per_warp;
    Place now = place(first + lane / P.lanes);
    fetch(now, 0);
    float wa[NS][VEC], wb[NS][VEC];
    int have = -1;                         // the side whose weights these are
    // whole warps walk together: a warp's first item decides
    while (first < total) {
        const Place next = place(first + stride + lane / P.lanes);
        const NormSide& S = P.side[now.w];
        float cs[NS][VEC], sn[NS][VEC];
        bool good = now.left > 0;
#pragma unroll
        for (int m = 0; m < NS; ++m) {
            const int slot = li + m * P.lanes;
            if (now.left && !load_angles<VEC>(P, now.t, slot, cs[m], sn[m])) {
                set_error(P.err, KDA_ERR_BAD_INDEX);
                good = false;
            }
            if (have != now.w) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) wa[m][i] = wb[m][i] = 1.0f;
                if (S.w && slot < slots) load_slot<VEC>(S.w, slot, P.half, P.inter, wa[m], wb[m]);
            }
        }
        have = now.w;
        T* z = static_cast<T*>(S.y) + ((long long)now.t * S.heads + now.h) * P.D;
#pragma unroll 1
        for (int j = 0; j < hb; j += R) {
            float a[R][NS][VEC], b[R][NS][VEC], sum[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sum[r] = 0.0f;
#pragma unroll
                for (int m = 0; m < NS; ++m) {     // slots past the row are zeros
                    spread<VEC>(raw[r][m], P.inter, a[r][m], b[r][m]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum[r] += a[r][m][i] * a[r][m][i] + b[r][m][i] * b[r][m][i];
                }
            }
            if (j + R < hb) fetch(now, j + R);
            else fetch(next, 0);
            for (int o = P.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < R; ++r) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!good || j + r >= now.left) continue;
                const float k = 1.0f / sqrtf(P.c * sum[r] + P.eps);
#pragma unroll
                for (int m = 0; m < NS; ++m) {
                    const int slot = li + m * P.lanes;
                    if (slot >= slots) continue;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float ya = a[r][m][i] * k * wa[m][i], yb = b[r][m][i] * k * wb[m][i];
                        a[r][m][i] = ya * cs[m][i] - yb * sn[m][i];
                        b[r][m][i] = yb * cs[m][i] + ya * sn[m][i];
                    }
                    store_slot<VEC>(z + (j + r) * P.D, slot, P.half, P.inter, a[r][m], b[r][m]);
                }
            }
        }
        now = next;
        first += stride;
    }
}

// Backward: the first blocks take the queries, the others the keys; a side's groups walk its items
// with a stride, a head at a time with the next head's row on its way.  Each lane sums its
// channels of dw over its rows, and the block writes one partial row of D sums (in a fixed order:
// results do not depend on scheduling).
template <typename T, int VEC, int NS, bool kRot, bool kW>
__global__ void __launch_bounds__(kNormThreads, bwd_per_sm(VEC, NS, kRot, kW)) qk_norm_bwd_kernel(NormProblem P, int hb) {
    __shared__ __align__(16) float part[kW ? kNormThreads / 32 : 1][kNormMaxDim];
    const int side = blockIdx.x >= P.side[0].blocks, block = blockIdx.x - (side ? P.side[0].blocks : 0);
    const NormSide& S = P.side[side];
    const int per_warp = 32 / P.lanes;
    const int lane = threadIdx.x & 31, li = lane % P.lanes, wid = threadIdx.x >> 5;
    const unsigned hblocks = head_blocks(S.heads, hb), items = P.T * hblocks;
    const unsigned stride = S.blocks * (kNormThreads / 32) * per_warp;
    const int slots = P.D / (2 * VEC);
    float wa[NS][VEC], wb[NS][VEC], ga[NS][VEC], gb[NS][VEC];
#pragma unroll
    for (int m = 0; m < NS; ++m) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            wa[m][i] = wb[m][i] = 1.0f;
            ga[m][i] = gb[m][i] = 0.0f;
        }
        const int slot = li + m * P.lanes;
        if (kW && S.w && slot < slots) load_slot<VEC>(S.w, slot, P.half, P.inter, wa[m], wb[m]);
    }
    Raw<T, VEC> rx[NS] = {}, rz[NS] = {};
    const auto fetch = [&](int t, int h) {
        const T* x = static_cast<const T*>(S.x) + t * S.stride + (long long)h * P.D;
        const T* dz = static_cast<const T*>(S.dz) + ((long long)t * S.heads + h) * P.D;
#pragma unroll
        for (int m = 0; m < NS; ++m)
            if (li + m * P.lanes < slots) {
                rx[m] = fetch_slot<VEC>(x, li + m * P.lanes, P.half, P.inter);
                rz[m] = fetch_slot<VEC>(dz, li + m * P.lanes, P.half, P.inter);
            }
    };
    // whole warps leave the loop together: a warp's first item decides, and the lanes of items past
    // the end repeat the last one without writing
    unsigned first = (block * (kNormThreads / 32) + wid) * per_warp;
    unsigned item = min(first + lane / P.lanes, items - 1);
    int t = (int)(item / hblocks), h = (int)(item % hblocks) * hb;
    if (first < items) fetch(t, h);
    while (first < items) {
        const bool there = first + lane / P.lanes < items;
        float cs[NS][VEC], sn[NS][VEC];
        bool good = there;
        if (kRot) {
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (!load_angles<VEC>(P, t, li + m * P.lanes, cs[m], sn[m])) {
                    if (there) set_error(P.err, KDA_ERR_BAD_INDEX);
                    good = false;
                }
        }
        // a warp's groups may have fewer heads left than others: all take hb turns
        const unsigned next = first + stride;
        const int t0 = t, h0 = h;
        if (next < items) {
            item = min(next + lane / P.lanes, items - 1);
            t = (int)(item / hblocks);
            h = (int)(item % hblocks) * hb;
        }
#pragma unroll 1
        for (int j = 0; j < hb; ++j) {
            const bool mine = good && h0 + j < S.heads;
            float a[NS][VEC], b[NS][VEC], da[NS][VEC], db[NS][VEC], sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                spread<VEC>(rx[m], P.inter, a[m], b[m]);
                spread<VEC>(rz[m], P.inter, da[m], db[m]);
            }
            if (j + 1 < hb) fetch(t0, min(h0 + j + 1, S.heads - 1));
            else if (next < items) fetch(t, h);
#pragma unroll
            for (int m = 0; m < NS; ++m) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (kRot) {
                        const float ya = da[m][i] * cs[m][i] + db[m][i] * sn[m][i];
                        db[m][i] = db[m][i] * cs[m][i] - da[m][i] * sn[m][i];
                        da[m][i] = ya;
                    }
                    sum += a[m][i] * a[m][i] + b[m][i] * b[m][i];
                    dot += a[m][i] * (wa[m][i] * da[m][i]) + b[m][i] * (wb[m][i] * db[m][i]);
                }
            }
            for (int o = P.lanes >> 1; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            }
            if (!mine) continue;
            const float r = 1.0f / sqrtf(P.c * sum + P.eps), k = P.c * r * r * dot;
            T* dx = static_cast<T*>(S.y) + ((long long)t0 * S.heads + h0 + j) * P.D;
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const int slot = li + m * P.lanes;
                if (slot >= slots) continue;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (kW) {
                        ga[m][i] += da[m][i] * (a[m][i] * r);
                        gb[m][i] += db[m][i] * (b[m][i] * r);
                    }
                    a[m][i] = r * (wa[m][i] * da[m][i] - a[m][i] * k);
                    b[m][i] = r * (wb[m][i] * db[m][i] - b[m][i] * k);
                }
                store_slot<VEC>(dx, slot, P.half, P.inter, a[m], b[m]);
            }
        }
        first = next;
    }
    if constexpr (kW) {
        if (!S.dw_part) return;
        // groups of a warp, then the block's warps
#pragma unroll
        for (int m = 0; m < NS; ++m)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int o = P.lanes; o < 32; o <<= 1) {
                    ga[m][i] += __shfl_xor_sync(0xFFFFFFFFu, ga[m][i], o);
                    gb[m][i] += __shfl_xor_sync(0xFFFFFFFFu, gb[m][i], o);
                }
        if (lane < P.lanes) {
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const int slot = li + m * P.lanes;
                if (slot < slots) store_slot<VEC>(part[wid], slot, P.half, P.inter, ga[m], gb[m]);
            }
        }
        __syncthreads();
        for (int ch = threadIdx.x; ch < P.D; ch += kNormThreads) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kNormThreads / 32; ++i) s += part[i][ch];
            S.dw_part[(size_t)block * P.D + ch] = s;
        }
    }
}

// dw[ch] = sum over blocks of part[block][ch]; one block of 32 warps per side and 32 channels
constexpr int kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads) qk_norm_dw_kernel(NormProblem P) {
    __shared__ float s[kDwThreads / 32][33];
    const NormSide& S = P.side[blockIdx.y];
    if (!S.dw_part) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, ch = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (ch < P.D)
#pragma unroll 8
        for (int i = w; i < S.blocks; i += kDwThreads / 32) sum += S.dw_part[(size_t)i * P.D + ch];
    s[w][lane] = sum;
    __syncthreads();
    if (w == 0 && ch < P.D) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kDwThreads / 32; ++i) sum += s[i][lane];
        S.dw[ch] = sum;
    }
}

// Calls f<T, VEC, NS>() for the widest access that the problem's sizes, strides and
// addresses allow: 16 bytes, or single elements (8,192 x 72 heads x 128 bf16: 56 against 128 us,
// fp32 99 against 142).
// NS slots per lane as a row needs them: a lane that could hold more has fewer registers for its rows
// (8,192 x 72 heads x 128 fp32 backwards with weights and angles: 169 us, with two 245).
template <class F>
cudaError_t with_width(const NormProblem& P, int dtype, bool wide, F&& f) {
    const int vec = !wide ? 1 : dtype == KDA_BF16 ? 8 : 4;
    const int slots = P.D / (2 * vec);
    if (dtype == KDA_BF16) {
        if (wide) return f.template operator()<__nv_bfloat16, 8, 1>(slots);
        return slots <= 64 ? f.template operator()<__nv_bfloat16, 1, 2>(slots) : f.template operator()<__nv_bfloat16, 1, 8>(slots);
    }
    if (wide) return slots <= 32 ? f.template operator()<float, 4, 1>(slots) : f.template operator()<float, 4, 2>(slots);
    return slots <= 64 ? f.template operator()<float, 1, 2>(slots) : f.template operator()<float, 1, 8>(slots);
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

long long blocks_for(long long items, int lanes) {
    const long long per_block = kNormThreads / lanes;
    return (items + per_block - 1) / per_block;
}

// Heads of an item: as many as share angles and weights well (8,192 x 72 heads: 8 for 2 at a time
// 60 us, always 2 at a time 93), but a group keeps four items at least, so that few rows are
// spread over all groups and the walk ends evenly (1,009 x 15 heads backwards: 1 for 8, 15 against 19 us).
int item_heads(long long rows, int least, int lanes, int blocks) {
    const long long groups = (long long)blocks * (kNormThreads / lanes);
    int hb = least;
    while (hb < kManyHeads && rows >= 4 * groups * 2 * hb) hb *= 2;
    return hb;
}

struct LaunchFwd {
    NormProblem P;
    int sms;
    cudaStream_t s;
    template <typename T, int VEC, int NS>
    cudaError_t operator()(int slots) {
        P.lanes = group_lanes(slots);
        const int room = fwd_per_sm(VEC, NS) * sms;
        const int hb = item_heads((long long)P.T * (P.side[0].heads + P.side[1].heads), rows_at_once(VEC), P.lanes, room);
        const long long items = (long long)P.T * (head_blocks(P.side[0].heads, hb) + head_blocks(P.side[1].heads, hb));
        qk_norm_kernel<T, VEC, NS><<<(unsigned)std::min<long long>(room, blocks_for(items, P.lanes)), kNormThreads, 0, s>>>(P, hb);
        return cudaGetLastError();
    }
};
struct LaunchBwd {
    NormProblem P;
    int sms;
    cudaStream_t s;
    // blocks between the sides by their rows, and no more than there are items for
    template <typename T, int VEC, int NS, bool kRot, bool kW>
    cudaError_t run() {
        const int heads = P.side[0].heads + P.side[1].heads, room = bwd_per_sm(VEC, NS, kRot, kW) * sms;
        const int hb = item_heads((long long)P.T * heads, 1, P.lanes, room);
        for (NormSide& S : P.side)
            S.blocks = S.heads ? (int)std::max<long long>(1, std::min<long long>((long long)room * S.heads / heads,
                                                                                 blocks_for((long long)P.T * head_blocks(S.heads, hb), P.lanes)))
                               : 0;
        const size_t parts = (size_t)P.side[0].blocks + P.side[1].blocks;
        float* part = nullptr;
        if (kW) {
            const cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&part), parts * P.D * 4, s);
            if (e != cudaSuccess) return e;
            P.side[0].dw_part = P.side[0].w ? part : nullptr;
            P.side[1].dw_part = P.side[1].w ? part + (size_t)P.side[0].blocks * P.D : nullptr;
        }
        cudaError_t e = timed_launch(KDA_KERNEL_QK_NORM_BWD, s, [&] {
            qk_norm_bwd_kernel<T, VEC, NS, kRot, kW><<<(unsigned)parts, kNormThreads, 0, s>>>(P, hb);
            return cudaGetLastError();
        });
        if (kW && e == cudaSuccess)
            e = timed_launch(KDA_KERNEL_QK_NORM_DW, s, [&] {
                qk_norm_dw_kernel<<<dim3((P.D + 31) / 32, 2), kDwThreads, 0, s>>>(P);
                return cudaGetLastError();
            });
        if (kW) cudaFreeAsync(part, s);
        return e;
    }
    template <typename T, int VEC, int NS>
    cudaError_t operator()(int slots) {
        P.lanes = group_lanes(slots);
        const bool w = P.side[0].w || P.side[1].w;
        if (P.cos) return w ? run<T, VEC, NS, true, true>() : run<T, VEC, NS, true, false>();
        return w ? run<T, VEC, NS, false, true>() : run<T, VEC, NS, false, false>();
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
    // items are counted in 32 bits, and a group's walk ends up to one stride (fewer than 2^18 items on
    // any GPU of this kind) after the last of them
    if ((long long)T * (Hq + Hk) >= (1LL << 32) - (1LL << 18)) return KDA_ERR_SHAPE;
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
                        interleaved, T, Hq, Hk, D, q_stride, k_stride, err), sms, s};
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
    LaunchBwd L{problem(q, k, norm, eps, q_weight, k_weight, cos, sin, positions, table_rows, rotary_dim,
                        interleaved, T, Hq, Hk, D, q_stride, k_stride, err), sms, s};
    L.P.side[0].dz = dq_out;
    L.P.side[1].dz = dk_out;
    L.P.side[0].y = dq;
    L.P.side[1].y = dk;
    L.P.side[0].dw = dq_weight;
    L.P.side[1].dw = dk_weight;
    e = with_width(L.P, dtype, wide_ok(L.P, dtype), L);
    if (e == cudaErrorMemoryAllocation) return cuda_fail(KDA_ERR_ALLOC, e);
    if (e != cudaSuccess) return cuda_fail(KDA_ERR_LAUNCH, e);
    return KDA_OK;
}

}  // extern "C"

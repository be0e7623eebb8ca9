// The gated delta rule token by token: a few new tokens for each of N sequences, applied to
// states held in HBM (kda_gdr_step).
//
// Bound by the states' traffic: 64 KB (fp32) in and, where it is wanted, 64 KB out per
// (sequence, value head), against ~2 flops per byte and token.  The columns of S are
// independent of one another, so a warp owns 16 columns for all 128 rows, in registers from
// its first read to its write: lane (rg, cq) = (lane / 4, lane % 4) holds rows rg + 8 i and
// the 4 columns 4 cq ..  A token needs S'^T k and S'^T q, both from the decayed state
// (o = scale (S'^T q + (k.q) d)), so its 9 sums over rows are one butterfly over the 8 row
// groups, and warps share nothing but a token's keys and queries.  Everything is fp32.
//
// Measured: one token for 256 sequences x 96 heads 464 us, 7.0 TB/s (more than a plain copy's
// 6.78).  Five tokens for 16 x 32 heads 19 us against a floor of 10: there the states stay in L2 on
// their way out and the 1,024 CTAs' instructions (half of all issue slots) count.  Pairs of fp32
// in one instruction (27 us) and keys straight from global memory (23) were no faster.
#include "kda_gdr.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 128;          // 4 warps: 64 columns
constexpr int kStepCols = 16;              // columns of a warp
constexpr int kStepParts = kDim / (kStepCols * kStepThreads / 32);   // CTAs of a state, next to one another
constexpr int kRowGroups = 8;
constexpr int kStepRows = kDim / kRowGroups;

__device__ __forceinline__ float4 load4(const void* base, int dtype, size_t i) {
    if (dtype == KDA_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + i);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ uint2 pack4(float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(void* base, int dtype, size_t i, float4 x) {
    if (dtype == KDA_F32) *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = x;
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + i) = pack4(x);
}

__global__ void __launch_bounds__(kStepThreads) gdr_step_kernel(GdrStep P) {
    __shared__ float s_k[2][kDim], s_q[2][kDim];
    const GdrInputs& I = P.in;
    const int tid = threadIdx.x, lane = tid & 31, rg = lane >> 2, cq = lane & 3;
    const int unit = blockIdx.x / kStepParts, h = unit % I.Hv, n = unit / I.Hv;
    const int col = blockIdx.x % kStepParts * (kStepThreads / 32) * kStepCols + (tid >> 5) * kStepCols + 4 * cq;
    const long long start = (long long)n * I.T;
    const int len = I.T;
    const int slot = P.slots ? P.slots[n] : n;
    const int keep = P.lengths ? P.lengths[n] : len;
    if (slot == -1) return;                      // a padding entry
    if (slot < -1 || slot >= P.pool || keep < 0 || keep > len) {
        if (tid == 0) set_error(P.err, KDA_ERR_BAD_INDEX);
        return;
    }
    const size_t base = ((size_t)slot * I.Hv + h) * kDim * kDim + col;
    float4 s[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i)
        s[i] = P.state_in ? load4(P.state_in, P.in_dtype, base + (size_t)(rg + kRowGroups * i) * kDim)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int hk = h / (I.Hv / I.Hk);
    const __nv_bfloat16* kp = I.k + start * I.k_stride + hk * kDim + tid;
    const __nv_bfloat16* qp = I.q + start * I.q_stride + hk * kDim + tid;
    const __nv_bfloat16* vp = I.v + start * I.v_stride + h * kDim + col;
    // without outputs only the tokens up to the kept state count
    const int end = P.out ? len : P.state_out ? keep : 0;
    __nv_bfloat16 kn, qn;
    uint2 vn;
    float gn = 0.0f, bn = 0.0f;
    auto fetch = [&](int t) {
        kn = kp[t * I.k_stride];
        qn = qp[t * I.q_stride];
        vn = *reinterpret_cast<const uint2*>(vp + t * I.v_stride);
        gn = load_gate(I.g, I.gate_dtype, (size_t)(start + t) * I.Hv + h);
        bn = load_gate(I.beta, I.gate_dtype, (size_t)(start + t) * I.Hv + h);
    };
    auto write = [&] {
#pragma unroll
        for (int i = 0; i < kStepRows; ++i)
            store4(P.state_out, P.out_dtype, base + (size_t)(rg + kRowGroups * i) * kDim, s[i]);
    };
    if (end > 0) fetch(0);
    if (P.state_out && keep == 0) write();
    for (int t = 0; t < end; ++t) {
        const int buf = t & 1;
        s_k[buf][tid] = __bfloat162float(kn);
        s_q[buf][tid] = __bfloat162float(qn);
        const float4 v = make_float4(__uint_as_float(vn.x << 16), __uint_as_float(vn.x & 0xFFFF0000u),
                                     __uint_as_float(vn.y << 16), __uint_as_float(vn.y & 0xFFFF0000u));
        const float a = expf(gn), b = bn;
        __syncthreads();   // one per token: a buffer is written again only after the next one
        if (t + 1 < end) fetch(t + 1);
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = r;
        float kq = 0.0f;
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const float k = s_k[buf][rg + kRowGroups * i], q = s_q[buf][rg + kRowGroups * i];
            s[i].x *= a; s[i].y *= a; s[i].z *= a; s[i].w *= a;
            r.x = fmaf(k, s[i].x, r.x); r.y = fmaf(k, s[i].y, r.y);
            r.z = fmaf(k, s[i].z, r.z); r.w = fmaf(k, s[i].w, r.w);
            o.x = fmaf(q, s[i].x, o.x); o.y = fmaf(q, s[i].y, o.y);
            o.z = fmaf(q, s[i].z, o.z); o.w = fmaf(q, s[i].w, o.w);
            kq = fmaf(k, q, kq);
        }
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
            r.x += __shfl_xor_sync(0xFFFFFFFFu, r.x, m); r.y += __shfl_xor_sync(0xFFFFFFFFu, r.y, m);
            r.z += __shfl_xor_sync(0xFFFFFFFFu, r.z, m); r.w += __shfl_xor_sync(0xFFFFFFFFu, r.w, m);
            o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, m); o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, m);
            o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, m); o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, m);
            kq += __shfl_xor_sync(0xFFFFFFFFu, kq, m);
        }
        const float4 d = make_float4(b * (v.x - r.x), b * (v.y - r.y), b * (v.z - r.z), b * (v.w - r.w));
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const float k = s_k[buf][rg + kRowGroups * i];
            s[i].x = fmaf(k, d.x, s[i].x); s[i].y = fmaf(k, d.y, s[i].y);
            s[i].z = fmaf(k, d.z, s[i].z); s[i].w = fmaf(k, d.w, s[i].w);
        }
        if (P.out && rg == 0)
            *reinterpret_cast<uint2*>(P.out + ((start + t) * I.Hv + h) * kDim + col) =
                pack4(make_float4(I.scale * fmaf(kq, d.x, o.x), I.scale * fmaf(kq, d.y, o.y),
                                  I.scale * fmaf(kq, d.z, o.z), I.scale * fmaf(kq, d.w, o.w)));
        if (P.state_out && t + 1 == keep) write();
    }
}

}  // namespace

cudaError_t launch_gdr_step(const GdrStep& P, cudaStream_t s) {
    const long long units = (long long)P.in.N * P.in.Hv;
    if (units == 0) return cudaSuccess;
    gdr_step_kernel<<<(unsigned)(units * kStepParts), kStepThreads, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace kda

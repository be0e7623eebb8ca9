// More of tcgen05, for kernels whose whole warp comes by where one thread issues, and the split of
// a CTA's registers between its warpgroups.
#pragma once
#include "kda_tcgen05.cuh"

namespace kda {
namespace tc {

// other forms of kind::f16: bf16 operands (type 1), an operand stored with its M (or N)
// index contiguous (major-ness 1)
constexpr uint32_t kIdBf16 = (1u << 7) | (1u << 10);
constexpr uint32_t kIdMnA = 1u << 15, kIdMnB = 1u << 16;
// MN-major 128-byte swizzle: rows of 128 bytes hold 64 consecutive M (or N) indices of one
// k; 8 rows (k) make an atom of 1024 bytes, sbo = step between atoms along k, lbo = step to
// the next 64 indices.

// moves the warpgroup's share of the CTA's registers up or down to kRegs a thread; the shares
// of all warpgroups add up to no more than what the CTA was launched with
template <int kRegs>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
// One thread of the warp, always the same.
__device__ __forceinline__ uint32_t elect() {
    uint32_t on;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(on));
    return on;
}
// The same where the whole warp comes by and `on` = elect() picks the thread that issues.
// With operands that the compiler knows to be the same in all lanes (a shuffle says so) an MMA
// then takes about 6 cycles of issue; behind a branch on the lane, or predicated on it, it
// took 46 (measured, 8 in a row).
__device__ __forceinline__ void mma_ts_on(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t on) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
__device__ __forceinline__ void mma_ss_on(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t on) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
__device__ __forceinline__ void commit_on(uint32_t mbar_smem, uint32_t on) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
        ::"r"(mbar_smem), "r"(on) : "memory");
}
// an arrival of the thread that `on` picks, beside its commit
__device__ __forceinline__ void arrive_on(uint32_t mbar_smem, uint32_t on) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n"
        ::"r"(mbar_smem), "r"(on) : "memory");
}
// 16 lanes x 32 columns as accumulator fragments of mma.sync: registers 4 j .. of a thread are
// (lane / 4, 8 j + 2 (lane % 4)), the column after it, and both 8 lanes further down
__device__ __forceinline__ void ld_fragments(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

}  // namespace tc
}  // namespace kda

// Shared-memory descriptors of MN-major operands and instruction descriptors
// with a choice of operand orders, next to the K-major ones of sm100.cuh.
#pragma once

#include "sm100.cuh"

namespace moe {
namespace sm100 {

// MN-major operand in the 128-byte swizzle layout: an atom is 8 rows of 128
// bytes, row = one K index, its 64 values consecutive along M or N (chunk c of
// row r stored at chunk c ^ (r % 8)).  mn_step: bytes between atoms 64 values
// apart along M or N; k_step: bytes between atoms 8 apart along K.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t mn_step, uint32_t k_step) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((mn_step >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((k_step >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// kind::f16, fp32 accumulators: operand type (0 fp16, 1 bf16, the same for
// both) and whether A and B are MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit(int bf16, int a_mn, int b_mn, int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
           (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A wait for the phase of the given parity with a limit in time: true once it
// has completed, false after limit_ns, or as soon as *stop is set.  The thread
// sleeps in the hardware's wait, which is longer than a limit below 20 us (a
// test's): with such a limit a phase that has not completed counts as late.
constexpr unsigned long long kWaitNs = 1000000000ull;        // the limit where no test sets one
__device__ __forceinline__ bool mbar_wait_ns(uint64_t *bar, uint32_t parity, unsigned long long limit_ns,
                                             const volatile int *stop) {
    if (mbar_test_wait(bar, parity)) return true;
    if (limit_ns < 20000ull) return false;
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    do {
        if (mbar_try_wait(bar, parity)) return true;
    } while (!(stop && *stop) && globaltimer_ns() - t0 < limit_ns);
    return false;
}

// 32 lanes x 8 columns of 32-bit accumulators (tmem_ld16 takes 16).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// One lane of the warp, the same one every time: 1 on it, 0 on the others.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t on;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(on));
    return on;
}
// The MMA and commit wrappers of sm100.cuh for a whole warp, issued by the lane
// whose `on` is 1: the operands stay warp-uniform, so that the compiler keeps
// them in uniform registers, where the instructions read them; under a branch
// on the lane it moves each of them there for every MMA (measured: 112 cycles
// an MMA against under 60).
__device__ __forceinline__ void mma_f16_on(uint32_t on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}
// The same with A in TMEM: lane = row, a 32-bit column two neighbouring K (K-major).
__device__ __forceinline__ void mma_f16_ts_on(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}
// Registers to TMEM: 16 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mma_commit_on(uint32_t on, uint64_t *bar) {
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0; "
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_addr(bar)),
        "r"(on)
        : "memory");
}

}  // namespace sm100
}  // namespace moe

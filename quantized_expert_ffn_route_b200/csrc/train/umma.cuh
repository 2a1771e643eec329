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

}  // namespace sm100
}  // namespace moe

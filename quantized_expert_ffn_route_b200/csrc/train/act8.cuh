// The 8-bit activation format: step byte, codes and their values.
#pragma once

#include "common.cuh"

namespace moe {

// Values 8i..8i+7 of an fp32 or bf16 array (16-byte aligned).
template <bool BF16>
__device__ __forceinline__ void load8(const void *x, long i, float (&v)[8]) {
    if constexpr (BF16) {
        const uint4 u = static_cast<const uint4 *>(x)[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4 a = static_cast<const float4 *>(x)[2 * i], b = static_cast<const float4 *>(x)[2 * i + 1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// The step byte of a block whose largest |value| has the bits `top`: 127 + e
// with e = floor(log2 max) - 6, one more where the largest code would round to
// 128 (a fraction of 127.5 / 64 and up: mantissa bits 0x7F0000 and up), held
// within [-126, 121]; 255 where the block is not finite.
__device__ __forceinline__ uint32_t act8_scale(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    const int e = static_cast<int>(top >> 23) - 6 + ((top & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0);
    return static_cast<uint32_t>(min(max(e, 1), 248));
}

// rint(v * inv), half to even, in the low byte: added to 1.5 * 2^23 the sum's
// last mantissa bits are the rounded value.  Only a step byte of 248 (the
// largest) can meet a code of 128, which stays at 127.
__device__ __forceinline__ uint32_t act8_code(float v, float inv, uint32_t b) {
    if (b == 255u) return 0u;
    float c = __fmul_rn(v, inv);
    if (b == 248u) c = fminf(fmaxf(c, -127.f), 127.f);
    return __float_as_uint(__fadd_rn(c, 12582912.0f)) & 0xFFu;
}

// 2^(b - 127); byte 255 gives +inf, which makes its blocks' values 0 * inf = NaN.
__device__ __forceinline__ float act8_step(uint8_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 23); }

// Four codes (one word) times the step, exact.
__device__ __forceinline__ void act8_values(uint32_t codes, float d, float *v) {
    const uint32_t u = codes ^ 0x80808080u;               // code + 128, unsigned
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u | j)) - 8388736.0f) * d;
}

}  // namespace moe

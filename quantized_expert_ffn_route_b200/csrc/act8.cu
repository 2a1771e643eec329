// 8-bit activation checkpoints: x <-> one int8 code per value and one
// power-of-two step per block of 32.
//
// With the step a power of two, x / step and code * step are exact, so that
// packing rounds once (half to even) and unpacking never: codes have 7 bits
// and a sign, and bf16 keeps 8.  A step of max / 127 would halve the largest
// rounding error, and would cost a division, a rounding in every unpacked
// value and an answer that depends on how the division rounds.
//
// Both kernels move bytes only: 2 + 1.03 bytes a value for bf16, 4 + 1.03 for
// fp32.  Four lanes hold a block, 8 values each, so that a warp's loads and
// stores are whole lines (two lanes with 16 values each write half sectors:
// unpacking 8192 x 2048 took 11.6 us against 7.1); two pieces a thread are in
// flight.
#include "common.cuh"
#include "train/act8.cuh"
#include "train/train.h"

namespace moe {

constexpr int kActThreads = 256;

// One piece of 8 values (four lanes hold a block): its codes and the block's step byte.
__device__ __forceinline__ uint2 pack_piece(const float (&v)[8], uint32_t &b) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);   // NaN above inf above all
    const unsigned lanes = 0xFu << (threadIdx.x & 28);
    top = max(top, __shfl_xor_sync(lanes, top, 1));
    top = max(top, __shfl_xor_sync(lanes, top, 2));
    b = act8_scale(top);
    const float inv = b == 255u ? 0.f : __uint_as_float((254u - b) << 23);              // 1 / step
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = act8_code(v[j], inv, b);
    return make_uint2(__byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
}

// n8: 8-value pieces, a multiple of 4: the four lanes of a block are in or out
// together.
template <bool BF16>
__global__ void __launch_bounds__(kActThreads) k_act_pack8(const void *__restrict__ x, long n8,
                                                           int8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const long step = static_cast<long>(gridDim.x) * kActThreads;
    for (long i = static_cast<long>(blockIdx.x) * kActThreads + threadIdx.x; i < n8; i += 2 * step) {
        const bool two = i + step < n8;
        float v[8], w[8];
        load8<BF16>(x, i, v);
        if (two) load8<BF16>(x, i + step, w);
        uint32_t b;
        reinterpret_cast<uint2 *>(codes)[i] = pack_piece(v, b);
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(b);
        if (two) {
            reinterpret_cast<uint2 *>(codes)[i + step] = pack_piece(w, b);
            if ((threadIdx.x & 3) == 0) scales[(i + step) >> 2] = static_cast<uint8_t>(b);
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kActThreads) k_act_unpack8(const int8_t *__restrict__ codes,
                                                             const uint8_t *__restrict__ scales, long n8,
                                                             void *__restrict__ x) {
    const long step = static_cast<long>(gridDim.x) * kActThreads;
#pragma unroll 2
    for (long i = static_cast<long>(blockIdx.x) * kActThreads + threadIdx.x; i < n8; i += step) {
        const uint2 c = reinterpret_cast<const uint2 *>(codes)[i];
        const float d = act8_step(scales[i >> 2]);
        float v[8];
        act8_values(c.x, d, v);
        act8_values(c.y, d, v + 4);
        if constexpr (BF16) {
            uint4 o;                                       // exact in bf16: the upper halves
            o.x = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x7632);
            o.y = __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x7632);
            o.z = __byte_perm(__float_as_uint(v[4]), __float_as_uint(v[5]), 0x7632);
            o.w = __byte_perm(__float_as_uint(v[6]), __float_as_uint(v[7]), 0x7632);
            static_cast<uint4 *>(x)[i] = o;
        } else {
            static_cast<float4 *>(x)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
            static_cast<float4 *>(x)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

static long act_blocks(long n8) {
    const long want = (n8 + kActThreads - 1) / kActThreads, cap = num_sms() * 8L;
    return want < cap ? want : cap;
}

int launch_act_pack8(const void *x, int x_dtype, size_t n, int8_t *codes, uint8_t *scales, cudaStream_t s) {
    const long n8 = static_cast<long>(n / 8);
    if (x_dtype == MOE_BF16) k_act_pack8<true><<<act_blocks(n8), kActThreads, 0, s>>>(x, n8, codes, scales);
    else k_act_pack8<false><<<act_blocks(n8), kActThreads, 0, s>>>(x, n8, codes, scales);
    count_launches(1);
    return cuda_status(cudaGetLastError(), "activation pack launch");
}

int launch_act_unpack8(const int8_t *codes, const uint8_t *scales, size_t n, void *x, int x_dtype, cudaStream_t s) {
    const long n8 = static_cast<long>(n / 8);
    if (x_dtype == MOE_BF16) k_act_unpack8<true><<<act_blocks(n8), kActThreads, 0, s>>>(codes, scales, n8, x);
    else k_act_unpack8<false><<<act_blocks(n8), kActThreads, 0, s>>>(codes, scales, n8, x);
    count_launches(1);
    return cuda_status(cudaGetLastError(), "activation unpack launch");
}

}  // namespace moe

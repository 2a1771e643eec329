// Tensor maps and tiled bulk copies (TMA) of the training kernels.
#pragma once

#include <cuda.h>

#include "sm100.cuh"

namespace moe {

// A map of a row-major [rows, cols] array of 16-bit values whose copies are
// box_rows x 64 values, written with the 128-byte swizzle (row r of a copy: 128
// bytes, 16-byte chunk c at c ^ (r % 8)); outside the array zeros are written.
// base 16-byte aligned, row_bytes a multiple of 16.  Returns a MOE_* status.
int make_tensor_map(CUtensorMap *map, const void *base, int bf16, uint64_t rows, uint64_t cols, uint64_t row_bytes,
                    uint32_t box_rows);

// The same for bytes without a swizzle: boxes of box_rows x box_bytes (a
// multiple of 16), rows one after another.
int make_byte_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t bytes, uint32_t box_rows,
                  uint32_t box_bytes);

namespace sm100 {

// A map made on the device: a copy of `like` (by one warp) for the array at
// `base`; 128-byte aligned in global memory.  A kernel after this one may use it
// once it has called map_acquire.
__device__ __forceinline__ void map_for(CUtensorMap *to, const CUtensorMap &like, const void *base) {
    const int lane = threadIdx.x & 31;
    reinterpret_cast<uint32_t *>(to)[lane] = reinterpret_cast<const uint32_t *>(&like)[lane];
    __syncwarp();
    if (lane == 0)
        asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(
                         __cvta_generic_to_global(to)),
                     "l"(base)
                     : "memory");
    __syncwarp();
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}
__device__ __forceinline__ void map_acquire(const CUtensorMap *map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

// A box of the map at (column x, row y) to shared memory, counted on `bar`, by
// the lane whose `on` is 1 (the whole warp calls, with the same operands: the
// instruction reads uniform registers, and operands that differ by lane make a
// loop over the lanes of it).  x a multiple of 8 values.
__device__ __forceinline__ void tma_load_on(uint32_t on, uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint64_t *bar) {
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %5, 0; "
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4]; }"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)), "r"(on)
        : "memory");
}
__device__ __forceinline__ void expect_tx_on(uint32_t on, uint64_t *bar, uint32_t bytes) {
    asm volatile(
        "{ .reg .pred q; .reg .b64 st; setp.ne.b32 q, %2, 0; "
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(smem_addr(bar)),
        "r"(bytes), "r"(on)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace sm100
}  // namespace moe

// Backward pass of the router: dx = dx_in + dl W, dW = dl^T x, db = sum_t dl.
//
// The form for any types and sizes: fp32 products on CUDA cores, 64 x 64
// tiles, 16 of the summed index at a time through shared memory.
#include "common.cuh"
#include "train/train.h"

namespace moe {

namespace {
__device__ __forceinline__ float at(const void *p, int dtype, size_t i) {
    return dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                             : static_cast<const float *>(p)[i];
}
}  // namespace

// C[m,n] = add[m,n] + sum_k A(m,k) B[k,n], A(m,k) = A[m,k], or A[k,m] with
// TRANS; B and C have N columns.
template <bool TRANS>
__global__ void __launch_bounds__(256) k_router_product(const void *__restrict__ A, int a_dtype,
                                                        const void *__restrict__ B, int b_dtype, const float *add,
                                                        int M, int N, int K, void *C, int c_dtype) {
    __shared__ float as[16][65], bs[16][65];
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            // the faster index along the row of the array that is read
            const int am = TRANS ? i & 63 : i >> 4, ak = TRANS ? i >> 6 : i & 15;
            const bool in = m0 + am < M && k0 + ak < K;
            as[ak][am] = in ? at(A, a_dtype, TRANS ? static_cast<size_t>(k0 + ak) * M + m0 + am
                                                   : static_cast<size_t>(m0 + am) * K + k0 + ak)
                            : 0.f;
            const int bn = i & 63, bk = i >> 6;
            bs[bk][bn] = n0 + bn < N && k0 + bk < K ? at(B, b_dtype, static_cast<size_t>(k0 + bk) * N + n0 + bn) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[kk][ty + 16 * i], bs[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= M || n >= N) continue;
            const size_t o = static_cast<size_t>(m) * N + n;
            const float v = acc[i][j] + (add ? add[o] : 0.f);
            if (c_dtype == MOE_BF16) static_cast<__nv_bfloat16 *>(C)[o] = __float2bfloat16_rn(v);
            else static_cast<float *>(C)[o] = v;
        }
}

// db[e] = sum_t dl[t,e]: a block per 32 columns, 32 rows at a time.
__global__ void __launch_bounds__(1024) k_router_bias(const void *__restrict__ dl, int dtype, int T, int E,
                                                      float *__restrict__ db) {
    __shared__ float part[32][33];
    const int e = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float a = 0.f;
    if (e < E)
        for (int t = warp; t < T; t += 32) a += at(dl, dtype, static_cast<size_t>(t) * E + e);
    part[warp][lane] = a;
    __syncthreads();
    const float v = warp_sum(part[lane][warp]);
    const int o = blockIdx.x * 32 + warp;
    if (lane == 0 && o < E) db[o] = v;
}

int launch_router_backward_simt(const RouterBackward &a, cudaStream_t s) {
    const auto tiles = [](int n) { return static_cast<unsigned>((n + 63) / 64); };
    if (a.dx && a.T) {
        // a grid's second axis ends at 65535 tiles: one launch per slice of tokens
        const size_t row = static_cast<size_t>(a.E) * (a.dl_dtype == MOE_BF16 ? 2 : 4);
        const size_t out = static_cast<size_t>(a.H) * (a.dx_dtype == MOE_BF16 ? 2 : 4);
        const int slice = 65535 * 64;
        for (int t0 = 0; t0 < a.T; t0 += slice) {
            const int n = a.T - t0 < slice ? a.T - t0 : slice;
            k_router_product<false><<<dim3(tiles(a.H), tiles(n)), 256, 0, s>>>(
                static_cast<const uint8_t *>(a.dl) + t0 * row, a.dl_dtype, a.w, a.w_dtype,
                a.dx_in ? a.dx_in + static_cast<size_t>(t0) * a.H : nullptr, n, a.H, a.E,
                static_cast<uint8_t *>(a.dx) + t0 * out, a.dx_dtype);
            count_launches(1);
        }
    }
    if (a.d_w) {
        k_router_product<true><<<dim3(tiles(a.H), tiles(a.E)), 256, 0, s>>>(a.dl, a.dl_dtype, a.x, a.x_dtype, nullptr,
                                                                            a.E, a.H, a.T, a.d_w, a.w_dtype);
        count_launches(1);
    }
    if (a.d_bias) {
        k_router_bias<<<(a.E + 31) / 32, 1024, 0, s>>>(a.dl, a.dl_dtype, a.T, a.E, a.d_bias);
        count_launches(1);
    }
    return cuda_status(cudaGetLastError(), "router backward launch");
}

}  // namespace moe

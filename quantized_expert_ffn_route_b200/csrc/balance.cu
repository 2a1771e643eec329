// Balance loss with per-expert counts, and the gradient of the router's logits.
//
// The loss needs no column sums: with the counts known, f is a constant and
//   sum_e f[e] mean_t p[t,e] = mean_t D[t],  D[t] = sum_e f[e] p[t,e],
// so that one pass over the logits gives each row's maximum, sum of
// exponentials, D and lse in registers, and the gradient of a row,
//   dl[e] = g p[e] (b (f[e] - D) + c lse)   b = balance_coef E / N, c = z_coef 2 / N,
// needs nothing but that row: the backward kernel recomputes the three sums
// from the row it has to read anyway, and nothing is kept between the calls.
// Both kernels move T E 4 bytes (plus the gradient out) and are bound by that
// at large T E, by launch latency below.
//
// Rows of up to 1024 experts: one warp each, the row in registers.  Longer
// rows (a model-wide pool): one block each, two reads of the row, the second
// one from L1 or L2.
#include "common.cuh"
#include "train/train.h"

#include <type_traits>

namespace moe {

namespace {
constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBigThreads = 512;
constexpr int kHistMax = 8192;                    // experts counted in shared memory (32 KB)

// (maximum, sum of exp(l - max), sum of f exp(l - max)) of a part of a row
struct Soft {
    float m, s, d;
};
__device__ __forceinline__ Soft soft_join(const Soft &a, const Soft &b) {
    const float m = fmaxf(a.m, b.m);
    // a part without a finite entry has s = d = 0 (or NaN, which stays)
    const float ea = a.m == m ? 1.f : expf(a.m - m), eb = b.m == m ? 1.f : expf(b.m - m);
    return {m, a.s * ea + b.s * eb, a.d * ea + b.d * eb};
}
// Adds N entries at a time.
template <int N>
__device__ __forceinline__ void soft_add(Soft &a, const float (&l)[N], const float (&f)[N]) {
    float m = a.m;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        m = fmaxf(m, l[i]);                       // drops NaN
        nan |= l[i] != l[i];
    }
    if (m == -INFINITY) {                         // nothing yet: exp(-inf - -inf) is no number
        if (nan) a.s = a.d = NAN;
        return;
    }
    const float e0 = a.m == m ? 1.f : expf(a.m - m);
    a.s *= e0;
    a.d *= e0;
    a.m = m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float e = expf(l[i] - m);
        a.s += e;
        a.d = fmaf(f[i], e, a.d);
    }
}
__device__ __forceinline__ Soft soft_warp(Soft a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Soft b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.d = __shfl_xor_sync(0xffffffffu, a.d, o);
        a = soft_join(a, b);
    }
    return a;
}
// The block's join, on every thread; `part` holds one entry per warp.
__device__ __forceinline__ Soft soft_block(Soft a, Soft *part) {
    a = soft_warp(a);
    const int lane = threadIdx.x & 31;
    __syncthreads();                              // the last row's readers are done with `part`
    if (lane == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : Soft{-INFINITY, 0.f, 0.f};
    return soft_warp(a);
}

// What one row adds: D and lse^2.  A row of -inf alone adds nothing.
struct RowSums {
    float d;
    double z;                                     // lse of a row of the type's lowest values squares out of fp32's range
};
__device__ __forceinline__ RowSums row_sums(const Soft &a, unsigned *err, bool leader) {
    if (a.m == -INFINITY && a.s == 0.f) return {0.f, 0.};
    const float lse = a.m + logf(a.s);
    if (leader && !isfinite(lse)) report(err, MOE_DEVERR_NONFINITE);
    return {a.d / a.s, static_cast<double>(lse) * lse};
}

__device__ __forceinline__ void block_add(float d, double z, double2 *out) {
    // one value per warp (lane 0), summed in warp order
    __shared__ double2 part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    if (lane == 0) part[warp] = make_double2(d, z);
    __syncthreads();
    if (threadIdx.x == 0) {
        double2 a = part[0];
        for (int i = 1; i < n; ++i) {
            a.x += part[i].x;
            a.y += part[i].y;
        }
        *out = a;
    }
}
}  // namespace

// counts[0..E-1] and counts[E], zero before: (token, slot) pairs and tokens.
__global__ void __launch_bounds__(kBalThreads) k_balance_counts(const int32_t *__restrict__ ids,
                                                                const uint8_t *__restrict__ mask, int T, int E, int k,
                                                                int32_t *counts, unsigned *err) {
    extern __shared__ int32_t hist[];
    const bool local = E <= kHistMax;
    if (local) {
        for (int e = threadIdx.x; e < E; e += kBalThreads) hist[e] = 0;
        __syncthreads();
    }
    const int n = T * k;
    int tokens = 0;
    for (int i = blockIdx.x * kBalThreads + threadIdx.x; i < n; i += gridDim.x * kBalThreads) {
        const int t = i / k;
        if (mask && !mask[t]) continue;
        tokens += i == t * k;
        const int e = ids[i];
        if (e < 0 || e >= E) report(err, MOE_DEVERR_BAD_EXPERT);
        else atomicAdd((local ? hist : counts) + e, 1);
    }
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(counts + E, tokens);
    if (local) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kBalThreads)
            if (hist[e]) atomicAdd(counts + e, hist[e]);
    }
}

// Four neighbouring entries of a row from column c on (fill beyond E).
template <bool VEC>
__device__ __forceinline__ void row4(const float *row, int c, int E, float fill, float (&v)[4]) {
    if constexpr (VEC) {
        if (c < E) {
            const float4 u = *reinterpret_cast<const float4 *>(row + c);
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c + i < E ? row[c + i] : fill;
        return;
    }
    v[0] = v[1] = v[2] = v[3] = fill;
}
template <bool VEC>
__device__ __forceinline__ void share4(const int32_t *counts, int c, int E, float unit, float (&f)[4]) {
    if constexpr (VEC) {
        if (c + 3 < E) {
            const int4 u = *reinterpret_cast<const int4 *>(counts + c);
            f[0] = u.x * unit, f[1] = u.y * unit, f[2] = u.z * unit, f[3] = u.w * unit;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = c + i < E ? counts[c + i] * unit : 0.f;
}

// One warp per row, NV float4 per lane (E <= 128 NV).
template <int NV, bool VEC>
__global__ void __launch_bounds__(kBalThreads) k_balance_rows(const float *__restrict__ logits,
                                                              const uint8_t *__restrict__ mask, int T, int E, int k,
                                                              const int32_t *__restrict__ counts,
                                                              double2 *__restrict__ part, unsigned *err) {
    const int lane = threadIdx.x & 31;
    const float unit = 1.f / (static_cast<float>(max(counts[E], 1)) * k);
    float f[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) share4<VEC>(counts, 4 * lane + 128 * i, E, unit, f[i]);
    float sd = 0.f;
    double sz = 0.;
    for (int t = blockIdx.x * kBalWarps + (threadIdx.x >> 5); t < T; t += gridDim.x * kBalWarps) {
        if (mask && !mask[t]) continue;
        const float *row = logits + static_cast<size_t>(t) * E;
        float l[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) row4<VEC>(row, 4 * lane + 128 * i, E, -INFINITY, l[i]);
        Soft a = {-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) soft_add(a, l[i], f[i]);
        const RowSums r = row_sums(soft_warp(a), err, lane == 0);
        sd += r.d;
        sz += r.z;
    }
    block_add(sd, sz, part + blockIdx.x);
}

// One block per row.
template <bool VEC>
__global__ void __launch_bounds__(kBigThreads) k_balance_rows_big(const float *__restrict__ logits,
                                                                  const uint8_t *__restrict__ mask, int T, int E,
                                                                  int k, const int32_t *__restrict__ counts,
                                                                  double2 *__restrict__ part, unsigned *err) {
    __shared__ Soft warps[kBigThreads / 32];
    const float unit = 1.f / (static_cast<float>(max(counts[E], 1)) * k);
    float sd = 0.f;
    double sz = 0.;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (mask && !mask[t]) continue;
        const float *row = logits + static_cast<size_t>(t) * E;
        Soft a = {-INFINITY, 0.f, 0.f};
        for (int c = 4 * threadIdx.x; c < E; c += 4 * kBigThreads) {
            float l[4], f[4];
            row4<VEC>(row, c, E, -INFINITY, l);
            share4<VEC>(counts, c, E, unit, f);
            soft_add(a, l, f);
        }
        const RowSums r = row_sums(soft_block(a, warps), err, threadIdx.x == 0);
        if (threadIdx.x == 0) {
            sd += r.d;
            sz += r.z;
        }
    }
    block_add(threadIdx.x == 0 ? sd : 0.f, threadIdx.x == 0 ? sz : 0., part + blockIdx.x);
}

// Sums the blocks' parts in a fixed order and writes the four losses.
__global__ void __launch_bounds__(256) k_balance_finish(const double2 *__restrict__ part, int n,
                                                        const int32_t *__restrict__ counts, int E, float balance_coef,
                                                        float z_coef, float *__restrict__ loss) {
    __shared__ double2 sum[256];
    double2 a = make_double2(0., 0.);
    for (int i = threadIdx.x; i < n; i += 256) {
        a.x += part[i].x;
        a.y += part[i].y;
    }
    sum[threadIdx.x] = a;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o) {
            sum[threadIdx.x].x += sum[threadIdx.x + o].x;
            sum[threadIdx.x].y += sum[threadIdx.x + o].y;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const double N = max(counts[E], 1);
        const double b = E * sum[0].x / N, z = sum[0].y / N;
        loss[0] = static_cast<float>(balance_coef * b + z_coef * z);
        loss[1] = static_cast<float>(b);
        loss[2] = static_cast<float>(z);
        loss[3] = static_cast<float>(counts[E]);
    }
}

// ---------------------------------------------------------------- backward
struct RouteGrad {
    const float *logits;
    const int32_t *ids;
    const float *w, *dw;
    const uint8_t *mask;
    const int32_t *counts;
    const float *d_loss;
    int T, E, k;
    float balance, z;      // coefficients
    void *dl;
    unsigned *err;
};

template <bool BF16>
__device__ __forceinline__ void put1(void *out, size_t i, float v) {
    if constexpr (BF16) static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(out)[i] = v;
}
template <bool BF16, bool VEC>
__device__ __forceinline__ void put4(void *out, size_t row, int c, int E, const float (&v)[4]) {
    if (c >= E) return;
    if constexpr (VEC) {
        if constexpr (BF16) {
            __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
            uint2 u;
            u.x = *reinterpret_cast<uint32_t *>(&a);
            u.y = *reinterpret_cast<uint32_t *>(&b);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + row + c) = u;
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + row + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < E) put1<BF16>(out, row + c + i, v[i]);
    }
}

// The loss term of one entry: p (alpha f + beta), the row's constants given.
struct RowGrad {
    float m, inv_s;        // maximum, 1 / sum
    float alpha, beta;     // g b, g (c lse - b D)
};
__device__ __forceinline__ RowGrad row_grad(const Soft &a, float gb, float gc, unsigned *err, bool leader) {
    if (a.m == -INFINITY && a.s == 0.f) return {0.f, 0.f, 0.f, 0.f};      // a row of -inf: no gradient
    const float lse = a.m + logf(a.s);
    if (leader && !isfinite(lse)) report(err, MOE_DEVERR_NONFINITE);
    return {a.m, 1.f / a.s, gb, gc * lse - gb * (a.d / a.s)};
}
__device__ __forceinline__ float loss_term(const RowGrad &r, float l, float f) {
    return expf(l - r.m) * r.inv_s * fmaf(r.alpha, f, r.beta);
}

// The gates' gradient: lane j < k writes the whole entry of its expert, the
// loss term included (equal ids write equal values).  The row is written.
template <bool BF16, bool LOSS>
__device__ __forceinline__ void gate_entries(const RouteGrad &a, int t, const RowGrad &r, float unit) {
    const int lane = threadIdx.x & 31;
    const size_t at = static_cast<size_t>(t) * a.k + lane;
    const bool in = lane < a.k;
    const int id = in ? a.ids[at] : -1;
    const float w = in ? a.w[at] : 0.f, dw = in ? a.dw[at] : 0.f;
    const float mean = warp_sum(in ? w * dw : 0.f);
    const float mine = w * (dw - mean);
    float g = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const float v = __shfl_sync(0xffffffffu, mine, j);
        if (__shfl_sync(0xffffffffu, id, j) == id) g += v;
    }
    if (!in) return;
    if (id < 0 || id >= a.E) {
        report(a.err, MOE_DEVERR_BAD_EXPERT);
        return;
    }
    if constexpr (LOSS) g += loss_term(r, a.logits[static_cast<size_t>(t) * a.E + id], a.counts[id] * unit);
    put1<BF16>(a.dl, static_cast<size_t>(t) * a.E + id, g);
}

// One warp per row, NV float4 per lane.
template <int NV, bool VEC, bool BF16, bool LOSS>
__global__ void __launch_bounds__(kBalThreads) k_route_backward(RouteGrad a) {
    const int lane = threadIdx.x & 31;
    float f[NV][4], gb = 0.f, gc = 0.f, unit = 0.f;
    if constexpr (LOSS) {
        const float n = static_cast<float>(max(a.counts[a.E], 1)), g = a.d_loss ? *a.d_loss : 1.f;
        unit = 1.f / (n * a.k);
        gb = g * a.balance * a.E / n;
        gc = g * a.z * 2.f / n;
#pragma unroll
        for (int i = 0; i < NV; ++i) share4<VEC>(a.counts, 4 * lane + 128 * i, a.E, unit, f[i]);
    }
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = blockIdx.x * kBalWarps + (threadIdx.x >> 5); t < a.T; t += gridDim.x * kBalWarps) {
        const size_t row = static_cast<size_t>(t) * a.E;
        const bool on = !a.mask || a.mask[t];
        RowGrad r = {0.f, 0.f, 0.f, 0.f};
        if (LOSS && on) {
            float l[NV][4];
#pragma unroll
            for (int i = 0; i < NV; ++i) row4<VEC>(a.logits + row, 4 * lane + 128 * i, a.E, -INFINITY, l[i]);
            Soft s = {-INFINITY, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i) soft_add(s, l[i], f[i]);
            r = row_grad(soft_warp(s), gb, gc, a.err, lane == 0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = loss_term(r, l[i][j], f[i][j]);
                put4<BF16, VEC>(a.dl, row, 4 * lane + 128 * i, a.E, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) put4<BF16, VEC>(a.dl, row, 4 * lane + 128 * i, a.E, zero);
        }
        if (on && a.dw) {
            __syncwarp();                          // the row is written before its entries are
            gate_entries<BF16, LOSS>(a, t, r, unit);
        }
    }
}

// One block per row.
template <bool VEC, bool BF16, bool LOSS>
__global__ void __launch_bounds__(kBigThreads) k_route_backward_big(RouteGrad a) {
    __shared__ Soft warps[kBigThreads / 32];
    float gb = 0.f, gc = 0.f, unit = 0.f;
    if constexpr (LOSS) {
        const float n = static_cast<float>(max(a.counts[a.E], 1)), g = a.d_loss ? *a.d_loss : 1.f;
        unit = 1.f / (n * a.k);
        gb = g * a.balance * a.E / n;
        gc = g * a.z * 2.f / n;
    }
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = static_cast<size_t>(t) * a.E;
        const bool on = !a.mask || a.mask[t];
        RowGrad r = {0.f, 0.f, 0.f, 0.f};
        if (LOSS && on) {
            Soft s = {-INFINITY, 0.f, 0.f};
            for (int c = 4 * threadIdx.x; c < a.E; c += 4 * kBigThreads) {
                float l[4], f[4];
                row4<VEC>(a.logits + row, c, a.E, -INFINITY, l);
                share4<VEC>(a.counts, c, a.E, unit, f);
                soft_add(s, l, f);
            }
            r = row_grad(soft_block(s, warps), gb, gc, a.err, threadIdx.x == 0);
            for (int c = 4 * threadIdx.x; c < a.E; c += 4 * kBigThreads) {
                float l[4], f[4], v[4];
                row4<VEC>(a.logits + row, c, a.E, -INFINITY, l);
                share4<VEC>(a.counts, c, a.E, unit, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = loss_term(r, l[j], f[j]);
                put4<BF16, VEC>(a.dl, row, c, a.E, v);
            }
        } else {
            for (int c = 4 * threadIdx.x; c < a.E; c += 4 * kBigThreads) put4<BF16, VEC>(a.dl, row, c, a.E, zero);
        }
        __syncthreads();                           // the row is written before its entries are
        if (on && a.dw && threadIdx.x < 32) gate_entries<BF16, LOSS>(a, t, r, unit);
    }
}

// ------------------------------------------------------------------ launch
static int row_blocks(int T) {
    const long want = (static_cast<long>(T) + kBalWarps - 1) / kBalWarps, cap = num_sms() * 8L;
    return static_cast<int>(want < cap ? want : cap);
}
static int big_blocks(int T) {
    const int cap = num_sms() * 3;
    return T < cap ? T : cap;
}

size_t balance_ws_bytes(int T, int E) {
    return static_cast<size_t>(E <= 1024 ? row_blocks(T) : big_blocks(T)) * sizeof(double2);
}

int launch_balance_loss(const float *logits, const int32_t *ids, const uint8_t *mask, int T, int E, int k,
                        float balance_coef, float z_coef, int32_t *counts, float *loss, void *ws, unsigned *err,
                        cudaStream_t s) {
    int rc = cuda_status(cudaMemsetAsync(counts, 0, (static_cast<size_t>(E) + 1) * sizeof(int32_t), s), "counts memset");
    if (rc) return rc;
    double2 *part = static_cast<double2 *>(ws);
    const long pairs = static_cast<long>(T) * k;
    long blocks = (pairs + 8L * kBalThreads - 1) / (8L * kBalThreads);
    if (blocks > num_sms()) blocks = num_sms();
    k_balance_counts<<<blocks, kBalThreads, E <= kHistMax ? E * sizeof(int32_t) : 0, s>>>(ids, mask, T, E, k, counts,
                                                                                          err);
    const int n = E <= 1024 ? row_blocks(T) : big_blocks(T);
    const bool vec = E % 4 == 0;
    if (E > 1024) {
        if (vec) k_balance_rows_big<true><<<n, kBigThreads, 0, s>>>(logits, mask, T, E, k, counts, part, err);
        else k_balance_rows_big<false><<<n, kBigThreads, 0, s>>>(logits, mask, T, E, k, counts, part, err);
    } else {
#define MOE_ROWS(NV)                                                                                            \
    do {                                                                                                        \
        if (vec) k_balance_rows<NV, true><<<n, kBalThreads, 0, s>>>(logits, mask, T, E, k, counts, part, err);  \
        else k_balance_rows<NV, false><<<n, kBalThreads, 0, s>>>(logits, mask, T, E, k, counts, part, err);     \
    } while (0)
        if (E <= 128) MOE_ROWS(1);
        else if (E <= 256) MOE_ROWS(2);
        else if (E <= 512) MOE_ROWS(4);
        else MOE_ROWS(8);
#undef MOE_ROWS
    }
    k_balance_finish<<<1, 256, 0, s>>>(part, n, counts, E, balance_coef, z_coef, loss);
    count_launches(3);
    return cuda_status(cudaGetLastError(), "balance loss launch");
}

template <bool BF16, bool LOSS, bool VEC>
static void route_backward_rows(const RouteGrad &a, cudaStream_t s) {
    if (a.E > 1024) {
        k_route_backward_big<VEC, BF16, LOSS><<<big_blocks(a.T), kBigThreads, 0, s>>>(a);
        return;
    }
    const int n = row_blocks(a.T);
    if (a.E <= 128) k_route_backward<1, VEC, BF16, LOSS><<<n, kBalThreads, 0, s>>>(a);
    else if (a.E <= 256) k_route_backward<2, VEC, BF16, LOSS><<<n, kBalThreads, 0, s>>>(a);
    else if (a.E <= 512) k_route_backward<4, VEC, BF16, LOSS><<<n, kBalThreads, 0, s>>>(a);
    else k_route_backward<8, VEC, BF16, LOSS><<<n, kBalThreads, 0, s>>>(a);
}

int launch_route_backward(const float *logits, const int32_t *ids, const float *w, const float *dw,
                          const uint8_t *mask, const int32_t *counts, const float *d_loss, int T, int E, int k,
                          float balance_coef, float z_coef, void *dl, int dl_dtype, unsigned *err, cudaStream_t s) {
    const RouteGrad a = {logits, ids, w, dw, mask, counts, d_loss, T, E, k, balance_coef, z_coef, dl, err};
    const bool bf16 = dl_dtype == MOE_BF16, loss = counts != nullptr, vec = E % 4 == 0;
    auto go = [&](auto b, auto l) {
        constexpr bool B = decltype(b)::value, L = decltype(l)::value;
        if (vec) route_backward_rows<B, L, true>(a, s);
        else route_backward_rows<B, L, false>(a, s);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (bf16) loss ? go(Yes{}, Yes{}) : go(Yes{}, No{});
    else loss ? go(No{}, Yes{}) : go(No{}, No{});
    count_launches(1);
    return cuda_status(cudaGetLastError(), "route backward launch");
}

}  // namespace moe

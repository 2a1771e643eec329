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
// at large T E, by the chain load - maximum - sums - store and by launches
// below; so the counts go without atomics and memsets (a block's part each,
// added where they are read), the last block to end adds the rows' sums, and
// up to 128 rows of up to 1024 experts are one block's work and one launch.
//
// Measured: 8192 x 512 in 6.3 us (counts) + 10.6 (rows) + 10.4 (gradient), 129 x
// 24,576 in 2.9 + 10.5 + 10.1.  The next row's loads issued before a row's sums
// cost registers and were slower (13.3 and 11.7 us).
//
// Rows of up to 1024 experts: one warp each, the row in registers.  Longer
// rows (a model-wide pool): one block each, up to 64 entries a thread.
#include "common.cuh"
#include "train/train.h"

#include <type_traits>

namespace moe {

namespace {
constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBigThreads = 1024;
constexpr int kOneThreads = 1024;                 // the one-block form
constexpr int kOneRows = 128;
constexpr int kCountThreads = 1024;
constexpr int kSlice = 4096;                      // experts a block counts, above 1024
constexpr int kParts = 8;                         // blocks that count at most, up to 1024

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A row's maximum, sum of exp(l - max) and sum of f exp(l - max).  fmaxf drops
// NaN; the exponential brings it back into the sums.  A row of -inf alone has
// m = -inf and is left out before its sums (which would be NaN) are used.
struct Soft {
    float m, s, d;
};

// What one row adds: D and lse^2.
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

// A lane's (thread's) N entries: exponentials in place, sums into s and d.  m
// is the whole row's maximum.
template <int N>
__device__ __forceinline__ void soft_exps(float (&l)[N], const float (&f)[N], float m, float &s, float &d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // nothing but -inf (and NaN) in the row: exp(-inf - -inf) is no number
        l[i] = m == -INFINITY ? (l[i] != l[i] ? l[i] : 0.f) : expf(l[i] - m);
        s += l[i];
        d = fmaf(f[i], l[i], d);
    }
}

// The block's sum of one value a warp (lane 0's), in warp order, on thread 0.
__device__ __forceinline__ double2 block_rows(float d, double z) {
    __shared__ double2 part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    if (lane == 0) part[warp] = make_double2(d, z);
    __syncthreads();
    double2 a = part[0];
    if (threadIdx.x == 0)
        for (int i = 1; i < n; ++i) {
            a.x += part[i].x;
            a.y += part[i].y;
        }
    return a;
}

struct LossOut {
    int E;
    float balance, z;      // coefficients
    float *loss;
};
__device__ __forceinline__ void write_loss(const LossOut &o, double2 sum, int tokens) {
    const double N = max(tokens, 1);
    const double b = o.E * sum.x / N, z = sum.y / N;
    o.loss[0] = static_cast<float>(o.balance * b + o.z * z);
    o.loss[1] = static_cast<float>(b);
    o.loss[2] = static_cast<float>(z);
    o.loss[3] = static_cast<float>(tokens);
}

// The last block to come adds all blocks' parts, in block order.
__device__ __forceinline__ void finish_loss(double2 mine, double2 *part, unsigned *ticket, const LossOut &o, int tokens) {
    __shared__ bool last;
    __shared__ double2 sum[32];
    if (threadIdx.x == 0) {
        part[blockIdx.x] = mine;
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double2 a = make_double2(0., 0.);
    for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += blockDim.x) {
        const double2 v = __ldcg(part + i);
        a.x += v.x;
        a.y += v.y;
    }
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, o2);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, o2);
    }
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i) {
            a.x += sum[i].x;
            a.y += sum[i].y;
        }
        write_loss(o, a, tokens);
    }
}

// Counts (token, slot) pairs first, first + step, .. of the experts e0 .. e1 - 1
// into hist (shared memory, zeroed: expert e at e - e0); returns the tokens met
// at their first slot, added over the warp.  Four pairs' loads are in flight.
__device__ __forceinline__ int count_pairs(const int32_t *ids, const uint8_t *mask, int T, int E, int k, int first,
                                           int step, int e0, int e1, int32_t *hist, unsigned *err) {
    const int n = T * k;
    int tokens = 0;
    for (int i0 = first; i0 < n; i0 += 4 * step) {
        int id[4], on[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long i = i0 + static_cast<long>(u) * step;
            const bool in = i < n;
            const int t = in ? static_cast<int>(i) / k : 0;
            id[u] = in ? ids[i] : 0;
            on[u] = in && (!mask || mask[t]);
            tokens += on[u] && i == static_cast<long>(t) * k;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!on[u]) continue;
            if (id[u] < 0 || id[u] >= E) report(err, MOE_DEVERR_BAD_EXPERT);
            else if (id[u] >= e0 && id[u] < e1) atomicAdd(hist + id[u] - e0, 1);
        }
    }
    return __reduce_add_sync(0xffffffffu, tokens);
}
}  // namespace

// Up to 1024 experts: each block counts its share of the pairs, out [blocks, E + 1].
__global__ void __launch_bounds__(kCountThreads) k_balance_parts(const int32_t *__restrict__ ids,
                                                                 const uint8_t *__restrict__ mask, int T, int E, int k,
                                                                 int32_t *__restrict__ out, unsigned *ticket,
                                                                 unsigned *err) {
    __shared__ int32_t hist[1024 + 1];
    for (int e = threadIdx.x; e <= E; e += kCountThreads) hist[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
    __syncthreads();
    const int tokens = count_pairs(ids, mask, T, E, k, blockIdx.x * kCountThreads + threadIdx.x,
                                   gridDim.x * kCountThreads, 0, E, hist, err);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(hist + E, tokens);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kCountThreads) out[static_cast<size_t>(blockIdx.x) * (E + 1) + e] = hist[e];
}

// More experts: each block reads all pairs and counts kSlice experts.
__global__ void __launch_bounds__(kCountThreads) k_balance_slices(const int32_t *__restrict__ ids,
                                                                  const uint8_t *__restrict__ mask, int T, int E, int k,
                                                                  int32_t *__restrict__ counts, unsigned *ticket,
                                                                  unsigned *err) {
    __shared__ int32_t hist[kSlice];
    __shared__ int32_t all;
    const int e0 = blockIdx.x * kSlice, e1 = min(E, e0 + kSlice);
    for (int e = threadIdx.x; e < kSlice; e += kCountThreads) hist[e] = 0;
    if (threadIdx.x == 0) {
        all = 0;
        if (blockIdx.x == 0) *ticket = 0;
    }
    __syncthreads();
    const int tokens = count_pairs(ids, mask, T, E, k, threadIdx.x, kCountThreads, e0, e1, hist, err);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(&all, tokens);
    __syncthreads();
    for (int e = e0 + threadIdx.x; e < e1; e += kCountThreads) counts[e] = hist[e - e0];
    if (blockIdx.x == 0 && threadIdx.x == 0) counts[E] = all;
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

// The sums of one row by a warp, NV float4 per lane (E <= 128 NV).
template <int NV, bool VEC>
__device__ __forceinline__ Soft warp_row(const float *row, int E, const float (&f)[NV][4], float (&l)[NV][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NV; ++i) row4<VEC>(row, 4 * lane + 128 * i, E, -INFINITY, l[i]);
    Soft a = {-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) a.m = fmaxf(a.m, fmaxf(fmaxf(l[i][0], l[i][1]), fmaxf(l[i][2], l[i][3])));
    a.m = warp_max(a.m);
#pragma unroll
    for (int i = 0; i < NV; ++i) soft_exps(l[i], f[i], a.m, a.s, a.d);
    a.s = warp_sum(a.s);
    a.d = warp_sum(a.d);
    return a;
}

// Rows r0, r0 + step, .. by this warp: their D and lse^2 added up.
template <int NV, bool VEC>
__device__ __forceinline__ RowSums warp_rows(const float *logits, const uint8_t *mask, int T, int E, float unit,
                                             const int32_t *counts, int r0, int step, unsigned *err) {
    const int lane = threadIdx.x & 31;
    float f[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) share4<VEC>(counts, 4 * lane + 128 * i, E, unit, f[i]);
    RowSums sum = {0.f, 0.};
    for (int t = r0; t < T; t += step) {
        if (mask && !mask[t]) continue;
        float l[NV][4];
        const RowSums r = row_sums(warp_row<NV, VEC>(logits + static_cast<size_t>(t) * E, E, f, l), err, lane == 0);
        sum.d += r.d;
        sum.z += r.z;
    }
    return sum;
}

// Rows of up to 1024 experts, the counts' parts added first.
template <int NV, bool VEC>
__global__ void __launch_bounds__(kBalThreads) k_balance_rows(const float *__restrict__ logits,
                                                              const uint8_t *__restrict__ mask, int T, int E, int k,
                                                              const int32_t *__restrict__ parts, int n_parts,
                                                              int32_t *__restrict__ counts, double2 *part,
                                                              unsigned *ticket, LossOut o, unsigned *err) {
    __shared__ __align__(16) int32_t n[1024 + 4];
    for (int e = threadIdx.x; e <= E; e += kBalThreads) {
        int c = 0;
#pragma unroll
        for (int p = 0; p < kParts; ++p) c += p < n_parts ? parts[static_cast<size_t>(p) * (E + 1) + e] : 0;
        n[e] = c;
        if (blockIdx.x == 0) counts[e] = c;
    }
    __syncthreads();
    const float unit = 1.f / (static_cast<float>(max(n[E], 1)) * k);
    const RowSums r = warp_rows<NV, VEC>(logits, mask, T, E, unit, n, blockIdx.x * kBalWarps + (threadIdx.x >> 5),
                                         gridDim.x * kBalWarps, err);
    finish_loss(block_rows(r.d, r.z), part, ticket, o, n[E]);
}

// Few rows of up to 1024 experts: counts, rows and losses by one block.
template <int NV, bool VEC>
__global__ void __launch_bounds__(kOneThreads) k_balance_one(const float *__restrict__ logits,
                                                             const int32_t *__restrict__ ids,
                                                             const uint8_t *__restrict__ mask, int T, int E, int k,
                                                             int32_t *__restrict__ counts, LossOut o, unsigned *err) {
    __shared__ __align__(16) int32_t n[1024 + 4];
    for (int e = threadIdx.x; e <= E; e += kOneThreads) n[e] = 0;
    __syncthreads();
    const int tokens = count_pairs(ids, mask, T, E, k, threadIdx.x, kOneThreads, 0, E, n, err);
    if ((threadIdx.x & 31) == 0 && tokens) atomicAdd(n + E, tokens);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kOneThreads) counts[e] = n[e];
    const float unit = 1.f / (static_cast<float>(max(n[E], 1)) * k);
    const RowSums r = warp_rows<NV, VEC>(logits, mask, T, E, unit, n, threadIdx.x >> 5, kOneThreads / 32, err);
    const double2 sum = block_rows(r.d, r.z);
    if (threadIdx.x == 0) write_loss(o, sum, n[E]);
}

// The sums of one row by a block, V float4 per thread (E <= 4096 V); on every thread.
template <int V, bool VEC>
__device__ __forceinline__ Soft block_row(const float *row, int E, const int32_t *counts, float unit,
                                          float (&l)[V][4]) {
    __shared__ float red[3][kBigThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < V; ++i) row4<VEC>(row, 4 * (threadIdx.x + kBigThreads * i), E, -INFINITY, l[i]);
    Soft a = {-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) a.m = fmaxf(a.m, fmaxf(fmaxf(l[i][0], l[i][1]), fmaxf(l[i][2], l[i][3])));
    a.m = warp_max(a.m);
    __syncthreads();                              // the last row's values are read
    if (lane == 0) red[0][warp] = a.m;
    __syncthreads();
    a.m = warp_max(lane < kBigThreads / 32 ? red[0][lane] : -INFINITY);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[4];
        share4<VEC>(counts, 4 * (threadIdx.x + kBigThreads * i), E, unit, f);
        soft_exps(l[i], f, a.m, a.s, a.d);
    }
    a.s = warp_sum(a.s);
    a.d = warp_sum(a.d);
    if (lane == 0) red[1][warp] = a.s, red[2][warp] = a.d;
    __syncthreads();
    a.s = warp_sum(lane < kBigThreads / 32 ? red[1][lane] : 0.f);
    a.d = warp_sum(lane < kBigThreads / 32 ? red[2][lane] : 0.f);
    return a;
}

template <int V, bool VEC>
__global__ void __launch_bounds__(kBigThreads) k_balance_rows_big(const float *__restrict__ logits,
                                                                  const uint8_t *__restrict__ mask, int T, int E,
                                                                  int k, const int32_t *__restrict__ counts,
                                                                  double2 *part, unsigned *ticket, LossOut o,
                                                                  unsigned *err) {
    const float unit = 1.f / (static_cast<float>(max(counts[E], 1)) * k);
    RowSums sum = {0.f, 0.};
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (mask && !mask[t]) continue;
        float l[V][4];
        const RowSums r = row_sums(block_row<V, VEC>(logits + static_cast<size_t>(t) * E, E, counts, unit, l), err,
                                   threadIdx.x == 0);
        sum.d += r.d;
        sum.z += r.z;
    }
    finish_loss(make_double2(sum.d, sum.z), part, ticket, o, counts[E]);
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
__device__ __forceinline__ float loss_term(const RowGrad &r, float e, float f) {
    return e * r.inv_s * fmaf(r.alpha, f, r.beta);
}

// Lane j < k's slot of a token, read before the row is.
struct Slot {
    int id;
    float w, dw;
};
__device__ __forceinline__ Slot slot_of(const RouteGrad &a, int t, bool on) {
    const int lane = threadIdx.x & 31;
    const bool in = on && a.dw && lane < a.k;
    const size_t at = static_cast<size_t>(t) * a.k + lane;
    return {in ? a.ids[at] : -1, in ? a.w[at] : 0.f, in ? a.dw[at] : 0.f};
}

// The gates' gradient: lane j < k writes the whole entry of its expert, the
// loss term included (equal ids write equal values).  The row is written.
template <bool BF16, bool LOSS>
__device__ __forceinline__ void gate_entries(const RouteGrad &a, int t, const Slot &s, const RowGrad &r, float unit) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < a.k, good = in && s.id >= 0 && s.id < a.E;
    const size_t at = static_cast<size_t>(t) * a.E + (good ? s.id : 0);
    float l = 0.f, n = 0.f;
    if (LOSS && good) l = a.logits[at], n = a.counts[s.id] * unit;
    const float mean = warp_sum(in ? s.w * s.dw : 0.f);
    const float mine = s.w * (s.dw - mean);
    float g = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const float v = __shfl_sync(0xffffffffu, mine, j);
        if (__shfl_sync(0xffffffffu, s.id, j) == s.id) g += v;
    }
    if (in && !good) report(a.err, MOE_DEVERR_BAD_EXPERT);
    if (!good) return;
    if constexpr (LOSS) g += loss_term(r, r.alpha == 0.f && r.inv_s == 0.f ? 0.f : expf(l - r.m), n);
    put1<BF16>(a.dl, at, g);
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
    for (int t = blockIdx.x * kBalWarps + (threadIdx.x >> 5); t < a.T; t += gridDim.x * kBalWarps) {
        const size_t row = static_cast<size_t>(t) * a.E;
        const bool on = !a.mask || a.mask[t];
        const Slot slot = slot_of(a, t, on);
        RowGrad r = {0.f, 0.f, 0.f, 0.f};
        float v[NV][4] = {};
        if (LOSS && on) {
            r = row_grad(warp_row<NV, VEC>(a.logits + row, a.E, f, v), gb, gc, a.err, lane == 0);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = loss_term(r, v[i][j], f[i][j]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) put4<BF16, VEC>(a.dl, row, 4 * lane + 128 * i, a.E, v[i]);
        if (on && a.dw) {
            __syncwarp();                          // the row is written before its entries are
            gate_entries<BF16, LOSS>(a, t, slot, r, unit);
        }
    }
}

// One block per row, V float4 per thread.
template <int V, bool VEC, bool BF16, bool LOSS>
__global__ void __launch_bounds__(kBigThreads) k_route_backward_big(RouteGrad a) {
    float gb = 0.f, gc = 0.f, unit = 0.f;
    if constexpr (LOSS) {
        const float n = static_cast<float>(max(a.counts[a.E], 1)), g = a.d_loss ? *a.d_loss : 1.f;
        unit = 1.f / (n * a.k);
        gb = g * a.balance * a.E / n;
        gc = g * a.z * 2.f / n;
    }
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = static_cast<size_t>(t) * a.E;
        const bool on = !a.mask || a.mask[t];
        const Slot slot = slot_of(a, t, on && threadIdx.x < 32);
        RowGrad r = {0.f, 0.f, 0.f, 0.f};
        float v[V][4] = {};
        if (LOSS && on) {
            r = row_grad(block_row<V, VEC>(a.logits + row, a.E, a.counts, unit, v), gb, gc, a.err, threadIdx.x == 0);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[4];                        // again, from L1
                share4<VEC>(a.counts, 4 * (threadIdx.x + kBigThreads * i), a.E, unit, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = loss_term(r, v[i][j], f[j]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) put4<BF16, VEC>(a.dl, row, 4 * (threadIdx.x + kBigThreads * i), a.E, v[i]);
        __syncthreads();                           // the row is written before its entries are
        if (on && a.dw && threadIdx.x < 32) gate_entries<BF16, LOSS>(a, t, slot, r, unit);
    }
}

// ------------------------------------------------------------------ launch
static int row_blocks(int T) {
    // (measured at 8192 x 512: 4 blocks an SM, two rows a warp, against 8)
    const long want = (static_cast<long>(T) + kBalWarps - 1) / kBalWarps, cap = num_sms() * 4L;
    return static_cast<int>(want < cap ? want : cap);
}
static int big_blocks(int T) {
    const int cap = num_sms();
    return T < cap ? T : cap;
}
// Blocks that count, up to 1024 experts: each with at least 4096 pairs.
static int count_parts(int T, int k) {
    const long n = (static_cast<long>(T) * k + 4095) / 4096;
    return static_cast<int>(n < 1 ? 1 : n < kParts ? n : kParts);
}

struct BalanceWs {
    unsigned *ticket;
    double2 *part;
    int32_t *counts;
};
static size_t carve(int T, int E, uint8_t *base, BalanceWs *out) {
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t *p = base ? base + at : nullptr;
        at += (n + 255) / 256 * 256;
        return p;
    };
    BalanceWs w;
    w.ticket = reinterpret_cast<unsigned *>(take(sizeof(unsigned)));
    w.part = reinterpret_cast<double2 *>(take((E <= 1024 ? row_blocks(T) : big_blocks(T)) * sizeof(double2)));
    w.counts = reinterpret_cast<int32_t *>(take(E <= 1024 ? kParts * (static_cast<size_t>(E) + 1) * 4 : 0));
    if (out) *out = w;
    return at;
}
size_t balance_ws_bytes(int T, int E) { return carve(T, E, nullptr, nullptr); }

// The instantiation for E <= 1024: float4 per lane, whether rows are aligned.
template <class F>
static void by_row(int E, F &&go) {
    using std::integral_constant;
    auto v = [&](auto nv) {
        if (E % 4 == 0) go(nv, std::true_type{});
        else go(nv, std::false_type{});
    };
    if (E <= 128) v(integral_constant<int, 1>{});
    else if (E <= 256) v(integral_constant<int, 2>{});
    else if (E <= 512) v(integral_constant<int, 4>{});
    else v(integral_constant<int, 8>{});
}
// And above: float4 per thread.
template <class F>
static void by_big_row(int E, F &&go) {
    using std::integral_constant;
    auto v = [&](auto nv) {
        if (E % 4 == 0) go(nv, std::true_type{});
        else go(nv, std::false_type{});
    };
    if (E <= 4096 * 2) v(integral_constant<int, 2>{});
    else v(integral_constant<int, 8>{});
}

int launch_balance_loss(const float *logits, const int32_t *ids, const uint8_t *mask, int T, int E, int k,
                        float balance_coef, float z_coef, int32_t *counts, float *loss, void *ws, unsigned *err,
                        cudaStream_t s) {
    BalanceWs w;
    carve(T, E, static_cast<uint8_t *>(ws), &w);
    const LossOut o = {E, balance_coef, z_coef, loss};
    if (E <= 1024 && T <= kOneRows) {
        by_row(E, [&](auto nv, auto vec) {
            k_balance_one<decltype(nv)::value, decltype(vec)::value>
                <<<1, kOneThreads, 0, s>>>(logits, ids, mask, T, E, k, counts, o, err);
        });
        count_launches(1);
        return cuda_status(cudaGetLastError(), "balance loss launch");
    }
    const int parts = E <= 1024 ? count_parts(T, k) : 1;
    if (E <= 1024) k_balance_parts<<<parts, kCountThreads, 0, s>>>(ids, mask, T, E, k, w.counts, w.ticket, err);
    else k_balance_slices<<<(E + kSlice - 1) / kSlice, kCountThreads, 0, s>>>(ids, mask, T, E, k, counts, w.ticket, err);
    if (E <= 1024)
        by_row(E, [&](auto nv, auto vec) {
            k_balance_rows<decltype(nv)::value, decltype(vec)::value><<<row_blocks(T), kBalThreads, 0, s>>>(
                logits, mask, T, E, k, w.counts, parts, counts, w.part, w.ticket, o, err);
        });
    else
        by_big_row(E, [&](auto nv, auto vec) {
            k_balance_rows_big<decltype(nv)::value, decltype(vec)::value><<<big_blocks(T), kBigThreads, 0, s>>>(
                logits, mask, T, E, k, counts, w.part, w.ticket, o, err);
        });
    count_launches(2);
    return cuda_status(cudaGetLastError(), "balance loss launch");
}

int launch_route_backward(const float *logits, const int32_t *ids, const float *w, const float *dw,
                          const uint8_t *mask, const int32_t *counts, const float *d_loss, int T, int E, int k,
                          float balance_coef, float z_coef, void *dl, int dl_dtype, unsigned *err, cudaStream_t s) {
    const RouteGrad a = {logits, ids, w, dw, mask, counts, d_loss, T, E, k, balance_coef, z_coef, dl, err};
    auto go = [&](auto bf16, auto with_loss) {
        constexpr bool B = decltype(bf16)::value, L = decltype(with_loss)::value;
        if (E <= 1024)
            by_row(E, [&](auto nv, auto vec) {
                k_route_backward<decltype(nv)::value, decltype(vec)::value, B, L><<<row_blocks(T), kBalThreads, 0, s>>>(a);
            });
        else
            by_big_row(E, [&](auto nv, auto vec) {
                k_route_backward_big<decltype(nv)::value, decltype(vec)::value, B, L>
                    <<<big_blocks(T), kBigThreads, 0, s>>>(a);
            });
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (dl_dtype == MOE_BF16) counts ? go(Yes{}, Yes{}) : go(Yes{}, No{});
    else counts ? go(No{}, Yes{}) : go(No{}, No{});
    count_launches(1);
    return cuda_status(cudaGetLastError(), "route backward launch");
}

}  // namespace moe

// Backward pass of the quantized experts on CUDA cores, fp32 throughout
// (MOE_MODE_GEMV): a few tokens, where reading the weights is the cost.
//
// Three passes over an expert's weights' codes, for up to kNT rows at a time:
//   1. g = Wg x, u = Wu x                       (dot products along a row)
//   2. q = Wd^T dy, then dg, du and the strip's share of <q, h>   (columns)
//   3. dxp = Wg^T dg + Wu^T du                                    (columns)
// and a gather of each token's rows, weighted by its gates.  Passes 2 and 3
// read a row's codes as they lie, four neighbouring blocks a row and eight
// rows a warp (64-byte pieces at 4 bits), each lane keeping the 32 sums of its
// block's columns in registers; lanes and warps are joined once at the end.
// A weight is decoded exactly (code minus offset is a small whole number) and
// once for all rows in flight.
#include "common.cuh"
#include "qdot.cuh"
#include "train/ffn_bwd.cuh"

namespace moe {

namespace {
constexpr int kBwThreads = 256;
constexpr int kBwWarps = kBwThreads / 32;
constexpr int kNT = 2;             // rows in flight
constexpr int kStrip = 128;        // columns of a pass 2 or 3 task: four blocks

struct GemvBwdWs {
    float *gu;      // [T*k + T, 2I]: g, u, then dg, du
    float *dwp;     // [T*k, I / kStrip]: shares of <q, h>
    float *dxp;     // [T*k + T, H]
    uint8_t *ok;    // [T*k]: the row's expert was computed
};

__host__ __device__ inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Four codes, one per byte of `q`, as whole numbers minus the offset: the
// float 1 + q/128 built from the code's bits, times 128, minus 128 + offset.
template <int BITS>
__device__ __forceinline__ void decode4(uint32_t q, float (&w)[4]) {
    q |= 0x80808080u;
    constexpr float off = 128.f + QT<BITS>::HALF;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = fmaf(magic(q, j), 128.f, -off);
}
// The four-value piece p (elements 4p .. 4p+3) of a block of 32.
template <int BITS>
__device__ __forceinline__ uint32_t block_piece(const uint32_t *w, int p) {
    if constexpr (BITS == 4) return (p < 4 ? w[p] : w[p - 4] >> 4) & 0x0F0F0F0Fu;
    else return (w[p & 1] >> (2 * (p >> 1))) & 0x03030303u;
}
}  // namespace

// Pass 1.  Task = (group, 16 weight rows): a warp takes two rows of both
// matrices, its lanes the row's chunks of 16 bytes.
template <int BITS>
__global__ void __launch_bounds__(kBwThreads) k_bwd_gateup(FfnBackward a, GemvBwdWs ws) {
    using Q = QT<BITS>;
    extern __shared__ float4 xs[];                 // [kNT][piece][chunk]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
    const int n_groups = n_act + (a.shared ? 1 : 0), row_blocks = a.I / 16;
    const int nch = a.H / Q::EPC, nsc = a.H / 32;
    const size_t rowb = static_cast<size_t>(a.H) * BITS / 8;
    for (int task = blockIdx.x; task < n_groups * row_blocks; task += gridDim.x) {
        const int g = task / row_blocks, rb = task - g * row_blocks;
        const BwdGroup G = bwd_group(a, g, n_act, threadIdx.x == 0 && rb == 0);
        if (G.n <= 0) continue;
        const BlobView bv = blob_view(G.blob, BITS, a.H, a.I);
        const int i0 = rb * 16 + warp * 2;
        if (rb == 0 && G.row0 >= 0)
            for (int r = threadIdx.x; r < G.n; r += kBwThreads) ws.ok[G.row0 + r] = 1;
        const size_t out0 = G.row0 >= 0 ? G.row0 : static_cast<size_t>(a.T) * a.k;
        for (int r0 = 0; r0 < G.n; r0 += kNT) {
            __syncthreads();
            for (int t = 0; t < kNT; ++t) {
                const bool in = r0 + t < G.n;
                const size_t tok = in ? bwd_token(a, G, r0 + t) : 0;
                for (int h4 = threadIdx.x; h4 < a.H / 4; h4 += kBwThreads)
                    xs[(t * Q::PPC + h4 % Q::PPC) * nch + h4 / Q::PPC] =
                        in ? bwd_load4(a.x, a.x_scales, a.x_dtype, tok, a.H, h4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            __syncthreads();
            float dot[4][kNT] = {};
            for (int cc = lane; cc < nch; cc += 32) {
                uint4 code[4];
                float d[4][Q::BPC];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const size_t i = i0 + (v >> 1);
                    code[v] = ldg_stream((v & 1 ? bv.cu : bv.cg) + i * rowb + static_cast<size_t>(cc) * 16);
                    load_scales<BITS>((v & 1 ? bv.su : bv.sg) + i * nsc, cc, true, d[v]);
                }
#pragma unroll
                for (int b = 0; b < Q::BPC; ++b) {
                    float acc[4][kNT] = {};
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        float4 x[kNT];
#pragma unroll
                        for (int t = 0; t < kNT; ++t) x[t] = xs[(t * Q::PPC + 8 * b + p) * nch + cc];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const uint32_t words[4] = {code[v].x, code[v].y, code[v].z, code[v].w};
                            float w[4];
                            decode4<BITS>(block_piece<BITS>(words + (BITS == 4 ? 0 : 2 * b), p), w);
#pragma unroll
                            for (int t = 0; t < kNT; ++t)
                                acc[v][t] = fmaf(w[3], x[t].w, fmaf(w[2], x[t].z,
                                            fmaf(w[1], x[t].y, fmaf(w[0], x[t].x, acc[v][t]))));
                        }
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v)
#pragma unroll
                        for (int t = 0; t < kNT; ++t) dot[v][t] = fmaf(d[v][b], acc[v][t], dot[v][t]);
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int t = 0; t < kNT; ++t) {
                    const float s = warp_sum(dot[v][t]);
                    if (lane == 0 && r0 + t < G.n)
                        ws.gu[(out0 + r0 + t) * 2 * a.I + (v & 1) * a.I + i0 + (v >> 1)] = s;
                }
        }
    }
}

// Passes 2 (DOWN: columns of Wd, along h) and 3 (columns of Wg, then Wu, along
// i).  Task = (group, strip of 128 columns).
template <int BITS, bool DOWN>
__global__ void __launch_bounds__(kBwThreads) k_bwd_columns(FfnBackward a, GemvBwdWs ws) {
    extern __shared__ float4 vmem[];
    const int M = DOWN ? a.H : 2 * a.I;            // rows summed over
    const int C = DOWN ? a.I : a.H;                // columns of the matrix
    float *vs = reinterpret_cast<float *>(vmem);   // [kNT][M]
    float *red = vs + kNT * M;                     // [warp][kNT][kStrip]
    __shared__ float wsum[kStrip * kNT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blk = lane & 3, sub = lane >> 2;
    const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
    const int n_groups = n_act + (a.shared ? 1 : 0), strips = C / kStrip;
    const size_t rowb = static_cast<size_t>(C) * BITS / 8;
    for (int task = blockIdx.x; task < n_groups * strips; task += gridDim.x) {
        const int g = task / strips, st = task - g * strips;
        const BwdGroup G = bwd_group(a, g, n_act, false);
        if (G.n <= 0) continue;
        const BlobView bv = blob_view(G.blob, BITS, a.H, a.I);
        const size_t out0 = G.row0 >= 0 ? G.row0 : static_cast<size_t>(a.T) * a.k;
        for (int r0 = 0; r0 < G.n; r0 += kNT) {
            __syncthreads();
            for (int t = 0; t < kNT; ++t) {
                const bool in = r0 + t < G.n;
                const size_t tok = in && DOWN ? bwd_token(a, G, r0 + t) : 0;
                for (int m4 = threadIdx.x; m4 < M / 4; m4 += kBwThreads) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in)
                        v = DOWN ? bwd_load4(a.dy, nullptr, a.dy_dtype, tok, a.H, m4)
                                 : load4(ws.gu + (out0 + r0 + t) * 2 * a.I + 4 * m4);
                    reinterpret_cast<float4 *>(vs + t * M)[m4] = v;
                }
            }
            __syncthreads();
            float acc[kNT][32] = {};
#pragma unroll 2
            for (int m = 8 * warp + sub; m < M; m += 8 * kBwWarps) {
                const uint8_t *codes;
                const __half *scl;
                int row = m;
                if (DOWN) codes = bv.cd, scl = bv.sd;
                else if (m < a.I) codes = bv.cg, scl = bv.sg;
                else codes = bv.cu, scl = bv.su, row = m - a.I;
                const uint8_t *src = codes + row * rowb + (st * kStrip + 32 * blk) * BITS / 8;
                uint32_t w[BITS];
                if constexpr (BITS == 4) {
                    const uint4 c = *reinterpret_cast<const uint4 *>(src);
                    w[0] = c.x, w[1] = c.y, w[2] = c.z, w[3] = c.w;
                } else {
                    const uint2 c = *reinterpret_cast<const uint2 *>(src);
                    w[0] = c.x, w[1] = c.y;
                }
                const float d = __half2float(scl[static_cast<size_t>(row) * (C / 32) + st * 4 + blk]);
                float vd[kNT];
#pragma unroll
                for (int t = 0; t < kNT; ++t) vd[t] = d * vs[t * M + m];
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    float q[4];
                    decode4<BITS>(block_piece<BITS>(w, p), q);
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t][4 * p + j] = fmaf(vd[t], q[j], acc[t][4 * p + j]);
                }
            }
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float v = acc[t][j];
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    if (sub == (j & 7)) red[(warp * kNT + t) * kStrip + 32 * blk + j] = v;
                }
            __syncthreads();
            // one thread per (row in flight, column): kNT * kStrip == kBwThreads
            const int t = threadIdx.x / kStrip, c = threadIdx.x % kStrip;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kBwWarps; ++w) v += red[(w * kNT + t) * kStrip + c];
            const bool in = r0 + t < G.n;
            if constexpr (DOWN) {
                float share = 0.f;
                if (in) {
                    float *gu = ws.gu + (out0 + r0 + t) * 2 * a.I + st * kStrip + c;
                    const float gv = gu[0], uv = gu[a.I], s = 1.f / (1.f + expf(-gv)), act = gv * s;
                    gu[0] = v * uv * fmaf(act, 1.f - s, s);
                    gu[a.I] = v * act;
                    share = v * act * uv;
                }
                share = warp_sum(share);
                if (lane == 0) wsum[warp] = share;
                __syncthreads();
                if (c == 0 && in && G.row0 >= 0) {
                    float sum = 0.f;
                    for (int w = 0; w < kStrip / 32; ++w) sum += wsum[t * (kStrip / 32) + w];
                    ws.dwp[(out0 + r0 + t) * strips + st] = sum;
                }
            } else if (in) {
                ws.dxp[(out0 + r0 + t) * a.H + st * kStrip + c] = v;
            }
        }
    }
}

// dx[t] = sum_j w[t,j] dxp[row(t,j)] + dxp[shared row t], in slot order, and
// d_topk_w[t,j] = the sum of its row's shares; with `scale`, times the token's
// sx sd and sx sx sd.  One block per token.
__global__ void __launch_bounds__(kBwThreads) k_bwd_gather(FfnBackward a, const float *__restrict__ dxp,
                                                           const float *__restrict__ dwp, int shares,
                                                           const uint8_t *__restrict__ ok,
                                                           const float2 *__restrict__ scale) {
    const size_t t = blockIdx.x;
    const float2 sc = scale ? scale[t] : make_float2(1.f, 1.f);
    __shared__ int row_s[32];
    __shared__ float w_s[32];
    const int j = threadIdx.x;
    if (j < a.k) {
        int row = a.perm_dst[t * a.k + j];
        if (row < 0 || row >= a.T * a.k) {
            report(a.err, MOE_DEVERR_BAD_ROW);
            row = -1;
        } else if (!ok[row]) {
            row = -1;
        }
        row_s[j] = row;
        w_s[j] = a.topk_w[t * a.k + j];
        float sum = 0.f;
        if (row >= 0)
            for (int i = 0; i < shares; ++i) sum += dwp[static_cast<size_t>(row) * shares + i];
        a.d_topk_w[t * a.k + j] = sum * sc.x * sc.y * sc.x;
    }
    __syncthreads();
    for (int h4 = threadIdx.x; h4 < a.H / 4; h4 += kBwThreads) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < a.k; ++i) {
            if (row_s[i] < 0) continue;
            const float4 v = load4(dxp + static_cast<size_t>(row_s[i]) * a.H + 4 * h4);
            acc.x = fmaf(w_s[i], v.x, acc.x);
            acc.y = fmaf(w_s[i], v.y, acc.y);
            acc.z = fmaf(w_s[i], v.z, acc.z);
            acc.w = fmaf(w_s[i], v.w, acc.w);
        }
        if (a.shared) {
            const float4 v = load4(dxp + (static_cast<size_t>(a.T) * a.k + t) * a.H + 4 * h4);
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        acc.x = acc.x * sc.x * sc.y, acc.y = acc.y * sc.x * sc.y;
        acc.z = acc.z * sc.x * sc.y, acc.w = acc.w * sc.x * sc.y;
        const size_t at = t * (a.H / 4) + h4;
        if (a.dx_dtype == MOE_BF16) {
            __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
            uint2 u;
            u.x = *reinterpret_cast<uint32_t *>(&lo);
            u.y = *reinterpret_cast<uint32_t *>(&hi);
            static_cast<uint2 *>(a.dx)[at] = u;
        } else {
            static_cast<float4 *>(a.dx)[at] = acc;
        }
    }
}

// ------------------------------------------------------------------ launch
static size_t carve(int T, int k, int H, int I, uint8_t *base, GemvBwdWs *out) {
    const size_t rows = static_cast<size_t>(T) * k, all = rows + T;
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t *p = base ? base + at : nullptr;
        at += align256(n);
        return p;
    };
    GemvBwdWs w;
    w.gu = reinterpret_cast<float *>(take(all * 2 * I * 4));
    w.dwp = reinterpret_cast<float *>(take(rows * (I / kStrip) * 4));
    w.dxp = reinterpret_cast<float *>(take(all * H * 4));
    w.ok = take(rows);
    if (out) *out = w;
    return at;
}

size_t ffn_backward_gemv_ws_bytes(int T, int k, int H, int I) { return carve(T, k, H, I, nullptr, nullptr); }

template <int BITS>
static int launch_gemv_bwd(const FfnBackward &a, const GemvBwdWs &w, cudaStream_t s) {
    const long rows = static_cast<long>(a.T) * a.k, groups = (rows < a.E ? rows : a.E) + (a.shared ? 1 : 0);
    const long cap = num_sms() * 8L;
    auto grid = [&](long per) { return groups * per < cap ? groups * per : cap; };
    const int sm1 = kNT * a.H * 4;
    auto columns = [&](int m) { return (kNT * m + kBwWarps * kNT * kStrip) * 4; };
    int rc = cuda_status(cudaFuncSetAttribute(k_bwd_gateup<BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm1),
                         "backward smem attribute");
    if (rc) return rc;
    k_bwd_gateup<BITS><<<grid(a.I / 16), kBwThreads, sm1, s>>>(a, w);
    rc = cuda_status(cudaFuncSetAttribute(k_bwd_columns<BITS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          columns(a.H)),
                     "backward smem attribute");
    if (rc) return rc;
    k_bwd_columns<BITS, true><<<grid(a.I / kStrip), kBwThreads, columns(a.H), s>>>(a, w);
    rc = cuda_status(cudaFuncSetAttribute(k_bwd_columns<BITS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          columns(2 * a.I)),
                     "backward smem attribute");
    if (rc) return rc;
    k_bwd_columns<BITS, false><<<grid(a.H / kStrip), kBwThreads, columns(2 * a.I), s>>>(a, w);
    count_launches(3);
    rc = cuda_status(cudaGetLastError(), "expert backward launch");
    if (rc) return rc;
    return launch_ffn_backward_gather(a, w.dxp, w.dwp, a.I / kStrip, w.ok, nullptr, s);
}

int launch_ffn_backward_gather(const FfnBackward &a, const float *dxp, const float *dwp, int shares,
                               const uint8_t *ok, const float2 *scale, cudaStream_t s) {
    k_bwd_gather<<<a.T, kBwThreads, 0, s>>>(a, dxp, dwp, shares, ok, scale);
    count_launches(1);
    return cuda_status(cudaGetLastError(), "expert backward gather launch");
}

int launch_ffn_backward_gemv(const FfnBackward &a, void *ws, cudaStream_t s) {
    GemvBwdWs w;
    carve(a.T, a.k, a.H, a.I, static_cast<uint8_t *>(ws), &w);
    int rc = cuda_status(cudaMemsetAsync(w.ok, 0, static_cast<size_t>(a.T) * a.k, s), "row flags memset");
    if (rc) return rc;
    return a.bits == 4 ? launch_gemv_bwd<4>(a, w, s) : launch_gemv_bwd<2>(a, w, s);
}

}  // namespace moe

// Backward pass of the quantized experts on CUDA cores, fp32 throughout
// (MOE_MODE_GEMV): a few tokens, where reading the weights is the cost.
//
// Two passes over an expert's weights' codes, for one or two rows at a time:
//   1. g = Wg x, u = Wu x (dot products along a row) and q = Wd^T dy (columns),
//      tasks of one launch, since neither needs the other
//   2. dg, du from them, then dxp = Wg^T dg + Wu^T du             (columns)
// and a gather of each token's rows, weighted by its gates.  Columns are summed
// over rows of codes as they lie, two (q) or four neighbouring blocks a row,
// each lane keeping the 32 sums of its block's columns in registers; lanes and
// warps are joined once at the end.  A weight is decoded exactly (code minus
// offset is a small whole number) and once for the rows in flight.
//
// At one token this is a chain of memory latencies: three kernels, each of
// which may start while the one before it runs (programmatic dependent launch).
// 28.5 us as a graph at one token, 512 experts of 2048 x 512, top-10 (3.0 at
// the bandwidth); with one row in flight in every task, four of its weight rows
// loaded at once in the column sums and halves exchanged in their join, the
// first kernel takes 12.7 us for 16.7 and the second 16.1 for 19.8.  Loads a
// step ahead, eight at once, or three blocks an SM were slower.  The shared
// expert's rows come first and split over tasks: left to one task each, they
// were the tail at 16 tokens.
#include "common.cuh"
#include "qdot.cuh"
#include "train/ffn_bwd.cuh"
#include "train/launch.cuh"

namespace moe {

namespace {
constexpr int kBwThreads = 256;
constexpr int kNT = 2;             // rows in flight
// Column sums: columns of a task (64 of Wd, which has the fewest and the longest
// sums, 128 of Wg and Wu).
template <bool DOWN> struct Strip {
    static constexpr int COLS = DOWN ? 64 : 128, BLOCKS = COLS / 32;
    static constexpr int SUBS = 32 / BLOCKS;       // weight rows a warp reads at once
};
constexpr int kBwWarps = kBwThreads / 32;

struct GemvBwdWs {
    float *guq;     // [T*k + T, 3I]: g, u, q
    float *dwp;     // [T*k]: <q, h>
    float *dxp;     // [T*k + T, H]
    uint8_t *ok;    // [T*k + T]: the row was computed
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

// A task's group and rows.  The shared expert's tasks come first, kNT rows
// each; a routed expert's take all its rows.
struct Rows {
    BwdGroup G;
    int r0, r1;
};
__device__ __forceinline__ Rows task_rows(const FfnBackward &a, int item, int n_act, int chunks, bool say) {
    if (item < chunks) {
        BwdGroup G = {a.shared, a.T, -1};
        return {G, item * kNT, min(a.T, (item + 1) * kNT)};
    }
    const BwdGroup G = bwd_group(a, item - chunks, n_act, say);
    return {G, 0, G.n};
}
}  // namespace

// Pass 1, gate and up: 16 weight rows of both matrices, a warp two of each, its
// lanes the row's chunks of 16 bytes.  The dot products of NT rows of x (xs:
// [NT][piece][chunk]); out(row in flight, matrix, weight row, sum) on lane 0.
template <int BITS, int NT, class Out>
__device__ __forceinline__ void gate_up_dots(const BlobView &bv, const float4 *xs, int H, int i0, Out out) {
    using Q = QT<BITS>;
    const int lane = threadIdx.x & 31, nch = H / Q::EPC, nsc = H / 32;
    const size_t rowb = static_cast<size_t>(H) * BITS / 8;
    float dot[4][NT] = {};
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
            float acc[4][NT] = {};
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                float4 x[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t] = xs[(t * Q::PPC + 8 * b + p) * nch + cc];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t words[4] = {code[v].x, code[v].y, code[v].z, code[v].w};
                    float w[4];
                    decode4<BITS>(block_piece<BITS>(words + (BITS == 4 ? 0 : 2 * b), p), w);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[v][t] = fmaf(w[3], x[t].w, fmaf(w[2], x[t].z,
                                    fmaf(w[1], x[t].y, fmaf(w[0], x[t].x, acc[v][t]))));
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int t = 0; t < NT; ++t) dot[v][t] = fmaf(d[v][b], acc[v][t], dot[v][t]);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float s = warp_sum(dot[v][t]);
            if (lane == 0) out(t, v & 1, i0 + (v >> 1), s);
        }
}
template <int BITS>
__device__ __forceinline__ void gate_up(const FfnBackward &a, const GemvBwdWs &ws, const Rows &R, int rb, float4 *xs) {
    using Q = QT<BITS>;
    const int nch = a.H / Q::EPC, i0 = rb * 16 + (threadIdx.x >> 5) * 2;
    const BwdGroup G = R.G;
    const BlobView bv = blob_view(G.blob, BITS, a.H, a.I);
    const size_t out0 = G.row0 >= 0 ? G.row0 : static_cast<size_t>(a.T) * a.k;
    for (int r0 = R.r0; r0 < R.r1; r0 += kNT) {
        const int nt = min(kNT, R.r1 - r0);
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const size_t tok = bwd_token(a, G, r0 + t);
            for (int h4 = threadIdx.x; h4 < a.H / 4; h4 += kBwThreads)
                xs[(t * Q::PPC + h4 % Q::PPC) * nch + h4 / Q::PPC] = bwd_load4(a.x, a.x_scales, a.x_dtype, tok, a.H, h4);
        }
        __syncthreads();
        auto out = [&](int t, int mat, int i, float v) { ws.guq[(out0 + r0 + t) * 3 * a.I + mat * a.I + i] = v; };
        if (nt == 1) gate_up_dots<BITS, 1>(bv, xs, a.H, i0, out);
        else gate_up_dots<BITS, kNT>(bv, xs, a.H, i0, out);
    }
}

// The sums of NT rows of v (shared memory, M values each) over a warp's weight
// rows, for the 32 columns of the lane's block.
template <int BITS, bool DOWN, int NT>
__device__ __forceinline__ void column_sums(const BlobView &bv, const float *vs, int M, int C, int I, int col0,
                                            float (&acc)[kNT][32]) {
    using S = Strip<DOWN>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blk = lane % S::BLOCKS, sub = lane / S::BLOCKS;
    const size_t rowb = static_cast<size_t>(C) * BITS / 8;
    const size_t cofs = static_cast<size_t>(col0 / 32 + blk) * 4 * BITS;
    constexpr int STEP = S::SUBS * kBwWarps;
    constexpr int kLoads = NT == 1 ? 4 : 2;        // weight rows a lane has in flight
    for (int m0 = S::SUBS * warp + sub; m0 < M; m0 += kLoads * STEP) {
        uint32_t w[kLoads][BITS];
        float d[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int m = m0 + u * STEP;
            d[u] = 0.f;
#pragma unroll
            for (int x = 0; x < BITS; ++x) w[u][x] = 0;
            if (m >= M) continue;
            const uint8_t *codes = DOWN ? bv.cd : m < I ? bv.cg : bv.cu;
            const __half *scl = DOWN ? bv.sd : m < I ? bv.sg : bv.su;
            const size_t row = DOWN || m < I ? m : m - I;
            if constexpr (BITS == 4) {
                const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes + row * rowb + cofs));
                w[u][0] = c.x, w[u][1] = c.y, w[u][2] = c.z, w[u][3] = c.w;
            } else {
                const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + row * rowb + cofs));
                w[u][0] = c.x, w[u][1] = c.y;
            }
            d[u] = __half2float(scl[row * (C / 32) + col0 / 32 + blk]);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int m = min(m0 + u * STEP, M - 1);           // beyond M: the step is zero
            float vd[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) vd[t] = m0 + u * STEP < M ? d[u] * vs[t * M + m] : 0.f;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                float q[4];
                decode4<BITS>(block_piece<BITS>(w[u], p), q);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][4 * p + j] = fmaf(vd[t], q[j], acc[t][4 * p + j]);
            }
        }
    }
}

// Column sums of the rows staged in vs, joined over the block: out(t, column,
// sum) for each row in flight and column of the strip.
template <int BITS, bool DOWN, class Out>
__device__ __forceinline__ void columns(const BlobView &bv, const float *vs, float *red, int nt, int M, int C, int I,
                                        int col0, Out out) {
    using S = Strip<DOWN>;                         // red: [warp][kNT][COLS]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blk = lane % S::BLOCKS;
    float acc[kNT][32] = {};
    if (nt == 1) column_sums<BITS, DOWN, 1>(bv, vs, M, C, I, col0, acc);
    else column_sums<BITS, DOWN, kNT>(bv, vs, M, C, I, col0, acc);
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
        if (t >= nt) break;
        // the lanes of a block exchange halves: each step halves the columns a lane holds
#pragma unroll
        for (int o = 16; o >= S::BLOCKS; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int e = 0; e < o; ++e) {
                const float give = up ? acc[t][e] : acc[t][e + o], keep = up ? acc[t][e + o] : acc[t][e];
                acc[t][e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
#pragma unroll
        for (int e = 0; e < S::BLOCKS; ++e)
            red[(warp * kNT + t) * S::COLS + 32 * blk + (lane & ~(S::BLOCKS - 1)) + e] = acc[t][e];
    }
    __syncthreads();
    const int t = threadIdx.x / S::COLS, c = threadIdx.x % S::COLS;
    if (t < nt) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kBwWarps; ++w) v += red[(w * kNT + t) * S::COLS + c];
        out(t, c, v);
    }
}

// Pass 1.  Tasks: first (rows, strip of Wd's columns), the longer ones, then
// (rows, 16 rows of Wg and Wu).
template <int BITS>
__global__ void __launch_bounds__(kBwThreads) k_bwd_first(FfnBackward a, GemvBwdWs ws) {
    using S = Strip<true>;
    extern __shared__ float4 mem[];                // x, or dy [kNT][H] and the joining sums
    const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
    const int chunks = a.shared ? (a.T + kNT - 1) / kNT : 0;
    const int n_items = n_act + chunks, strips = a.I / S::COLS, row_blocks = a.I / 16;
    pdl_next();
    for (long r = static_cast<long>(blockIdx.x) * kBwThreads + threadIdx.x; r < static_cast<long>(a.T) * (a.k + 1);
         r += static_cast<long>(gridDim.x) * kBwThreads)
        ws.ok[r] = 0;                              // pass 2 marks the rows it computes
    const long n_q = static_cast<long>(n_items) * strips, n_all = n_q + static_cast<long>(n_items) * row_blocks;
    for (long task = blockIdx.x; task < n_all; task += gridDim.x) {
        const bool down = task < n_q;
        const long v = down ? task : task - n_q;
        const int per = down ? strips : row_blocks;
        const int item = static_cast<int>(v / per), part = static_cast<int>(v - static_cast<long>(item) * per);
        const Rows R = task_rows(a, item, n_act, chunks, threadIdx.x == 0 && down && part == 0);
        if (R.G.n <= 0) continue;
        if (!down) {
            gate_up<BITS>(a, ws, R, part, mem);
            continue;
        }
        const BlobView bv = blob_view(R.G.blob, BITS, a.H, a.I);
        const size_t out0 = R.G.row0 >= 0 ? R.G.row0 : static_cast<size_t>(a.T) * a.k;
        float *vs = reinterpret_cast<float *>(mem);
        for (int r0 = R.r0; r0 < R.r1; r0 += kNT) {
            const int nt = min(kNT, R.r1 - r0);
            __syncthreads();
            for (int t = 0; t < nt; ++t) {
                const size_t tok = bwd_token(a, R.G, r0 + t);
                for (int h4 = threadIdx.x; h4 < a.H / 4; h4 += kBwThreads)
                    reinterpret_cast<float4 *>(vs + t * a.H)[h4] = bwd_load4(a.dy, nullptr, a.dy_dtype, tok, a.H, h4);
            }
            __syncthreads();
            columns<BITS, true>(bv, vs, vs + kNT * a.H, nt, a.H, a.I, a.I, part * S::COLS, [&](int t, int c, float q) {
                ws.guq[(out0 + r0 + t) * 3 * a.I + 2 * a.I + part * S::COLS + c] = q;
            });
        }
    }
}

// Pass 2.  Task = (rows, strip of Wg's and Wu's columns).
template <int BITS>
__global__ void __launch_bounds__(kBwThreads) k_bwd_second(FfnBackward a, GemvBwdWs ws) {
    using S = Strip<false>;
    extern __shared__ float4 mem[];
    float *vs = reinterpret_cast<float *>(mem);    // [kNT][2I]: dg, du
    __shared__ float wsum[kBwWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, M = 2 * a.I;
    const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
    const int chunks = a.shared ? (a.T + kNT - 1) / kNT : 0;
    const int n_items = n_act + chunks, strips = a.H / S::COLS;
    pdl_next();
    pdl_wait();
    for (long task = blockIdx.x; task < static_cast<long>(n_items) * strips; task += gridDim.x) {
        const int item = static_cast<int>(task / strips), st = static_cast<int>(task - static_cast<long>(item) * strips);
        const Rows R = task_rows(a, item, n_act, chunks, false);
        const BwdGroup G = R.G;
        if (G.n <= 0) continue;
        const BlobView bv = blob_view(G.blob, BITS, a.H, a.I);
        const size_t out0 = G.row0 >= 0 ? G.row0 : static_cast<size_t>(a.T) * a.k;
        for (int r0 = R.r0; r0 < R.r1; r0 += kNT) {
            const int nt = min(kNT, R.r1 - r0);
            for (int t = 0; t < nt; ++t) {
                const float *guq = ws.guq + (out0 + r0 + t) * 3 * a.I;
                __syncthreads();
                float share = 0.f;
                for (int i = threadIdx.x; i < a.I; i += kBwThreads) {
                    const float g = guq[i], u = guq[a.I + i], q = guq[2 * a.I + i];
                    const float sg = 1.f / (1.f + expf(-g)), act = g * sg;
                    vs[t * M + i] = q * u * fmaf(act, 1.f - sg, sg);
                    vs[t * M + a.I + i] = q * act;
                    share = fmaf(q * act, u, share);
                }
                if (st == 0 && G.row0 >= 0) {      // the same for the whole block
                    share = warp_sum(share);
                    if (lane == 0) wsum[warp] = share;
                    __syncthreads();
                    if (threadIdx.x == 0) {
                        float sum = 0.f;
#pragma unroll
                        for (int w = 0; w < kBwWarps; ++w) sum += wsum[w];
                        ws.dwp[out0 + r0 + t] = sum;
                        ws.ok[out0 + r0 + t] = 1;
                    }
                } else if (st == 0 && threadIdx.x == 0) {
                    ws.ok[out0 + r0 + t] = 1;
                }
            }
            __syncthreads();
            columns<BITS, false>(bv, vs, vs + kNT * M, nt, M, a.H, a.I, st * S::COLS, [&](int t, int c, float v) {
                ws.dxp[(out0 + r0 + t) * a.H + st * S::COLS + c] = v;
            });
        }
    }
}

// dx[t] = sum_j w[t,j] dxp[row(t,j)] + dxp[shared row t], in slot order, and
// d_topk_w[t,j] = the sum of its row's shares, over the rows that were computed; with `scale`, times the token's
// sx sd / r and sx sx sd.  One block per token.
__global__ void __launch_bounds__(kBwThreads) k_bwd_gather(FfnBackward a, const float *__restrict__ dxp,
                                                           const float *__restrict__ dwp, int shares,
                                                           const uint8_t *__restrict__ ok,
                                                           const float4 *__restrict__ scale) {
    const size_t t = blockIdx.x;
    pdl_wait();
    const float4 sc = scale ? scale[t] : make_float4(1.f, 1.f, 1.f, 1.f);
    const size_t own = static_cast<size_t>(a.T) * a.k + t;     // the shared expert's row
    __shared__ int row_s[32];
    __shared__ float w_s[32];
    // what a column needs once, at its end, is read from shared memory there: in
    // registers it leaves room for four blocks an SM instead of five (156 us for
    // 144 at 8192 x 2048, top-10)
    __shared__ float end_s[4];                     // 1 where the shared row was computed; 1/r, sx, sd
    const volatile float *end = end_s;
    if (threadIdx.x == 32) {
        end_s[0] = a.shared && ok[own] ? 1.f : 0.f;
        end_s[1] = sc.w, end_s[2] = sc.x, end_s[3] = sc.y;
    }
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
        // eight slots' rows in flight, added in slot order
        for (int i0 = 0; i0 < a.k; i0 += 8) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = i0 + u < a.k && row_s[i0 + u] >= 0 ? load4(dxp + static_cast<size_t>(row_s[i0 + u]) * a.H + 4 * h4)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (i0 + u >= a.k || row_s[i0 + u] < 0) continue;
                const float w = w_s[i0 + u];
                acc.x = fmaf(w, v[u].x, acc.x);
                acc.y = fmaf(w, v[u].y, acc.y);
                acc.z = fmaf(w, v[u].z, acc.z);
                acc.w = fmaf(w, v[u].w, acc.w);
            }
        }
        if (end[0] != 0.f) {
            const float4 v = load4(dxp + own * a.H + 4 * h4);
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float f = end[i];
            acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
        }
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
    w.guq = reinterpret_cast<float *>(take(all * 3 * I * 4));
    w.dwp = reinterpret_cast<float *>(take(rows * 4));
    w.dxp = reinterpret_cast<float *>(take(all * H * 4));
    w.ok = take(all);
    if (out) *out = w;
    return at;
}

size_t ffn_backward_gemv_ws_bytes(int T, int k, int H, int I) { return carve(T, k, H, I, nullptr, nullptr); }

template <int BITS>
static int launch_gemv_bwd(const FfnBackward &a, const GemvBwdWs &w, cudaStream_t s) {
    const long rows = static_cast<long>(a.T) * a.k;
    const long items = (rows < a.E ? rows : a.E) + (a.shared ? (a.T + kNT - 1) / kNT : 0);
    const long cap = num_sms() * 8L;
    auto grid = [&](long per) { return items * per < cap ? items * per : cap; };
    using D = Strip<true>;
    using U = Strip<false>;
    static_assert(kNT * U::COLS <= kBwThreads, "a thread per row in flight and column");
    const int sm1 = (kNT * a.H + kBwWarps * kNT * D::COLS) * 4, sm2 = (kNT * 2 * a.I + kBwWarps * kNT * U::COLS) * 4;
    auto smem = [](const void *f, int n) {
        return cuda_status(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, n), "backward smem attribute");
    };
    int rc = smem(reinterpret_cast<const void *>(k_bwd_first<BITS>), sm1);
    if (!rc) rc = smem(reinterpret_cast<const void *>(k_bwd_second<BITS>), sm2);
    if (rc) return rc;
    k_bwd_first<BITS><<<grid(a.I / D::COLS + a.I / 16), kBwThreads, sm1, s>>>(a, w);
    count_launches(1);
    rc = cuda_status(cudaGetLastError(), "expert backward launch");
    if (rc) return rc;
    rc = cuda_status(launch_after(k_bwd_second<BITS>, dim3(grid(a.H / U::COLS)), kBwThreads, sm2, s, a, w),
                     "expert backward launch");
    if (rc) return rc;
    count_launches(1);
    return launch_ffn_backward_gather(a, w.dxp, w.dwp, 1, w.ok, nullptr, s);
}

int launch_ffn_backward_gather(const FfnBackward &a, const float *dxp, const float *dwp, int shares,
                               const uint8_t *ok, const float4 *scale, cudaStream_t s) {
    const int rc = cuda_status(launch_after(k_bwd_gather, dim3(a.T), kBwThreads, 0, s, a, dxp, dwp, shares, ok, scale),
                               "expert backward gather launch");
    if (!rc) count_launches(1);
    return rc;
}

int launch_ffn_backward_gemv(const FfnBackward &a, void *ws, cudaStream_t s) {
    GemvBwdWs w;
    carve(a.T, a.k, a.H, a.I, static_cast<uint8_t *>(ws), &w);
    return a.bits == 4 ? launch_gemv_bwd<4>(a, w, s) : launch_gemv_bwd<2>(a, w, s);
}

}  // namespace moe

// Backward pass of a bf16 router on the 5th-generation tensor cores:
//   dx^T [H, T]  = W^T dl^T (+ dx_in)     K = E
//   dW^T [H, E]  = x^T dl                 K = T, split over blocks
//   db   [E]     = sum_t dl               read beside the products
// in one persistent launch, and a second one that adds the splits.
//
// Both products put h on the M side (the accumulator's lanes), where W and x
// are MN-major as they lie, so that neighbouring lanes read dx_in and write dx
// and dW at neighbouring addresses.  The N side is dl: tokens (K-major) for
// dx, experts (MN-major) for dW.  All operands come by TMA, 64 of K a stage;
// zeros outside the arrays make ragged T, H and E exact.
//
// Bound: the bytes (dx_in in fp32 is the largest part), then the tensor cores.
// K = T is split so that there is a unit of dW for nearly every SM: at 8192
// tokens, 512 experts and 2048 hidden the 64 tiles of dW alone would take 128
// k-steps each on 64 SMs.
//
// Measured at 8192 x 512 x 2048: 56 us and 5 for the second launch (22.4 at the
// bandwidth); a stage of 32 KB takes 530 cycles, 61 bytes a cycle into an SM,
// where its MMAs take 256, and the epilogue's fp32 dx_in comes on top.
//
// Roles: warp 0 TMA, warp 1 MMA, warps 2 on epilogue (they sum their block's
// rows of dl for db before their first tile).  Waits are bounded.
#include "common.cuh"
#include "kernels.h"
#include "train/tma.cuh"
#include "train/train.h"
#include "train/umma.cuh"

namespace moe {
using namespace sm100;

namespace {
constexpr int kRM = 128, kRK = 64;
constexpr int kRN = 128;                           // N of a tile: tokens (dx), experts (dW)
constexpr int kRStages = 6, kRAcc = 4;
constexpr int kREpi = 16;
constexpr int kRThreads = 32 * (2 + kREpi);
constexpr uint32_t kRA = kRM * kRK * 2, kRStage = kRA + kRN * kRK * 2;
constexpr uint32_t kROffBar = kRStages * kRStage;
constexpr uint32_t kRSmem = kROffBar + 24 * 8 + 16 + 1024;
static_assert(2 * kRStages + 2 * kRAcc + 1 <= 24 && kRAcc * kRN <= 512, "barriers and TMEM columns");
constexpr int kBiasRows = 64;                      // rows of dl a block sums at least

struct RouterArgs {
    const __nv_bfloat16 *dl;
    const float *dx_in;
    void *dx, *dw;
    float *db, *dw_part, *db_part;                 // [splits, E, H], [bias_parts, E]
    int T, H, E, dx_bf16;
    int mt, et, splits, per_split;                 // tiles of h and e; k-steps of a split
    int units_w, units;                            // dW's units come first: they are the longer ones
    int bias_parts;
    unsigned *err;
    unsigned long long limit_ns;                   // of a pipeline wait
};

struct Unit {
    bool w;            // dW (else dx)
    int m0, n0, N;
    int k0, nk;        // first k-step, k-steps
    int split;
};
__device__ __forceinline__ Unit unit_of(const RouterArgs &a, int u) {
    Unit j;
    j.w = u < a.units_w;
    const int v = j.w ? u : u - a.units_w, r = v / a.mt;
    j.m0 = (v - r * a.mt) * kRM;
    if (j.w) {
        j.split = r / a.et;
        j.n0 = (r - j.split * a.et) * kRN;
        j.N = min(kRN, (a.E - j.n0 + 15) & ~15);
        j.k0 = j.split * a.per_split;
        j.nk = min(a.per_split, (a.T + kRK - 1) / kRK - j.k0);
    } else {
        j.split = 0;
        j.n0 = r * kRN;
        j.N = min(kRN, (a.T - j.n0 + 15) & ~15);
        j.k0 = 0;
        j.nk = (a.E + kRK - 1) / kRK;
    }
    return j;
}
}  // namespace

__global__ void __launch_bounds__(kRThreads, 1) k_router_bwd(const RouterArgs a, const __grid_constant__ CUtensorMap map_w,
                                                             const __grid_constant__ CUtensorMap map_x,
                                                             const __grid_constant__ CUtensorMap map_dl_k,
                                                             const __grid_constant__ CUtensorMap map_dl_mn) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kROffBar);
    uint64_t *full = bars, *empty = bars + kRStages, *accF = bars + 2 * kRStages, *accE = accF + kRAcc, *drain = accE + kRAcc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 24);
    volatile int &abort_s = *(reinterpret_cast<int *>(bars + 24) + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < kRStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kRAcc; ++i) {
            mbar_init(accF + i, 1);
            mbar_init(accE + i, kREpi);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        fence_proxy_async();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int bid = blockIdx.x, grid = gridDim.x;
    auto wait = [&](uint64_t *bar, uint32_t parity) {         // bounded; the same answer on every lane
        const bool ok = mbar_wait_ns(bar, parity, a.limit_ns, &abort_s);
        if (!ok && !abort_s) {
            report(a.err, MOE_DEVERR_TIMEOUT);
            abort_s = 1;
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };

    if (warp == 0) {
        // -------------------------------------------------------------- TMA
        const uint32_t on = elect_one();
        int st = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int u = bid; u < a.units && ok; u += grid) {
            const Unit j = unit_of(a, u);
            for (int s = 0; s < j.nk; ++s) {
                if (!(ok = wait(empty + st, phase))) break;
                const uint32_t sa = smem_addr(smem + st * kRStage), sb = sa + kRA;
                const int k = (j.k0 + s) * kRK;
                expect_tx_on(on, full + st, kRStage);
                // two boxes of 64 h; dl: one box of 128 tokens, or two of 64 experts
                if (j.w) {
                    tma_load_on(on, sa, &map_x, j.m0, k, full + st);
                    tma_load_on(on, sa + 8192, &map_x, j.m0 + 64, k, full + st);
                    tma_load_on(on, sb, &map_dl_mn, j.n0, k, full + st);
                    tma_load_on(on, sb + 8192, &map_dl_mn, j.n0 + 64, k, full + st);
                } else {
                    tma_load_on(on, sa, &map_w, j.m0, k, full + st);
                    tma_load_on(on, sa + 8192, &map_w, j.m0 + 64, k, full + st);
                    tma_load_on(on, sb, &map_dl_k, k, j.n0, full + st);
                }
                if (++st == kRStages) st = 0, phase ^= 1;
                ++issued;
            }
        }
        // no copy is in flight when the block leaves, also when another role gave up
        for (int f = max(0, issued - kRStages); f < issued; ++f)
            (void)mbar_wait_ns(full + f % kRStages, (f / kRStages) & 1, kWaitNs, nullptr);
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA
        const uint32_t on = elect_one(), ring = smem_addr(smem), tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t mn = desc_mn_sw128(ring, 8192, 1024), km = desc_sw128(ring);
        int st = 0, i = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = bid; u < a.units && ok; u += grid, ++i) {
            const Unit j = unit_of(a, u);
            const uint32_t idesc = idesc_16bit(1, 1, j.w, kRM, j.N), d = tm + (i % kRAcc) * kRN;
            if (!(ok = wait(accE + i % kRAcc, ((i / kRAcc) & 1) ^ 1))) break;
            tc_fence_after();
            for (int s = 0; s < j.nk; ++s) {
                if (!(ok = wait(full + st, phase))) break;
                tc_fence_after();
                const uint64_t as = (st * kRStage) >> 4, bs = as + (kRA >> 4);
#pragma unroll
                for (int kk = 0; kk < kRK / 16; ++kk)
                    mma_f16_on(on, d, mn + as + kk * 128, j.w ? mn + bs + kk * 128 : km + bs + kk * 2, idesc, (s | kk) != 0);
                mma_commit_on(on, empty + st);
                if (++st == kRStages) st = 0, phase ^= 1;
            }
            mma_commit_on(on, accF + i % kRAcc);
        }
        mma_commit_on(on, drain);
        if (!mbar_wait_ns(drain, 0, kWaitNs, nullptr)) report(a.err, MOE_DEVERR_TIMEOUT);
        __syncwarp();
    } else {
        // --------------------------------------------------------- epilogue
        const int ew = warp - 2, q = warp & 3, m = 32 * q + lane;     // TMEM lanes 32q .. 32q + 31
        if (a.db && bid < a.bias_parts) {
            // rows of dl of this block's part, two columns a thread
            const int rows = (a.T + a.bias_parts - 1) / a.bias_parts;
            const int t0 = bid * rows, t1 = min(a.T, t0 + rows);
            float *out = a.bias_parts > 1 ? a.db_part + static_cast<size_t>(bid) * a.E : a.db;
            for (int e = 2 * (tid - 64); e < a.E; e += 2 * 32 * kREpi) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
                for (int t = t0; t < t1; ++t) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(a.dl + static_cast<size_t>(t) * a.E + e);
                    s0 += __uint_as_float(v << 16);
                    s1 += __uint_as_float(v & 0xFFFF0000u);
                }
                out[e] = s0;
                out[e + 1] = s1;
            }
        }
        // A warp has every (kREpi / 4)th chunk of 16 columns of its lanes.  dx_in is what it waits for: a
        // unit's lines are brought to L2 a unit ahead, a chunk's values to registers a chunk ahead.
        // (The loop stays rolled: unrolled with two units' values in registers it was slower, its code
        // being read by eight warps.)
        const int part = ew >> 2;
        auto prefetch = [&](const Unit &j) {
            // 128 tokens x 512 bytes: the warp's share of tokens, a line a lane
            if (j.w || !a.dx_in) return;
            for (int e = lane >> 2; e < kRN / kREpi; e += 8) {
                const int t = j.n0 + kRN / kREpi * ew + e, h = j.m0 + 32 * (lane & 3);
                if (t < a.T && h < a.H)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.dx_in + static_cast<size_t>(t) * a.H + h));
            }
        };
        Unit j = {};
        if (bid < a.units) {
            j = unit_of(a, bid);
            prefetch(j);
        }
        int i = 0;
        for (int u = bid; u < a.units; u += grid, ++i) {
            Unit next = j;
            if (u + grid < a.units) {
                next = unit_of(a, u + grid);
                prefetch(next);
            }
            const int h = j.m0 + m, ncol = h < a.H ? (j.w ? a.E : a.T) - j.n0 : 0;      // columns to write
            const bool add = !j.w && a.dx_in, wide = j.w ? a.splits > 1 : !a.dx_bf16;
            const float *src = a.dx_in + static_cast<size_t>(j.n0) * a.H + h;
            void *dst = j.w ? (wide ? static_cast<void *>(a.dw_part) : a.dw) : a.dx;
            const size_t at = static_cast<size_t>((j.w && wide ? static_cast<size_t>(j.split) * a.E : 0) + j.n0) * a.H + h;
            float in[16];
            auto fetch = [&](int c0) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    in[e] = add && c0 + e < ncol ? src[static_cast<size_t>(c0 + e) * a.H] : 0.f;
            };
            fetch(16 * part);
            if (!wait(accF + i % kRAcc, (i / kRAcc) & 1)) break;
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + (i % kRAcc) * kRN;
#pragma unroll 1
            for (int c0 = 16 * part; c0 < j.N; c0 += 4 * kREpi) {
                float v[16];
                tmem_ld16(base + c0, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] += in[e];
                fetch(c0 + 4 * kREpi);
                const size_t o = at + static_cast<size_t>(c0) * a.H;
                if (wide) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c0 + e < ncol) static_cast<float *>(dst)[o + static_cast<size_t>(e) * a.H] = v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c0 + e < ncol)
                            static_cast<__nv_bfloat16 *>(dst)[o + static_cast<size_t>(e) * a.H] = __float2bfloat16_rn(v[e]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(accE + i % kRAcc);
            j = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dW from its splits (four neighbouring values a thread), then db from its
// parts (the last blocks: one warp per expert), both in order.
__global__ void __launch_bounds__(256) k_router_join(RouterArgs a, int w_blocks) {
    const size_t n4 = static_cast<size_t>(a.E) * a.H / 4;
    if (static_cast<int>(blockIdx.x) < w_blocks) {
        const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
        if (i >= n4) return;
        float4 s = reinterpret_cast<const float4 *>(a.dw_part)[i];
        for (int p = 1; p < a.splits; ++p) {
            const float4 v = reinterpret_cast<const float4 *>(a.dw_part)[p * n4 + i];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        uint2 o;
        o.x = *reinterpret_cast<uint32_t *>(&lo);
        o.y = *reinterpret_cast<uint32_t *>(&hi);
        static_cast<uint2 *>(a.dw)[i] = o;
    } else {
        const int e = (blockIdx.x - w_blocks) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        if (e >= a.E) return;
        float s = 0.f;
        for (int p = lane; p < a.bias_parts; p += 32) s += a.db_part[static_cast<size_t>(p) * a.E + e];
        s = warp_sum(s);
        if (lane == 0) a.db[e] = s;
    }
}

// ------------------------------------------------------------------ launch
namespace {
struct RouterPlan {
    int mt, et, splits, per_split, bias_parts;
    size_t dw_bytes, db_bytes;
};
RouterPlan router_plan(int T, int H, int E) {
    RouterPlan p;
    p.mt = (H + kRM - 1) / kRM;
    p.et = (E + kRN - 1) / kRN;
    const int steps = (T + kRK - 1) / kRK;
    // as many splits as give every SM a unit, each of at least 8 k-steps (a
    // split costs E x H x 8 bytes of traffic)
    const long tiles = static_cast<long>(p.mt) * p.et;
    int s = static_cast<int>(num_sms() / tiles);
    if (s > steps / 8) s = steps / 8;
    if (s < 1) s = 1;
    p.per_split = (steps + s - 1) / s;
    if (p.per_split < 1) p.per_split = 1;
    p.splits = steps > 0 ? (steps + p.per_split - 1) / p.per_split : 1;
    const int parts = (T + kBiasRows - 1) / kBiasRows;
    p.bias_parts = parts < 1 ? 1 : parts < num_sms() ? parts : num_sms();
    p.dw_bytes = p.splits > 1 ? static_cast<size_t>(p.splits) * E * H * 4 : 0;
    p.db_bytes = p.bias_parts > 1 ? static_cast<size_t>(p.bias_parts) * E * 4 : 0;
    return p;
}
}  // namespace

bool router_backward_tc_supported(int T, int H, int E, int dl_dtype, int x_dtype, int w_dtype) {
    return T > 0 && E % 8 == 0 && H % 8 == 0 && dl_dtype == MOE_BF16 && x_dtype == MOE_BF16 && w_dtype == MOE_BF16;
}

size_t router_backward_tc_ws_bytes(int T, int H, int E) {
    const RouterPlan p = router_plan(T, H, E);
    return (p.dw_bytes + 255) / 256 * 256 + p.db_bytes;
}

int launch_router_backward_tc(const RouterBackward &b, void *ws, cudaStream_t s) {
    const RouterPlan p = router_plan(b.T, b.H, b.E);
    RouterArgs a = {};
    a.dl = static_cast<const __nv_bfloat16 *>(b.dl);
    a.dx_in = b.dx_in;
    a.dx = b.dx, a.dw = b.d_w, a.db = b.d_bias;
    a.dw_part = static_cast<float *>(ws);
    a.db_part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + (p.dw_bytes + 255) / 256 * 256);
    a.T = b.T, a.H = b.H, a.E = b.E, a.dx_bf16 = b.dx_dtype == MOE_BF16;
    a.mt = p.mt, a.et = p.et, a.splits = p.splits, a.per_split = p.per_split;
    a.bias_parts = p.bias_parts;
    a.units_w = b.d_w ? p.mt * p.et * p.splits : 0;
    a.units = a.units_w + (b.dx ? p.mt * ((b.T + kRN - 1) / kRN) : 0);
    a.err = b.err;
    const long long hook = test_hook_value(MOE_HOOK_WAIT_LIMIT_NS);
    a.limit_ns = hook > 0 ? static_cast<unsigned long long>(hook) : kWaitNs;
    const uint64_t hb = static_cast<uint64_t>(b.H) * 2, eb = static_cast<uint64_t>(b.E) * 2;
    CUtensorMap mw = {}, mx = {}, mk = {}, mm = {};
    int rc = MOE_OK;
    if (b.dx && ((rc = make_tensor_map(&mw, b.w, 1, b.E, b.H, hb, kRK)) ||
                 (rc = make_tensor_map(&mk, b.dl, 1, b.T, b.E, eb, kRN))))
        return rc;
    if (b.d_w && ((rc = make_tensor_map(&mx, b.x, 1, b.T, b.H, hb, kRK)) ||
                  (rc = make_tensor_map(&mm, b.dl, 1, b.T, b.E, eb, kRK))))
        return rc;
    rc = cuda_status(cudaFuncSetAttribute(k_router_bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, kRSmem),
                     "router backward smem attribute");
    if (rc) return rc;
    int grid = a.units;
    if (b.d_bias && grid < p.bias_parts) grid = p.bias_parts;
    if (grid > num_sms()) grid = num_sms();
    k_router_bwd<<<grid, kRThreads, kRSmem, s>>>(a, mw, mx, mk, mm);
    count_launches(1);
    rc = cuda_status(cudaGetLastError(), "router backward launch");
    if (rc) return rc;
    const int w_blocks = b.d_w && p.splits > 1 ? static_cast<int>((static_cast<size_t>(b.E) * b.H / 4 + 255) / 256) : 0;
    const int b_blocks = b.d_bias && p.bias_parts > 1 ? (b.E + 7) / 8 : 0;
    if (w_blocks + b_blocks == 0) return MOE_OK;
    k_router_join<<<w_blocks + b_blocks, 256, 0, s>>>(a, w_blocks);
    count_launches(1);
    return cuda_status(cudaGetLastError(), "router backward join launch");
}

}  // namespace moe

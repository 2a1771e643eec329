// Backward pass of the quantized experts on the 5th-generation tensor cores
// (MOE_MODE_GEMM).
//
// Per expert, over its rows (tokens on the N side, weights on the M side):
//   phase 1   g = Wg x, u = Wu x, q = Wd^T dy      three products of K = H,
//             then dg = q u (s + a (1 - s)), du = q a and each row's <q, a u>
//   phase 2   dxp = Wg^T dg + Wu^T du              one product of K = 2I
// and a gather of each token's rows.  Wg and Wu enter phase 1 as they lie
// (K-major); every transposed use takes the codes as they lie too, a row of
// the matrix being one K index and its values consecutive along M: the
// MN-major operand layout, so that nothing is ever transposed.
//
// Operands are fp16.  x and dy rows are divided by a power of two of their own
// (largest value in [1, 2)) before they are rounded, which makes the products'
// range independent of either's scale; g is scaled back in fp32 before the
// activation, and dg, du are kept in the scaled form,
//   dg / (sx sd) = q' u' (s + a (1 - s)),   du / (sx sd) = q' a',
// until the gather multiplies by w sx sd in fp32.
//
// One persistent block per SM.  Roles:
//   dequantising warps read codes straight to registers, one step of 128 K
//       values ahead, and write fp16 tiles to the A stages; the four lanes of
//       a row read its 64 (4-bit) or 32 bytes, so that whole sectors are used
//       and no shared memory is spent on codes;
//   loader warps gather the rows (cp.async) into the B stages;
//   one thread issues tcgen05.mma; four warps read the accumulators.
// Every wait is bounded (MOE_DEVERR_TIMEOUT; all roles then leave their loops
// and TMEM is freed).
#include "common.cuh"
#include "kernels.h"
#include "train/ffn_bwd.cuh"
#include "train/umma.cuh"

namespace moe {
using namespace sm100;

namespace {
constexpr int kBM = 128;                    // weight rows of one product (MMA M)
constexpr int kBK = 64;                     // K per stage: 128 bytes of fp16
constexpr long kSpin = 1L << 22;            // polls before a wait gives up (about a second)
constexpr uint32_t kMat = kBM * 128;        // bytes of one A tile
constexpr size_t kSmemMax = 232448;

// A token tile: rows n0 .. n0 + n - 1 of one group.
struct __align__(16) TokTile {
    const uint8_t *blob;
    int row0;      // first permuted row of the group, or -1 for the shared expert
    int n0, n;
    int pad[3];
};

struct TcArgs {
    FfnBackward a;
    const __half *x16, *dy16;     // [T, H], scaled
    const float2 *scale;          // [T]: sx, sd
    __half *gu16;                 // [T*k + T, 2I]: dg, du, scaled
    float *dwp;                   // [T*k, I/32]
    float *dxp;                   // [T*k + T, H]
    uint8_t *ok;                  // [T*k]
    const TokTile *tiles;         // this phase's token tiles
    const int *n_tiles;
    long spin;
};

// MAXN: tokens a tile holds.
template <int BITS, int PHASE, int MAXN_>
struct Cfg {
    static constexpr int MAXN = MAXN_;
    static constexpr int NM = PHASE == 1 ? 3 : 2;             // A tiles per stage: g, u, q, or two halves of 256 rows
    static constexpr int NB = PHASE == 1 ? 2 : 1;             // B tiles per stage: x and dy, or [dg | du]
    static constexpr int DEQ = PHASE == 1 ? 12 : 8;           // dequantising warps
    static constexpr int LOAD = 4;                            // loader warps
    static constexpr int THREADS = 32 * (DEQ + 4 + 1 + LOAD);
    static constexpr uint32_t A_STAGE = NM * kMat;
    static constexpr uint32_t B_TILE = MAXN * 128;
    static constexpr uint32_t B_STAGE = NB * B_TILE;
    static constexpr int SA = PHASE == 1 ? (MAXN > 64 ? 2 : 3) : 3;
    static constexpr int SB = PHASE == 1 ? (MAXN > 64 ? 3 : 4) : 3;
    static constexpr int ACC = 2 * NM * MAXN <= 512 ? 2 : 1;  // accumulator sets
    static constexpr int TMEM = ACC * NM * MAXN <= 256 ? 256 : 512;
    static constexpr uint32_t OFF_B = SA * A_STAGE;
    static constexpr uint32_t OFF_TOK = OFF_B + SB * B_STAGE;
    static constexpr uint32_t OFF_SX = OFF_TOK + MAXN * 4;
    static constexpr uint32_t OFF_BAR = (OFF_SX + (PHASE == 1 ? 4 * MAXN * 4 : 0) + 15) / 16 * 16;   // a copy per epilogue warp
    static constexpr uint32_t SMEM = OFF_BAR + 24 * 8 + 16 + 1024;
    static_assert(SMEM <= kSmemMax, "shared memory per block");
    static_assert(2 * SA + 2 * SB + 5 <= 24, "barrier slots");
    static_assert(ACC * NM * MAXN <= 512, "TMEM columns");
    static_assert(MAXN % (4 * LOAD) == 0 && MAXN % 16 == 0 && MAXN <= 256, "rows per loader warp");
};

// One block's codes as read: four words (4 bits) or two.
template <int BITS> struct Codes { uint32_t w[BITS]; };
template <int BITS>
__device__ __forceinline__ Codes<BITS> load_codes(const uint8_t *p) {
    Codes<BITS> c;
    if constexpr (BITS == 4)
        asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]) : "l"(p));
    else
        asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[1]) : "l"(p));
    return c;
}

// (1024 + a, 1024 + b) from the bytes of `bytes` that sel names, less 1024 and
// the offset (exact), times the step: one rounding.
__device__ __forceinline__ uint32_t weight2(uint32_t bytes, uint32_t sel, __half2 off, __half2 d) {
    const uint32_t m = __byte_perm(bytes, 0x64646464u, sel);
    __half2 h = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&m), off), d);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Writes a block's 32 values into 16-byte chunks c0 .. c0+3 of the 128-byte row
// at `row`, chunk c at c ^ sw.  Values 8j..8j+7 go to chunk j; with FLIP the
// two halves are written in the other order (the same bytes), which keeps the
// lanes of a quarter warp on different banks where two of them write the same
// chunk of different tiles.
template <int BITS>
__device__ __forceinline__ void put_block(Codes<BITS> c, __half d, uint32_t row, int c0, int sw, bool flip) {
    const __half2 d2 = __half2half2(d), off = __float2half2_rn(BITS == 4 ? 1032.f : 1026.f);
    if (flip) {
#pragma unroll
        for (int i = 0; i < BITS; ++i) c.w[i] = ((c.w[i] >> 4) & 0x0F0F0F0Fu) | ((c.w[i] << 4) & 0xF0F0F0F0u);
    }
    const int x = flip ? sw ^ 2 : sw;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;                       // values 8j..8j+3 and 8j+4..8j+7, one per byte
        if constexpr (BITS == 4) {
            lo = (j < 2 ? c.w[2 * j] : c.w[2 * j - 4] >> 4) & 0x0F0F0F0Fu;
            hi = (j < 2 ? c.w[2 * j + 1] : c.w[2 * j - 3] >> 4) & 0x0F0F0F0Fu;
        } else {
            lo = (c.w[0] >> (2 * j)) & 0x03030303u;
            hi = (c.w[1] >> (2 * j)) & 0x03030303u;
        }
        st_shared16(row + (((c0 + j) ^ x) << 4), weight2(lo, 0x5140u, off, d2), weight2(lo, 0x5342u, off, d2),
                    weight2(hi, 0x5140u, off, d2), weight2(hi, 0x5342u, off, d2));
    }
}

__device__ __forceinline__ __half half_of(uint2 v, int i) {
    const uint32_t w = i & 2 ? v.y : v.x;
    return __ushort_as_half(static_cast<unsigned short>(i & 1 ? w >> 16 : w));
}
}  // namespace

template <int BITS, int PHASE, int MAXN>
__global__ void __launch_bounds__(Cfg<BITS, PHASE, MAXN>::THREADS, 1) k_bwd_tc(TcArgs p) {
    using C = Cfg<BITS, PHASE, MAXN>;
    constexpr int SA = C::SA, SB = C::SB, ACC = C::ACC, NM = C::NM, DEQ = C::DEQ;
    constexpr int kEpi0 = DEQ, kMma = DEQ + 4, kLoad0 = DEQ + 5;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int32_t *tok_s = reinterpret_cast<int32_t *>(smem + C::OFF_TOK);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *fullA = bars, *emptyA = bars + SA, *fullB = bars + 2 * SA, *emptyB = bars + 2 * SA + SB;
    uint64_t *accF = bars + 2 * SA + 2 * SB, *accE = accF + 2, *drain = accF + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 24);
    volatile int &abort_s = *(reinterpret_cast<int *>(bars + 24) + 1);
    const FfnBackward &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.H, I = a.I;
    const int MT = PHASE == 1 ? I / kBM : (H + 2 * kBM - 1) / (2 * kBM);
    const int nk = (PHASE == 1 ? H : 2 * I) / kBK;
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < SA; ++i) {
            mbar_init(fullA + i, DEQ);
            mbar_init(emptyA + i, 1);
        }
        for (int i = 0; i < SB; ++i) {
            mbar_init(fullB + i, C::LOAD);
            mbar_init(emptyB + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accF + i, 1);
            mbar_init(accE + i, 4);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        fence_proxy_async();
    }
    if (warp == kMma) {
        tmem_alloc(tmem_slot, C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // tiles: all weight rows of a token tile first, dealt to blocks round robin
    const int total = *p.n_tiles * MT, grid = static_cast<int>(gridDim.x), bid = static_cast<int>(blockIdx.x);
    const int n_my = bid < total ? (total - 1 - bid) / grid + 1 : 0;
    auto tile_of = [&](int i, int &m0) {
        const int t = bid + i * grid, g = t / MT;
        m0 = (t - g * MT) * (PHASE == 1 ? kBM : 2 * kBM);
        return p.tiles[g];
    };
    auto fail = [&]() {
        report(a.err, MOE_DEVERR_TIMEOUT);
        abort_s = 1;
    };
    auto aborted = [&]() { return __shfl_sync(0xffffffffu, abort_s, 0) != 0; };
    // one lane polls, the warp follows
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(bar, parity, p.spin);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) fail();
        return ok != 0;
    };

    if (warp < DEQ) {
        // ------------------------------------------------- dequantisation
        const uint32_t sA = smem_addr(smem);
        const int b = lane & 3, rl = lane >> 2, w4 = warp & 3;
        constexpr int BB = 4 * BITS;                          // bytes of a block's codes
        if constexpr (PHASE == 1) {
            // matrix g, u or q = warp / 4; steps of 128 K values, two stages each
            const int mat = warp >> 2, nslot = nk / 2;
            const bool trans = mat == 2;
            const bool odd = b >= 2;                          // takes the odd row of a pair
            struct Slot {
                Codes<BITS> c[4];
                uint2 s[2];                                   // steps: two rows of four, or four rows of one
            } cur, nxt;
            const int U = n_my * nslot;
            auto issue = [&](int u, Slot &o) {
                int m0;
                const TokTile te = tile_of(u / nslot, m0);
                const int sl = u % nslot;
                const BlobView bv = blob_view(te.blob, BITS, H, I);
                if (!trans) {
                    const uint8_t *codes = (mat ? bv.cu : bv.cg) + (4 * sl + b) * BB;
                    const size_t rowb = static_cast<size_t>(H) * BITS / 8;
                    const __half *sc = (mat ? bv.su : bv.sg) + 4 * sl;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o.c[i] = load_codes<BITS>(codes + (m0 + 32 * w4 + 16 * (i >> 1) + 2 * rl + (i & 1)) * rowb);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        o.s[i] = __ldg(reinterpret_cast<const uint2 *>(
                            sc + static_cast<size_t>(m0 + 32 * w4 + 16 * i + 2 * rl + odd) * (H / 32)));
                } else {
                    const uint8_t *codes = bv.cd + (m0 / 32 + b) * BB;
                    const size_t rowb = static_cast<size_t>(I) * BITS / 8;
                    const unsigned short *sc = reinterpret_cast<const unsigned short *>(bv.sd) + m0 / 32 + b;
                    uint32_t s[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const size_t h = 128 * sl + 32 * i + 8 * w4 + rl;
                        o.c[i] = load_codes<BITS>(codes + h * rowb);
                        s[i] = __ldg(sc + h * (I / 32));
                    }
                    o.s[0] = make_uint2(s[0] | s[1] << 16, s[2] | s[3] << 16);
                }
            };
            if (U) issue(0, cur);
            for (int u = 0; u < U && !aborted(); ++u) {
                if (u + 1 < U) issue(u + 1, nxt);
                if (!trans) {
                    // lanes 0, 1 of a row's four take the even row of each pair (their own block of the
                    // first stage, the neighbour's of the second), lanes 2, 3 the odd row
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
#pragma unroll
                        for (int x = 0; x < BITS; ++x) {
                            const uint32_t give = odd ? cur.c[i].w[x] : cur.c[i + 1].w[x];
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 2);
                            if (odd) cur.c[i].w[x] = got;
                            else cur.c[i + 1].w[x] = got;
                        }
                }
                bool ok = true;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const int j = 2 * u + ks, sa = j % SA;
                    ok = ok && wait(emptyA + sa, ((j / SA) & 1) ^ 1);
                    if (!ok) break;
                    const uint32_t tile = sA + sa * C::A_STAGE + mat * kMat;
                    if (!trans) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = 32 * w4 + 16 * i + 2 * rl + odd;
                            put_block<BITS>(cur.c[2 * i + ks], half_of(cur.s[i], 2 * ks + (b & 1)), tile + row * 128,
                                            4 * (b & 1), row & 7, false);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int k = 32 * i + 8 * w4 + rl;
                            put_block<BITS>(cur.c[2 * ks + i], half_of(cur.s[0], 2 * ks + i),
                                            tile + (b >> 1) * 8192 + k * 128, 4 * (b & 1), k & 7, odd);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fullA + sa);
                }
                if (!ok) break;
                cur = nxt;
            }
        } else {
            // 64 rows of Wg, then Wu, a stage: 256 columns, two tiles of 128
            struct Step {
                Codes<BITS> c[2];
                uint32_t s;
            } ring[2];
            const int J = n_my * nk;
            auto issue = [&](int j, Step &o) {
                int m0;
                const TokTile te = tile_of(j / nk, m0);
                const BlobView bv = blob_view(te.blob, BITS, H, I);
                int i = (j % nk) * kBK + 8 * warp + rl;
                const bool up = i >= I;
                if (up) i -= I;
                const uint8_t *codes = (up ? bv.cu : bv.cg) + i * (static_cast<size_t>(H) * BITS / 8) + (m0 / 32 + b) * BB;
                const unsigned short *sc = reinterpret_cast<const unsigned short *>(up ? bv.su : bv.sg) +
                                           static_cast<size_t>(i) * (H / 32) + m0 / 32 + b;
                const bool two = m0 + kBM < H;
                o.c[0] = load_codes<BITS>(codes);
                o.s = __ldg(sc);
                if (two) {
                    o.c[1] = load_codes<BITS>(codes + 4 * BB);
                    o.s |= static_cast<uint32_t>(__ldg(sc + 4)) << 16;
                } else {
                    o.c[1] = o.c[0];                          // a ragged last tile: written, not used
                }
            };
            if (J > 0) issue(0, ring[0]);
            if (J > 1) issue(1, ring[1]);
            for (int j = 0; j < J && !aborted(); ++j) {
                const Step cur = ring[0];
                ring[0] = ring[1];
                if (j + 2 < J) issue(j + 2, ring[1]);
                const int sa = j % SA;
                if (!wait(emptyA + sa, ((j / SA) & 1) ^ 1)) break;
                const uint32_t row = sA + sa * C::A_STAGE + (b >> 1) * 8192 + (8 * warp + rl) * 128;
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    put_block<BITS>(cur.c[m], half_of(make_uint2(cur.s, 0), m), row + m * kMat, 4 * (b & 1), rl, b >= 2);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(fullA + sa);
            }
        }
    } else if (warp >= kLoad0) {
        // --------------------------------------------------- rows of x, dy or [dg | du]
        const int lw = warp - kLoad0, c = lane & 7;
        constexpr int ROWS = MAXN / C::LOAD;
        int32_t *tok = tok_s + lw * ROWS;
        const size_t rowb = static_cast<size_t>(PHASE == 1 ? H : 2 * I) * 2;
        const uint8_t *src0 = reinterpret_cast<const uint8_t *>(PHASE == 1 ? p.x16 : p.gu16) + c * 16;
        const uint8_t *src1 = reinterpret_cast<const uint8_t *>(p.dy16) + c * 16;
        const int J = n_my * nk;
        constexpr int D = 1;                                  // steps of copies in flight beyond the one issued
        int cur = -1, N = 0, n = 0;
        for (int j = 0; j < J + D; ++j) {
            if (aborted()) break;
            if (j < J) {
                const int i = j / nk, s = j - i * nk;
                if (i != cur) {
                    int m0;
                    const TokTile te = tile_of(i, m0);
                    cur = i;
                    n = te.n;
                    N = (n + 15) & ~15;
                    __syncwarp();
                    for (int r = lane; r < ROWS; r += 32) {
                        const int q = lw * ROWS + r;
                        int v = 0;
                        if (q < n) {
                            if (PHASE == 2) v = (te.row0 >= 0 ? te.row0 : a.T * a.k) + te.n0 + q;
                            else v = te.row0 >= 0
                                         ? guard_index(a.perm_src[te.row0 + te.n0 + q], a.T, a.err, MOE_DEVERR_BAD_ROW)
                                         : te.n0 + q;
                        }
                        tok[r] = v;
                    }
                    __syncwarp();
                }
                const int sb = j % SB;
                if (!wait(emptyB + sb, ((j / SB) & 1) ^ 1)) break;
                const uint32_t dst = smem_addr(smem + C::OFF_B + sb * C::B_STAGE);
#pragma unroll 4
                for (int r = lane >> 3; r < ROWS; r += 4) {
                    const int q = lw * ROWS + r;
                    if (q < N) {
                        const size_t off = static_cast<size_t>(tok[r]) * rowb + static_cast<size_t>(s) * 128;
                        const uint32_t to = dst + q * 128 + ((c ^ (q & 7)) << 4), bytes = q < n ? 16u : 0u;
                        cp_async16(to, src0 + off, bytes);
                        if (PHASE == 1) cp_async16(to + C::B_TILE, src1 + off, bytes);
                    }
                }
            }
            cp_async_commit();
            if (j >= D) {
                cp_async_wait<D>();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(fullB + (j - D) % SB);
            }
        }
        cp_async_wait<0>();
    } else if (warp < kMma) {
        // -------------------------------------------------------- epilogue
        const int q = warp - kEpi0;                           // TMEM lanes 32q .. 32q + 31
        // a warp reads the lanes of its rank modulo four
        static_assert(kEpi0 % 4 == 0, "TMEM lanes follow the warp's rank");
        const int m = 32 * q + lane;
        // each warp has its own table of the tile's scales: no barrier among
        // the four, of which one may leave early
        float *sx_s = reinterpret_cast<float *>(smem + C::OFF_SX) + q * MAXN;
        for (int i = 0; i < n_my && !aborted(); ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const size_t row0 = static_cast<size_t>(te.row0 >= 0 ? te.row0 : a.T * a.k) + te.n0;
            if constexpr (PHASE == 1) {
                __syncwarp();                                 // the last tile's scales are read
                for (int r = lane; r < te.n; r += 32) {
                    const int t = te.row0 >= 0 ? guard_index(a.perm_src[te.row0 + te.n0 + r], a.T, nullptr, 0) : te.n0 + r;
                    sx_s[r] = p.scale[t].x;
                    if (te.row0 >= 0 && m0 == 0 && q == 0) p.ok[row0 + r] = 1;
                }
                __syncwarp();
            }
            const int acc = i % ACC;
            if (!wait(accF + acc, (i / ACC) & 1)) break;
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * NM * MAXN;
            if constexpr (PHASE == 1) {
                for (int c0 = 0; c0 < te.n; c0 += 16) {
                    float gv[16], uv[16], qv[16];
                    tmem_ld16(base + c0, gv);
                    tmem_ld16(base + MAXN + c0, uv);
                    tmem_ld16(base + 2 * MAXN + c0, qv);
                    tmem_ld_wait();
                    __half *out = p.gu16 + (row0 + c0) * 2 * I + m0 + m;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const bool in = c0 + e < te.n;
                        const float g = gv[e] * (in ? sx_s[c0 + e] : 0.f);
                        const float s = __fdividef(1.f, 1.f + __expf(-g));
                        const float qu = qv[e] * uv[e], act = gv[e] * s;       // a / sx
                        if (in) {
                            out[static_cast<size_t>(e) * 2 * I] = __float2half_rn(qu * fmaf(g * s, 1.f - s, s));
                            out[static_cast<size_t>(e) * 2 * I + I] = __float2half_rn(qv[e] * act);
                        }
                        qv[e] = in ? qu * act : 0.f;
                    }
                    // sixteen rows' sums over the warp's 32 lanes: halves are exchanged, so that each
                    // step halves the values a lane holds
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) {
                        const bool up = lane & (2 * o);
#pragma unroll
                        for (int e = 0; e < o; ++e) {
                            const float give = up ? qv[e] : qv[e + o], keep = up ? qv[e + o] : qv[e];
                            qv[e] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * o);
                        }
                    }
                    const float sum = qv[0] + __shfl_xor_sync(0xffffffffu, qv[0], 1);
                    const int r = c0 + (lane >> 1);
                    if (!(lane & 1) && te.row0 >= 0 && r < te.n) p.dwp[(row0 + r) * (I / 32) + m0 / 32 + q] = sum;
                }
            } else {
                for (int mat = 0; mat < 2; ++mat) {
                    const int h = m0 + kBM * mat + m;
                    if (m0 + kBM * mat >= H) break;
                    for (int c0 = 0; c0 < te.n; c0 += 16) {
                        float v[16];
                        tmem_ld16(base + mat * MAXN + c0, v);
                        tmem_ld_wait();
                        float *out = p.dxp + (row0 + c0) * H + h;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c0 + e < te.n) out[static_cast<size_t>(e) * H] = v[e];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(accE + acc);
        }
    } else {
        // ------------------------------------------------------ MMA issuer
        for (int i = 0; i < n_my && !aborted(); ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const int N = (te.n + 15) & ~15, acc = i % ACC;
            const int nmat = PHASE == 1 || m0 + kBM < H ? NM : 1;
            const uint32_t id_k = idesc_16bit(0, 0, 0, kBM, N), id_mn = idesc_16bit(0, 1, 0, kBM, N);
            if (lane == 0) {
                if (!mbar_wait(accE + acc, ((i / ACC) & 1) ^ 1, p.spin)) fail();
                tc_fence_after();
                for (int s = 0; s < nk && !abort_s; ++s) {
                    const int j = i * nk + s, sa = j % SA, sb = j % SB;
                    if (!mbar_spin(fullB + sb, (j / SB) & 1, p.spin * 16) ||
                        !mbar_spin(fullA + sa, (j / SA) & 1, p.spin * 16)) {
                        fail();
                        break;
                    }
                    tc_fence_after();
                    const uint32_t bs = smem_addr(smem + C::OFF_B + sb * C::B_STAGE);
                    const uint32_t as = smem_addr(smem + sa * C::A_STAGE);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        for (int mat = 0; mat < nmat; ++mat) {
                            const bool mn = PHASE == 2 || mat == 2;
                            const uint32_t at = as + mat * kMat;
                            mma_f16(tmem + (acc * NM + mat) * MAXN,
                                    mn ? desc_mn_sw128(at + kk * 2048, 8192, 1024) : desc_sw128(at + kk * 32),
                                    desc_sw128(bs + (PHASE == 1 && mat == 2 ? C::B_TILE : 0) + kk * 32),
                                    mn ? id_mn : id_k, (s | kk) != 0);
                        }
                    }
                    mma_commit(emptyA + sa);
                    mma_commit(emptyB + sb);
                }
                mma_commit(accF + acc);
            }
            __syncwarp();
        }
        if (lane == 0) {                                      // TMEM is released once every MMA is done
            mma_commit(drain);
            if (!mbar_wait(drain, 0, kSpin)) report(a.err, MOE_DEVERR_TIMEOUT);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// ------------------------------------------------------------------ prepare
namespace {
constexpr int kPrepThreads = 256;

struct Prep {
    __half *x16, *dy16;
    float2 *scale;
    TokTile *tiles1, *tiles2;
    int *counts;                  // token tiles of phase 1 and 2
    int max1, max2;               // tokens per tile
    int cap1, cap2;               // entries of the lists
};

// 2^-e and 2^e with e = floor(log2 top) of the row's largest |value| (bits
// `top`), held where both are normal numbers; 1 for a row of zeros or one that
// is not finite (its NaN or infinity goes through as it is).
__device__ __forceinline__ float2 row_scale(uint32_t top) {
    if (top == 0u || top >= 0x7F800000u) return make_float2(1.f, 1.f);
    const uint32_t e = min(max(top >> 23, 1u), 253u);
    return make_float2(__uint_as_float((254u - e) << 23), __uint_as_float(e << 23));
}

// Tiles of a group of n rows: as few as hold it, of equal size (a multiple of
// 16), so that no tile is left with a few rows.
__device__ __forceinline__ int tile_rows(int n, int most) {
    const int tiles = (n + most - 1) / most;
    return ((n + tiles - 1) / tiles + 15) & ~15;
}
}  // namespace

// Block 0 lists both phases' token tiles; each other block scales and rounds
// one token's x and dy.
__global__ void __launch_bounds__(kPrepThreads) k_bwd_prepare(FfnBackward a, Prep p) {
    __shared__ uint32_t part[kPrepThreads / 32];
    __shared__ int2 sums[kPrepThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0) {
        const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
        const int ng = n_act + (a.shared ? 1 : 0);
        int2 done = make_int2(0, 0);
        for (int g0 = 0; g0 < ng; g0 += kPrepThreads) {
            const int g = g0 + tid;
            BwdGroup G = {nullptr, 0, -1};
            if (g < ng) G = bwd_group(a, g, n_act, true);
            int2 r = make_int2(16, 16), c = make_int2(0, 0);
            if (G.n > 0) {
                r = make_int2(tile_rows(G.n, p.max1), tile_rows(G.n, p.max2));
                c = make_int2((G.n + r.x - 1) / r.x, (G.n + r.y - 1) / r.y);
            }
            int2 in = c;                                      // inclusive sums over the warp, then the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, in.x, o), y = __shfl_up_sync(0xffffffffu, in.y, o);
                if (lane >= o) in.x += x, in.y += y;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = in;
            __syncthreads();
            int2 at = make_int2(done.x + in.x - c.x, done.y + in.y - c.y);
            for (int w = 0; w < kPrepThreads / 32; ++w) {
                if (w < warp) at.x += sums[w].x, at.y += sums[w].y;
                done.x += sums[w].x, done.y += sums[w].y;
            }
            // consistent offsets never reach the lists' ends
            if (at.x + c.x > p.cap1 || at.y + c.y > p.cap2) {
                report(a.err, MOE_DEVERR_BAD_ROW);
                c = make_int2(0, 0);
            }
            for (int i = 0; i < c.x; ++i)
                p.tiles1[at.x + i] = {G.blob, G.row0, i * r.x, min(r.x, G.n - i * r.x), {0, 0, 0}};
            for (int i = 0; i < c.y; ++i)
                p.tiles2[at.y + i] = {G.blob, G.row0, i * r.y, min(r.y, G.n - i * r.y), {0, 0, 0}};
        }
        const bool fits = done.x <= p.cap1 && done.y <= p.cap2;
        if (tid == 0) p.counts[0] = fits ? done.x : 0, p.counts[1] = fits ? done.y : 0;
        return;
    }
    const size_t t = blockIdx.x - 1;
    const int h4n = a.H / 4;
    constexpr int V = 8192 / 4 / kPrepThreads;
    float2 scale[2];
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const void *src = which ? a.dy : a.x;
        const uint8_t *steps = which ? nullptr : a.x_scales;
        const int kind = which ? a.dy_dtype : a.x_dtype;
        float4 v[V];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int h4 = tid + i * kPrepThreads;
            if (h4 < h4n) {
                v[i] = bwd_load4(src, steps, kind, t, a.H, h4);
                top = max(max(top, __float_as_uint(fabsf(v[i].x))), __float_as_uint(fabsf(v[i].y)));
                top = max(max(top, __float_as_uint(fabsf(v[i].z))), __float_as_uint(fabsf(v[i].w)));
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        __syncthreads();
        if (lane == 0) part[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kPrepThreads / 32; ++w) top = max(top, part[w]);
        const float2 sc = row_scale(top);
        scale[which] = sc;
        uint2 *out = reinterpret_cast<uint2 *>((which ? p.dy16 : p.x16) + t * a.H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int h4 = tid + i * kPrepThreads;
            if (h4 < h4n) {
                __half2 lo = __floats2half2_rn(v[i].x * sc.x, v[i].y * sc.x), hi = __floats2half2_rn(v[i].z * sc.x, v[i].w * sc.x);
                uint2 u;
                u.x = *reinterpret_cast<uint32_t *>(&lo);
                u.y = *reinterpret_cast<uint32_t *>(&hi);
                out[h4] = u;
            }
        }
    }
    if (tid == 0) p.scale[t] = make_float2(scale[0].y, scale[1].y);
}

// ------------------------------------------------------------------ launch
namespace {
struct TcPlan {
    bool large;
    int max1, max2;
    size_t tiles1, tiles2;        // bounds on the token tiles
};
constexpr int kSmallN = 64, kLargeN1 = 160, kLargeN2 = 256;

TcPlan plan_of(int T, int k, int E) {
    const long rows = static_cast<long>(T) * k, groups = rows < E ? rows : E;
    TcPlan p;
    p.large = rows > 32L * groups;
    p.max1 = p.large ? kLargeN1 : kSmallN;
    p.max2 = p.large ? kLargeN2 : kSmallN;
    // a group of n rows has at most n / most + 1 tiles, and rounding a tile up to 16 rows adds none
    auto bound = [&](int most) { return static_cast<size_t>(rows / most + groups + T / most + 1); };
    p.tiles1 = bound(p.max1);
    p.tiles2 = bound(p.max2);
    return p;
}

struct TcWs {
    __half *x16, *dy16, *gu16;
    float2 *scale;
    float *dwp, *dxp;
    uint8_t *ok;
    TokTile *tiles1, *tiles2;
    int *counts;
};

size_t carve(int T, int k, int H, int I, int E, uint8_t *base, TcWs *out) {
    const size_t rows = static_cast<size_t>(T) * k, all = rows + T;
    const TcPlan p = plan_of(T, k, E);
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t *q = base ? base + at : nullptr;
        at += (n + 255) / 256 * 256;
        return q;
    };
    TcWs w;
    w.x16 = reinterpret_cast<__half *>(take(static_cast<size_t>(T) * H * 2));
    w.dy16 = reinterpret_cast<__half *>(take(static_cast<size_t>(T) * H * 2));
    w.gu16 = reinterpret_cast<__half *>(take(all * 2 * I * 2));
    w.scale = reinterpret_cast<float2 *>(take(static_cast<size_t>(T) * sizeof(float2)));
    w.dwp = reinterpret_cast<float *>(take(rows * (I / 32) * 4));
    w.dxp = reinterpret_cast<float *>(take(all * H * 4));
    w.ok = take(rows);
    w.tiles1 = reinterpret_cast<TokTile *>(take(p.tiles1 * sizeof(TokTile)));
    w.tiles2 = reinterpret_cast<TokTile *>(take(p.tiles2 * sizeof(TokTile)));
    w.counts = reinterpret_cast<int *>(take(2 * sizeof(int)));
    if (out) *out = w;
    return at;
}

template <int BITS, int PHASE, int MAXN>
int launch_phase(const TcArgs &p, cudaStream_t s) {
    using C = Cfg<BITS, PHASE, MAXN>;
    int rc = cuda_status(cudaFuncSetAttribute(k_bwd_tc<BITS, PHASE, MAXN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(C::SMEM)),
                         "backward gemm smem attribute");
    if (rc) return rc;
    k_bwd_tc<BITS, PHASE, MAXN><<<num_sms(), C::THREADS, C::SMEM, s>>>(p);
    count_launches(1);
    return cuda_status(cudaGetLastError(), "backward gemm launch");
}
}  // namespace

size_t ffn_backward_gemm_ws_bytes(int T, int k, int H, int I, int E) { return carve(T, k, H, I, E, nullptr, nullptr); }

bool ffn_backward_gemm_supported(int T, int k, int H, int I, int E) {
    // tile and step numbers are ints
    const TcPlan p = plan_of(T, k, E);
    const double n1 = static_cast<double>(p.tiles1) * (I / kBM), n2 = static_cast<double>(p.tiles2) * ((H + 255) / 256);
    return n1 < 2e9 && n2 < 2e9 && n1 / num_sms() * (H / kBK) < 2e9 && n2 / num_sms() * (2 * I / kBK) < 2e9;
}

int launch_ffn_backward_gemm(const FfnBackward &a, void *ws, cudaStream_t s) {
    TcWs w;
    carve(a.T, a.k, a.H, a.I, a.E, static_cast<uint8_t *>(ws), &w);
    const TcPlan plan = plan_of(a.T, a.k, a.E);
    int rc = cuda_status(cudaMemsetAsync(w.ok, 0, static_cast<size_t>(a.T) * a.k, s), "row flags memset");
    if (rc) return rc;
    const Prep prep = {w.x16, w.dy16, w.scale, w.tiles1, w.tiles2, w.counts, plan.max1, plan.max2,
                       static_cast<int>(plan.tiles1), static_cast<int>(plan.tiles2)};
    k_bwd_prepare<<<a.T + 1, kPrepThreads, 0, s>>>(a, prep);
    count_launches(1);
    rc = cuda_status(cudaGetLastError(), "backward prepare launch");
    if (rc) return rc;
    const long hook = static_cast<long>(test_hook_value(MOE_HOOK_GEMM_SPIN));
    TcArgs p = {a, w.x16, w.dy16, w.scale, w.gu16, w.dwp, w.dxp, w.ok, w.tiles1, w.counts, hook > 0 ? hook : kSpin};
    TcArgs p2 = p;
    p2.tiles = w.tiles2, p2.n_tiles = w.counts + 1;
    if (a.bits == 4) {
        rc = plan.large ? launch_phase<4, 1, kLargeN1>(p, s) : launch_phase<4, 1, kSmallN>(p, s);
        if (!rc) rc = plan.large ? launch_phase<4, 2, kLargeN2>(p2, s) : launch_phase<4, 2, kSmallN>(p2, s);
    } else {
        rc = plan.large ? launch_phase<2, 1, kLargeN1>(p, s) : launch_phase<2, 1, kSmallN>(p, s);
        if (!rc) rc = plan.large ? launch_phase<2, 2, kLargeN2>(p2, s) : launch_phase<2, 2, kSmallN>(p2, s);
    }
    if (rc) return rc;
    return launch_ffn_backward_gather(a, w.dxp, w.dwp, a.I / 32, w.ok, w.scale, s);
}

}  // namespace moe

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
// times c r, until the gather multiplies by w sx sd / r in fp32.  c (a power of
// two of the expert, undone as phase 2 writes its fp32 rows) and r (one of the
// token) hold them in fp16's range whatever the weights are: with D the largest
// magnitude of a code,
//   |u'|, |a'| <= D max|step of Wg, Wu| |x'|_1,   |q'| <= D max|step of Wd| |dy'|_1,
// the weights' part and the rows' are taken up to a power of two, c r times
// these is 2^15, and |s + a (1 - s)| < 1.1.  So none is infinite, and one that is
// 2^-27 of the bound still has all its bits: for random weights of one size
// values lie about 2^13 to 2^15 below it.  The steps' largest are read ahead, with the
// rows: a sixteenth of a weight a byte (4 bits: 1/9 of the weights' bytes).
// They lie transposed between the phases, [2I] x rows, a group's rows padded
// to 16: a thread of phase 1 holds one i and 16 rows, 32 bytes to store, and
// phase 2 takes its N side MN-major as it takes the weights.
//
// One persistent block per SM.  Roles:
//   dequantising warps, two groups that take alternate stages, write fp16 tiles
//       to the A stages, four blocks of 32 a thread between two barriers.  g's
//       and u's A tiles go to TMEM, a row a lane (848 us for 775 at 8192 tokens:
//       in shared memory they were half of its traffic); transposed tiles lie in
//       shared memory.  The codes come by TMA to a ring of raw tiles in phase 1
//       (loaded by the threads, the 32-byte pieces of a K-major tile's rows kept
//       the load unit busy: 208 of 1047 us at 8192 tokens, 148 of 396 at 64), in
//       phase 2, whose rows are longer, straight to registers two stages ahead;
//   one warp of phase 1 issues those copies, through a map per expert and
//       matrix that the kernel in front makes from the blob's address;
//   loader warps fill the B stages: phase 1 gathers the tokens' rows with
//       cp.async (TMA's four-row gathers took 50 cycles each here: 1842 us for
//       1047 at 8192 tokens), phase 2 one warp with TMA boxes of 128 K rows x 64
//       tokens;
//   one thread issues tcgen05.mma; four warps read the accumulators.
// Every wait is bounded (MOE_DEVERR_TIMEOUT; all roles then leave their loops
// and TMEM is freed).
//
// Measured (512 experts of 2048 x 512 and a shared one, top-10, 4 bits, 8192
// tokens): preparation 56 us (33 of it the rows, the rest 100 MB of steps), phase
// 1 790, phase 2 527, gather 144; 945 GFLOP at 623 TFLOP/s.  No role alone bounds the two phases: of phase 1's, copying no rows
// saves 27, writing no transposed tiles 37, the epilogue's work 120, the MMAs 34;
// of phase 2's, its stores 78, its codes 55, its B copies 55, its MMAs 65.  A tile
// of 128 rows (phase 1) leaves room for three B stages and fills TMEM with its
// accumulators and A (96 rows and three A stages: 862 us); of 256 (phase 2) reads
// the weights least (192: 564 us for 526, 128: 605).  The gather moves its 770 MB
// at 5.5 TB/s.  At 16 tokens (phases 94 and 67 at 2 bits) the transposed tile's warps take
// longest; twice as many of them gained 4 us there and cost 80 at 8192, in
// registers.
#include "common.cuh"
#include "kernels.h"
#include "train/ffn_bwd.cuh"
#include "train/launch.cuh"
#include "train/tma.cuh"
#include "train/umma.cuh"
#include "train/ws.h"

namespace moe {
using namespace sm100;

namespace {
constexpr int kBM = 128;                    // weight rows of one product (MMA M)
constexpr int kBK = 64;                     // K per stage: 128 bytes of fp16
constexpr uint32_t kMat = kBM * 128;        // bytes of one A tile
constexpr size_t kSmemMax = 232448;
constexpr int kBars = 28;                   // barrier slots

// A token tile: rows n0 .. n0 + n - 1 of one group.
struct __align__(16) TokTile {
    const uint8_t *blob;
    int row0;      // first permuted row of the group, or -1 for the shared expert
    int n0, n;
    int at;        // column of gu16 of the first row
    int g;         // the group's number
    int pad;
};

struct TcArgs {
    FfnBackward a;
    const float4 *scale;          // [T]: sx, sd, r, 1/r
    const uint32_t *steps;        // [groups, 32]: largest steps of Wg and Wu (16), of Wd (16), by parts
    int gu_parts, d_parts;
    __half *gu16;                 // [2I, cols]: dg, du, scaled, a column per row of a group
    int cols;
    const __half *x16, *dy16;     // [T, H], scaled
    float *dwp;                   // [T*k, I/32]
    float *dxp;                   // [T*k + T, H]
    uint8_t *ok;                  // [T*k + T]
    const CUtensorMap *maps;      // [groups, 3]: Wg, Wu, Wd as bytes
    const TokTile *tiles;         // this phase's token tiles
    const int *n_tiles;
    unsigned long long limit_ns;  // of a pipeline wait
};

// MAXN: tokens a tile holds.
template <int BITS, int PHASE, int MAXN_>
struct Cfg {
    static constexpr int MAXN = MAXN_;
    // phase 1: a stage is 64 of K, three A tiles (g, u, q; an accumulator each)
    // and two B tiles (x, dy); phase 2: 128 of K, two A and two B tiles of 64,
    // one accumulator
    static constexpr int NM = PHASE == 1 ? 3 : 2;
    static constexpr int NB = 2;
    static constexpr int ND = PHASE == 1 ? 3 : 1;
    static constexpr int KSTAGE = PHASE == 1 ? kBK : 2 * kBK;
    static constexpr int GROUP = PHASE == 1 ? 6 : 4;          // warps of a dequantising group: 4 blocks a thread
    static constexpr int DEQ = 2 * GROUP;
    static constexpr int EPI = 4;
    static constexpr int LOAD = PHASE == 2 ? 1 : MAXN > 64 ? 6 : 3;      // loader warps
    static constexpr int RAW = PHASE == 1 ? 1 : 0;            // the warp that copies codes
    static constexpr int THREADS = 32 * (DEQ + EPI + 1 + LOAD + RAW);
    // phase 1: g's and u's A tiles lie in TMEM, 32 columns each
    static constexpr int NS = PHASE == 1 ? 1 : NM;            // A tiles in shared memory
    static constexpr uint32_t A_STAGE = NS * kMat;
    static constexpr uint32_t B_TILE = MAXN * 128;
    static constexpr uint32_t B_STAGE = NB * B_TILE;
    static constexpr int SA = PHASE == 1 ? 2 : (MAXN > 64 ? 3 : 4);
    static constexpr int SB = PHASE == 1 ? 3 : (MAXN > 64 ? 2 : 4);
    // raw code slots, a stage each (phase 2: unused); an even number, so that a
    // slot is always the same group's: a group may be a stage ahead of the other,
    // and the parity it waits for would tell it that the other's stage is its own
    static constexpr int SR = PHASE == 1 && MAXN <= 64 ? 4 : 2;
    static constexpr uint32_t RAW_TILE = kBM * kBK * BITS / 8, RAW_SLOT = 3 * RAW_TILE;
    static constexpr int TA = PHASE == 1 ? 64 * SA : 0;       // TMEM columns of A
    static constexpr int ACC = 2 * ND * MAXN + TA <= 512 ? 2 : 1;         // accumulator sets
    static constexpr int COLS = ACC * ND * MAXN + TA, TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr uint32_t OFF_B = SA * A_STAGE;
    static constexpr uint32_t OFF_RAW = OFF_B + SB * B_STAGE;
    static constexpr uint32_t OFF_SX = OFF_RAW + (PHASE == 1 ? SR * RAW_SLOT : 0);
    static constexpr uint32_t OFF_BAR = OFF_SX + (PHASE == 1 ? EPI * MAXN * 8 : 0);   // a copy per epilogue warp
    static constexpr uint32_t SMEM = OFF_BAR + kBars * 8 + 16 + 1024;
    static_assert(SMEM <= kSmemMax, "shared memory per block");
    static_assert(2 * SA + 2 * SB + 2 * SR + 5 <= kBars, "barrier slots");
    static_assert(SR % 2 == 0, "raw slots of a group");
    static_assert(COLS <= 512, "TMEM columns");
    static_assert(MAXN % 16 == 0 && MAXN <= 256 && (PHASE == 1 || MAXN % 64 == 0), "tokens a tile");
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

// A block's 32 values are written in the order in which its codes come out with
// the fewest steps, two at a time from bits 16 apart: position p of the 32
// holds value block_order(p).  Whatever meets them follows: x's columns (K of
// g and u), Wg's and Wu's rows against q's (M of phase 1), the lanes' h (M of
// phase 2).
template <int BITS>
__device__ __forceinline__ int block_order(int p) {
    const int c = p >> 3, in4 = ((p & 1) << 1) | ((p >> 1) & 1);                // 0, 2, 1, 3
    if (BITS == 4) return 4 * c + 4 * (p & 4) + in4;                            // + 16 in the chunk's second half
    return 4 * (c >> 1) + 8 * (2 * (c & 1) + ((p >> 2) & 1)) + in4;
}
// Its inverse for four neighbouring values 4f .. 4f+3: the position of the first.
__device__ __forceinline__ int block_place(int bits, int f) {
    if (bits == 4) return f < 4 ? 8 * f : 8 * (f - 4) + 4;
    return 8 * (2 * (f & 1) + (f >> 2)) + 4 * ((f >> 1) & 1);
}

// The same from a raw tile in shared memory.
template <int BITS>
__device__ __forceinline__ Codes<BITS> raw_codes(const uint8_t *p) {
    Codes<BITS> c;
    if constexpr (BITS == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        c.w[0] = v.x, c.w[1] = v.y, c.w[2] = v.z, c.w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        c.w[0] = v.x, c.w[1] = v.y;
    }
    return c;
}

// Two codes at bit SHIFT of w's halves, as fp16 weights: 1024 + 2^SHIFT q from
// the bits, back to q less the offset (exact), times the step (one rounding).
template <int BITS, int SHIFT>
__device__ __forceinline__ uint32_t weight2(uint32_t w, __half2 d) {
    constexpr uint32_t mask = ((1u << BITS) - 1) << SHIFT;
    const uint32_t m = (w & (mask | mask << 16)) | 0x64006400u;
    __half2 h = *reinterpret_cast<const __half2 *>(&m);
    constexpr float unit = 1.f / (1 << SHIFT), off = 1024.f * unit + (1 << (BITS - 1));
    if constexpr (SHIFT == 0) h = __hsub2(h, __float2half2_rn(off));
    else h = __hfma2(h, __float2half2_rn(unit), __float2half2_rn(-off));
    h = __hmul2(h, d);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Writes a block's 32 values into 16-byte chunks c0 .. c0+3 of the 128-byte row
// at `row`, chunk c at c ^ sw, in block_order.  With FLIP the two halves are
// written in the other order (the same bytes), which keeps the lanes of a
// quarter warp on different banks where two of them write the same chunk of
// different tiles.
template <int BITS>
__device__ __forceinline__ void put_block(const Codes<BITS> &c, __half d, uint32_t row, int c0, int sw, bool flip) {
    const __half2 d2 = __half2half2(d);
    const int x = flip ? sw ^ 2 : sw;
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = flip ? c.w[j ^ 2] : c.w[j], v = w >> 8;
            st_shared16(row + (((c0 + j) ^ x) << 4), weight2<4, 0>(w, d2), weight2<4, 0>(v, d2), weight2<4, 4>(w, d2),
                        weight2<4, 4>(v, d2));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w = flip ? c.w[j ^ 1] : c.w[j], v = w >> 8;
            st_shared16(row + (((c0 + 2 * j) ^ x) << 4), weight2<2, 0>(w, d2), weight2<2, 0>(v, d2), weight2<2, 2>(w, d2),
                        weight2<2, 2>(v, d2));
            st_shared16(row + (((c0 + 2 * j + 1) ^ x) << 4), weight2<2, 4>(w, d2), weight2<2, 4>(v, d2),
                        weight2<2, 6>(w, d2), weight2<2, 6>(v, d2));
        }
    }
}

// A block's 32 values as 16 words, in block_order.
template <int BITS>
__device__ __forceinline__ void block_words(const Codes<BITS> &c, __half d, uint32_t (&o)[16]) {
    const __half2 d2 = __half2half2(d);
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = c.w[j], v = w >> 8;
            o[4 * j] = weight2<4, 0>(w, d2), o[4 * j + 1] = weight2<4, 0>(v, d2);
            o[4 * j + 2] = weight2<4, 4>(w, d2), o[4 * j + 3] = weight2<4, 4>(v, d2);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w = c.w[j], v = w >> 8;
            o[8 * j] = weight2<2, 0>(w, d2), o[8 * j + 1] = weight2<2, 0>(v, d2);
            o[8 * j + 2] = weight2<2, 2>(w, d2), o[8 * j + 3] = weight2<2, 2>(v, d2);
            o[8 * j + 4] = weight2<2, 4>(w, d2), o[8 * j + 5] = weight2<2, 4>(v, d2);
            o[8 * j + 6] = weight2<2, 6>(w, d2), o[8 * j + 7] = weight2<2, 6>(v, d2);
        }
    }
}

// e with c = 2^e of a group's inner gradients (a warp's call): 15 less the
// exponent of the weights' part of the bound.  0 where no bound is to be had (a step
// that is infinite or NaN) or none is needed (all steps of a side are 0).
template <int BITS>
__device__ __forceinline__ int group_exponent(const TcArgs &p, int g) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    const uint32_t v = part < (lane < 16 ? p.gu_parts : p.d_parts) ? p.steps[32 * static_cast<size_t>(g) + lane] : 0u;
    const uint32_t gu = __reduce_max_sync(0xffffffffu, lane < 16 ? v : 0u);
    const uint32_t d = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : v);
    if (gu == 0u || d == 0u || gu >= 0x7C00u || d >= 0x7C00u) return 0;
    const float both = __half2float(__ushort_as_half(static_cast<unsigned short>(gu))) *
                       __half2float(__ushort_as_half(static_cast<unsigned short>(d)));     // exact, 2^-48 to 2^32
    return 15 - 2 * (BITS - 1) - (static_cast<int>(__float_as_uint(both) >> 23) - 126);
}
__device__ __forceinline__ float exp2_of(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// What a dequantising thread reads for one stage: four blocks and their steps.
template <int BITS> struct Step {
    Codes<BITS> c[4];
    unsigned short s[4];
};
}  // namespace

template <int BITS, int PHASE, int MAXN>
__global__ void __launch_bounds__(Cfg<BITS, PHASE, MAXN>::THREADS, 1) k_bwd_tc(
    TcArgs p, const __grid_constant__ CUtensorMap map) {
    using C = Cfg<BITS, PHASE, MAXN>;
    constexpr int SA = C::SA, SB = C::SB, ACC = C::ACC, NM = C::NM, ND = C::ND;
    constexpr int kEpi0 = C::DEQ, kMma = kEpi0 + C::EPI, kLoad0 = kMma + 1;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *fullA = bars, *emptyA = bars + SA, *fullB = bars + 2 * SA, *emptyB = bars + 2 * SA + SB;
    uint64_t *accF = bars + 2 * SA + 2 * SB, *accE = accF + 2, *drain = accF + 4;
    uint64_t *fullR = drain + 1, *emptyR = fullR + C::SR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int &abort_s = *(reinterpret_cast<int *>(bars + kBars) + 1);
    const FfnBackward &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.H, I = a.I;
    const int MT = (PHASE == 1 ? I : H) / kBM;                // weight tiles of 128 rows
    const int nk = (PHASE == 1 ? H : 2 * I) / C::KSTAGE;      // stages of a tile (even)
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < SA; ++i) {
            mbar_init(fullA + i, C::GROUP);
            mbar_init(emptyA + i, 1);
        }
        for (int i = 0; i < SB; ++i) {
            mbar_init(fullB + i, PHASE == 1 ? C::LOAD : 1);   // phase 2: and the copies' bytes
            mbar_init(emptyB + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accF + i, 1);
            mbar_init(accE + i, C::EPI);
        }
        for (int i = 0; i < C::SR; ++i) {
            mbar_init(fullR + i, 1);
            mbar_init(emptyR + i, C::GROUP);
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
    pdl_wait();                                               // the lists and rows of the kernel before
    // tiles: all weight rows of a token tile first, dealt to blocks round robin
    const int total = *p.n_tiles * MT, grid = static_cast<int>(gridDim.x), bid = static_cast<int>(blockIdx.x);
    const int n_my = bid < total ? (total - 1 - bid) / grid + 1 : 0;
    auto tile_of = [&](int i, int &m0) {
        const int t = bid + i * grid, g = t / MT;
        m0 = (t - g * MT) * kBM;
        return p.tiles[g];
    };
    auto fail = [&]() {
        report(a.err, MOE_DEVERR_TIMEOUT);
        abort_s = 1;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {         // a warp's wait: the same answer on every lane
        const bool ok = mbar_wait_ns(bar, parity, p.limit_ns, &abort_s);
        if (!ok && !abort_s) fail();
        return __all_sync(0xffffffffu, ok) != 0;
    };

    if (warp < C::DEQ) {
        // ------------------------------------------------- dequantisation
        // Group 0 takes the even stages, group 1 the odd ones.
        const int group = warp / C::GROUP, t = tid - group * 32 * C::GROUP;
        constexpr int BB = 4 * BITS;                          // bytes of a block's codes
        // phase 1: four warps g and u, a thread a row of the warp's TMEM lanes (its two blocks of g, then of
        // u), two warps q; q and phase 2: (K index + KS i, block of columns), neighbouring lanes the blocks
        // of a row.
        const bool trans = PHASE == 2 || t >= 128;
        constexpr int KS = PHASE == 1 ? 16 : 32;
        const int tt = PHASE == 1 ? t - 128 : t, b = tt & 3, r = tt >> 2;
        const int row_m = 32 * (warp & 3) + block_order<BITS>(lane);          // g and u: the row of the tile
        // the source of the next stage: pointers of the first block, distances of the others and of stages
        const uint8_t *cp = nullptr;
        const unsigned short *sp = nullptr;
        const int rowb = (PHASE == 1 && trans ? I : H) * BITS / 8, rows = (PHASE == 1 && trans ? I : H) / 32;
        const int cs = KS * rowb, ss = KS * rows;
        const int sstep = trans ? 2 * kBK * rows : 4;         // phase 1
        const size_t u_off = static_cast<size_t>(I) * H / 32; // from g's steps to u's
        int st = nk, next = 0, m0 = 0;                        // the next stage, the tile after this one
        BlobView bv = {};
        auto fetch = [&](Step<BITS> &o) {
            const bool start = st >= nk;
            if (start) {
                const TokTile te = tile_of(next++, m0);
                bv = blob_view(te.blob, BITS, H, I);
                st = group;
            }
            if (PHASE == 2 || start) {
                // phase 2: Wg's I / 128 stages, then Wu's
                const bool up = PHASE == 2 && st * C::KSTAGE >= I;
                const uint8_t *codes = up ? bv.cu : bv.cg;
                const __half *steps = PHASE == 2 ? (up ? bv.su : bv.sg) : trans ? bv.sd : bv.sg;
                const size_t row = trans ? st * C::KSTAGE - (up ? I : 0) + r : m0 + row_m;
                const int col = trans ? m0 / 32 + b : 2 * group;
                if (PHASE == 2) cp = codes + row * rowb + col * BB;
                sp = reinterpret_cast<const unsigned short *>(steps) + row * rows + col;
            }
            st += 2;
            if (trans) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (PHASE == 2) o.c[i] = load_codes<BITS>(cp + static_cast<size_t>(i) * cs);
                    o.s[i] = __ldg(sp + static_cast<size_t>(i) * ss);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t two = __ldg(reinterpret_cast<const unsigned *>(sp + i * u_off));
                    o.s[2 * i] = static_cast<unsigned short>(two), o.s[2 * i + 1] = static_cast<unsigned short>(two >> 16);
                }
            }
            if (PHASE == 1) sp += sstep;
        };
        // where the thread's blocks go within a stage
        const uint32_t sA = smem_addr(smem);
        const uint32_t to = (b >> 1) * 8192 + r * 128;
        const int c0 = 4 * (b & 1), sw = r & 7;
        const bool flip = b >= 2;
        const uint32_t to_t = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + C::COLS - C::TA;
        int sa = group % SA;
        uint32_t phase = 1;                                   // the first pass over the ring finds it empty
        auto put = [&](const Step<BITS> &o) {
            if (!wait(emptyA + sa, phase)) return false;
            if (trans) {
                const uint32_t at = sA + sa * C::A_STAGE + to;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // K rows KS i on: 128 bytes each, 64 rows a tile
                    const uint32_t off = PHASE == 1 ? i * KS * 128 : (i >> 1) * kMat + (i & 1) * KS * 128;
                    put_block<BITS>(o.c[i], __ushort_as_half(o.s[i]), at + off, c0, sw, flip);
                }
                fence_proxy_async();
            } else {
                tc_fence_after();                             // the MMAs that read the stage are done
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t words[16];
                    block_words<BITS>(o.c[i], __ushort_as_half(o.s[i]), words);
                    tmem_st16(to_t + sa * 64 + i * 16, words);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fullA + sa);
            sa += 2;
            if (sa >= SA) sa -= SA, phase ^= 1;
            return true;
        };
        const int n = n_my * (nk / 2);
        if constexpr (PHASE == 1) {
            Step<BITS> s0;
            // the thread's blocks of the raw tiles, as they lie in the matrices: four a row of Wd's, two of
            // the others', where half of the lanes read the second first (other banks)
            const uint8_t *raw = smem + C::OFF_RAW + (trans ? 2 * C::RAW_TILE + (r * 4 + b) * BB : row_m * 2 * BB);
            const bool second = lane & 4;
            int sr = group;
            uint32_t pr = 0;
            if (n > 0) fetch(s0);
            for (int i = 0; i < n; ++i) {
                if (!wait(fullR + sr, pr)) break;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int at = trans ? x * KS * 4 * BB : (x >> 1) * C::RAW_TILE + ((x & 1) ^ second) * BB;
                    s0.c[x] = raw_codes<BITS>(raw + sr * C::RAW_SLOT + at);
                }
                if (!trans && second) {
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        const Codes<BITS> c = s0.c[x];
                        s0.c[x] = s0.c[x + 1], s0.c[x + 1] = c;
                    }
                }
                // the reads are done before the next copy, of the asynchronous proxy, may write here
                // (the arrival alone does not wait for them)
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(emptyR + sr);
                sr += 2;
                if (sr >= C::SR) sr -= C::SR, pr ^= 1;
                if (!put(s0)) break;
                if (i + 1 < n) fetch(s0);
            }
        } else {
            // two ahead: a stage is shorter here (194 us one ahead, 167 two, at 64 tokens)
            Step<BITS> s0, s1;
            if (n > 0) fetch(s0);
            if (n > 1) fetch(s1);
            for (int i = 0; i < n; i += 2) {
                if (!put(s0)) break;
                if (i + 2 < n) fetch(s0);
                if (i + 1 >= n || !put(s1)) break;
                if (i + 3 < n) fetch(s1);
            }
        }
    } else if (PHASE == 1 && warp == kLoad0 + C::LOAD) {
        // ------------------------------------------------------------ codes
        const uint32_t on = elect_one();
        int sr = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int i = 0; i < n_my && ok; ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const int y = __shfl_sync(0xffffffffu, m0, 0);
            const CUtensorMap *maps = p.maps + 3 * static_cast<size_t>(__shfl_sync(0xffffffffu, te.g, 0));
#pragma unroll
            for (int m = 0; m < 3; ++m) map_acquire(maps + m);
            for (int s = 0; s < nk; ++s) {
                if (!(ok = wait(emptyR + sr, phase))) break;
                const uint32_t dst = smem_addr(smem + C::OFF_RAW + sr * C::RAW_SLOT);
                expect_tx_on(on, fullR + sr, C::RAW_SLOT);
                tma_load_on(on, dst, maps, s * kBK * BITS / 8, y, fullR + sr);
                tma_load_on(on, dst + C::RAW_TILE, maps + 1, s * kBK * BITS / 8, y, fullR + sr);
                tma_load_on(on, dst + 2 * C::RAW_TILE, maps + 2, y * BITS / 8, s * kBK, fullR + sr);
                if (++sr == C::SR) sr = 0, phase ^= 1;
                ++issued;
            }
        }
        // no copy is in flight when the block leaves, also when another role gave up
        for (int f = max(0, issued - C::SR); f < issued; ++f)
            (void)mbar_wait_ns(fullR + f % C::SR, (f / C::SR) & 1, kWaitNs, nullptr);
        __syncwarp();
    } else if (PHASE == 1 && warp >= kLoad0) {
        // ------------------------------------------------- rows of x and dy
        // A warp instruction copies 128 bytes of four rows.
        const int lw = warp - kLoad0, c = lane & 7, r0 = 4 * lw + (lane >> 3);
        constexpr int RSTEP = 4 * C::LOAD, R = (MAXN + RSTEP - 1) / RSTEP;     // rows of a lane: r0 + RSTEP r
        constexpr int D = 1;                                  // stages of copies in flight beyond the one issued
        int sb = 0, pub = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        auto publish = [&]() {                                // the stage issued D stages ago has landed
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(fullB + pub);
            if (++pub == SB) pub = 0;
        };
        for (int i = 0; i < n_my && ok; ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const int N = (te.n + 15) & ~15;
            size_t off[R];                                    // values from x16's (dy16's) start to the row's
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int q = r0 + RSTEP * r;
                int v = 0;
                if (q < te.n)
                    v = te.row0 >= 0 ? guard_index(a.perm_src[te.row0 + te.n0 + q], a.T, a.err, MOE_DEVERR_BAD_ROW)
                                     : te.n0 + q;
                off[r] = static_cast<size_t>(v) * H + 8 * c;
            }
            for (int s = 0; s < nk; ++s) {
                if (!(ok = wait(emptyB + sb, phase))) break;
                const uint32_t dst = smem_addr(smem + C::OFF_B + sb * C::B_STAGE);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int q = r0 + RSTEP * r;
                    if (q < N) {
                        const uint32_t to = dst + q * 128 + ((c ^ (q & 7)) << 4), bytes = q < te.n ? 16u : 0u;
                        const size_t at = off[r] + static_cast<uint32_t>(s * kBK);
                        cp_async16(to, p.x16 + at, bytes);
                        cp_async16(to + C::B_TILE, p.dy16 + at, bytes);
                    }
                }
                if (++sb == SB) sb = 0, phase ^= 1;
                cp_async_commit();
                if (issued++ >= D) {
                    cp_async_wait<D>();
                    publish();
                }
            }
        }
        cp_async_wait<0>();
        for (int i = 0; i < D && i < issued && ok; ++i) publish();
    } else if (PHASE == 2 && warp >= kLoad0) {
        // ------------------------------------------------- [dg | du] by TMA
        int sb = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        const uint32_t on = elect_one();
        if (lane == 0) tma_prefetch_map(&map);
        for (int i = 0; i < n_my && ok; ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const int n = __shfl_sync(0xffffffffu, te.n, 0), at = __shfl_sync(0xffffffffu, te.at, 0);
            for (int s = 0; s < nk; ++s) {
                if (!(ok = wait(emptyB + sb, phase))) break;
                const uint32_t dst = smem_addr(smem + C::OFF_B + sb * C::B_STAGE);
                expect_tx_on(on, fullB + sb, (n + 63) / 64 * 128 * 128);
                for (int n0 = 0; n0 < n; n0 += 64)            // 128 K rows of 64 tokens
                    tma_load_on(on, dst + n0 * 256, &map, at + n0, s * C::KSTAGE, fullB + sb);
                if (++sb == SB) sb = 0, phase ^= 1;
                ++issued;
            }
        }
        // no copy is in flight when the block leaves, also when another role gave up
        for (int f = max(0, issued - SB); f < issued; ++f)
            (void)mbar_wait_ns(fullB + f % SB, (f / SB) & 1, kWaitNs, nullptr);
        __syncwarp();
    } else if (warp < kMma) {
        // -------------------------------------------------------- epilogue
        static_assert(kEpi0 % 4 == 0, "TMEM lanes follow the warp's rank");
        const int ew = warp - kEpi0, q = ew & 3;              // TMEM lanes 32q .. 32q + 31
        const int m = 32 * q + block_order<BITS>(lane);       // the weight row (column) of this lane
        // each warp has its own table of the tile's scales (sx, c r): no barrier
        // among them, of which one may leave early
        float2 *sx_s = reinterpret_cast<float2 *>(smem + C::OFF_SX) + ew * MAXN;
        for (int i = 0; i < n_my; ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const size_t row0 = static_cast<size_t>(te.row0 >= 0 ? te.row0 : a.T * a.k) + te.n0;
            const int ce = group_exponent<BITS>(p, te.g);
            if constexpr (PHASE == 1) {
                __syncwarp();                                 // the last tile's scales are read
                for (int r = lane; r < ((te.n + 15) & ~15); r += 32) {
                    float2 sx = make_float2(0.f, 0.f);
                    if (r < te.n) {
                        const int t = te.row0 >= 0 ? guard_index(a.perm_src[te.row0 + te.n0 + r], a.T, nullptr, 0) : te.n0 + r;
                        const float4 sc = p.scale[t];
                        sx = make_float2(sc.x, exp2_of(ce) * sc.z);
                        if (m0 == 0 && ew == 0) p.ok[row0 + r] = 1;
                    }
                    sx_s[r] = sx;
                }
                __syncwarp();
            }
            const int acc = i % ACC;
            if (!wait(accF + acc, (i / ACC) & 1)) break;
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * ND * MAXN;
            if constexpr (PHASE == 1) {
                // eight columns at a time (sixteen: 943 us for 817 at 8192 tokens)
                for (int c0 = 0; c0 < te.n; c0 += 8) {
                    float gv[8], uv[8], qv[8];
                    tmem_ld8(base + c0, gv);
                    tmem_ld8(base + MAXN + c0, uv);
                    tmem_ld8(base + 2 * MAXN + c0, qv);
                    tmem_ld_wait();
                    uint32_t dg[4], du[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 sx = *reinterpret_cast<const float4 *>(sx_s + c0 + e);
                        float vg[2], vu[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float g = gv[e + x] * (x ? sx.z : sx.x);
                            const float s = __fdividef(1.f, 1.f + __expf(-g));
                            const float q2 = qv[e + x] * (x ? sx.w : sx.y);
                            const float qu = q2 * uv[e + x], act = gv[e + x] * s;               // a / sx
                            vg[x] = qu * fmaf(g * s, 1.f - s, s);
                            vu[x] = q2 * act;
                            qv[e + x] = qu * act;
                        }
                        const __half2 hg = __floats2half2_rn(vg[0], vg[1]), hu = __floats2half2_rn(vu[0], vu[1]);
                        dg[e / 2] = *reinterpret_cast<const uint32_t *>(&hg);
                        du[e / 2] = *reinterpret_cast<const uint32_t *>(&hu);
                    }
                    __half *og = p.gu16 + static_cast<size_t>(m0 + m) * p.cols + te.at + c0;
                    *reinterpret_cast<uint4 *>(og) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
                    *reinterpret_cast<uint4 *>(og + static_cast<size_t>(I) * p.cols) = make_uint4(du[0], du[1], du[2], du[3]);
                    if (te.row0 >= 0) {
                        // eight rows' sums over the warp's 32 lanes: halves are exchanged, so that each
                        // step halves the values a lane holds
#pragma unroll
                        for (int o = 4; o > 0; o >>= 1) {
                            const bool up = lane & (4 * o);
#pragma unroll
                            for (int e = 0; e < o; ++e) {
                                const float give = up ? qv[e] : qv[e + o], keep = up ? qv[e + o] : qv[e];
                                qv[e] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * o);
                            }
                        }
                        float sum = qv[0] + __shfl_xor_sync(0xffffffffu, qv[0], 2);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        const int r = c0 + (lane >> 2);
                        if (!(lane & 3) && r < te.n) {
                            const float inv = __uint_as_float(0x7F000000u - __float_as_uint(sx_s[r].y));   // 1 / (c r)
                            p.dwp[(row0 + r) * (I / 32) + m0 / 32 + q] = sum * inv;
                        }
                    }
                }
            } else {
                const float inv = exp2_of(-ce);
                for (int c0 = 0; c0 < te.n; c0 += 16) {
                    float v[16];
                    tmem_ld16(base + c0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= inv;
                    float *out = p.dxp + (row0 + c0) * H + m0 + m;
                    if (c0 + 16 <= te.n) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) out[static_cast<size_t>(e) * H] = v[e];
                    } else {
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
        const uint32_t on = elect_one();
        const uint32_t ring = smem_addr(smem), tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t mn = desc_mn_sw128(ring, 8192, 1024), km = desc_sw128(ring);
        const uint64_t mnb = desc_mn_sw128(ring, 16384, 1024);          // phase 2's B: atoms of 128 K rows
        int sa = 0, sb = 0;
        uint32_t pa = 0, pb = 0;
        bool ok = true;
        for (int i = 0; i < n_my && ok; ++i) {
            int m0;
            const TokTile te = tile_of(i, m0);
            const int N = __shfl_sync(0xffffffffu, (te.n + 15) & ~15, 0), acc = i % ACC;
            const uint32_t id_k = idesc_16bit(0, 0, 0, kBM, N), id_mn = idesc_16bit(0, 1, PHASE == 2, kBM, N);
            const uint32_t d = tm + acc * ND * MAXN;
            if (!(ok = wait(accE + acc, ((i / ACC) & 1) ^ 1))) break;
            tc_fence_after();
            for (int s = 0; s < nk; ++s) {
                if (!(ok = wait(fullB + sb, pb)) || !(ok = wait(fullA + sa, pa))) break;
                tc_fence_after();
                // descriptors count in 16 bytes from the ring's start
                const uint64_t as = (sa * C::A_STAGE) >> 4, bs = (C::OFF_B + sb * C::B_STAGE) >> 4;
#pragma unroll
                for (int mat = 0; mat < NM; ++mat) {
                    const bool trans = PHASE == 2 || mat == 2;
                    const uint64_t am = as + (PHASE == 1 ? 0 : mat * (kMat >> 4));
                    const uint64_t bm = bs + (PHASE == 1 ? (mat == 2) * (C::B_TILE >> 4) : mat * (8192 >> 4));
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        const uint64_t bk = PHASE == 2 ? mnb + bm + kk * 128 : km + bm + kk * 2;
                        const uint32_t dm = d + (PHASE == 1 ? mat : 0) * MAXN;
                        const uint32_t more = PHASE == 1 ? s | kk : s | kk | mat;
                        if (trans) mma_f16_on(on, dm, mn + am + kk * 128, bk, id_mn, more != 0);
                        else mma_f16_ts_on(on, dm, tm + C::COLS - C::TA + sa * 64 + mat * 32 + kk * 8, bk, id_k, more != 0);
                    }
                }
                mma_commit_on(on, emptyA + sa);
                mma_commit_on(on, emptyB + sb);
                if (++sa == SA) sa = 0, pa ^= 1;
                if (++sb == SB) sb = 0, pb ^= 1;
            }
            mma_commit_on(on, accF + acc);
        }
        mma_commit_on(on, drain);                             // TMEM is released once every MMA is done
        if (!mbar_wait_ns(drain, 0, kWaitNs, nullptr)) report(a.err, MOE_DEVERR_TIMEOUT);
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
constexpr int kStepLoads = 8;     // 16-byte loads of steps a thread has in flight

struct Prep {
    __half *x16, *dy16;
    float4 *scale;
    uint8_t *ok;
    uint32_t *steps;              // [groups, 32]
    int gu_parts, d_parts;        // parts of a group's steps, a block each
    TokTile *tiles1, *tiles2;
    int *counts;                  // token tiles of phase 1 and 2
    int max1, max2;               // tokens per tile
    int cap1, cap2;               // entries of the lists
    int cols;                     // columns of gu16
    CUtensorMap *maps;
};

// 2^-e and 2^e with e = floor(log2 top) of the row's largest |value| (bits
// `top`), held where both are normal numbers; 1 for a row of zeros or one that
// is not finite (its NaN or infinity goes through as it is).
__device__ __forceinline__ float2 row_scale(uint32_t top) {
    if (top == 0u || top >= 0x7F800000u) return make_float2(1.f, 1.f);
    const uint32_t e = min(max(top >> 23, 1u), 253u);
    return make_float2(__uint_as_float((254u - e) << 23), __uint_as_float(e << 23));
}

// The sum of the scaled row's |values| (its largest is in [1, 2), but for the
// ends of the range) from the plain row's; 2^15 covers H = 8192 where the plain
// sum is beyond fp32.  Nothing below 1, for rows of next to nothing.
__device__ __forceinline__ float scaled_sum(float sum, float inv_scale) {
    return fminf(fmaxf(sum * inv_scale, 1.f), 32768.f);
}

// Tiles of a group of n rows: as few as hold it, of equal size (a multiple of
// 16), so that no tile is left with a few rows.
__device__ __forceinline__ int tile_rows(int n, int most) {
    const int tiles = (n + most - 1) / most;
    return ((n + tiles - 1) / tiles + 15) & ~15;
}
}  // namespace

// Block 0 lists both phases' token tiles, the next T blocks scale and round one
// token's x and dy each, and the rest find the experts' largest steps, a part of
// a group's each, and make the maps of their codes.
// V: float4 a thread holds of a row.
// V = 2 is held to seven blocks an SM, a few registers spilled: the rows take
// 33 us at 8192 x 2048, for 48 with five blocks and none spilled.  Eight loads of
// steps in flight: 56 us with 512 experts' steps, 59 with four, 71 with two.
template <int V>
__global__ void __launch_bounds__(kPrepThreads, V <= 2 ? 7 : 1) k_bwd_prepare(FfnBackward a, Prep p,
                                                              const __grid_constant__ CUtensorMap rows_map,
                                                              const __grid_constant__ CUtensorMap down_map) {
    __shared__ uint32_t part[2][kPrepThreads / 32];
    __shared__ float part_sum[2][kPrepThreads / 32];
    __shared__ int3 sums[kPrepThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0) {
        const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), a.err);
        const int ng = n_act + (a.shared ? 1 : 0);
        int3 done = make_int3(0, 0, 0);                       // tiles of phase 1 and 2, columns of gu16
        for (int g0 = 0; g0 < ng; g0 += kPrepThreads) {
            const int g = g0 + tid;
            BwdGroup G = {nullptr, 0, -1};
            if (g < ng) G = bwd_group(a, g, n_act, true);
            int2 r = make_int2(16, 16);
            int3 c = make_int3(0, 0, 0);
            if (G.n > 0) {
                r = make_int2(tile_rows(G.n, p.max1), tile_rows(G.n, p.max2));
                c = make_int3((G.n + r.x - 1) / r.x, (G.n + r.y - 1) / r.y, (G.n + 15) & ~15);
            }
            int3 in = c;                                      // inclusive sums over the warp, then the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, in.x, o), y = __shfl_up_sync(0xffffffffu, in.y, o);
                const int z = __shfl_up_sync(0xffffffffu, in.z, o);
                if (lane >= o) in.x += x, in.y += y, in.z += z;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = in;
            __syncthreads();
            int3 at = make_int3(done.x + in.x - c.x, done.y + in.y - c.y, done.z + in.z - c.z);
            for (int w = 0; w < kPrepThreads / 32; ++w) {
                if (w < warp) at.x += sums[w].x, at.y += sums[w].y, at.z += sums[w].z;
                done.x += sums[w].x, done.y += sums[w].y, done.z += sums[w].z;
            }
            // consistent offsets never reach the lists' ends
            if (at.x + c.x > p.cap1 || at.y + c.y > p.cap2 || at.z + c.z > p.cols) {
                report(a.err, MOE_DEVERR_BAD_ROW);
                c = make_int3(0, 0, 0);
            }
            for (int i = 0; i < c.x; ++i)
                p.tiles1[at.x + i] = {G.blob, G.row0, i * r.x, min(r.x, G.n - i * r.x), at.z + i * r.x, g, 0};
            for (int i = 0; i < c.y; ++i)
                p.tiles2[at.y + i] = {G.blob, G.row0, i * r.y, min(r.y, G.n - i * r.y), at.z + i * r.y, g, 0};
        }
        pdl_next();
        const bool fits = done.x <= p.cap1 && done.y <= p.cap2 && done.z <= p.cols;
        if (tid == 0) p.counts[0] = fits ? done.x : 0, p.counts[1] = fits ? done.y : 0;
        return;
    }
    pdl_next();
    if (static_cast<int>(blockIdx.x) > a.T) {
        const int parts = p.gu_parts + p.d_parts, v = static_cast<int>(blockIdx.x) - a.T - 1;
        const int g = v / parts, at = v - g * parts;
        const int n_act = guard_count(a.active[0], min(a.E, a.T * a.k), nullptr);
        if (g >= n_act + (a.shared ? 1 : 0)) return;
        const BwdGroup G = bwd_group(a, g, n_act, false);
        if (G.n <= 0) return;
        const BlobView bv = blob_view(G.blob, a.bits, a.H, a.I);
        if (at == 0 && warp == 0) {                           // the maps of the three matrices' codes
            CUtensorMap *to = p.maps + 3 * static_cast<size_t>(g);
            map_for(to, rows_map, bv.cg);
            map_for(to + 1, rows_map, bv.cu);
            map_for(to + 2, down_map, bv.cd);
        }
        const bool down = at >= p.gu_parts;
        const int i = down ? at - p.gu_parts : at, most = down ? p.d_parts : p.gu_parts;
        const long n8 = static_cast<long>(down ? 1 : 2) * a.H * a.I / 32 / 8;               // eight steps a load
        const uint4 *steps = reinterpret_cast<const uint4 *>(down ? bv.sd : bv.sg);         // Wu's lie behind Wg's
        const long end = n8 * (i + 1) / most;
        uint32_t top2 = 0;
        for (long j = n8 * i / most + tid; j < end; j += kStepLoads * kPrepThreads) {
            uint4 u[kStepLoads];
#pragma unroll
            for (int x = 0; x < kStepLoads; ++x)
                u[x] = j + x * kPrepThreads < end ? __ldg(steps + j + x * kPrepThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < kStepLoads; ++x) {
                top2 = __vmaxu2(__vmaxu2(top2, u[x].x & 0x7FFF7FFFu), u[x].y & 0x7FFF7FFFu);
                top2 = __vmaxu2(__vmaxu2(top2, u[x].z & 0x7FFF7FFFu), u[x].w & 0x7FFF7FFFu);
            }
        }
        const uint32_t most1 = __reduce_max_sync(0xffffffffu, max(top2 & 0xFFFFu, top2 >> 16));
        if (lane == 0) part[0][warp] = most1;
        __syncthreads();
        if (tid == 0) {
            uint32_t m = 0;
            for (int w = 0; w < kPrepThreads / 32; ++w) m = max(m, part[0][w]);
            p.steps[32 * static_cast<size_t>(g) + (down ? 16 : 0) + i] = m;
            // a step whose lowest code's weight is beyond fp16: 65504 / 2^(bits - 1) and up
            if (m > 0x7BFFu - (static_cast<uint32_t>(a.bits - 1) << 10)) report(a.err, MOE_DEVERR_NONFINITE);
        }
        return;
    }
    const size_t t = blockIdx.x - 1;
    const int h4n = a.H / 4;
    if (tid < a.k) p.ok[t * a.k + tid] = 0;
    if (tid == 0) p.ok[static_cast<size_t>(a.T) * a.k + t] = 0;
    float4 v[2][V];                                           // x and dy, both rows' loads in flight
    uint32_t top[2] = {0, 0};
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int h4 = tid + i * kPrepThreads;
        if (h4 >= h4n) continue;
        v[0][i] = bwd_load4(a.x, a.x_scales, a.x_dtype, t, a.H, h4);
        v[1][i] = bwd_load4(a.dy, nullptr, a.dy_dtype, t, a.H, h4);
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (tid + i * kPrepThreads >= h4n) continue;
            const float4 &u = v[which][i];
            top[which] = max(max(top[which], __float_as_uint(fabsf(u.x))), __float_as_uint(fabsf(u.y)));
            top[which] = max(max(top[which], __float_as_uint(fabsf(u.z))), __float_as_uint(fabsf(u.w)));
            sum[which] += (fabsf(u.x) + fabsf(u.y)) + (fabsf(u.z) + fabsf(u.w));
        }
        top[which] = __reduce_max_sync(0xffffffffu, top[which]);
        sum[which] = warp_sum(sum[which]);
        if (lane == 0) part[which][warp] = top[which], part_sum[which][warp] = sum[which];
    }
    __syncthreads();
    float2 scale[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int w = 0; w < kPrepThreads / 32; ++w) top[which] = max(top[which], part[which][w]);
        const float2 sc = scale[which] = row_scale(top[which]);
        // x in the order of the blocks that it meets as K of g and u
        uint2 *out = reinterpret_cast<uint2 *>((which ? p.dy16 : p.x16) + t * a.H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int h4 = tid + i * kPrepThreads;
            if (h4 >= h4n) continue;
            const float4 &u = v[which][i];
            const float y = which ? u.y : u.z, z = which ? u.z : u.y;
            __half2 lo = __floats2half2_rn(u.x * sc.x, y * sc.x), hi = __floats2half2_rn(z * sc.x, u.w * sc.x);
            uint2 o;
            o.x = *reinterpret_cast<uint32_t *>(&lo);
            o.y = *reinterpret_cast<uint32_t *>(&hi);
            out[which ? h4 : (h4 & ~7) + block_place(a.bits, h4 & 7) / 4] = o;
        }
    }
    if (tid == 0) {
        float both = 1.f;                                     // the two sums' product
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kPrepThreads / 32; ++w) s += part_sum[which][w];
            if (top[which] < 0x7F800000u) both *= scaled_sum(s, scale[which].x);
        }
        const int e = static_cast<int>(__float_as_uint(both) >> 23) - 126;     // the product is below 2^e
        p.scale[t] = make_float4(scale[0].y, scale[1].y, exp2_of(-e), exp2_of(e));
    }
}

// ------------------------------------------------------------------ launch
namespace {
struct TcPlan {
    bool large;
    int max1, max2;
    size_t tiles1, tiles2;        // bounds on the token tiles
    size_t cols;                  // and on the rows, each group's padded to 16
    size_t groups;
    int gu_parts, d_parts;        // blocks that look through a group's steps
};
constexpr int kSmallN = 64, kLargeN1 = 128, kLargeN2 = 256;

TcPlan plan_of(int T, int k, int H, int I, int E) {
    const long rows = static_cast<long>(T) * k, groups = rows < E ? rows : E;
    TcPlan p;
    p.large = rows > 32L * groups;
    p.max1 = p.large ? kLargeN1 : kSmallN;
    p.max2 = p.large ? kLargeN2 : kSmallN;
    // a group of n rows has at most n / most + 1 tiles, and rounding a tile up to 16 rows adds none
    auto bound = [&](int most) { return static_cast<size_t>(rows / most + groups + T / most + 1); };
    p.tiles1 = bound(p.max1);
    p.tiles2 = bound(p.max2);
    p.groups = static_cast<size_t>(groups + 1);
    p.cols = static_cast<size_t>((rows + T + 15 * (groups + 1) + 63) / 64 * 64);
    // a part is one round of a block's loads (32 KB), or a sixteenth
    auto parts = [&](long steps) {
        const long n = (steps / 8 + kStepLoads * kPrepThreads - 1) / (kStepLoads * kPrepThreads);
        return static_cast<int>(n < 16 ? n : 16);
    };
    p.gu_parts = parts(2L * H * I / 32);
    p.d_parts = parts(1L * H * I / 32);
    return p;
}

struct TcWs {
    __half *x16, *dy16, *gu16;
    float4 *scale;
    uint32_t *steps;
    float *dwp, *dxp;
    uint8_t *ok;
    TokTile *tiles1, *tiles2;
    int *counts;
    CUtensorMap *maps;
};

// The parts of a workspace at `base` (a multiple of kWsAlign: the maps' addresses
// need 128), each at a multiple of kWsAlign; returns their bytes.
size_t carve(int T, int k, int H, int I, int E, uint8_t *base, TcWs *out) {
    const size_t rows = static_cast<size_t>(T) * k, all = rows + T;
    const TcPlan p = plan_of(T, k, H, I, E);
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t *q = base ? base + at : nullptr;
        at += (n + kWsAlign - 1) / kWsAlign * kWsAlign;
        return q;
    };
    TcWs w;
    w.x16 = reinterpret_cast<__half *>(take(static_cast<size_t>(T) * H * 2));
    w.dy16 = reinterpret_cast<__half *>(take(static_cast<size_t>(T) * H * 2));
    w.gu16 = reinterpret_cast<__half *>(take(p.cols * 2 * I * 2));
    w.scale = reinterpret_cast<float4 *>(take(static_cast<size_t>(T) * sizeof(float4)));
    w.steps = reinterpret_cast<uint32_t *>(take(p.groups * 32 * sizeof(uint32_t)));
    w.dwp = reinterpret_cast<float *>(take(rows * (I / 32) * 4));
    w.dxp = reinterpret_cast<float *>(take(all * H * 4));
    w.ok = take(all);
    w.tiles1 = reinterpret_cast<TokTile *>(take(p.tiles1 * sizeof(TokTile)));
    w.tiles2 = reinterpret_cast<TokTile *>(take(p.tiles2 * sizeof(TokTile)));
    w.counts = reinterpret_cast<int *>(take(2 * sizeof(int)));
    w.maps = reinterpret_cast<CUtensorMap *>(take(p.groups * 3 * sizeof(CUtensorMap)));
    if (out) *out = w;
    return at;
}

template <int BITS, int PHASE, int MAXN>
int launch_phase(const TcArgs &p, const CUtensorMap &map, cudaStream_t s) {
    using C = Cfg<BITS, PHASE, MAXN>;
    int rc = cuda_status(cudaFuncSetAttribute(k_bwd_tc<BITS, PHASE, MAXN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(C::SMEM)),
                         "backward gemm smem attribute");
    if (rc) return rc;
    rc = cuda_status(launch_after(k_bwd_tc<BITS, PHASE, MAXN>, dim3(num_sms()), C::THREADS, C::SMEM, s, p, map),
                     "backward gemm launch");
    if (!rc) count_launches(1);
    return rc;
}
}  // namespace

size_t ffn_backward_gemm_ws_bytes(int T, int k, int H, int I, int E) {
    return carve(T, k, H, I, E, nullptr, nullptr) + kWsSlack;
}

bool ffn_backward_gemm_supported(int T, int k, int H, int I, int E) {
    // tile and step numbers are ints
    const TcPlan p = plan_of(T, k, H, I, E);
    const double n1 = static_cast<double>(p.tiles1) * (I / kBM), n2 = static_cast<double>(p.tiles2) * (H / kBM);
    if (p.cols > 2000000000u) return false;
    return n1 < 2e9 && n2 < 2e9 && (n1 / num_sms() + 1) * (H / kBK) < 2e9 && (n2 / num_sms() + 1) * (I / kBK) < 2e9;
}

int launch_ffn_backward_gemm(const FfnBackward &a, void *ws, cudaStream_t s) {
    TcWs w;
    carve(a.T, a.k, a.H, a.I, a.E, ws_start(ws), &w);
    const TcPlan plan = plan_of(a.T, a.k, a.H, a.I, a.E);
    const Prep prep = {w.x16, w.dy16, w.scale, w.ok, w.steps, plan.gu_parts, plan.d_parts, w.tiles1, w.tiles2, w.counts, plan.max1, plan.max2,
                       static_cast<int>(plan.tiles1), static_cast<int>(plan.tiles2),
                       static_cast<int>(plan.cols), w.maps};
    // (the base is a stand-in: each group's maps get their own)
    CUtensorMap rows_map, down_map;
    const uint64_t rowb = static_cast<uint64_t>(a.H) * a.bits / 8, downb = static_cast<uint64_t>(a.I) * a.bits / 8;
    int rc = make_byte_map(&rows_map, w.x16, a.I, rowb, kBM, kBK * a.bits / 8);
    if (!rc) rc = make_byte_map(&down_map, w.x16, a.H, downb, kBK, kBM * a.bits / 8);
    if (rc) return rc;
    const unsigned blocks = static_cast<unsigned>(a.T + 1 + plan.groups * (plan.gu_parts + plan.d_parts));
    if (a.H <= 2048) k_bwd_prepare<2><<<blocks, kPrepThreads, 0, s>>>(a, prep, rows_map, down_map);
    else k_bwd_prepare<8><<<blocks, kPrepThreads, 0, s>>>(a, prep, rows_map, down_map);
    count_launches(1);
    rc = cuda_status(cudaGetLastError(), "backward prepare launch");
    if (rc) return rc;
    const long long hook = test_hook_value(MOE_HOOK_WAIT_LIMIT_NS);
    const unsigned long long limit = hook > 0 ? static_cast<unsigned long long>(hook) : kWaitNs;
    const TcArgs p = {a, w.scale, w.steps, plan.gu_parts, plan.d_parts, w.gu16, static_cast<int>(plan.cols), w.x16, w.dy16, w.dwp, w.dxp, w.ok, w.maps,
                      w.tiles1, w.counts, limit};
    TcArgs p2 = p;
    p2.tiles = w.tiles2, p2.n_tiles = w.counts + 1;
    CUtensorMap map;
    rc = make_tensor_map(&map, w.gu16, 0, 2 * static_cast<uint64_t>(a.I), plan.cols, plan.cols * 2, 2 * kBK);
    if (rc) return rc;
    if (a.bits == 4) {
        rc = plan.large ? launch_phase<4, 1, kLargeN1>(p, map, s) : launch_phase<4, 1, kSmallN>(p, map, s);
        if (!rc) rc = plan.large ? launch_phase<4, 2, kLargeN2>(p2, map, s) : launch_phase<4, 2, kSmallN>(p2, map, s);
    } else {
        rc = plan.large ? launch_phase<2, 1, kLargeN1>(p, map, s) : launch_phase<2, 1, kSmallN>(p, map, s);
        if (!rc) rc = plan.large ? launch_phase<2, 2, kLargeN2>(p2, map, s) : launch_phase<2, 2, kSmallN>(p2, map, s);
    }
    if (rc) return rc;
    return launch_ffn_backward_gather(a, w.dxp, w.dwp, a.I / 32, w.ok, w.scale, s);
}

}  // namespace moe

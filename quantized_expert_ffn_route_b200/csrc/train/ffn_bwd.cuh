// What the two forms of the experts' backward pass share: the groups of a
// step, reading x and dy rows, and the final gather.
#pragma once

#include "common.cuh"
#include "train/act8.cuh"
#include "train/train.h"

namespace moe {

// One expert's rows (or every token, for the shared expert).
struct BwdGroup {
    const uint8_t *blob;
    int n;       // rows
    int row0;    // first permuted row, or -1 for the shared expert
};

// Group g: active expert g, or the shared expert when g == n_act.  n = 0 where
// there is nothing to do; what is wrong is reported by the thread with `say`.
__device__ __forceinline__ BwdGroup bwd_group(const FfnBackward &a, int g, int n_act, bool say) {
    BwdGroup G = {nullptr, 0, -1};
    unsigned bad = 0;
    if (g < n_act) {
        const int e = a.active[1 + g];
        if (e < 0 || e >= a.E) {
            bad = MOE_DEVERR_BAD_EXPERT;
        } else {
            const int r0 = a.offsets[e], r1 = a.offsets[e + 1];
            G.blob = a.blobs[e];
            if (r0 < 0 || r1 < r0 || r1 > a.T * a.k) bad = MOE_DEVERR_BAD_ROW;
            else if (!G.blob) bad = MOE_DEVERR_NULL_BLOB;
            else if (reinterpret_cast<uintptr_t>(G.blob) & 15u) bad = MOE_DEVERR_MISALIGNED;
            G.row0 = r0;
            G.n = r1 - r0;
        }
    } else {
        G.blob = a.shared;
        G.n = a.T;
    }
    if (bad) {
        if (say) report(a.err, bad);
        G.n = 0;
    }
    return G;
}

// The token of row r of a group.
__device__ __forceinline__ int bwd_token(const FfnBackward &a, const BwdGroup &G, int r) {
    return G.row0 >= 0 ? guard_index(a.perm_src[G.row0 + r], a.T, a.err, MOE_DEVERR_BAD_ROW) : r;
}

// Values 4 h4 .. 4 h4 + 3 of a token's x or dy row (kind MOE_F32, MOE_BF16 or MOE_Q8).
__device__ __forceinline__ float4 bwd_load4(const void *x, const uint8_t *scales, int kind, size_t tok, int H,
                                            int h4) {
    const size_t i = tok * (H / 4) + h4;
    if (kind == MOE_F32) return load4(static_cast<const float *>(x) + 4 * i);
    if (kind == MOE_BF16) return load4(static_cast<const __nv_bfloat16 *>(x) + 4 * i);
    float v[4];
    act8_values(static_cast<const uint32_t *>(x)[i], act8_step(scales[i >> 3]), v);
    return make_float4(v[0], v[1], v[2], v[3]);
}

}  // namespace moe

// Internal launchers of libmoe's training side (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_train.h"

namespace moe {

int launch_act_pack8(const void *x, int x_dtype, size_t n, int8_t *codes, uint8_t *scales, cudaStream_t s);
int launch_act_unpack8(const int8_t *codes, const uint8_t *scales, size_t n, void *x, int x_dtype, cudaStream_t s);

size_t balance_ws_bytes(int T, int E);
int launch_balance_loss(const float *logits, const int32_t *ids, const uint8_t *mask, int T, int E, int k,
                        float balance_coef, float z_coef, int32_t *counts, float *loss, void *ws, unsigned *err,
                        cudaStream_t s);
int launch_route_backward(const float *logits, const int32_t *ids, const float *w, const float *dw,
                          const uint8_t *mask, const int32_t *counts, const float *d_loss, int T, int E, int k,
                          float balance_coef, float z_coef, void *dl, int dl_dtype, unsigned *err, cudaStream_t s);

// Arguments of the experts' backward pass, as the caller gave them.
struct FfnBackward {
    const uint8_t *const *blobs;
    const int32_t *offsets, *active, *perm_src, *perm_dst;
    const float *topk_w;
    const void *x;
    const uint8_t *x_scales;
    const void *dy;
    const uint8_t *shared;
    void *dx;
    float *d_topk_w;
    int bits, x_dtype, dy_dtype, dx_dtype, T, k, H, I, E;
    unsigned *err;
};
size_t ffn_backward_gemv_ws_bytes(int T, int k, int H, int I);
int launch_ffn_backward_gemv(const FfnBackward &a, void *ws, cudaStream_t s);
size_t ffn_backward_gemm_ws_bytes(int T, int k, int H, int I, int E);
bool ffn_backward_gemm_supported(int T, int k, int H, int I, int E);
int launch_ffn_backward_gemm(const FfnBackward &a, void *ws, cudaStream_t s);
// dx and d_topk_w from the rows' parts: dxp [T*k + T, H], dwp [T*k, shares], ok
// [T*k + T] (rows that were computed: the others' parts are not read); scale
// [T] (sx, sd, r, 1/r) where dxp is kept times r / (sx sd) and dwp divided by
// sx sx sd, or NULL.
int launch_ffn_backward_gather(const FfnBackward &a, const float *dxp, const float *dwp, int shares,
                               const uint8_t *ok, const float4 *scale, cudaStream_t s);

struct RouterBackward {
    const void *dl, *x, *w;
    const float *dx_in;
    void *dx, *d_w;
    float *d_bias;
    int dl_dtype, x_dtype, w_dtype, dx_dtype, T, H, E;
    unsigned *err;
};
int launch_router_backward_simt(const RouterBackward &a, cudaStream_t s);
bool router_backward_tc_supported(int T, int H, int E, int dl_dtype, int x_dtype, int w_dtype);
size_t router_backward_tc_ws_bytes(int T, int H, int E);
int launch_router_backward_tc(const RouterBackward &a, void *ws, cudaStream_t s);

}  // namespace moe

// C ABI of libmoe's training side: argument validation, workspace sizing and dispatch.
#include "common.cuh"
#include "train/train.h"

using namespace moe;

namespace {
bool float_dtype(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
}  // namespace

extern "C" {

// ------------------------------------------------ activation checkpoints
int moe_act_pack8(const void *x, int x_dtype, int T, int H, int8_t *codes, uint8_t *scales, moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_act_pack8");
    set_error("%s", "");
    REQUIRE(T >= 0, "T must be >= 0 (got %d)", T);
    REQUIRE(H >= 32 && H % 32 == 0, "H must be a positive multiple of 32 (got %d)", H);
    REQUIRE(float_dtype(x_dtype), "x_dtype must be MOE_F32 or MOE_BF16");
    if (T == 0) return MOE_OK;
    REQUIRE(x && codes && scales, "x/codes/scales must not be NULL");
    REQUIRE(x != static_cast<const void *>(codes), "x and codes must not be the same buffer");
    REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales), "x/codes/scales must be 16-byte aligned");
    return launch_act_pack8(x, x_dtype, static_cast<size_t>(T) * H, codes, scales, reinterpret_cast<cudaStream_t>(s));
}

int moe_act_unpack8(const int8_t *codes, const uint8_t *scales, int T, int H, void *x, int x_dtype, moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_act_unpack8");
    set_error("%s", "");
    REQUIRE(T >= 0, "T must be >= 0 (got %d)", T);
    REQUIRE(H >= 32 && H % 32 == 0, "H must be a positive multiple of 32 (got %d)", H);
    REQUIRE(float_dtype(x_dtype), "x_dtype must be MOE_F32 or MOE_BF16");
    if (T == 0) return MOE_OK;
    REQUIRE(x && codes && scales, "x/codes/scales must not be NULL");
    REQUIRE(x != static_cast<const void *>(codes), "x and codes must not be the same buffer");
    REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales), "x/codes/scales must be 16-byte aligned");
    return launch_act_unpack8(codes, scales, static_cast<size_t>(T) * H, x, x_dtype, reinterpret_cast<cudaStream_t>(s));
}

// ----------------------------------------------------------- balance loss
size_t moe_balance_ws_size(int T, int E) { return T <= 0 || E <= 0 ? 0 : balance_ws_bytes(T, E); }

static int check_routing(int T, int E, int k) {
    REQUIRE(T >= 0, "T must be >= 0 (got %d)", T);
    REQUIRE(E >= 1 && E <= 32768, "E must be in [1, 32768] (got %d)", E);
    REQUIRE(k >= 1 && k <= 32 && k <= E, "k must be in [1, min(E, 32)] (got k=%d, E=%d)", k, E);
    REQUIRE(static_cast<long>(T) * k <= (1L << 30), "T*k too large");
    return MOE_OK;
}

int moe_balance_loss(const float *logits, const int32_t *topk_ids, const uint8_t *token_mask, int T, int E, int k,
                     float balance_coef, float z_coef, int32_t *counts, float *loss, void *ws, size_t ws_bytes,
                     moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_balance_loss");
    set_error("%s", "");
    const int rc = check_routing(T, E, k);
    if (rc) return rc;
    REQUIRE(counts && loss, "counts/loss must not be NULL");
    REQUIRE(aligned16(counts) && aligned16(loss), "counts/loss must be 16-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    if (T == 0) {
        const int m = cuda_status(cudaMemsetAsync(counts, 0, (static_cast<size_t>(E) + 1) * 4, st), "counts memset");
        return m ? m : cuda_status(cudaMemsetAsync(loss, 0, 16, st), "loss memset");
    }
    REQUIRE(logits && topk_ids, "logits/topk_ids must not be NULL");
    REQUIRE(aligned16(logits) && aligned16(topk_ids), "logits/topk_ids must be 16-byte aligned");
    REQUIRE(ws && ws_bytes >= balance_ws_bytes(T, E) && aligned16(ws), "workspace too small: need %zu bytes",
            balance_ws_bytes(T, E));
    unsigned *err = device_error_word();
    if (!err) return cuda_status(cudaErrorInvalidDevice, "device error word");
    return launch_balance_loss(logits, topk_ids, token_mask, T, E, k, balance_coef, z_coef, counts, loss, ws, err, st);
}

int moe_route_backward(const float *logits, const int32_t *topk_ids, const float *topk_w, const float *d_topk_w,
                       const uint8_t *token_mask, const int32_t *counts, const float *d_loss, int T, int E, int k,
                       float balance_coef, float z_coef, void *d_logits, int dl_dtype, moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_route_backward");
    set_error("%s", "");
    const int rc = check_routing(T, E, k);
    if (rc) return rc;
    REQUIRE(float_dtype(dl_dtype), "dl_dtype must be MOE_F32 or MOE_BF16");
    if (T == 0) return MOE_OK;
    REQUIRE(d_logits && aligned16(d_logits), "d_logits must be given and 16-byte aligned");
    REQUIRE((topk_w != nullptr) == (d_topk_w != nullptr), "topk_w and d_topk_w go together (both or neither)");
    REQUIRE(d_logits != static_cast<const void *>(logits), "d_logits must not be logits");
    REQUIRE(!counts || logits, "logits is NULL while counts asks for the loss's gradient");
    REQUIRE(!d_topk_w || topk_ids, "topk_ids is NULL while d_topk_w is given");
    REQUIRE((!logits || aligned16(logits)) && (!topk_ids || aligned16(topk_ids)) && (!topk_w || aligned16(topk_w)) &&
                (!d_topk_w || aligned16(d_topk_w)) && (!counts || aligned16(counts)),
            "logits/topk_ids/topk_w/d_topk_w/counts must be 16-byte aligned");
    REQUIRE((reinterpret_cast<uintptr_t>(d_loss) & 3u) == 0, "d_loss must be 4-byte aligned");
    unsigned *err = device_error_word();
    if (!err) return cuda_status(cudaErrorInvalidDevice, "device error word");
    if (balance_coef == 0.f && z_coef == 0.f) counts = nullptr;          // no loss term
    return launch_route_backward(logits, topk_ids, topk_w, d_topk_w, token_mask, counts, d_loss, T, E, k, balance_coef,
                                 z_coef, d_logits, dl_dtype, err, reinterpret_cast<cudaStream_t>(s));
}

// ---------------------------------------------------------------- experts
// Up to four tokens on CUDA cores: a group has a row or two then, and the tensor
// cores' form pays three launches' latencies and tiles of 64 rows.  Measured as
// graphs with a shared expert, us on CUDA cores : on tensor cores, 4 bits | 2 bits:
//                              1 token         4 tokens          6 tokens         16 tokens
//   2048 x 512, top-10 of 512  29:46 | 29:45    73:82 | 67:77   108:96 | 96:88    247:183 | 231:171
//   2048 x 512, top-4 of 64    21:40 | 20:38    34:45 | 34:44    48:49 | 48:47    111:57  | 107:53
//   4096 x 1536, top-4 of 32   58:83 | 57:80   153:149 | 141:135 225:169 | 211:154 481:245 | 465:229
// Rows an expert and a blob's bytes move the crossing by a token or two; nowhere
// here does the rule cost more than 4 %.  From five tokens on the operands are
// thereby rounded to fp16, as the forward pass's are in its GEMM mode; fp32
// throughout at 16 tokens would take 1.3 to 2 times as long, and MOE_MODE_GEMV
// asks for it.
static int backward_mode(int mode, int T) {
    if (mode == MOE_MODE_AUTO) return T <= 4 ? MOE_MODE_GEMV : MOE_MODE_GEMM;
    return mode;
}

size_t moe_expert_ffn_backward_ws_size(int bits, int T, int k, int H, int I, int E, int mode) {
    if ((bits != 2 && bits != 4) || T <= 0 || k <= 0 || H <= 0 || I <= 0 || E <= 0) return 0;
    mode = backward_mode(mode, T);
    return mode == MOE_MODE_GEMM ? ffn_backward_gemm_ws_bytes(T, k, H, I, E) : ffn_backward_gemv_ws_bytes(T, k, H, I);
}

int moe_expert_ffn_backward(int bits, const void *const *expert_blobs, const int32_t *expert_offsets,
                            const int32_t *active, const int32_t *perm_src, const int32_t *perm_dst,
                            const float *topk_w, const void *x, int x_dtype, const uint8_t *x_scales,
                            const void *dy, int dy_dtype, int T, int k, int H, int I, int E,
                            const void *shared_blob, void *dx, int dx_dtype, float *d_topk_w, int mode, void *ws,
                            size_t ws_bytes, moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_expert_ffn_backward");
    set_error("%s", "");
    REQUIRE(bits == 4 || bits == 2, "bits must be 4 or 2 (got %d)", bits);
    const int rc = check_routing(T, E, k);
    if (rc) return rc;
    REQUIRE(H >= 128 && H % 128 == 0 && H <= 8192, "H must be a multiple of 128 in [128, 8192] (got %d)", H);
    REQUIRE(I >= 128 && I % 128 == 0 && I <= 4096, "I must be a multiple of 128 in [128, 4096] (got %d)", I);
    REQUIRE(mode == MOE_MODE_AUTO || mode == MOE_MODE_GEMV || mode == MOE_MODE_GEMM, "bad mode %d", mode);
    REQUIRE(float_dtype(x_dtype) || x_dtype == MOE_Q8, "x_dtype must be MOE_F32, MOE_BF16 or MOE_Q8");
    REQUIRE(float_dtype(dy_dtype) && float_dtype(dx_dtype), "dy_dtype/dx_dtype must be MOE_F32 or MOE_BF16");
    if (T == 0) return MOE_OK;
    REQUIRE(expert_blobs && expert_offsets && active && perm_src && perm_dst && topk_w && x && dy && dx && d_topk_w,
            "expert_blobs/expert_offsets/active/perm_src/perm_dst/topk_w/x/dy/dx/d_topk_w must not be NULL");
    REQUIRE((x_dtype == MOE_Q8) == (x_scales != nullptr), "x_scales goes with x_dtype MOE_Q8, and only with it");
    REQUIRE(aligned16(expert_blobs) && aligned16(expert_offsets) && aligned16(active) && aligned16(perm_src) &&
                aligned16(perm_dst) && aligned16(topk_w) && aligned16(x) && aligned16(x_scales) && aligned16(dy) &&
                aligned16(dx) && aligned16(d_topk_w) && aligned16(shared_blob),
            "the buffers must be 16-byte aligned");
    REQUIRE(dx != dy && dx != x, "dx must not be x or dy");
    mode = backward_mode(mode, T);
    REQUIRE(mode == MOE_MODE_GEMV || ffn_backward_gemm_supported(T, k, H, I, E), "too many tiles for GEMM mode");
    const size_t need = moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, mode);
    REQUIRE(ws && ws_bytes >= need && aligned16(ws), "workspace too small: need %zu bytes", need);
    unsigned *err = device_error_word();
    if (!err) return cuda_status(cudaErrorInvalidDevice, "device error word");
    FfnBackward a;
    a.blobs = reinterpret_cast<const uint8_t *const *>(expert_blobs);
    a.offsets = expert_offsets, a.active = active, a.perm_src = perm_src, a.perm_dst = perm_dst;
    a.topk_w = topk_w;
    a.x = x, a.x_scales = x_scales, a.dy = dy;
    a.shared = static_cast<const uint8_t *>(shared_blob);
    a.dx = dx, a.d_topk_w = d_topk_w;
    a.bits = bits, a.x_dtype = x_dtype, a.dy_dtype = dy_dtype, a.dx_dtype = dx_dtype;
    a.T = T, a.k = k, a.H = H, a.I = I, a.E = E;
    a.err = err;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    return mode == MOE_MODE_GEMM ? launch_ffn_backward_gemm(a, ws, st) : launch_ffn_backward_gemv(a, ws, st);
}

// ----------------------------------------------------------------- router
size_t moe_router_backward_ws_size(int T, int H, int E, int dl_dtype, int x_dtype, int w_dtype) {
    if (T <= 0 || H <= 0 || E <= 0 || !router_backward_tc_supported(T, H, E, dl_dtype, x_dtype, w_dtype)) return 0;
    return router_backward_tc_ws_bytes(T, H, E);
}

int moe_router_backward(const void *d_logits, int dl_dtype, const void *x, int x_dtype, const void *w_router,
                        int w_dtype, const float *dx_in, int T, int H, int E, void *dx, int dx_dtype, void *d_w,
                        float *d_bias, void *ws, size_t ws_bytes, moe_stream_t s) {
    moe::NvtxRange nvtx_range("moe_router_backward");
    set_error("%s", "");
    REQUIRE(T >= 0, "T must be >= 0 (got %d)", T);
    REQUIRE(T <= (1 << 30), "T too large (got %d)", T);
    REQUIRE(E >= 1 && E <= 32768, "E must be in [1, 32768] (got %d)", E);
    REQUIRE(H >= 8 && H % 8 == 0, "H must be a positive multiple of 8 (got %d)", H);
    REQUIRE(float_dtype(dl_dtype) && float_dtype(x_dtype) && float_dtype(w_dtype) && float_dtype(dx_dtype),
            "dl_dtype/x_dtype/w_dtype/dx_dtype must be MOE_F32 or MOE_BF16");
    REQUIRE(dx || d_w || d_bias, "dx, d_w and d_bias are all NULL");
    REQUIRE(T == 0 || d_logits, "d_logits is NULL");
    REQUIRE(T == 0 || !dx || w_router, "w_router is NULL while dx is asked for");
    REQUIRE(T == 0 || !d_w || x, "x is NULL while d_w is asked for");
    REQUIRE(aligned16(d_logits) && aligned16(x) && aligned16(w_router) && aligned16(dx_in) && aligned16(dx) &&
                aligned16(d_w) && aligned16(d_bias),
            "d_logits/x/w_router/dx_in/dx/d_w/d_bias must be 16-byte aligned");
    REQUIRE(!dx || dx != static_cast<const void *>(dx_in) || dx_dtype == MOE_F32, "dx may be dx_in only in MOE_F32");
    REQUIRE(!dx || (dx != d_logits && dx != x && dx != w_router), "dx must not be d_logits, x or w_router");
    REQUIRE(!d_w || (d_w != d_logits && d_w != x && d_w != w_router && d_w != dx && d_w != static_cast<const void *>(dx_in)),
            "d_w must not be d_logits, x, w_router, dx_in or dx");
    const size_t need = moe_router_backward_ws_size(T, H, E, dl_dtype, x_dtype, w_dtype);
    REQUIRE(need == 0 || (ws && ws_bytes >= need && aligned16(ws)), "workspace too small: need %zu bytes", need);
    unsigned *err = device_error_word();
    if (!err) return cuda_status(cudaErrorInvalidDevice, "device error word");
    const RouterBackward a = {d_logits, x, w_router, dx_in, dx, d_w, d_bias, dl_dtype, x_dtype, w_dtype, dx_dtype,
                              T, H, E, err};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    if (router_backward_tc_supported(T, H, E, dl_dtype, x_dtype, w_dtype)) return launch_router_backward_tc(a, ws, st);
    return launch_router_backward_simt(a, st);
}

}  // extern "C"

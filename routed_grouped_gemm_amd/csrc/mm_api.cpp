// C ABI of the 16-bit and block-scaled FP8 grouped products, the block
// quantisers and the checkpointed activation: argument validation only
// (nothing is launched before a call is found valid; the workspace a product
// needs follows from its plan, which asks for the device's compute units).
#include <hip/hip_runtime.h>
#include "mm_check.h"

namespace {

int32_t check_glu(const moe_epilogue* e) {
    if (!e) return MOE_OK;
    if (e->act != MOE_ACT_SWIGLU && e->act != MOE_ACT_GEGLU && e->act != MOE_ACT_SRELU) return MOE_ERR_UNSUPPORTED;
    if (e->bias || e->save_pre) return MOE_ERR_UNSUPPORTED;
    if (!(e->beta > 0.0f) || !isfinite(e->beta) || !(e->limit >= 0.0f) || !isfinite(e->limit)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

}  // namespace

MOE_EXPORT size_t moe_grouped_mm_workspace_size(int32_t R_max, int32_t G, int32_t N, int32_t K) {
    if (check_dims(R_max, N, K, G, 8)) return 0;
    return moe_mm_workspace_bytes(0, false, R_max, G, N, K);
}

MOE_EXPORT int32_t moe_grouped_mm(const void* x, int32_t x_rows, int32_t ldx, const int32_t* row_src, const void* w,
                                  int32_t dtype, const int32_t* offsets, int32_t R_max, int32_t N, int32_t K,
                                  int32_t G, uint32_t flags, void* y, int32_t ldy, void* ws, size_t ws_bytes,
                                  hipStream_t stream) {
    if (!t16(dtype) || (flags & ~MOE_MM_W_KN)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_dims(R_max, N, K, G, 8);
    if (st) return st;
    if (ldy < N || ldy % 4 || ldy > kMaxLd) return MOE_ERR_SHAPE;
    if ((st = check_rows(x, x_rows, K, ldx, 2, row_src, R_max))) return st;
    if (R_max == 0) return MOE_OK;
    if (!w || !offsets || !y) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(y, 8)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_grouped_mm_workspace_size(R_max, G, N, K), ws, ws_bytes))) return st;
    MmCall c{};
    c.kind = (flags & MOE_MM_W_KN) ? 1 : 0;
    c.dtype = dtype;
    c.x = x; c.x_rows = x_rows; c.ldx = ldx; c.x_src = row_src;
    c.w = w; c.offsets = offsets;
    c.R_max = R_max; c.N = N; c.K = K; c.G = G;
    c.out = y; c.ldy = ldy; c.ws = ws; c.ws_bytes = ws_bytes;
    return hip_status(moe_launch_mm(c, stream));
}

MOE_EXPORT size_t moe_grouped_wgrad_workspace_size(int32_t R_max, int32_t G, int32_t N, int32_t K) {
    if (check_dims(R_max, N, K, G, 8)) return 0;
    return moe_mm_workspace_bytes(2, false, R_max, G, N, K);
}

MOE_EXPORT int32_t moe_grouped_wgrad(const void* dy, int32_t dy_rows, int32_t ld_dy, const int32_t* dy_src,
                                     const void* x, int32_t x_rows, int32_t ldx, const int32_t* x_src,
                                     const float* xs, int32_t dtype, const int32_t* offsets, int32_t R_max,
                                     int32_t N, int32_t K, int32_t G, uint32_t flags, void* dw, void* ws,
                                     size_t ws_bytes, hipStream_t stream) {
    if (!t16(dtype) || (flags & ~(MOE_WGRAD_ACCUMULATE | MOE_WGRAD_F32))) return MOE_ERR_UNSUPPORTED;
    // (codes times scales reach past fp16's range, and the product's operands
    // are of one type: 8-bit rows are decoded to bf16, with bf16 gradients)
    if (xs && dtype != MOE_T_BF16) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_dims(R_max, N, K, G, 8);
    if (st) return st;
    if ((st = check_rows(dy, dy_rows, N, ld_dy, 2, dy_src, R_max))) return st;
    if (xs) {
        // 8-bit rows are read in pieces of 8 bytes
        if (x_rows < 0 || ldx < K || ldx % 8 || ldx > kMaxLd) return MOE_ERR_SHAPE;
        if (x_rows < (x_src ? (R_max > 0 ? 1 : 0) : R_max)) return MOE_ERR_SHAPE;
        if (x_src && (int64_t)x_rows * ldx >= kGatherBytes) return MOE_ERR_SHAPE;
        if (R_max > 0 && !x) return MOE_ERR_NULL;
        if (!aligned(x, 8)) return MOE_ERR_SHAPE;
    } else if ((st = check_rows(x, x_rows, K, ldx, 2, x_src, R_max))) {
        return st;
    }
    if (!offsets || !dw) return MOE_ERR_NULL;
    if (!aligned(dw, (flags & MOE_WGRAD_F32) ? 16 : 8)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_grouped_wgrad_workspace_size(R_max, G, N, K), ws, ws_bytes))) return st;
    MmCall c{};
    c.kind = 2;
    c.dtype = dtype;
    c.x = x; c.x_rows = x_rows; c.ldx = ldx; c.x_src = x_src; c.xs = xs;
    c.dy = dy; c.dy_rows = dy_rows; c.ld_dy = ld_dy; c.dy_src = dy_src;
    c.offsets = offsets;
    c.R_max = R_max; c.N = N; c.K = K; c.G = G;
    c.out = dw; c.out_f32 = (flags & MOE_WGRAD_F32) != 0; c.accumulate = (flags & MOE_WGRAD_ACCUMULATE) != 0;
    c.ws = ws; c.ws_bytes = ws_bytes;
    return hip_status(moe_launch_mm(c, stream));
}

MOE_EXPORT int32_t moe_quantize_block(const void* x, int32_t dtype, int32_t rows, int32_t K, int32_t ld,
                                      const int32_t* n_rows, uint8_t* q, float* s, hipStream_t stream) {
    if (!t16(dtype) && dtype != MOE_T_F32) return MOE_ERR_UNSUPPORTED;
    const int eb = dtype == MOE_T_F32 ? 4 : 2;
    if (rows < 0 || K < 8 || K % 8 || K > MOE_MM_MAX_DIM || ld < K || ((int64_t)ld * eb) % 16) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !s) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 8)) return MOE_ERR_SHAPE;
    return hip_status(moe_launch_quantize_block(x, dtype, rows, K, ld, n_rows, q, s, stream));
}

MOE_EXPORT int32_t moe_quantize_block_weights(const void* w, int32_t dtype, int32_t G, int32_t N, int32_t K,
                                              uint8_t* q, float* s, hipStream_t stream) {
    if (!t16(dtype) && dtype != MOE_T_F32) return MOE_ERR_UNSUPPORTED;
    if (G < 0 || G > MOE_MAX_EXPERTS + 1 || N < 1 || N > MOE_MM_MAX_DIM || K < 8 || K % 8 || K > MOE_MM_MAX_DIM)
        return MOE_ERR_SHAPE;
    if (G == 0) return MOE_OK;
    if (!w || !q || !s) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(q, 8)) return MOE_ERR_SHAPE;
    return hip_status(moe_launch_quantize_block_weights(w, dtype, G, N, K, q, s, stream));
}

MOE_EXPORT size_t moe_grouped_mm_fp8_workspace_size(int32_t R_max, int32_t G, int32_t N, int32_t K) {
    if (check_dims(R_max, N, K, G, 16)) return 0;
    return moe_mm_workspace_bytes(0, true, R_max, G, N, K);
}

MOE_EXPORT int32_t moe_grouped_mm_fp8(const uint8_t* xq, const float* xs, int32_t x_rows, const int32_t* row_src,
                                      const uint8_t* wq, const float* wscale, const int32_t* offsets, int32_t R_max,
                                      int32_t N, int32_t K, int32_t G, int32_t dtype, void* y, int32_t ldy, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
    if (!t16(dtype)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_dims(R_max, N, K, G, 16);
    if (st) return st;
    if (ldy < N || ldy % 4 || ldy > kMaxLd) return MOE_ERR_SHAPE;
    if ((st = check_rows(xq, x_rows, K, K, 1, row_src, R_max))) return st;
    if (R_max == 0) return MOE_OK;
    if (!xs || !wq || !wscale || !offsets || !y) return MOE_ERR_NULL;
    if (!aligned(wq, 16) || !aligned(y, 8)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_grouped_mm_fp8_workspace_size(R_max, G, N, K), ws, ws_bytes))) return st;
    MmCall c{};
    c.kind = 0;
    c.dtype = dtype; c.fp8 = true;
    c.x = xq; c.x_rows = x_rows; c.ldx = K; c.x_src = row_src; c.xs = xs;
    c.w = wq; c.wscale = wscale; c.offsets = offsets;
    c.R_max = R_max; c.N = N; c.K = K; c.G = G;
    c.out = y; c.ldy = ldy; c.ws = ws; c.ws_bytes = ws_bytes;
    return hip_status(moe_launch_mm(c, stream));
}

MOE_EXPORT int32_t moe_grouped_mm_plan(int32_t R_max, int32_t G, int32_t N, int32_t K, int32_t fp8,
                                       int32_t* tile_rows, int32_t* parts) {
    const int32_t st = check_dims(R_max, N, K, G, fp8 ? 16 : 8);
    if (st) return st;
    if (!tile_rows || !parts) return MOE_ERR_NULL;
    moe_mm_plan(fp8 != 0, R_max, G, N, K, tile_rows, parts);
    return MOE_OK;
}

MOE_EXPORT int32_t moe_grouped_wgrad_plan(int32_t R_max, int32_t G, int32_t N, int32_t K, int32_t* part_rows) {
    const int32_t st = check_dims(R_max, N, K, G, 8);
    if (st) return st;
    if (!part_rows) return MOE_ERR_NULL;
    *part_rows = moe_wgrad_plan(R_max, G, N, K);
    return MOE_OK;
}

MOE_EXPORT int32_t moe_glu_checkpoint(const void* pre, int32_t dtype, int32_t rows, int32_t I, int32_t ld,
                                      const float* row_w, const int32_t* n_rows, const moe_epilogue* epi, void* h,
                                      uint8_t* q, float* s, hipStream_t stream) {
    if (!t16(dtype)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_glu(epi);
    if (st) return st;
    if (rows < 0 || I < 8 || I % 8 || I > MOE_MM_MAX_DIM || ld < 2 * I || ld % 8) return MOE_ERR_SHAPE;
    if ((q == nullptr) != (s == nullptr)) return MOE_ERR_NULL;
    if (rows == 0) return MOE_OK;
    if (!pre || !h) return MOE_ERR_NULL;
    if (!aligned(pre, 16) || !aligned(h, 16) || !aligned(q, 8)) return MOE_ERR_SHAPE;
    GluCall c{};
    c.dtype = dtype; c.rows = rows; c.I = I; c.ld = ld; c.row_w = row_w; c.n_rows = n_rows;
    c.act = epi ? epi->act : MOE_ACT_SWIGLU; c.beta = epi ? epi->beta : 1.0f; c.limit = epi ? epi->limit : 0.0f;
    c.in = pre; c.h = h; c.q = q; c.s = s;
    return hip_status(moe_launch_glu_forward(c, stream));
}

MOE_EXPORT int32_t moe_glu_checkpoint_backward(const uint8_t* q, const float* s, const void* dh, int32_t dtype,
                                               int32_t rows, int32_t I, int32_t ld_dh, const float* row_w,
                                               const int32_t* n_rows, const moe_epilogue* epi, void* dpre, void* h,
                                               float* dw, hipStream_t stream) {
    if (!t16(dtype)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_glu(epi);
    if (st) return st;
    if (rows < 0 || I < 8 || I % 8 || I > MOE_MM_MAX_DIM || ld_dh < I || ld_dh % 8) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!q || !s || !dh || !dpre) return MOE_ERR_NULL;
    if (!aligned(q, 8) || !aligned(dh, 16) || !aligned(dpre, 16) || !aligned(h, 16)) return MOE_ERR_SHAPE;
    GluCall c{};
    c.dtype = dtype; c.rows = rows; c.I = I; c.ld = ld_dh; c.row_w = row_w; c.n_rows = n_rows;
    c.act = epi ? epi->act : MOE_ACT_SWIGLU; c.beta = epi ? epi->beta : 1.0f; c.limit = epi ? epi->limit : 0.0f;
    c.in = dh; c.q_in = q; c.s_in = s; c.dpre = dpre; c.h = h; c.dw = dw;
    return hip_status(moe_launch_glu_backward(c, stream));
}

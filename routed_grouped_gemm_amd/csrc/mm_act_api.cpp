// C ABI of the products with an epilogue and their gradients, the layer for a
// few tokens and the router's gradient: argument validation only (nothing is
// launched before a call is found valid).
#include <hip/hip_runtime.h>

#include "mm_check.h"

namespace {

// activation, slope and limit of an epilogue (NULL: the call's default)
int32_t check_act(const moe_epilogue* e) {
    if (!e) return MOE_OK;
    if (e->act < MOE_ACT_SWIGLU || e->act > MOE_ACT_NONE) return MOE_ERR_UNSUPPORTED;
    if (!(e->beta > 0.0f) || !isfinite(e->beta) || !(e->limit >= 0.0f) || !isfinite(e->limit)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int32_t check_few_sizes(int32_t T, int32_t k, int32_t E_loc, int32_t s) {
    if (T < 0 || T > MOE_FEW_MAX_TOKENS || k < 1 || E_loc < 1 || E_loc > MOE_MAX_EXPERTS) return MOE_ERR_SHAPE;
    return s < 0 || s > 1 || k > MOE_MAX_SLOTS - s ? MOE_ERR_SHAPE : MOE_OK;
}

// largest hidden and inner size of moe_layer_few, and bound on the values of h
constexpr int32_t kFewMaxDim = 65536;
constexpr int64_t kFewMaxH = 1ll << 26;

}  // namespace

MOE_EXPORT size_t moe_layer_few_workspace_size(int32_t T, int32_t k, int32_t E_loc, int32_t H, int32_t I,
                                               int32_t s) {
    if (check_few_sizes(T, k, E_loc, s) || H < 8 || H > kFewMaxDim || I < 8 || I > kFewMaxDim) return 0;
    if ((int64_t)T * (k + s) * I >= kFewMaxH) return 0;
    return moe_few_bytes(T, k, E_loc + s, s, I);
}

MOE_EXPORT int32_t moe_layer_few(const moe_few_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!a) return MOE_ERR_NULL;
    if (!t16(a->dtype) || (a->flags & ~MOE_ROUTE_RENORM)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_act(a->epi);
    if (st) return st;
    if (a->epi && a->epi->save_pre) return MOE_ERR_UNSUPPORTED;
    if ((a->shared_w1 == nullptr) != (a->shared_w2 == nullptr)) return MOE_ERR_NULL;
    const int32_t s = a->shared_w1 ? 1 : 0;
    if ((st = check_few_sizes(a->T, a->k, a->E_loc, s))) return st;
    if (a->E_tot < a->k || a->E_tot > MOE_MAX_EXPERTS || a->e0 < 0 || a->e0 > MOE_MAX_EXPERTS - a->E_loc) return MOE_ERR_SHAPE;
    // scales of every weight array, or of none
    const bool eight = a->w1_scales != nullptr;
    if ((a->w2_scales != nullptr) != eight) return MOE_ERR_NULL;
    if ((a->shared_w1_scales != nullptr) != (eight && s) || (a->shared_w2_scales != nullptr) != (eight && s)) return MOE_ERR_NULL;
    const int32_t mult = eight ? 16 : 8;
    if (a->H < mult || a->H % mult || a->H > kFewMaxDim || a->I < mult || a->I % mult || a->I > kFewMaxDim) return MOE_ERR_SHAPE;
    if ((int64_t)2 * a->I * a->H * (eight ? 1 : 2) >= kGatherBytes) return MOE_ERR_SHAPE;
    if ((int64_t)a->T * (a->k + s) * a->I >= kFewMaxH) return MOE_ERR_SHAPE;
    if (a->ldx < a->H || a->ldx % 8 || a->ldx > kMaxLd || a->ld_out < a->H || (a->residual && a->ld_res < a->H)) return MOE_ERR_SHAPE;
    if (a->T == 0) return MOE_OK;
    if (!a->logits || !a->x || !a->w1 || !a->w2 || !a->out) return MOE_ERR_NULL;
    if (!aligned(a->x, 16) || !aligned(a->w1, 16) || !aligned(a->w2, 16) || !aligned(a->shared_w1, 16) || !aligned(a->shared_w2, 16))
        return MOE_ERR_SHAPE;
    if (!aligned(a->logits, a->E_tot % 4 ? 4 : 16) || !aligned(a->out, 2) || !aligned(a->residual, 2)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_few_bytes(a->T, a->k, a->E_loc + s, s, a->I), ws, ws_bytes))) return st;
    return hip_status(moe_launch_few(*a, ws, stream));
}

// a 16-bit array that is read or written beside the operands: 8-byte pieces of rows
static bool bad_rows(const void* p, int32_t ld, int32_t cols) { return ld < cols || ld % 4 || ld > kMaxLd || !aligned(p, 8); }

// sizes of a product with an epilogue; n: its output columns
static int32_t check_act_dims(int32_t R_max, int32_t N, int32_t K, int32_t G, uint32_t flags) {
    const int32_t st = check_dims(R_max, N, K, G, 8);
    if (st) return st;
    if (!(flags & MOE_MM_GATED)) return MOE_OK;
    // gate and up rows of a group are addressed together, by 32-bit offsets
    return N % 16 || (int64_t)N * K * 2 >= kGatherBytes ? MOE_ERR_SHAPE : MOE_OK;
}

MOE_EXPORT int32_t moe_grouped_mm_act_plan(int32_t R_max, int32_t G, int32_t N, int32_t K, uint32_t flags,
                                           int32_t plan[6]) {
    if (flags & ~MOE_MM_GATED) return MOE_ERR_UNSUPPORTED;
    const int32_t st = check_act_dims(R_max, N, K, G, flags);
    if (st) return st;
    if (!plan) return MOE_ERR_NULL;
    moe_mm_act_plan(R_max, G, (flags & MOE_MM_GATED) ? N / 2 : N, K, (flags & MOE_MM_GATED) != 0, plan);
    return MOE_OK;
}

MOE_EXPORT size_t moe_grouped_mm_act_workspace_size(int32_t R_max, int32_t G, int32_t N, int32_t K) {
    if (check_dims(R_max, N, K, G, 8)) return 0;
    return moe_mm_act_bytes(R_max, G, N, K);
}

MOE_EXPORT int32_t moe_grouped_mm_act(const void* x, int32_t x_rows, int32_t ldx, const int32_t* row_src, const void* w,
                                      int32_t dtype, const int32_t* offsets, int32_t R_max, int32_t N, int32_t K,
                                      int32_t G, uint32_t flags, const moe_epilogue* epi, const float* row_w,
                                      const void* residual, int32_t ld_res, void* y, int32_t ldy, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
    const bool gated = (flags & MOE_MM_GATED) != 0, kn = (flags & MOE_MM_W_KN) != 0;
    if (!t16(dtype) || (flags & ~(MOE_MM_W_KN | MOE_MM_GATED)) || (gated && kn)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_act(epi);
    if (st) return st;
    if ((st = check_act_dims(R_max, N, K, G, flags))) return st;
    const int32_t cols = gated ? N / 2 : N;
    if (ldy < cols || ldy % 4 || ldy > kMaxLd) return MOE_ERR_SHAPE;
    if (residual && bad_rows(residual, ld_res, cols)) return MOE_ERR_SHAPE;
    if ((st = check_rows(x, x_rows, K, ldx, 2, row_src, R_max))) return st;
    if (R_max == 0) return MOE_OK;
    if (!w || !offsets || !y) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(y, 8)) return MOE_ERR_SHAPE;
    if (epi && (!aligned(epi->bias, 16) || !aligned(epi->save_pre, 16))) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_mm_act_bytes(R_max, G, N, K), ws, ws_bytes))) return st;
    MmActCall c{};
    c.dtype = dtype; c.gated = gated; c.kn = kn;
    c.x = x; c.x_rows = x_rows; c.ldx = ldx; c.x_src = row_src;
    c.w = w; c.offsets = offsets;
    c.R_max = R_max; c.N = cols; c.K = K; c.G = G;
    c.act = epi ? epi->act : (gated ? MOE_ACT_SWIGLU : MOE_ACT_NONE);
    c.beta = epi ? epi->beta : 1.0f; c.limit = epi ? epi->limit : 0.0f;
    c.bias = epi ? epi->bias : nullptr; c.pre = epi ? epi->save_pre : nullptr;
    c.row_w = row_w; c.res = residual; c.ld_res = ld_res;
    c.out = y; c.ldy = ldy; c.ws = ws;
    return hip_status(moe_launch_mm_act(c, stream));
}

MOE_EXPORT size_t moe_grouped_mm_dact_workspace_size(int32_t R_max, int32_t G, int32_t N, int32_t K) {
    if (check_dims(R_max, N, K, G, 8)) return 0;
    return moe_mm_dact_bytes(R_max, G, N, K);
}

MOE_EXPORT int32_t moe_grouped_mm_dact(const void* dy, int32_t dy_rows, int32_t ld_dy, const int32_t* dy_src,
                                       const void* w, int32_t dtype, const int32_t* offsets, int32_t R_max, int32_t N,
                                       int32_t K, int32_t G, uint32_t flags, const moe_epilogue* epi, const void* pre,
                                       int32_t ld_pre, const float* row_w, void* dpre, void* h, float* dw, void* ws,
                                       size_t ws_bytes, hipStream_t stream) {
    const bool gated = (flags & MOE_MM_GATED) != 0;
    if (!t16(dtype) || (flags & ~(MOE_MM_W_KN | MOE_MM_GATED))) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_act(epi);
    if (st) return st;
    if ((st = check_dims(R_max, N, K, G, 8))) return st;
    if (bad_rows(pre, ld_pre, gated ? 2 * N : N)) return MOE_ERR_SHAPE;
    if ((st = check_rows(dy, dy_rows, K, ld_dy, 2, dy_src, R_max))) return st;
    if (R_max == 0) return MOE_OK;
    if (!w || !offsets || !pre || !dpre) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(dpre, 16) || !aligned(h, 16)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_mm_dact_bytes(R_max, G, N, K), ws, ws_bytes))) return st;
    MmActCall c{};
    c.dtype = dtype; c.grad = true; c.gated = gated; c.kn = (flags & MOE_MM_W_KN) != 0;
    c.x = dy; c.x_rows = dy_rows; c.ldx = ld_dy; c.x_src = dy_src;
    c.w = w; c.offsets = offsets;
    c.R_max = R_max; c.N = N; c.K = K; c.G = G;
    c.act = epi ? epi->act : (gated ? MOE_ACT_SWIGLU : MOE_ACT_NONE);
    c.beta = epi ? epi->beta : 1.0f; c.limit = epi ? epi->limit : 0.0f;
    c.row_w = row_w; c.pre = const_cast<void*>(pre); c.ld_pre = ld_pre;
    c.out = dpre; c.h = h; c.dw = dw; c.ws = ws;
    return hip_status(moe_launch_mm_dact(c, stream));
}

MOE_EXPORT size_t moe_grouped_bias_grad_workspace_size(int32_t R_max, int32_t G, int32_t N) {
    if (check_dims(R_max, N, 8, G, 8)) return 0;
    return moe_bias_grad_bytes(R_max, N);
}

MOE_EXPORT int32_t moe_grouped_bias_grad(const void* dy, int32_t dy_rows, int32_t ld_dy, const int32_t* dy_src,
                                         const float* row_w, int32_t dtype, const int32_t* offsets, int32_t R_max,
                                         int32_t N, int32_t G, uint32_t flags, float* db, void* ws, size_t ws_bytes,
                                         hipStream_t stream) {
    if (!t16(dtype) || (flags & ~MOE_WGRAD_ACCUMULATE)) return MOE_ERR_UNSUPPORTED;
    int32_t st = check_dims(R_max, N, 8, G, 8);
    if (st) return st;
    if ((st = check_rows(dy, dy_rows, N, ld_dy, 2, dy_src, R_max))) return st;
    if (!offsets || !db) return MOE_ERR_NULL;
    if (!aligned(db, 16)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_bias_grad_bytes(R_max, N), ws, ws_bytes))) return st;
    BiasGradCall c{};
    c.dtype = dtype;
    c.dy = dy; c.dy_rows = dy_rows; c.ld_dy = ld_dy; c.dy_src = dy_src; c.row_w = row_w; c.offsets = offsets;
    c.R_max = R_max; c.N = N; c.G = G; c.accumulate = (flags & MOE_WGRAD_ACCUMULATE) != 0;
    c.out = db; c.ws = ws;
    return hip_status(moe_launch_bias_grad(c, stream));
}

MOE_EXPORT int32_t moe_route_backward(const float* logits, int32_t T, int32_t E_tot, int32_t k, uint32_t flags,
                                      const int32_t* topk_idx, const float* dw, int32_t dw_rows,
                                      const int32_t* slot_row, int32_t ld_slot, const float* prob_grad, float z_coef,
                                      float* dlogits, hipStream_t stream) {
    if (flags & ~MOE_ROUTE_RENORM) return MOE_ERR_UNSUPPORTED;
    if (T < 0 || E_tot < 1 || E_tot > MOE_MAX_EXPERTS || k < 1 || k > E_tot || k > MOE_MAX_SLOTS) return MOE_ERR_SHAPE;
    if (dw_rows < 0 || (slot_row && ld_slot < k) || (!slot_row && dw_rows < (int64_t)T * k)) return MOE_ERR_SHAPE;
    if (!isfinite(z_coef)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || (!dw && dw_rows > 0) || !dlogits) return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(dlogits, 4)) return MOE_ERR_SHAPE;
    RouteGradCall c{};
    c.logits = logits; c.T = T; c.E_tot = E_tot; c.k = k; c.flags = flags;
    c.topk_idx = topk_idx; c.dw = dw; c.dw_rows = dw_rows; c.slot_row = slot_row; c.ld_slot = ld_slot;
    c.prob_grad = prob_grad; c.z_coef = z_coef; c.dlogits = dlogits;
    return hip_status(moe_launch_route_backward(c, stream));
}

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

// largest hidden and inner size of moe_layer_few
constexpr int32_t kFewMaxDim = 65536;

}  // namespace

MOE_EXPORT size_t moe_layer_few_workspace_size(int32_t T, int32_t k, int32_t E_loc, int32_t I, int32_t s) {
    if (check_few_sizes(T, k, E_loc, s) || I < 8 || I > kFewMaxDim) return 0;
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
    if (a->ldx < a->H || a->ldx % 8 || a->ldx > kMaxLd || a->ld_out < a->H || (a->residual && a->ld_res < a->H)) return MOE_ERR_SHAPE;
    if (a->T == 0) return MOE_OK;
    if (!a->logits || !a->x || !a->w1 || !a->w2 || !a->out) return MOE_ERR_NULL;
    if (!aligned(a->x, 16) || !aligned(a->w1, 16) || !aligned(a->w2, 16) || !aligned(a->shared_w1, 16) || !aligned(a->shared_w2, 16))
        return MOE_ERR_SHAPE;
    if (!aligned(a->logits, a->E_tot % 4 ? 4 : 16) || !aligned(a->out, 2) || !aligned(a->residual, 2)) return MOE_ERR_SHAPE;
    if ((st = check_ws(moe_few_bytes(a->T, a->k, a->E_loc + s, s, a->I), ws, ws_bytes))) return st;
    return hip_status(moe_launch_few(*a, ws, stream));
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

// The router's gradient: from the gradients of the routing weights to those of
// the logits. For one token with p = softmax(l) over its E logits, the chosen
// experts e_j and D_j the gradient of weight j (0 where the expert is not here):
//
//   weights p_{e_j}:          dl_e = p_e (sum_{j: e_j = e} D_j - sum_j D_j p_{e_j})
//   divided by their sum S:   dl_e = sum_{j: e_j = e} w_j (D_j - sum_i D_i w_i),  w_j = p_{e_j} / S
//   balance term sum_e c_e p_e:   + p_e (c_e - sum_i c_i p_i)
//   z term z lse^2:               + 2 z lse p_e
//
// Bound by HBM where there are many tokens (the logits in, their gradient out,
// each once), by latency below. 16, 32 or 64 lanes hold a token's logits, 4
// consecutive ones to a lane and round, so its sums are a few DPP steps and a
// wave reads whole lines. Measured: 16384 tokens of 64
// experts with both terms, and 4099 tokens of 250, 10 us a call, which is host
// time.
#include "grouped_mm.h"

namespace {

constexpr int kRgThreads = 256;

struct RouteGradP {
    const float* logits; const int32_t* idx; const float* dw; const int32_t* slot;
    const float* prob_grad; float* out;
    int T, E, k, ld_slot, dw_rows, renorm, vec;             // vec: rows at multiples of 16 bytes
    float z;
};

// LPT lanes a token, 4 * NV logits a lane: logit 4 (LPT n + lane) + v
template <int LPT, int NV>
__global__ __launch_bounds__(kRgThreads)
void route_grad_kernel(RouteGradP p) {
    constexpr int TPB = kRgThreads / LPT;
    const int li = threadIdx.x & (LPT - 1);
    const int E = p.E;
    const int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / LPT;
    const bool here = t < p.T;
    const float* row = p.logits + (here ? t : 0) * E;
    const bool vec = p.vec != 0;
    f32x4 l[NV];
    #pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int e = 4 * (LPT * n + li);
        if (vec && e < E) l[n] = *(const f32x4*)(row + e);
        else {
            #pragma unroll
            for (int v = 0; v < 4; ++v) l[n][v] = e + v < E ? row[e + v] : -INFINITY;
        }
    }
    // the chosen experts: lane j holds number j (k <= LPT)
    int e_j = -1;
    float d_j = 0.f;
    if (here && li < p.k) {
        e_j = p.idx[t * p.k + li];
        if ((uint32_t)e_j >= (uint32_t)E) e_j = -1;
        const int64_t at = p.slot ? p.slot[t * p.ld_slot + li] : t * p.k + li;
        if (e_j >= 0 && (!p.slot || (uint64_t)at < (uint64_t)p.dw_rows)) d_j = p.dw[at];
    }
    const float l_j = e_j >= 0 ? row[e_j] : -INFINITY;

    float m = -INFINITY;
    #pragma unroll
    for (int n = 0; n < NV; ++n)
        #pragma unroll
        for (int v = 0; v < 4; ++v) m = fmaxf(m, l[n][v]);
    m = group_max<LPT>(m);
    if (m == -INFINITY) m = 0.f;                             // every expert masked: all p are 0, and the gradient
    float total = 0.f;
    #pragma unroll
    for (int n = 0; n < NV; ++n)
        #pragma unroll
        for (int v = 0; v < 4; ++v) {
            l[n][v] = expf(l[n][v] - m);
            total += l[n][v];
        }
    total = group_sum<LPT>(total);
    const float inv = total > 0.f ? 1.0f / total : (total == 0.f ? 0.f : total);
    const float lse = total == 0.f ? 0.f : m + logf(total);
    float w_j;
    if (p.renorm) {
        // (relative to the largest of the chosen: choices need not hold the row's largest
        // logit, and far below it their exponentials have few bits, or none)
        float mc = group_max<LPT>(l_j);
        if (mc == -INFINITY) mc = 0.f;
        const float x = e_j >= 0 ? expf(l_j - mc) : 0.f, s = group_sum<LPT>(x);
        w_j = s == 0.f ? 0.f : x / s;
        // a NaN or +inf elsewhere in the row makes its weights NaN here too
        if (!(total < INFINITY)) w_j = e_j >= 0 ? total - total : 0.f;
    } else {
        w_j = e_j >= 0 ? expf(l_j - m) * inv : 0.f;
    }
    const float mean = group_sum<LPT>(d_j * w_j);
    // what number j adds to its expert: scaled by p_e with the other terms, or by itself
    const float add_j = p.renorm ? w_j * (d_j - mean) : d_j;

    float cmean = 0.f;
    f32x4 c[NV];
    if (p.prob_grad) {
        #pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int e = 4 * (LPT * n + li);
            #pragma unroll
            for (int v = 0; v < 4; ++v) {
                c[n][v] = e + v < E ? p.prob_grad[e + v] : 0.f;
                l[n][v] *= inv;
                cmean += c[n][v] * l[n][v];
            }
        }
        cmean = group_sum<LPT>(cmean);
    } else {
        #pragma unroll
        for (int n = 0; n < NV; ++n)
            #pragma unroll
            for (int v = 0; v < 4; ++v) { c[n][v] = 0.f; l[n][v] *= inv; }
    }
    const float all = (p.renorm ? 0.f : -mean) - cmean + 2.0f * p.z * lse;
    f32x4 own[NV];
    #pragma unroll
    for (int n = 0; n < NV; ++n) own[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int first = threadIdx.x & 63 & ~(LPT - 1);
    for (int j = 0; j < p.k; ++j) {
        const int e = __shfl(e_j, first + j, 64);
        const float a = __shfl(add_j, first + j, 64);
        #pragma unroll
        for (int n = 0; n < NV; ++n)
            #pragma unroll
            for (int v = 0; v < 4; ++v) own[n][v] += 4 * (LPT * n + li) + v == e ? a : 0.f;
    }
    if (!here) return;
    float* out = p.out + t * E;
    #pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int e = 4 * (LPT * n + li);
        f32x4 o;
        #pragma unroll
        for (int v = 0; v < 4; ++v)
            o[v] = p.renorm ? fmaf(l[n][v], c[n][v] + all, own[n][v]) : l[n][v] * (own[n][v] + (c[n][v] + all));
        if (vec) {
            if (e < E) *(f32x4*)(out + e) = o;
        } else {
            #pragma unroll
            for (int v = 0; v < 4; ++v)
                if (e + v < E) out[e + v] = o[v];
        }
    }
}

template <int LPT, int NV>
int launch(const RouteGradP& p, hipStream_t stream) {
    const int tpb = kRgThreads / LPT;
    route_grad_kernel<LPT, NV><<<(unsigned)(((int64_t)p.T + tpb - 1) / tpb), kRgThreads, 0, stream>>>(p);
    return (int)hipGetLastError();
}

}  // namespace

int moe_launch_route_backward(const RouteGradCall& c, hipStream_t stream) {
    RouteGradP p{};
    p.logits = c.logits; p.idx = c.topk_idx; p.dw = c.dw; p.slot = c.slot_row; p.prob_grad = c.prob_grad;
    p.out = c.dlogits;
    p.T = c.T; p.E = c.E_tot; p.k = c.k; p.ld_slot = c.ld_slot; p.dw_rows = c.dw_rows;
    p.renorm = (c.flags & MOE_ROUTE_RENORM) != 0; p.z = c.z_coef;
    p.vec = c.E_tot % 4 == 0 && (((uintptr_t)c.logits | (uintptr_t)c.dlogits) & 15) == 0;
    // the fewest lanes that hold a token's logits in one round (16 also hold
    // up to 16 chosen experts), 64 lanes and more rounds for more
    if (c.E_tot <= 64 && c.k <= 16) return launch<16, 1>(p, stream);
    if (c.E_tot <= 128) return launch<32, 1>(p, stream);
    if (c.E_tot <= 256) return launch<64, 1>(p, stream);
    if (c.E_tot <= 512) return launch<64, 2>(p, stream);
    if (c.E_tot <= 1024) return launch<64, 4>(p, stream);
    return launch<64, 8>(p, stream);
}

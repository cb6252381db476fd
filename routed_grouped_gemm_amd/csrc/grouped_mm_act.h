// The products with an epilogue: kernel choice and launches, shared by the
// forward (grouped_mm_act.hip) and gradient (grouped_mm_dact.hip) files, which
// are apart so that they compile side by side. Internal to libmoe.
#pragma once
#include <algorithm>

#include "grouped_mm_rows.h"
#include "grouped_mm_tiled.h"

namespace {

template <int EL, int MODE, int EPI>
int launch_part(MmP& p, int rows, int cols, hipStream_t stream) {
    const int tile = rows > 64 ? a_tile(EPI) : rows_a(EPI);
    p.at = (cols + tile - 1) / tile;
    if (rows > 128) return launch_mm<EL, MODE, 8, EPI>(p, mm_items(p, 256, a_tile(EPI)), stream);
    if (rows > 64) return launch_mm<EL, MODE, 4, EPI>(p, mm_items(p, 128, a_tile(EPI)), stream);
    return rows > 32 ? launch_rows<EL, MODE, 4, EPI>(p, stream) : launch_rows<EL, MODE, 2, EPI>(p, stream);
}

// How a product with an epilogue runs: mm_plan's kernel and split (weight rows:
// gated 2 N), and for one group on the LDS-tiled kernel whether the last, mostly
// empty tiles of rows or columns (up to 64 of either) go to the weight-streaming
// kernel in launches of their own. A tile that is mostly empty takes as long as a
// full one, so that pays where they make for another round of workgroups: 8191 x
// 4104 x 4096 (8 columns past 16 tiles) 340 -> 314 us, 4099 x 4096 x 2040 (3 rows past
// 16 tiles) 141 -> 126. Times in rounds as mm_plan's; a tail's launch costs about 4
// us. (Several groups: how full their last tiles are is not known here.)
struct EpiPlan { int rows, parts; bool row_tail, col_tail; };
inline EpiPlan epi_plan(int R_max, int G, int N, int K, bool gated) {
    EpiPlan best{};
    moe_mm_plan(false, R_max, G, gated ? 2 * N : N, K, &best.rows, &best.parts);
    if (G > 1 || best.rows <= 64) return best;
    const int64_t cus = device_cu_count(), nk = (K + 63) / 64, at = gated ? kATile / 2 : kATile, thin = gated ? kRowsA / 2 : kRowsA;
    double least = 1e30;
    for (int rows = 256; rows >= 128; rows /= 2)
        for (int tails = 0; tails < 4; ++tails) {
            const bool rt = tails & 1, ct = tails & 2;
            const int r = R_max % rows, c = (int)(N % at);
            if ((rt && (r == 0 || r > 64 || r == R_max)) || (ct && (c == 0 || c > 64 || c == N))) continue;
            const int64_t items = ((R_max + rows - 1) / rows - rt) * ((N + at - 1) / at - ct);
            double t = (double)((items + cus - 1) / cus) * ((double)nk * (rows == 256 ? 1.6 : 1.0) + 8.0);
            if (rt) t += 4.0 + (double)((((N + thin - 1) / thin) + 2 * cus - 1) / (2 * cus)) * (double)nk * 0.5;
            if (ct) t += 4.0 + (double)(((int64_t)((R_max + 63) / 64) * ((c + thin - 1) / thin) + 2 * cus - 1) / (2 * cus)) * (double)nk * 0.54;
            if (t < least) { least = t; best = EpiPlan{rows, 1, rt, ct}; }
        }
    return best;
}
// columns of the main launch
inline int epi_main_cols(const EpiPlan& plan, int N, bool gated) {
    return plan.col_tail ? N - N % (gated ? kATile / 2 : kATile) : N;
}

// (three stages of 128 rows leave LDS for the tables of 2047 groups: mm_plan)
template <int EL, int MODE, int EPI>
int launch_epi(MmP& p, const EpiPlan& plan, hipStream_t stream) {
    const int main = epi_main_cols(plan, p.N, EPI == kEpiGated);
    p.row_tile = plan.rows;
    p.row_part = plan.row_tail ? 1 : 0;
    int e = launch_part<EL, MODE, EPI>(p, plan.rows, main, stream);
    if (e) return e;
    if (plan.col_tail) {
        MmP q = p;
        q.col0 = main;
        q.dw_slot0 = 4 * p.at;
        // 32 rows to a tile where 64 leave compute units without one (8 columns of 8191 x
        // 4096: 51.5 -> 43.5 us)
        const int64_t items = (int64_t)((p.R_max + 63) / 64) * ((p.N - main + rows_a(EPI) - 1) / rows_a(EPI));
        if ((e = launch_part<EL, MODE, EPI>(q, items <= device_cu_count() ? 32 : 64, p.N - main, stream))) return e;
    }
    if (plan.row_tail) {
        MmP q = p;
        q.row_part = 2;      // (3 rows of 4096 x 2040, 32 against 64 to a tile: 27.3 -> 24.3 us)
        if ((e = launch_part<EL, MODE, EPI>(q, p.R_max % plan.rows <= 32 ? 32 : 64, p.N, stream))) return e;
    }
    return 0;
}

// rows [lo, end) of all groups
MOE_DEV void all_rows(const MmP& p, int& lo, int& end) {
    int hi, a;
    group_rows(p, 0, lo, hi);
    group_rows(p, p.G - 1, a, end);
}

// the sum of the parts of 4 values, in the order of the parts
MOE_DEV f32x4 join_parts(const float* src, size_t stride, int parts) {
    f32x4 v = *(const f32x4*)src;
    for (int s = 1; s < parts; ++s) {
        const f32x4 e = *(const f32x4*)(src + (size_t)s * stride);
        v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]};
    }
    return v;
}

// parameters of a call (c: checked by the caller)
inline MmP epi_params(const MmActCall& c, const void* x, int x_rows, int ldx, const int32_t* src) {
    MmP p{};
    p.x = (const uint8_t*)x; p.x_ld = (uint32_t)(ldx * 2); p.x_src = src; p.x_rows = (uint32_t)x_rows;
    if (src) p.x_bytes = (uint32_t)((int64_t)(x_rows - 1) * ldx * 2 + (int64_t)c.K * 2);
    p.offsets = c.offsets;
    p.G = c.G; p.N = c.N; p.K = c.K; p.R_max = c.R_max;
    const int64_t wide = (int64_t)c.N * (c.gated && !c.grad ? 2 : 1);        // weight rows of a group
    p.w = (const uint8_t*)c.w; p.w_group = (size_t)(wide * c.K * 2);
    p.w_ld = (uint32_t)((c.kn ? c.N : c.K) * 2);
    p.act = c.act; p.beta = c.beta; p.limit = c.limit; p.gated = c.gated;
    p.bias = c.bias; p.row_w = c.row_w;
    p.out_f16 = c.dtype == MOE_T_F16;
    return p;
}

}  // namespace

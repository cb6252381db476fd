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
// kernel in launches of their own, which may be split along K and joined. A tile
// that is mostly empty takes as long as a full one, so that pays where they make
// for another round of workgroups: 8191 x 4104 x 4096 (8 columns past 16 tiles)
// 340 -> 314 us, its gradient at 4099 x 4096 x 2040 (3 rows past 16 tiles) 141 ->
// 126, and split 300 -> 288 and 111 -> 101. Times in rounds as mm_plan's; a tail's
// launch costs about 4 us. (Several groups: how full their last tiles are is not
// known here.)
struct EpiTail { bool on; int rows, parts; };                // rows to a tile, parts along K
struct EpiPlan { int rows, parts; EpiTail row, col; };

// a tail of R rows and n columns: 32 rows to a tile where 64 leave compute units
// without one (8 columns of 8191 x 4096: 51.5 -> 43.5 us, 3 rows of 4096 x 2040:
// 27.3 -> 24.3); as many parts as fill two workgroups on each, at least 8 K-tiles
// to a part, where that saves more than the joining launch (about 8 K-tiles)
inline EpiTail epi_tail(int64_t R, int64_t n, int64_t thin, int64_t nk, double& t) {
    const int64_t cus = device_cu_count(), at = (n + thin - 1) / thin;
    const int rows = (R + 63) / 64 * at <= cus ? 32 : 64;
    const int64_t items = (R + rows - 1) / rows * at;
    int64_t parts = std::min<int64_t>({2 * cus / std::max<int64_t>(items, 1), nk / 8, 8});
    if (parts < 2 || nk - nk / parts < 12) parts = 1;
    t += 4.0 + (double)((items * parts + 2 * cus - 1) / (2 * cus)) * (double)(nk / parts) * 0.5 + (parts > 1 ? 4.0 : 0.0);
    return EpiTail{true, rows, (int)parts};
}
inline EpiPlan epi_plan(int R_max, int G, int N, int K, bool gated) {
    EpiPlan best{};
    moe_mm_plan(false, R_max, G, gated ? 2 * N : N, K, &best.rows, &best.parts);
    if (best.rows <= 64) return best;
    const int64_t cus = device_cu_count(), nk = (K + 63) / 64, at = gated ? kATile / 2 : kATile, thin = gated ? kRowsA / 2 : kRowsA;
    double least = 1e30;
    if (G > 1) {
        // Tile height for groups that are not equal: half a tile more for each than
        // its rows make (4096 rows in 16 uneven groups, gated 2816 x 2048: 107 us with
        // 256 rows, 84 with 128). With 128 the tables of at most 2047 groups fit LDS.
        for (int rows = 256; rows >= 128 && G <= 2047; rows /= 2) {
            const int64_t items = ((int64_t)R_max / rows + (std::min(G, R_max) + 1) / 2) * ((N + at - 1) / at);
            const double t = (double)((items + cus - 1) / cus) * ((double)nk * (rows == 256 ? 1.6 : 1.0) + 8.0);
            if (t < least) { least = t; best.rows = rows; }
        }
        return best;
    }
    for (int rows = 256; rows >= 128; rows /= 2)
        for (int tails = 0; tails < 4; ++tails) {
            const bool rt = tails & 1, ct = tails & 2;
            const int r = R_max % rows, c = (int)(N % at);
            if ((rt && (r == 0 || r > 64 || r == R_max)) || (ct && (c == 0 || c > 64 || c == N))) continue;
            const int64_t items = ((R_max + rows - 1) / rows - rt) * ((N + at - 1) / at - ct);
            double t = (double)((items + cus - 1) / cus) * ((double)nk * (rows == 256 ? 1.6 : 1.0) + 8.0);
            EpiPlan plan{rows, 1, {}, {}};
            if (rt) plan.row = epi_tail(r, N, thin, nk, t);
            if (ct) plan.col = epi_tail(rt ? R_max - r : R_max, c, thin, nk, t);
            if (t < least) { least = t; best = plan; }
        }
    return best;
}
// columns of the main launch
inline int epi_main_cols(const EpiPlan& plan, int N, bool gated) {
    return plan.col.on ? N - N % (gated ? kATile / 2 : kATile) : N;
}
// bytes of the partial sums. (A tail of rows is what lies past the whole tiles of
// the group's rows, which the device knows: up to a tile's.)
inline size_t epi_partial_bytes(const EpiPlan& plan, int R_max, int N, bool gated) {
    const size_t wide = gated ? 2 : 1;
    size_t n = plan.parts > 1 ? plan.parts * (size_t)R_max * N * wide : 0;
    if (plan.col.on && plan.col.parts > 1) n = std::max(n, plan.col.parts * (size_t)R_max * (N - epi_main_cols(plan, N, gated)) * wide);
    if (plan.row.on && plan.row.parts > 1) n = std::max(n, plan.row.parts * (size_t)plan.rows * N * wide);
    return n * 4;
}

// join(p): the launch that joins a split one. (three stages of 128 rows leave
// LDS for the tables of 2047 groups: mm_plan)
template <int EL, int MODE, int EPI, typename Join>
int launch_epi(MmP& p, const EpiPlan& plan, hipStream_t stream, Join&& join) {
    const size_t wide = EPI == kEpiGated ? 2 : 1;
    const int main = epi_main_cols(plan, p.N, EPI == kEpiGated);
    p.row_tile = plan.rows;
    p.row_part = plan.row.on ? 1 : 0;
    p.parts = plan.parts;
    p.part_rows = (size_t)p.R_max;
    p.part_ld = (size_t)p.N * wide;
    int e = launch_part<EL, MODE, EPI>(p, plan.rows, main, stream);
    if (!e && p.parts > 1) e = join(p);
    if (!e && plan.col.on) {
        MmP q = p;
        q.col0 = main;
        q.dw_slot0 = 4 * p.at;
        q.parts = plan.col.parts;
        q.part_ld = (size_t)(p.N - main) * wide;
        e = launch_part<EL, MODE, EPI>(q, plan.col.rows, p.N - main, stream);
        if (!e && q.parts > 1) e = join(q);
    }
    if (!e && plan.row.on) {
        MmP q = p;
        q.row_part = 2;
        q.parts = plan.row.parts;
        q.part_rows = (size_t)plan.rows;
        e = launch_part<EL, MODE, EPI>(q, plan.row.rows, p.N, stream);
        if (!e && q.parts > 1) e = join(q);
    }
    return e;
}

// rows [lo, end) of all groups
MOE_DEV void all_rows(const MmP& p, int& lo, int& end) {
    int hi, a;
    group_rows(p, 0, lo, hi);
    group_rows(p, p.G - 1, a, end);
}
// those that a launch computes, and the first row of its partial sums
MOE_DEV void joined_rows(const MmP& p, int& lo, int& end, int& row0) {
    all_rows(p, lo, end);
    part_rows<true>(p, lo, end);
    row0 = first_part_row(p);
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

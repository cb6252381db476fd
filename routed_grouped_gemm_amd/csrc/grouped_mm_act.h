// The products with an epilogue: kernel choice and launches, shared by the
// forward (grouped_mm_act.hip) and gradient (grouped_mm_dact.hip) files, which
// are apart so that they compile side by side. Internal to libmoe.
#pragma once
#include <algorithm>

#include "grouped_mm_rows.h"
#include "grouped_mm_tiled.h"

namespace {

template <int EL, int MODE, int EPI>
int launch_epi(const MmP& p, int rows, hipStream_t stream) {
    if (rows > 128) return launch_mm<EL, MODE, 8, EPI>(p, mm_items(p, 256, a_tile(EPI)), stream);
    if (rows > 64) return launch_mm<EL, MODE, 4, EPI>(p, mm_items(p, 128, a_tile(EPI)), stream);
    return rows > 32 ? launch_rows<EL, MODE, 4, EPI>(p, stream) : launch_rows<EL, MODE, 2, EPI>(p, stream);
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

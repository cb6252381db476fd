// Grouped 16-bit products with bias, activation, row weight and residual in
// their epilogue (grouped_mm_epi.h): on the LDS-tiled kernel, on the
// weight-streaming kernel for few rows per group, or split along K there and
// joined by act_join_kernel (epi_plan).
//
// The matrix instructions bound the large calls. Measured: gated 24576 x 2816 x
// 2048 in 16 uneven groups, gathered, with bias, weights and kept
// pre-activation 324 us (875 TFLOP/s), 8191 x 4104 x 4096 in FP16 with bias and
// residual, W [K, N] 288 us (955 TFLOP/s).
#include "grouped_mm_act.h"

namespace {

template <int F16, int EPI>
__global__ __launch_bounds__(256)
void act_join_kernel(MmP p) {
    constexpr int PER = EPI == kEpiGated ? 2 : 4;            // outputs of 4 sums
    int lo, end, row0;
    joined_rows(p, lo, end, row0);
    const int n4 = (p.N - p.col0) / PER;
    const int64_t total = (int64_t)(end - row0) * n4, stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
        const int at = (int)(i / n4), a = (int)(i - (int64_t)at * n4), row = row0 + at;
        if (row < lo) continue;
        int g = 0;
        if (p.bias) {                                        // the last group that starts at or before the row
            int top = p.G - 1;
            while (g < top) {
                const int mid = (g + top + 1) >> 1;
                if (p.offsets[mid] <= row) g = mid;
                else top = mid - 1;
            }
        }
        const f32x4 z = join_parts(p.partial + (size_t)at * p.part_ld + 4 * a, p.part_rows * p.part_ld, p.parts);
        rows_forward<F16, EPI>(p, g, (size_t)row, p.col0 + PER * a, z);
    }
}

template <int EL, int MODE, int EPI>
int launch_act(MmP& p, const EpiPlan& plan, hipStream_t stream) {
    return launch_epi<EL, MODE, EPI>(p, plan, stream, [&](const MmP& q) {
        const int64_t rows = q.row_part == 2 ? q.row_tile : q.R_max, lanes = rows * ((q.N - q.col0) / (EPI == kEpiGated ? 2 : 4));
        const int grid = (int)std::min<int64_t>((lanes + 255) / 256, 4 * device_cu_count());
        act_join_kernel<EL == kElF16, EPI><<<grid, 256, 0, stream>>>(q);
        return (int)hipGetLastError();
    });
}

template <int EL>
int launch_type(const MmActCall& c, MmP& p, const EpiPlan& plan, hipStream_t stream) {
    if (c.gated) return launch_act<EL, kMmNK, kEpiGated>(p, plan, stream);
    return c.kn ? launch_act<EL, kMmKN, kEpiAct>(p, plan, stream) : launch_act<EL, kMmNK, kEpiAct>(p, plan, stream);
}

}  // namespace

void moe_mm_act_plan(int R_max, int G, int N, int K, bool gated, int32_t* plan) {
    const EpiPlan p = epi_plan(R_max, G, N, K, gated);
    const int32_t v[6] = {p.rows, p.parts, p.row.rows, p.row.parts, p.col.rows, p.col.parts};
    std::copy(v, v + 6, plan);
}

// (gated or not: the plans differ in their tails)
size_t moe_mm_act_bytes(int R_max, int G, int weight_rows, int K) {
    if (R_max <= 0) return 0;
    const size_t plain = epi_partial_bytes(epi_plan(R_max, G, weight_rows, K, false), R_max, weight_rows, false);
    if (weight_rows % 16) return plain;
    return std::max(plain, epi_partial_bytes(epi_plan(R_max, G, weight_rows / 2, K, true), R_max, weight_rows / 2, true));
}

int moe_launch_mm_act(const MmActCall& c, hipStream_t stream) {
    MmP p = epi_params(c, c.x, c.x_rows, c.ldx, c.x_src);
    p.out = (uint8_t*)c.out; p.out_ld = (size_t)c.ldy;
    p.res = (const uint8_t*)c.res; p.res_ld = (size_t)c.ld_res;
    p.pre = (uint8_t*)c.pre; p.pre_ld = (size_t)c.N * (c.gated ? 2 : 1);
    p.partial = (float*)c.ws;
    const EpiPlan plan = epi_plan(c.R_max, c.G, c.N, c.K, c.gated);
    return c.dtype == MOE_T_F16 ? launch_type<kElF16>(c, p, plan, stream) : launch_type<kElBf16>(c, p, plan, stream);
}

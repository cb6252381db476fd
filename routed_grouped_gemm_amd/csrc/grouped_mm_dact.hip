// The backward pass of the products with an activation, up to the
// pre-activation: the product dh = dy W with the activation's gradient in its
// epilogue (grouped_mm_epi.h), so dh is never in memory. The rows' sums (the
// gradient of the routing weight) come from partial sums per 64 columns (16 on
// the weight-streaming kernel), added in their order by a second launch; a
// product split along K has its epilogue in the launch that joins it.
//
// Measured: 24576 x 1408 x 2048 in 16 uneven groups, gathered, gated 265 us;
// 4099 x 4096 x 2040 in FP16, squared ReLU 163 us.
#include "grouped_mm_act.h"

namespace {

// one wave a row
template <int F16>
__global__ __launch_bounds__(256)
void grad_join_kernel(MmP p) {
    int lo, end;
    all_rows(p, lo, end);
    const int lane = threadIdx.x & 63;
    for (int64_t row = lo + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < end; row += (int64_t)gridDim.x * 4) {
        float sum = 0.f;
        for (int a = lane * 4; a < p.N; a += 256)
            sum += rows_grad<F16>(p, (size_t)row, a, join_parts(p.partial + (size_t)row * p.N + a, (size_t)p.R_max * p.N, p.parts));
        sum = wave_sum(sum);
        if (p.dw && lane == 0) p.dw[row] = sum;
    }
}

// n: partial sums of a row; tail_n: of the rows past the whole passes of one
// group (0: none apart). 64 rows to a workgroup, a quarter of the sums to each
// wave, the quarters joined in their order.
__global__ __launch_bounds__(256)
void grad_sum_kernel(MmP p, int n, int tail_n) {
    __shared__ float part[3][64];
    int lo, end;
    all_rows(p, lo, end);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t row = lo + (int64_t)blockIdx.x * 64 + lane;
    const bool in = row < end;
    if (tail_n && row >= end - (end - lo) % p.row_tile) n = tail_n;
    float sum = 0.f;
    if (in) {
        #pragma unroll 8
        for (int i = n * w / 4; i < n * (w + 1) / 4; ++i) sum += p.dw_part[(size_t)i * p.R_max + row];
    }
    if (w > 0) part[w - 1][lane] = sum;
    __syncthreads();
    if (w == 0 && in) p.dw[row] = ((sum + part[0][lane]) + part[1][lane]) + part[2][lane];
}

// partial sums of a row: 4 a tile of columns of either kernel
struct GradSums { int n, tail_n; };
GradSums grad_sums(const EpiPlan& plan, int N) {
    const int thin = 4 * ((N + kRowsA - 1) / kRowsA), main = epi_main_cols(plan, N, false);
    if (plan.rows <= 64) return GradSums{thin, 0};
    const int n = 4 * ((main + kATile - 1) / kATile) + 4 * ((N - main + kRowsA - 1) / kRowsA);
    return GradSums{n, plan.row_tail ? thin : 0};
}

template <int EL, int MODE>
int launch_dact(MmP& p, const EpiPlan& plan, hipStream_t stream) {
    int e = launch_epi<EL, MODE, kEpiGrad>(p, plan, stream);
    if (e) return e;
    if (p.parts > 1) {
        grad_join_kernel<EL == kElF16><<<(int)std::min<int64_t>(((int64_t)p.R_max + 3) / 4, 8 * device_cu_count()), 256, 0, stream>>>(p);
        return (int)hipGetLastError();
    }
    if (!p.dw) return 0;
    const GradSums s = grad_sums(plan, p.N);
    grad_sum_kernel<<<(unsigned)(((int64_t)p.R_max + 63) / 64), 256, 0, stream>>>(p, s.n, s.tail_n);
    return (int)hipGetLastError();
}

}  // namespace

size_t moe_mm_dact_bytes(int R_max, int G, int N, int K) {
    if (R_max <= 0) return 0;
    const EpiPlan plan = epi_plan(R_max, G, N, K, false);
    if (plan.parts > 1) return (size_t)plan.parts * R_max * N * 4;
    const GradSums s = grad_sums(plan, N);
    return (size_t)std::max(s.n, s.tail_n) * R_max * 4;
}

int moe_launch_mm_dact(const MmActCall& c, hipStream_t stream) {
    MmP p = epi_params(c, c.x, c.x_rows, c.ldx, c.x_src);
    p.out = (uint8_t*)c.out;
    p.pre = (uint8_t*)c.pre; p.pre_ld = (size_t)c.ld_pre;
    p.h = (uint8_t*)c.h; p.dw = c.dw;
    const EpiPlan plan = epi_plan(c.R_max, c.G, c.N, c.K, false);
    p.parts = plan.parts;
    if (plan.parts > 1) p.partial = (float*)c.ws;
    else if (c.dw) p.dw_part = (float*)c.ws;
    if (c.dtype == MOE_T_F16) return c.kn ? launch_dact<kElF16, kMmKN>(p, plan, stream) : launch_dact<kElF16, kMmNK>(p, plan, stream);
    return c.kn ? launch_dact<kElBf16, kMmKN>(p, plan, stream) : launch_dact<kElBf16, kMmNK>(p, plan, stream);
}

// The backward pass of the products with an activation, up to the
// pre-activation: the product dh = dy W with the activation's gradient in its
// epilogue (grouped_mm_epi.h), so dh is never in memory. The rows' sums (the
// gradient of the routing weight) come from partial sums per 64 columns (16 on
// the weight-streaming kernel), added in their order by a second launch; a
// product split along K has its epilogue in the launch that joins it.
//
// Bound by HBM in its epilogues, which all workgroups reach together: a gated
// tile's moves 640 KiB (pre, dpre and h), about 30 us a round at the rate of a
// large copy, while the matrix instructions wait (as compiled, for its stores too:
// the K loop begins with a wait for all that is in flight); by those between.
// Measured: 24576 x 1408 x 2048 in 16 uneven groups, gathered, gated 262 us;
// 4099 x 4096 x 2040 in FP16, squared ReLU 101 us.
#include "grouped_mm_act.h"

namespace {

// The parts of a split product joined and its epilogue: 16 lanes a row of at most
// 64 columns, else a workgroup a row. The row's sum is whole, or with dw_part one
// of the row's.
constexpr int kJoinThreads = 1024;

template <int F16>
MOE_DEV float grad_join_row(const MmP& p, int64_t row, int row0, int first, int step) {
    const float* const src = p.partial + (size_t)(row - row0) * p.part_ld;
    float sum = 0.f;
    for (int a = p.col0 + first; a < p.N; a += step)
        sum += rows_grad<F16>(p, (size_t)row, a, join_parts(src + (a - p.col0), p.part_rows * p.part_ld, p.parts));
    return sum;
}
MOE_DEV void grad_join_sum(const MmP& p, int64_t row, float sum) {
    if (p.dw_part) p.dw_part[(size_t)p.dw_slot0 * p.R_max + row] = sum;
    else if (p.dw) p.dw[row] = sum;
}

template <int F16>
__global__ __launch_bounds__(kJoinThreads)
void grad_join_kernel(MmP p) {
    __shared__ float part[kJoinThreads / 64];
    int lo, end, row0;
    joined_rows(p, lo, end, row0);
    for (int64_t row = lo + (int64_t)blockIdx.x; row < end; row += gridDim.x) {
        const float sum = wave_sum(grad_join_row<F16>(p, row, row0, (int)threadIdx.x * 4, kJoinThreads * 4));
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            float all = 0.f;
            #pragma unroll
            for (int i = 0; i < kJoinThreads / 64; ++i) all += part[i];
            grad_join_sum(p, row, all);
        }
        __syncthreads();
    }
}
template <int F16>
__global__ __launch_bounds__(256)
void grad_join_narrow_kernel(MmP p) {
    int lo, end, row0;
    joined_rows(p, lo, end, row0);
    const int li = threadIdx.x & 15;
    const int64_t row = lo + (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const float sum = group_sum<16>(row < end ? grad_join_row<F16>(p, row, row0, li * 4, 64) : 0.f);
    if (li == 0 && row < end) grad_join_sum(p, row, sum);
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

// partial sums of a row: 4 a tile of columns of either kernel, one of a split launch
struct GradSums { int n, tail_n; };
GradSums grad_sums(const EpiPlan& plan, int N) {
    const auto thin = [](int n) { return 4 * ((n + kRowsA - 1) / kRowsA); };
    if (plan.rows <= 64) return GradSums{thin(N), 0};
    const int main = epi_main_cols(plan, N, false), n = 4 * ((main + kATile - 1) / kATile);
    return GradSums{n + (plan.col.on ? plan.col.parts > 1 ? 1 : thin(N - main) : 0),
                    plan.row.on ? plan.row.parts > 1 ? 1 : thin(N) : 0};
}
// bytes of the rows' partial sums, before those of the products
size_t dw_bytes(const EpiPlan& plan, int R_max, int N) {
    if (plan.parts > 1) return 0;
    const GradSums s = grad_sums(plan, N);
    return ((size_t)std::max(s.n, s.tail_n) * R_max * 4 + 15) / 16 * 16;
}

template <int EL, int MODE>
int launch_dact(MmP& p, const EpiPlan& plan, hipStream_t stream) {
    const int e = launch_epi<EL, MODE, kEpiGrad>(p, plan, stream, [&](const MmP& q) {
        const int64_t rows = q.row_part == 2 ? q.row_tile : q.R_max;
        if (q.N - q.col0 <= 64) grad_join_narrow_kernel<EL == kElF16><<<(unsigned)((rows + 15) / 16), 256, 0, stream>>>(q);
        else grad_join_kernel<EL == kElF16><<<(unsigned)std::min<int64_t>(rows, 4 * device_cu_count()), kJoinThreads, 0, stream>>>(q);
        return (int)hipGetLastError();
    });
    if (e || !p.dw_part) return e;
    const GradSums s = grad_sums(plan, p.N);
    grad_sum_kernel<<<(unsigned)(((int64_t)p.R_max + 63) / 64), 256, 0, stream>>>(p, s.n, s.tail_n);
    return (int)hipGetLastError();
}

}  // namespace

size_t moe_mm_dact_bytes(int R_max, int G, int N, int K) {
    if (R_max <= 0) return 0;
    const EpiPlan plan = epi_plan(R_max, G, N, K, false);
    return dw_bytes(plan, R_max, N) + epi_partial_bytes(plan, R_max, N, false);
}

int moe_launch_mm_dact(const MmActCall& c, hipStream_t stream) {
    MmP p = epi_params(c, c.x, c.x_rows, c.ldx, c.x_src);
    p.out = (uint8_t*)c.out;
    p.pre = (uint8_t*)c.pre; p.pre_ld = (size_t)c.ld_pre;
    p.h = (uint8_t*)c.h; p.dw = c.dw;
    const EpiPlan plan = epi_plan(c.R_max, c.G, c.N, c.K, false);
    if (c.dw && plan.parts == 1) p.dw_part = (float*)c.ws;
    p.partial = (float*)((uint8_t*)c.ws + dw_bytes(plan, c.R_max, c.N));
    if (c.dtype == MOE_T_F16) return c.kn ? launch_dact<kElF16, kMmKN>(p, plan, stream) : launch_dact<kElF16, kMmNK>(p, plan, stream);
    return c.kn ? launch_dact<kElBf16, kMmKN>(p, plan, stream) : launch_dact<kElBf16, kMmNK>(p, plan, stream);
}

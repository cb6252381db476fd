// Bias gradients of the grouped products: db_g[n] = sum of w_r dy[s(r)][n] over
// the rows r of group g.
//
// Bound by HBM: dy is read once. A group's rows go in passes of `pass` rows, a
// workgroup sums 512 columns of one pass: 8 columns (16 bytes) to a lane, every
// fourth row to a wave, 8 rows requested at a time, in fp32, the four waves
// joined in LDS. A group of one pass is done with that; the sums of longer
// ones go to the workspace and a second launch adds them in the order of the
// passes, so results are the same bits every time. `pass` follows from R_max
// and N alone: about 1024 workgroups (4 on a compute unit, 32 KiB in flight
// each), at least 32 rows of work for each; up to 256 rows are one pass.
// Measured: 24576 rows of 2816 in 16 uneven groups 33 us (4.2 TB/s), 8191
// gathered rows of 4104 in one group 18 us.
#include <algorithm>

#include "grouped_mm.h"

namespace {

constexpr int kBgThreads = 256;
constexpr int kBgCols = 512;
constexpr int kBgJoinCols = 256;

struct BiasP {
    const uint8_t* dy; size_t ld;                            // bytes per row
    const int32_t* src; uint32_t rows;                       // rows of dy
    const float* w; const int32_t* offsets;
    int G, N, R_max, pass, max_slots, accumulate, f16;
    float* out; float* partial;
};

MOE_DEV void bias_rows(const BiasP& p, int g, int& lo, int& hi) {
    lo = min(max(p.offsets[g], 0), p.R_max);
    hi = min(max(p.offsets[g + 1], lo), p.R_max);
}

// For every group: at[g] passes before it (an empty group has one, which
// writes its zeros), slots[g] the workspace rows before its passes (groups of
// several passes only). One wave; a barrier must follow. False where groups
// overlap so far that the workspace does not hold their passes.
MOE_DEV bool bias_tables(const BiasP& p, int lane, int* at, int* slots) {
    int64_t run = 0, srun = 0;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
        int lo = 0, hi = 0;
        if (g0 + lane < p.G) bias_rows(p, g0 + lane, lo, hi);
        const int n = g0 + lane < p.G ? max(1, (hi - lo + p.pass - 1) / p.pass) : 0, m = n > 1 ? n : 0;
        const int inc = wave_incl_scan(n), sinc = wave_incl_scan(m);
        if (g0 + lane < p.G) {
            at[g0 + lane] = (int)run + inc - n;
            slots[g0 + lane] = (int)srun + sinc - m;
        }
        run += __builtin_amdgcn_readlane(inc, 63);
        srun += __builtin_amdgcn_readlane(sinc, 63);
    }
    if (lane == 0) at[p.G] = (int)run;
    return srun <= p.max_slots;
}

template <int F16>
MOE_DEV void add8(float (&acc)[8], const i32x4& v, float w, bool keep) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = keep ? (uint32_t)v[i] : 0u;
        acc[2 * i] = fmaf(lo16(u, F16), w, acc[2 * i]);
        acc[2 * i + 1] = fmaf(hi16(u, F16), w, acc[2 * i + 1]);
    }
}

template <int F16>
__global__ __launch_bounds__(kBgThreads)
void bias_grad_kernel(BiasP p) {
    extern __shared__ int tab[];                             // at [G + 1], slots [G]
    __shared__ float part[3][kBgCols];
    __shared__ int fits;
    int* const slots = tab + p.G + 1;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (w == 0) {
        const bool ok = bias_tables(p, lane, tab, slots);
        if (lane == 0) fits = ok;
    }
    __syncthreads();
    const int blocks = (p.N + kBgCols - 1) / kBgCols;
    const int unit = blockIdx.x / blocks, c0 = (int)(blockIdx.x % blocks) * kBgCols + lane * 8;
    if (unit >= tab[p.G] || !fits) return;
    // the group of this pass: the last one that starts at or before it
    int g = 0;
    for (int i0 = 0; i0 < p.G; i0 += 64) {
        const int here = __builtin_popcountll(__ballot(i0 + lane < p.G && tab[i0 + lane] <= unit));
        g += here;
        if (here < 64) break;
    }
    g = __builtin_amdgcn_readfirstlane(g) - 1;
    const int first = __builtin_amdgcn_readfirstlane(tab[g]), passes = __builtin_amdgcn_readfirstlane(tab[g + 1]) - first;
    int lo, hi;
    bias_rows(p, g, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo) + (unit - first) * p.pass;
    hi = min(__builtin_amdgcn_readfirstlane(hi), lo + p.pass);

    const bool in = c0 < p.N;
    const uint8_t* const base = p.dy + (size_t)(in ? c0 : 0) * 2;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // 64 of this wave's rows (lo + w + 4 i) at a time: sources and weights one to a lane
    for (int r0 = lo + w; r0 < hi; r0 += 256) {
        const int r = r0 + 4 * lane, n = min(64, (hi - r0 + 3) / 4);
        uint32_t s = 0;
        float wt = 0.f;
        if (r < hi) {
            s = p.src ? (uint32_t)p.src[r] : (uint32_t)r;
            wt = p.w ? p.w[r] : 1.f;
        }
        for (int i0 = 0; i0 < n; i0 += 8) {
            i32x4 v[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = min(i0 + i, n - 1);           // (past the end: the last row again, not added)
                const uint32_t row = (uint32_t)__builtin_amdgcn_readlane((int)s, at);
                v[i] = *(const i32x4*)(base + (size_t)(row < p.rows ? row : 0u) * p.ld);
            }
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = min(i0 + i, n - 1);
                const uint32_t row = (uint32_t)__builtin_amdgcn_readlane((int)s, at);
                const float rw = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(wt), at));
                const bool keep = i0 + i < n && row < p.rows;
                add8<F16>(acc, v[i], keep ? rw : 0.f, keep);
            }
        }
    }
    if (w > 0) {
        #pragma unroll
        for (int i = 0; i < 8; ++i) part[w - 1][i * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (w > 0 || !in) return;
    #pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = (acc[i] + part[0][i * 64 + lane]) + (part[1][i * 64 + lane] + part[2][i * 64 + lane]);
    float* d = passes > 1 ? p.partial + ((size_t)slots[g] + (unit - first)) * p.N + c0 : p.out + (size_t)g * p.N + c0;
    f32x4 a = {acc[0], acc[1], acc[2], acc[3]}, b = {acc[4], acc[5], acc[6], acc[7]};
    if (p.accumulate && passes == 1) {
        const f32x4 oa = ((const f32x4*)d)[0], ob = ((const f32x4*)d)[1];
        #pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] += oa[i]; b[i] += ob[i]; }
    }
    ((f32x4*)d)[0] = a;
    ((f32x4*)d)[1] = b;
}

// The passes of a long group: 256 columns to a workgroup, a quarter of the
// passes to each wave, the quarters joined in their order.
__global__ __launch_bounds__(kBgThreads)
void bias_join_kernel(BiasP p) {
    __shared__ f32x4 part[3][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = blockIdx.y;
    int lo, hi;
    bias_rows(p, g, lo, hi);
    const int n = (hi - lo + p.pass - 1) / p.pass;
    if (n <= 1) return;
    int slot = 0;
    int64_t all = 0;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
        int a = 0, b = 0;
        if (g0 + lane < p.G) bias_rows(p, g0 + lane, a, b);
        const int m = (b - a + p.pass - 1) / p.pass, k = m > 1 ? m : 0;
        slot += __builtin_amdgcn_readlane(wave_incl_scan(g0 + lane < g ? k : 0), 63);
        all += __builtin_amdgcn_readlane(wave_incl_scan(k), 63);
    }
    if (all > p.max_slots) return;
    const int c = blockIdx.x * kBgJoinCols + lane * 4;
    const bool in = c < p.N;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const int i0 = n * w / 4, i1 = n * (w + 1) / 4;
    if (in) {
        const float* src = p.partial + (size_t)slot * p.N + c;
        #pragma unroll 8
        for (int i = i0; i < i1; ++i) {
            const f32x4 v = *(const f32x4*)(src + (size_t)i * p.N);
            sum = f32x4{sum[0] + v[0], sum[1] + v[1], sum[2] + v[2], sum[3] + v[3]};
        }
    }
    if (w > 0) part[w - 1][lane] = sum;
    __syncthreads();
    if (w > 0 || !in) return;
    f32x4* d = (f32x4*)(p.out + (size_t)g * p.N + c);
    #pragma unroll
    for (int i = 0; i < 3; ++i) {
        const f32x4 v = part[i][lane];
        sum = f32x4{sum[0] + v[0], sum[1] + v[1], sum[2] + v[2], sum[3] + v[3]};
    }
    if (p.accumulate) {
        const f32x4 v = *d;
        sum = f32x4{sum[0] + v[0], sum[1] + v[1], sum[2] + v[2], sum[3] + v[3]};
    }
    *d = sum;
}

// Rows of a pass. Few rows go in one, which spares the second launch and the
// workspace (128 rows of 816 in 27 groups 12.6 -> 9.0 us a call, 4.8 -> 3.4 in a
// graph; 256 rows of 4104 in one group 12.6 -> 8.8 and 6.3 -> 8.2).
int bias_pass(int R_max, int N) {
    if (R_max <= 256) return 256;
    const int64_t blocks = (N + kBgCols - 1) / kBgCols;
    const int64_t rows = ((int64_t)R_max * blocks / 1024 + 15) / 16 * 16;
    return (int)std::min<int64_t>(std::max<int64_t>(rows, 32), 4096);
}
// passes that groups of several passes can have (each but a group's last is full)
int64_t bias_slots(int R_max, int N) {
    const int pass = bias_pass(R_max, N);
    return R_max > pass ? 2ll * (R_max / pass) : 0;
}

}  // namespace

size_t moe_bias_grad_bytes(int R_max, int N) { return (size_t)bias_slots(R_max, N) * N * 4; }

int moe_launch_bias_grad(const BiasGradCall& c, hipStream_t stream) {
    BiasP p{};
    p.dy = (const uint8_t*)c.dy; p.ld = (size_t)c.ld_dy * 2; p.src = c.dy_src; p.rows = (uint32_t)c.dy_rows;
    p.w = c.row_w; p.offsets = c.offsets;
    p.G = c.G; p.N = c.N; p.R_max = c.R_max; p.pass = bias_pass(c.R_max, c.N);
    p.max_slots = (int)bias_slots(c.R_max, c.N);
    p.accumulate = c.accumulate; p.out = c.out; p.partial = (float*)c.ws;
    const int64_t blocks = (c.N + kBgCols - 1) / kBgCols;
    const int64_t units = (int64_t)c.R_max / p.pass + c.G;
    const size_t lds = (size_t)(2 * c.G + 1) * 4;
    const unsigned grid = (unsigned)(units * blocks);
    if (c.dtype == MOE_T_F16) bias_grad_kernel<1><<<grid, kBgThreads, lds, stream>>>(p);
    else bias_grad_kernel<0><<<grid, kBgThreads, lds, stream>>>(p);
    const int e = (int)hipGetLastError();
    if (e || p.max_slots == 0) return e;
    bias_join_kernel<<<dim3((unsigned)((c.N + kBgJoinCols - 1) / kBgJoinCols), (unsigned)c.G), kBgThreads, 0, stream>>>(p);
    return (int)hipGetLastError();
}

// The routed layer for a few tokens (T <= 32) on 16-bit token rows and weights in
// 16 bits or in E4M3 with a scale per 128 x 128, in two launches:
//
//   few_w1  every workgroup routes and groups the tokens (a few thousand
//           cycles), then  h[r] = a(clamp(g)) clamp(u) w_r  for the rows r of the
//           experts that have tokens, [g | u] = x[src r] W1_g^T + b1_g
//   few_w2  out[t] = residual[t] + sum over t's rows r of (h[r] W2_g^T + w_r b2_g)
//
// Bound by the weights of the active experts, read once. Both kernels give 16
// rows of weights to a workgroup of 8 waves, which split the reduction axis:
// unit i (128 bytes of each row, so that the eight take 1 KiB of a row side by
// side) goes to wave i % 8. A lane's 16 bytes are its operand of the 16x16x32
// matrix instruction as they come (any order of k serves if both operands have
// it), so weights pass through registers alone, with two batches of units in
// flight in each wave and no barrier but the one that joins the eight waves'
// sums. E4M3 codes become 16-bit values exactly, the scale of a unit's 128
// columns multiplies its fp32 sums.
//
// few_w1's 16 rows are 8 of the gate and the same 8 of the up projection, in
// the order 2 gate, 2 up, so that a lane ends with both halves of its outputs.
// few_w2's 16 columns of the 16x16 result are the tokens themselves: a unit's
// sums are added for the tokens that chose its expert (a choice, not a product
// with 0: another token's infinities stay out), so the sum over experts stays in
// fp32 registers and nothing has to be combined afterwards.
//
// Measured: one token on 6 of 64 experts of 2048 x 1408 in BF16 (104 MB) 36 us;
// 16 tokens on 32 local experts of 256, 7168 x 2048 in E4M3 (about 560 MB) 146
// us; 8 tokens on 9 experts of 512 x 264 22 us, host time.
#include <algorithm>

#include "epilogue_act.h"
#include "grouped_mm.h"
#include "permute_block.h"

namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;

struct FewP {
    const float* logits;
    int T, E, k, e0, E_loc, s, G, renorm;
    const uint8_t* x; uint32_t x_ld, x_bytes;                // bytes
    int H, I;
    const uint8_t* w1[2]; const uint8_t* w2[2];              // routed groups, shared group
    const float* s1[2]; const float* s2[2];
    int act; float beta, limit;
    const float* b1; const float* b2;
    const uint16_t* res; size_t ld_res;
    uint16_t* out; size_t ld_out;
    // workspace
    uint16_t* h;                                             // [R, I]
    float* row_w;                                            // [R]
    int32_t* slot;                                           // [T, k + s] row of each slot, -1
    int32_t* active;                                         // number of groups with rows, then they
    int16_t* rowmap;                                         // [active][T] row of a token in the group, -1
};

// Reads the units (128 bytes of 16 weight rows, and the matching k of NT x 16
// token rows) of one wave. A batch is UB units.
template <bool F8, int NT>
struct FewGeom {
    static constexpr int UB = NT == 1 ? 2 : 1;
    static constexpr int NB = F8 ? 4 : 2;                    // 16-byte pieces of a token row in a unit
    static constexpr int UK = F8 ? 128 : 64;                 // k of a unit
};
template <bool F8, int NT>
struct FewBatch {
    using Geo = FewGeom<F8, NT>;
    i32x4 a[Geo::UB][2];
    i32x4 b[Geo::UB][NT][Geo::NB];
    float sc[Geo::UB][2];                                    // scales (few_w1: gate, up; few_w2: the first)
    int row[Geo::UB][NT];                                    // few_w2: the token's row, -1
};

// E4M3 codes (8 of them) as 16-bit values, exactly
template <int EL>
MOE_DEV i32x4 few_decode(int lo, int hi) {
    i32x4 v;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = i < 2 ? lo : hi;
        if constexpr (EL == kElBf16) {
            const auto d = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true)
                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
            v[i] = __builtin_bit_cast(int, d);
        } else {
            const auto d = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
            v[i] = __builtin_bit_cast(int, d);
        }
    }
    return v;
}

// the products of one unit with one tile of 16 token rows
template <int EL, bool F8>
MOE_DEV f32x4 few_unit(const i32x4 (&a)[2], const i32x4* b) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (F8) {
            d = mfma16x16x32<EL>(few_decode<EL>(a[h][0], a[h][1]), b[2 * h], d);
            d = mfma16x16x32<EL>(few_decode<EL>(a[h][2], a[h][3]), b[2 * h + 1], d);
        } else {
            d = mfma16x16x32<EL>(a[h], b[h], d);
        }
    }
    return d;
}

MOE_DEV i32x4 few_load(const rsrc_t& r, uint32_t o) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}
// weights: each byte is used once
MOE_DEV i32x4 few_load_w(const rsrc_t& r, uint32_t o) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 2));
}

// byte offset in a weight row of this lane's piece h of unit u, and of piece i
// of a token row; past the row: kMmInvalid
template <bool F8>
MOE_DEV uint32_t few_koff_w(int u, int h, int q, int K) {
    const int b = u * 128 + 64 * h + 16 * q;
    return b < (F8 ? K : 2 * K) ? (uint32_t)b : kMmInvalid;
}
template <bool F8>
MOE_DEV uint32_t few_koff_x(int u, int i, int q, int K) {
    const int k = F8 ? u * 128 + 64 * (i >> 1) + 16 * q + 8 * (i & 1) : u * 64 + 32 * i + 8 * q;
    return k < K ? (uint32_t)(2 * k) : kMmInvalid;
}
// the sum of two offsets, past every resource if one of them is
MOE_DEV uint32_t few_add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Routes the T tokens and groups their local assignments, by the whole
// workgroup, into LDS. Returns the layout's tables.
struct FewTables { int *sidx; float* sw; int *counts, *offsets, *row_src; float* row_w; int *slot, *active, *scratch; };

__host__ __device__ inline size_t few_table_ints(int T, int k, int G, int s) {
    const size_t R = (size_t)T * (k + s);
    return 2 * (size_t)T * k + (size_t)G + (G + 1) + 2 * R + R + ((size_t)G < R ? G : R) + 1;
}
MOE_DEV FewTables few_tables(int* lds, int T, int k, int G, int s) {
    const int R = T * (k + s);
    FewTables t;
    t.sidx = lds; lds += T * k;
    t.sw = (float*)lds; lds += T * k;
    t.counts = lds; lds += G;
    t.offsets = lds; lds += G + 1;
    t.row_src = lds; lds += R;
    t.row_w = (float*)lds; lds += R;
    t.slot = lds; lds += R;
    t.active = lds; lds += min(G, R) + 1;
    t.scratch = lds;
    return t;
}

MOE_DEV void few_route(const FewP& p, const FewTables& t) {
    if (p.E <= 64 && p.k <= 32) route_block<kFewWaves, 32, 2>(p.logits, p.T, p.E, p.k, p.renorm != 0, t.sidx, t.sw, nullptr, nullptr);
    else if (p.E <= 256 && p.k <= 32) route_block<kFewWaves, 32, 8>(p.logits, p.T, p.E, p.k, p.renorm != 0, t.sidx, t.sw, nullptr, nullptr);
    else if (p.E <= 512) route_block<kFewWaves, 64, 8>(p.logits, p.T, p.E, p.k, p.renorm != 0, t.sidx, t.sw, nullptr, nullptr);
    else route_block<kFewWaves, 64, 32>(p.logits, p.T, p.E, p.k, p.renorm != 0, t.sidx, t.sw, nullptr, nullptr);
    __syncthreads();
    permute_in_block<kFewWaves>([&](int a) { return t.sidx[a]; }, [&](int a) { return t.sw[a]; }, p.T, p.k, p.e0, p.E_loc,
                                p.s, t.counts, t.offsets, nullptr, t.row_src, t.row_w, t.slot, t.scratch);
    __syncthreads();
    // the groups with rows, in their order (at most one a row)
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int n = 0;
        for (int g0 = 0; g0 < p.G; g0 += 64) {
            const bool has = g0 + lane < p.G && t.counts[g0 + lane] > 0;
            const uint64_t m = __ballot(has);
            if (has) t.active[1 + n + __popcll(m & lanemask_lt(lane))] = g0 + lane;
            n += __popcll(m);
        }
        if (lane == 0) t.active[0] = n;
    }
    __syncthreads();
}

// ------------------------------------------------------------------ few_w1
template <int EL, bool F8, int NT>
__global__ __launch_bounds__(kFewThreads, 4)
void few_w1_kernel(FewP p) {
    using Geo = FewGeom<F8, NT>;
    constexpr int UB = Geo::UB;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* const part = (float*)smem;                        // [2][8 waves][NT][4][64]
    const FewTables tb = few_tables((int*)(smem + 2 * kFewWaves * NT * 1024), p.T, p.k, p.G, p.s);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;

    few_route(p, tb);
    const int n_act = __builtin_amdgcn_readfirstlane(tb.active[0]);
    if (blockIdx.x == 0) {                                   // for few_w2
        for (int i = threadIdx.x; i <= n_act; i += kFewThreads) p.active[i] = tb.active[i];
        for (int i = threadIdx.x; i < p.T * (p.k + p.s); i += kFewThreads) p.slot[i] = tb.slot[i];
        const int R = tb.offsets[p.G];
        for (int i = threadIdx.x; i < R; i += kFewThreads) p.row_w[i] = tb.row_w[i];
        for (int i = threadIdx.x; i < n_act * p.T; i += kFewThreads) {
            const int g = tb.active[1 + i / p.T], t = i % p.T;
            int row = -1;
            for (int r = tb.offsets[g]; r < tb.offsets[g] + tb.counts[g]; ++r) row = tb.row_src[r] == t ? r : row;
            p.rowmap[i] = (int16_t)row;
        }
    }
    const int cb = p.I / 8, n_items = n_act * cb, grid = gridDim.x;
    if ((int)blockIdx.x >= n_items) return;

    const int wrow = p.H * (F8 ? 1 : 2);                     // bytes of a weight row
    const int units = (p.H + Geo::UK - 1) / Geo::UK;
    const int nb = ((units + kFewWaves - 1) / kFewWaves + UB - 1) / UB, batches = (nb + 1) & ~1;
    const int nsb = (2 * p.I + 127) >> 7, ksb = (p.H + 127) >> 7;

    // the loader: one batch after another through all items
    struct { int item, b; bool live; const uint8_t* w; const float* s; int up_s; uint32_t ro, xo[NT]; } L;
    auto open = [&]() __attribute__((always_inline)) {
        L.b = 0;
        L.live = L.item < n_items;
        const int item = L.live ? L.item : 0;
        const int ai = __builtin_amdgcn_readfirstlane(item / cb), c0 = (item - ai * cb) * 8;
        const int g = __builtin_amdgcn_readfirstlane(tb.active[1 + ai]);
        const int sh = g < p.E_loc ? 0 : 1, gi = sh ? 0 : g;
        L.w = p.w1[sh] + (size_t)gi * (size_t)(2 * p.I) * (size_t)wrow;
        const int col = c0 + 2 * (j >> 2) + (j & 1);
        L.ro = (uint32_t)(((j >> 1) & 1) * p.I + col) * (uint32_t)wrow;
        if constexpr (F8) {
            L.s = p.s1[sh] + ((size_t)gi * nsb + (c0 >> 7)) * ksb;
            L.up_s = (((p.I + c0) >> 7) - (c0 >> 7)) * ksb;
        }
        const int lo = tb.offsets[g], n = tb.counts[g];
        #pragma unroll
        for (int i = 0; i < NT; ++i)
            L.xo[i] = 16 * i + j < n ? (uint32_t)tb.row_src[min(lo + 16 * i + j, p.T * (p.k + p.s) - 1)] * p.x_ld : kMmNoRow;
    };
    auto load = [&](FewBatch<F8, NT>& B) __attribute__((always_inline)) {
        const rsrc_t rw = make_rsrc(L.w, L.live ? (uint32_t)(2 * p.I) * (uint32_t)wrow : 0u);
        const rsrc_t rx = make_rsrc(p.x, L.live ? p.x_bytes : 0u);
        #pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int u = (L.b * UB + i) * kFewWaves + w;
            #pragma unroll
            for (int h = 0; h < 2; ++h) B.a[i][h] = few_load_w(rw, few_add(L.ro, few_koff_w<F8>(u, h, q, p.H)));
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                #pragma unroll
                for (int h = 0; h < Geo::NB; ++h) B.b[i][t][h] = few_load(rx, few_add(L.xo[t], few_koff_x<F8>(u, h, q, p.H)));
            if constexpr (F8) {
                const rsrc_t rs = make_rsrc(L.s, L.live ? (uint32_t)(L.up_s + ksb) * 4u : 0u);
                const int kb = min(u, ksb - 1);
                B.sc[i][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, kb * 4, 0, 0));
                B.sc[i][1] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (L.up_s + kb) * 4, 0, 0));
            }
        }
        if (++L.b == batches) {
            L.item += grid;
            open();
        }
    };
    f32x4 acc[NT];
    auto multiply = [&](const FewBatch<F8, NT>& B) __attribute__((always_inline)) {
        #pragma unroll
        for (int i = 0; i < UB; ++i)
            #pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 d = few_unit<EL, F8>(B.a[i], B.b[i][t]);
                #pragma unroll
                for (int v = 0; v < 4; ++v) acc[t][v] = F8 ? fmaf(d[v], B.sc[i][v >> 1], acc[t][v]) : acc[t][v] + d[v];
            }
    };

    FewBatch<F8, NT> b0, b1;
    L.item = blockIdx.x;
    open();
    load(b0);
    int turn = 0;
    for (int item = blockIdx.x; item < n_items; item += grid, turn ^= 1) {
        #pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        #pragma unroll 1
        for (int b = 0; b < batches; b += 2) {
            load(b1);
            multiply(b0);
            load(b0);                                        // the next item's first, at the end
            multiply(b1);
        }
        // the waves' sums through LDS, two buffers in turn: one barrier an item
        float* const mine = part + turn * (kFewWaves * NT * 256);
        #pragma unroll
        for (int t = 0; t < NT; ++t)
            #pragma unroll
            for (int v = 0; v < 4; ++v) mine[(w * NT + t) * 256 + v * 64 + lane] = acc[t][v];
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        bare_barrier();
        const int ai = __builtin_amdgcn_readfirstlane(item / cb), c0 = (item - ai * cb) * 8;
        const int g = __builtin_amdgcn_readfirstlane(tb.active[1 + ai]);
        const int lo = tb.offsets[g], n = tb.counts[g];
        // thread (tile, output v of a pair, lane of the result): gate v, up v + 2
        for (int e = threadIdx.x; e < NT * 128; e += kFewThreads) {
            const int t = e >> 7, v = (e >> 6) & 1, l = e & 63, r = 16 * t + (l & 15), c = c0 + 2 * (l >> 4) + v;
            if (r >= n) continue;
            float z = 0.f, u = 0.f;
            #pragma unroll
            for (int i = 0; i < kFewWaves; ++i) {
                z += mine[(i * NT + t) * 256 + v * 64 + l];
                u += mine[(i * NT + t) * 256 + (v + 2) * 64 + l];
            }
            if (p.b1) {
                z += p.b1[(size_t)g * 2 * p.I + c];
                u += p.b1[(size_t)g * 2 * p.I + p.I + c];
            }
            z = epi_clamp(z, p.limit);
            float a = 0.f;
            with_act(p.act, [&](auto act) { a = epi_act<decltype(act)::value>(z, p.beta); });
            const float o = a * epi_clamp(u, p.limit) * tb.row_w[lo + r];
            p.h[(size_t)(lo + r) * p.I + c] = (uint16_t)pack16(o, 0.f, EL == kElF16);
        }
    }
}

// ------------------------------------------------------------------ few_w2
template <int EL, bool F8, int NT>
__global__ __launch_bounds__(kFewThreads, 4)
void few_w2_kernel(FewP p) {
    using Geo = FewGeom<F8, NT>;
    constexpr int UB = Geo::UB;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* const part = (float*)smem;                        // [8 waves][NT][4][64]
    int* const active = (int*)(smem + kFewWaves * NT * 1024);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    const int n_act = __builtin_amdgcn_readfirstlane(p.active[0]);
    int16_t* const map = (int16_t*)(active + n_act);
    for (int i = threadIdx.x; i < n_act; i += kFewThreads) active[i] = p.active[1 + i];
    for (int i = threadIdx.x; i < n_act * p.T; i += kFewThreads) map[i] = p.rowmap[i];
    __syncthreads();

    const int n0 = blockIdx.x * 16;
    const int wrow = p.I * (F8 ? 1 : 2);
    const int upg = (p.I + Geo::UK - 1) / Geo::UK;           // units of a group
    const int units = n_act * upg;
    const int nb = ((units + kFewWaves - 1) / kFewWaves + UB - 1) / UB;
    const int nsb = (p.H + 127) >> 7, ksb = (p.I + 127) >> 7;
    // (rows past H read the last row: their sums are not stored)
    const uint32_t ro = (uint32_t)min(n0 + j, p.H - 1) * (uint32_t)wrow;
    const size_t h_rows = (size_t)p.T * (p.k + p.s);

    int ai = w / upg, ku = w - ai * upg;                     // this wave's next unit
    auto load = [&](FewBatch<F8, NT>& B) __attribute__((always_inline)) {
        #pragma unroll
        for (int i = 0; i < UB; ++i) {
            const bool live = ai < n_act;
            const int g = live ? __builtin_amdgcn_readfirstlane(active[ai]) : 0;
            const int sh = g < p.E_loc ? 0 : 1, gi = sh ? 0 : g;
            const rsrc_t rw = make_rsrc(p.w2[sh] + (size_t)gi * (size_t)p.H * (size_t)wrow, live ? (uint32_t)p.H * (uint32_t)wrow : 0u);
            const rsrc_t rh = make_rsrc(p.h, live ? (uint32_t)(h_rows * p.I * 2) : 0u);
            #pragma unroll
            for (int h = 0; h < 2; ++h) B.a[i][h] = few_load_w(rw, few_add(ro, few_koff_w<F8>(ku, h, q, p.I)));
            #pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = live && 16 * t + j < p.T ? map[ai * p.T + 16 * t + j] : -1;
                B.row[i][t] = row;
                const uint32_t o = row >= 0 ? (uint32_t)row * (uint32_t)(p.I * 2) : kMmNoRow;
                #pragma unroll
                for (int h = 0; h < Geo::NB; ++h) B.b[i][t][h] = few_load(rh, few_add(o, few_koff_x<F8>(ku, h, q, p.I)));
            }
            if constexpr (F8) {
                const rsrc_t rs = make_rsrc(p.s2[sh] + ((size_t)gi * nsb + (n0 >> 7)) * ksb, live ? (uint32_t)ksb * 4u : 0u);
                B.sc[i][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, ku * 4, 0, 0));
            }
            ku += kFewWaves;
            while (ku >= upg) { ku -= upg; ++ai; }
            ai = __builtin_amdgcn_readfirstlane(ai);
            ku = __builtin_amdgcn_readfirstlane(ku);
        }
    };
    f32x4 acc[NT];
    #pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const FewBatch<F8, NT>& B) __attribute__((always_inline)) {
        #pragma unroll
        for (int i = 0; i < UB; ++i)
            #pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 d = few_unit<EL, F8>(B.a[i], B.b[i][t]);
                const bool in = B.row[i][t] >= 0;
                #pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float s = F8 ? fmaf(d[v], B.sc[i][0], acc[t][v]) : acc[t][v] + d[v];
                    acc[t][v] = in ? s : acc[t][v];
                }
            }
    };
    FewBatch<F8, NT> b0, b1;
    load(b0);
    #pragma unroll 1
    for (int b = 0; b < nb; b += 2) {
        load(b1);
        multiply(b0);
        load(b0);
        multiply(b1);
    }
    #pragma unroll
    for (int t = 0; t < NT; ++t)
        #pragma unroll
        for (int v = 0; v < 4; ++v) part[(w * NT + t) * 256 + v * 64 + lane] = acc[t][v];
    __syncthreads();
    // thread (token, column): the waves' sums in their order
    for (int e = threadIdx.x; e < NT * 256; e += kFewThreads) {
        const int t = e >> 4, c = e & 15, n = n0 + c;
        if (t >= p.T || n >= p.H) continue;
        float o = 0.f;
        #pragma unroll
        for (int i = 0; i < kFewWaves; ++i) o += part[(i * NT + (t >> 4)) * 256 + (c & 3) * 64 + (c >> 2) * 16 + (t & 15)];
        if (p.b2) {
            for (int a = 0; a < n_act; ++a) {
                const int row = map[a * p.T + t];
                if (row >= 0) o = fmaf(p.row_w[row], p.b2[(size_t)active[a] * p.H + n], o);
            }
        }
        if (p.res) o += lo16(p.res[(size_t)t * p.ld_res + n], EL == kElF16);
        p.out[(size_t)t * p.ld_out + n] = (uint16_t)pack16(o, 0.f, EL == kElF16);
    }
}

template <typename K>
int few_ready(K* k, bool (&ready)[64]) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return (int)e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        const hipError_t f = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, kMmLds);
        if (f != hipSuccess) return (int)f;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    return 0;
}

template <int EL, bool F8, int NT>
int launch_few(const FewP& p, hipStream_t stream) {
    static bool ready1[64] = {false}, ready2[64] = {false};
    auto* k1 = &few_w1_kernel<EL, F8, NT>;
    auto* k2 = &few_w2_kernel<EL, F8, NT>;
    int e = few_ready(k1, ready1);
    if (e || (e = few_ready(k2, ready2))) return e;
    const int64_t rows = (int64_t)p.T * (p.k + p.s), most = std::min<int64_t>(p.G, rows);
    const int64_t items = most * (p.I / 8);
    const int grid = (int)std::min<int64_t>(items, 2 * device_cu_count());
    const size_t scratch = block_lds_ints(kFewWaves, p.G, p.E_loc);
    const size_t lds1 = (size_t)2 * kFewWaves * NT * 1024 + (few_table_ints(p.T, p.k, p.G, p.s) + scratch) * 4;
    const size_t lds2 = (size_t)kFewWaves * NT * 1024 + (size_t)most * 4 + (((size_t)most * p.T * 2 + 3) & ~(size_t)3);
    k1<<<grid, kFewThreads, lds1, stream>>>(p);
    if ((e = (int)hipGetLastError())) return e;
    k2<<<(unsigned)((p.H + 15) / 16), kFewThreads, lds2, stream>>>(p);
    return (int)hipGetLastError();
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// byte offsets of the workspace's regions: h, row_w, slot, active, rowmap, end
void few_regions(int T, int k, int G, int s, int I, size_t (&at)[6]) {
    const size_t R = (size_t)T * (k + s), most = std::min<size_t>(G, R);
    at[0] = 0;
    at[1] = at[0] + up16(R * I * 2);
    at[2] = at[1] + up16(R * 4);
    at[3] = at[2] + up16(R * 4);
    at[4] = at[3] + up16((most + 1) * 4);
    at[5] = at[4] + up16(most * T * 2);
}

}  // namespace

size_t moe_few_bytes(int T, int k, int G, int s, int I) {
    size_t at[6];
    few_regions(T, k, G, s, I, at);
    return at[5];
}

int moe_launch_few(const moe_few_args& a, void* ws, hipStream_t stream) {
    FewP p{};
    p.logits = a.logits;
    p.T = a.T; p.E = a.E_tot; p.k = a.k; p.e0 = a.e0; p.E_loc = a.E_loc; p.s = a.shared_w1 ? 1 : 0;
    p.G = p.E_loc + p.s; p.renorm = (a.flags & MOE_ROUTE_RENORM) != 0;
    p.x = (const uint8_t*)a.x; p.x_ld = (uint32_t)a.ldx * 2; p.x_bytes = (uint32_t)(a.T - 1) * p.x_ld + (uint32_t)a.H * 2;
    p.H = a.H; p.I = a.I;
    p.w1[0] = (const uint8_t*)a.w1; p.w1[1] = (const uint8_t*)a.shared_w1;
    p.w2[0] = (const uint8_t*)a.w2; p.w2[1] = (const uint8_t*)a.shared_w2;
    p.s1[0] = a.w1_scales; p.s1[1] = a.shared_w1_scales;
    p.s2[0] = a.w2_scales; p.s2[1] = a.shared_w2_scales;
    p.act = a.epi ? a.epi->act : MOE_ACT_SWIGLU; p.beta = a.epi ? a.epi->beta : 1.0f; p.limit = a.epi ? a.epi->limit : 0.0f;
    p.b1 = a.epi ? a.epi->bias : nullptr; p.b2 = a.bias2;
    p.res = (const uint16_t*)a.residual; p.ld_res = (size_t)a.ld_res;
    p.out = (uint16_t*)a.out; p.ld_out = (size_t)a.ld_out;
    size_t at[6];
    few_regions(p.T, p.k, p.G, p.s, p.I, at);
    uint8_t* b = (uint8_t*)ws;
    p.h = (uint16_t*)(b + at[0]); p.row_w = (float*)(b + at[1]); p.slot = (int32_t*)(b + at[2]);
    p.active = (int32_t*)(b + at[3]); p.rowmap = (int16_t*)(b + at[4]);
    const bool f8 = a.w1_scales != nullptr, two = a.T > 16;
    if (a.dtype == MOE_T_F16) {
        if (f8) return two ? launch_few<kElF16, true, 2>(p, stream) : launch_few<kElF16, true, 1>(p, stream);
        return two ? launch_few<kElF16, false, 2>(p, stream) : launch_few<kElF16, false, 1>(p, stream);
    }
    if (f8) return two ? launch_few<kElBf16, true, 2>(p, stream) : launch_few<kElBf16, true, 1>(p, stream);
    return two ? launch_few<kElBf16, false, 2>(p, stream) : launch_few<kElBf16, false, 1>(p, stream);
}

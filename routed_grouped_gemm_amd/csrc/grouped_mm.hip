// Grouped products of 16-bit and block-scaled FP8 operands and their weight
// gradients: the plain ones of the LDS-tiled kernel (grouped_mm_tiled.h; few
// rows per group: grouped_mm_rows.hip), the choice of a kernel and its split,
// and the launches.
#include <algorithm>

#include "grouped_mm_tiled.h"

namespace {

// The partial sums of split groups into the gradient, in the order of the
// parts: 64 rows of one tile per workgroup. Bound by HBM (each partial tile is
// read once).
__global__ __launch_bounds__(256)
void wgrad_join_kernel(MmP p) {
    const int bt = (p.N + 255) / 256, at = (p.K + 255) / 256, tiles = at * bt;
    const int g = blockIdx.y, tile = blockIdx.x >> 2, quarter = blockIdx.x & 3;
    const int lane = threadIdx.x & 63;
    const int parts = wgrad_parts(p, group_ktiles(p, g));
    if (parts == 1) return;
    int slot = 0, all = 0;                                   // slots of the groups before this one, and of all
    for (int g0 = 0; g0 < p.G; g0 += 64) {
        const int m = g0 + lane < p.G ? wgrad_parts(p, group_ktiles(p, g0 + lane)) : 0, n = m > 1 ? m * tiles : 0;
        slot += __builtin_amdgcn_readlane(wave_incl_scan(g0 + lane < g ? n : 0), 63);
        all += __builtin_amdgcn_readlane(wave_incl_scan(n), 63);
    }
    if (all > p.max_slots) return;
    // the tile's place, as the product's items count them
    const int band = tile / (4 * at), h = min(4, bt - 4 * band), l2 = tile - band * 4 * at;
    const int a0 = (l2 / h) * 256, b0 = (4 * band + l2 % h) * 256;
    const float* src = p.partial + ((size_t)slot + tile) * 65536;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int row = quarter * 64 + (i >> 6), col = (i & 63) * 4;
        if (b0 + row >= p.N || a0 + col >= p.K) continue;
        f32x4 v = *(const f32x4*)(src + row * 256 + col);
        for (int s = 1; s < parts; ++s) {
            const f32x4 e = *(const f32x4*)(src + (size_t)s * tiles * 65536 + row * 256 + col);
            v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]};
        }
        const size_t o = ((size_t)g * p.N + b0 + row) * p.K + a0 + col;
        if (p.out_f32) {
            f32x4* d = (f32x4*)((float*)p.out + o);
            if (p.accumulate) { const f32x4 e = *d; v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]}; }
            *d = v;
        } else {
            u32x2_t* d = (u32x2_t*)((uint16_t*)p.out + o);
            if (p.accumulate) {
                const u32x2_t e = *d;
                v[0] += lo16(e.x, p.out_f16); v[1] += hi16(e.x, p.out_f16);
                v[2] += lo16(e.y, p.out_f16); v[3] += hi16(e.y, p.out_f16);
            }
            *d = u32x2_t{pack16(v[0], v[1], p.out_f16), pack16(v[2], v[3], p.out_f16)};
        }
    }
}

// launchers
template <int EL, int MODE>
int launch_mm_rows(const MmP& p, int kind, int rows, hipStream_t stream) {
    if (rows <= 64) return moe_launch_mm_rows(&p, EL, kind, rows, stream);
    return rows > 128 ? launch_mm<EL, MODE, 8>(p, mm_items(p, 256), stream)
                      : launch_mm<EL, MODE, 4>(p, mm_items(p, 128), stream);
}

// The kernel of a product and its split along K, from sizes alone (uniform
// groups assumed: the counts are on the device). Time in rounds of workgroups,
// nk K-tiles each, at the measured microseconds per K-tile (G = 1, K = 4096,
// N = 4096 and 1024, R from 16 to 16384; W [K, N] and FP8 cost 1.1 to 1.3 times
// as much in all four, so their choice is the same):
//   256 rows x 256   1.6 (1.3 with few workgroups)   1 workgroup per CU
//   128 rows x 256   1.0 (0.9)                       1
//    64 rows x  64   0.54 for two on a CU (0.5)      2
//    32 rows x  64   0.48 for two on a CU (0.45)     2
// e.g. 512 x 4096 x 4096: 84, 58, 40 and 67 us; 4096 x 4096 x 4096: 109, 127,
// 281, 496. Splitting (64- and 32-row tiles only) costs the joining launch and
// its partial sums, about 5 us.
struct MmPlan { int rows, parts; };
MmPlan mm_plan(bool fp8, int R_max, int G, int N, int K) {
    static const int kRowsOf[4] = {256, 128, 64, 32};
    static const double kTile[4] = {1.6, 1.0, 0.54, 0.48}, kFew[4] = {1.3, 0.9, 0.5, 0.45};
    if (R_max <= 0) return MmPlan{32, 1};
    const int cus = device_cu_count(), active = std::max(1, std::min(G, R_max));
    const int64_t per = ((int64_t)R_max + active - 1) / active;          // rows of a group
    const int nk = (K + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
    MmPlan best{256, 1};
    double least = 1e30;
    for (int i = 0; i < 4; ++i) {
        const int cols = i < 2 ? 256 : 64, slots = i < 2 ? cus : 2 * cus;
        const int64_t items = active * ((per + kRowsOf[i] - 1) / kRowsOf[i]) * ((N + cols - 1) / cols);
        const int most = i < 2 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({slots / items, nk / 8, 16}));
        for (int parts = 1; parts <= most; parts = parts < most && 2 * parts > most ? most : 2 * parts) {
            const int64_t rounds = (items * parts + slots - 1) / slots;
            const double tile = items * parts <= cus ? kFew[i] : kTile[i];
            const double t = (double)rounds * ((nk + parts - 1) / parts * tile + (i < 2 ? 4.0 : 1.0)) + (parts > 1 ? 5.0 : 0.0);
            if (t < least) { least = t; best = MmPlan{kRowsOf[i], parts}; }
        }
    }
    // (three stages of 128 rows leave LDS for the tables of 2047 groups)
    const int lds = fp8 ? MmGeom<kElFp8, 4>::Lds(G, false) : MmGeom<kElBf16, 4>::Lds(G, false);
    if (best.rows == 128 && lds > kMmLds) best.rows = 256;
    return best;
}

// K-tiles per part of a weight gradient (0: no group can be longer): groups
// longer than that are split, so that few tiles, or one large group, do not
// leave most workgroups idle. For groups of equal size, the number of parts
// with the least time in rounds of workgroups (1.5 us a K-tile, 10 a tile) and
// in joining (256 KiB written and read per part and tile, at 4 TB/s); at least
// a workgroup's even share of the whole, for the groups that are larger. E.g.
// one group of 16384 rows, 2816 x 2048 (88 tiles, 256 K-tiles): 2 parts.
int wgrad_part(int R_max, int G, int N, int K) {
    if (R_max <= 0) return 0;
    const int64_t tiles = (int64_t)((N + 255) / 256) * ((K + 255) / 256), most = ((int64_t)R_max + 63) / 64;
    const int64_t cus = device_cu_count(), active = std::min(G, R_max);
    const int64_t share = (tiles * (most + active / 2) + cus - 1) / cus, nk = (most + active - 1) / active;
    int64_t part = nk;
    double least = 1e30;
    for (int64_t n = 1; n <= 64 && n * 8 <= nk + 7; ++n) {
        const int64_t items = tiles * active * n;
        const double t = (double)((items + cus - 1) / cus) * (1.5 * (double)((nk + n - 1) / n) + 10.0) +
                         (n > 1 ? 5.0 + (double)items * 0.131 : 0.0);
        if (t < least) { least = t; part = (nk + n - 1) / n; }
    }
    if (part == nk) part = std::max<int64_t>({nk, share, 8});
    return part >= most ? 0 : (int)part;
}

template <int EL, int KIND>
int launch_wgrad(const MmP& p, int items, hipStream_t stream) {
    if (p.x_src && p.dy_src) return launch_mm<EL, KIND | kGatherX | kGatherDy, 8>(p, items, stream);
    if (p.x_src) return launch_mm<EL, KIND | kGatherX, 8>(p, items, stream);
    if (p.dy_src) return launch_mm<EL, KIND | kGatherDy, 8>(p, items, stream);
    return launch_mm<EL, KIND, 8>(p, items, stream);
}

}  // namespace

void moe_mm_plan(bool fp8, int R_max, int G, int N, int K, int* tile_rows, int* parts) {
    const MmPlan plan = mm_plan(fp8, R_max, G, N, K);
    *tile_rows = plan.rows;
    *parts = plan.parts;
}
int moe_wgrad_plan(int R_max, int G, int N, int K) { return wgrad_part(R_max, G, N, K) * 64; }

size_t moe_mm_workspace_bytes(int kind, bool fp8, int R_max, int G, int N, int K) {
    if (kind == 2) {
        const int part = wgrad_part(R_max, G, N, K);
        if (part == 0) return 0;
        // groups longer than a part are split into fewer than twice as many
        // parts as their K-tiles make whole ones (partly filled K-tiles, one a
        // group, included)
        const int64_t tiles = (int64_t)((N + 255) / 256) * ((K + 255) / 256);
        const int64_t ktiles = ((int64_t)R_max + 63) / 64 + std::min(G, R_max);
        return (size_t)(tiles * (2 * ktiles / part)) * 65536 * 4;
    }
    const MmPlan plan = mm_plan(fp8, R_max, G, N, K);
    return plan.parts > 1 ? (size_t)plan.parts * R_max * N * 4 : 0;
}

int moe_launch_mm(const MmCall& c, hipStream_t stream) {
    const int eb = c.fp8 ? 1 : 2;
    MmP p{};
    p.x = (const uint8_t*)c.x; p.x_ld = (uint32_t)(c.ldx * eb); p.x_src = c.x_src;
    p.x_rows = (uint32_t)c.x_rows;
    if (c.x_src) p.x_bytes = (uint32_t)((int64_t)(c.x_rows - 1) * c.ldx * eb + (int64_t)c.K * eb);
    p.offsets = c.offsets;
    p.G = c.G; p.N = c.N; p.K = c.K; p.R_max = c.R_max;
    p.out = (uint8_t*)c.out; p.out_ld = (size_t)c.ldy;
    p.out_f16 = c.dtype == MOE_T_F16; p.out_f32 = c.out_f32; p.accumulate = c.accumulate;
    const bool f16 = c.dtype == MOE_T_F16;
    if (c.kind == 2) {
        if (c.xs) {                                          // x in 8 bits
            p.x_ld = (uint32_t)c.ldx;
            p.xs = c.xs; p.kb = (c.K + 127) / 128;
            if (c.x_src) {
                p.x_bytes = (uint32_t)((int64_t)(c.x_rows - 1) * c.ldx + c.K);
                p.xs_bytes = (uint32_t)((int64_t)c.x_rows * p.kb * 4);
            }
        }
        p.dy = (const uint8_t*)c.dy; p.dy_ld = (uint32_t)(c.ld_dy * 2); p.dy_src = c.dy_src;
        p.dy_rows = (uint32_t)c.dy_rows;
        if (c.dy_src) p.dy_bytes = (uint32_t)((int64_t)(c.dy_rows - 1) * c.ld_dy * 2 + (int64_t)c.N * 2);
        const int64_t tiles = (int64_t)c.G * ((c.N + 255) / 256) * ((c.K + 255) / 256);
        const int items = (int)std::min<int64_t>(tiles, 1 << 30);
        p.part = wgrad_part(c.R_max, c.G, c.N, c.K);
        p.partial = (float*)c.ws;
        p.max_slots = (int)(moe_mm_workspace_bytes(2, false, c.R_max, c.G, c.N, c.K) / (65536 * 4));
        int e;
        const int grid = p.part > 0 ? 1 << 30 : items;       // (split groups have more items than tiles)
        if (c.xs) e = launch_wgrad<kElBf16, kWgrad8>(p, grid, stream);
        else e = f16 ? launch_wgrad<kElF16, kWgrad>(p, grid, stream) : launch_wgrad<kElBf16, kWgrad>(p, grid, stream);
        if (e || p.part == 0) return e;
        const dim3 join((unsigned)(tiles / c.G * 4), (unsigned)c.G);
        wgrad_join_kernel<<<join, 256, 0, stream>>>(p);
        return (int)hipGetLastError();
    }
    const MmPlan plan = mm_plan(c.fp8, c.R_max, c.G, c.N, c.K);
    p.parts = plan.parts;
    p.partial = (float*)c.ws;
    p.w = (const uint8_t*)c.w;
    p.w_group = (size_t)c.N * c.K * eb;
    p.w_ld = (uint32_t)((c.kind == 1 ? c.N : c.K) * eb);
    if (c.fp8) {
        p.kb = (c.K + 127) / 128; p.nb = (c.N + 127) / 128;
        p.xs = c.xs; p.ws = c.wscale;
        if (c.x_src) p.xs_bytes = (uint32_t)((int64_t)c.x_rows * p.kb * 4);
        return launch_mm_rows<kElFp8, kMmNK>(p, 0, plan.rows, stream);
    }
    if (c.kind == 0)
        return f16 ? launch_mm_rows<kElF16, kMmNK>(p, 0, plan.rows, stream) : launch_mm_rows<kElBf16, kMmNK>(p, 0, plan.rows, stream);
    return f16 ? launch_mm_rows<kElF16, kMmKN>(p, 1, plan.rows, stream) : launch_mm_rows<kElBf16, kMmKN>(p, 1, plan.rows, stream);
}

// Grouped products (see grouped_mm.hip) for few rows per group, where the
// weights' bytes bound the call: every weight is read once per pass of BT rows.
//
// A workgroup of 4 waves computes 64 values of the a axis (n) for 32 or 64
// rows; wave w owns 16 of the 64 and all rows. 64, not 256: a decode batch on
// a few experts then gives about as many work items as two workgroups per CU
// take at once (8 groups of N = 4096: 512), and the K loop needs no split.
// K-tiles (64 x 128 bytes of weights, BT x 128 bytes of rows) are staged in
// LDS by loads that write it directly, through a ring of NST stages, so that
// about 40 KB of weights per workgroup are on their way; one barrier per
// K-tile. Layouts and swizzles as in grouped_mm.hip.
//
// Measured, weights not in any cache: 2 rows on each of 8 experts, 4096 x 7168
// in BF16 (470 MB) 76 us, 6.2 TB/s, in FP8 (235 MB) 41 us, 5.7 TB/s, W [K, N]
// 95 us; 16 rows of one expert, 1024 x 7168 (15 MB), 16 us of which about 5 are
// the joining launch, against 47 us unsplit.
#include <algorithm>

#include "grouped_mm.h"

namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsA = 64;

template <int EL, int NB>
struct RowsGeom {
    static constexpr int BT = 16 * NB;
    static constexpr int NQ = BT / 32;                       // requests of a wave for the rows
    static constexpr int QOff = kRowsA * 128;
    static constexpr int SOff = QOff + BT * 128;             // fp8: row scales, 256 bytes per wave
    static constexpr int Stage = SOff + (EL == kElFp8 ? 1024 : 0);
    static constexpr int NST = (kMmLds / 2 - 4096) / Stage;  // two workgroups per CU
    static constexpr int Loads = 2 + NQ + (EL == kElFp8 ? 1 : 0);
};

// the requests of a wave, one K-tile after another through all items
template <int NQ>
struct RowsReq {
    int item, kt, k1, step;             // K-tiles [kt, k1) of the item are still to come
    bool live;
    MmItem c;
    uint32_t row[NQ], srow;
};

// Item number `item`: its tile, and the K-tiles [k0, k1) of its part. A part's
// tiles go one after another before the next part's.
template <int EL, int MODE, int BT>
MOE_DEV MmItem rows_item(const MmP& p, const MmTables& tb, const MmWhere& wh, int item, int& part, int& k0, int& k1) {
    const int tiles = wh.n_items / p.parts;
    part = __builtin_amdgcn_readfirstlane(item / tiles);
    const MmItem c = mm_scalar(mm_decode<EL, MODE, BT, kRowsA>(p, tb, wh.at, item - part * tiles));
    k0 = __builtin_amdgcn_readfirstlane(c.nk * part / p.parts);
    k1 = __builtin_amdgcn_readfirstlane(c.nk * (part + 1) / p.parts);
    return c;
}

template <int EL, int MODE, int NB, int NQ>
MOE_DEV void rows_open(const MmP& p, const MmTables& tb, const MmWhere& wh, RowsReq<NQ>& R) {
    constexpr int BT = 16 * NB;
    R.live = R.item < wh.n_items;
    if (!R.live) return;
    int part;
    R.c = rows_item<EL, MODE, BT>(p, tb, wh, R.item, part, R.kt, R.k1);
    R.item += wh.grid;
    // source rows without a branch: past the item (and without a source
    // array, whose resource is then empty) the loads return 0
    const rsrc_t rm = make_rsrc(p.x_src + R.c.r0, p.x_src ? (uint32_t)(R.c.nrows * 4) : 0u);
    const int first = (BT / 4) * wh.w;
    #pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int row = first + 8 * i + (wh.lane >> 3);
        const uint32_t s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, row * 4, 0, 0);
        R.row[i] = row < R.c.nrows && s < p.x_rows ? (p.x_src ? s : (uint32_t)row) * p.x_ld : kMmNoRow;
    }
    if constexpr (EL == kElFp8) {
        const int row = first + wh.lane;
        const uint32_t s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, row * 4, 0, 0);
        R.srow = wh.lane < BT / 4 && row < R.c.nrows && s < p.x_rows ? (p.x_src ? s : (uint32_t)row) * (uint32_t)(p.kb * 4)
                                                                    : kMmNoRow;
    }
}

// request one K-tile into its stage, then move on (nothing once the items have
// ended). Tiles of 32 rows serve groups of about one pass each, whose weights
// are then read once: their weight loads are non-temporal (83 -> 77 us for the
// BF16 decode above; 128 rows on one of 33 groups and 4 on the others, 2816 x
// 2048, 89 -> 83). Where such a tile is chosen for a group of many passes that
// costs little (264 x 520, 94 passes 11.7 -> 11.5 us; 264 x 1544, 10 passes 15.7
// -> 16.2; 200 of 256 rows on one of 8 groups, 4096 x 4096, 75.7 -> 79.0). With
// 64 rows several passes share the weights through the caches (512 x 4096 x
// 4096: 40 us, non-temporal 43).
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void rows_request(const MmP& p, const MmTables& tb, const MmWhere& wh, RowsReq<NQ>& R, uint8_t* smem) {
    using Geo = RowsGeom<EL, NB>;
    constexpr int EB = EL == kElFp8 ? 1 : 2, BT = Geo::BT;
    if (!R.live) return;
    const int lane = mm_fresh(wh.lane), w = wh.w;
    const MmItem& c = R.c;
    uint8_t* st = smem + (R.step % Geo::NST) * Geo::Stage;
    if constexpr (MODE == kMmNK) {
        const rsrc_t r = make_rsrc(p.w + (size_t)c.g * p.w_group + (size_t)c.a0 * p.w_ld,
                                   (uint32_t)min(kRowsA, p.N - c.a0) * p.w_ld);
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int kb = R.kt * 128 + 16 * ((lane & 7) ^ ((lane >> 4) | (4 * i)));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (mm_lds_void_t*)(st + (16 * w + 8 * i) * 128), 16,
                kb < p.K * EB ? (uint32_t)(16 * w + 8 * i + (lane >> 3)) * p.w_ld + (uint32_t)kb : kMmInvalid, 0, 0, NB == 2 ? 2 : 0);
        }
    } else {
        const int krem = p.K - R.kt * 64;
        const rsrc_t r = make_rsrc(p.w + (size_t)c.g * p.w_group + (size_t)R.kt * 64 * p.w_ld + (size_t)c.a0 * 2,
                                   (uint32_t)(min(krem, 64) - 1) * p.w_ld + (uint32_t)(min(kRowsA, p.N - c.a0) * 2));
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = 16 * w + 8 * i + (lane >> 3);
            const int col = (((lane & 7) >> 1) ^ (k & 3)) * 16 + (lane & 1) * 8;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (mm_lds_void_t*)(st + (16 * w + 8 * i) * 128), 16,
                k < krem && c.a0 + col < p.N ? (uint32_t)k * p.w_ld + (uint32_t)(col * 2) : kMmInvalid, 0, 0, NB == 2 ? 2 : 0);
        }
    }
    // gathered rows are addressed from the array's start, a group's own rows from the tile's first
    const rsrc_t rx = make_rsrc(p.x_src ? p.x : p.x + (size_t)c.r0 * p.x_ld,
                                p.x_src ? p.x_bytes : (uint32_t)(c.nrows - 1) * p.x_ld + (uint32_t)(p.K * EB));
    const int first = (BT / 4) * w;
    #pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int kb = R.kt * 128 + 16 * ((lane & 7) ^ ((lane >> 4) | (4 * (((first >> 3) + i) & 1))));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (mm_lds_void_t*)(st + Geo::QOff + (first + 8 * i) * 128), 16,
                                                 kb < p.K * EB ? R.row[i] + (uint32_t)kb : kMmInvalid, 0, 0, 0);
    }
    if constexpr (EL == kElFp8) {
        const rsrc_t rs = make_rsrc(p.x_src ? p.xs : p.xs + (size_t)c.r0 * p.kb,
                                    p.x_src ? p.xs_bytes : (uint32_t)(c.nrows * p.kb * 4));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (mm_lds_void_t*)(st + Geo::SOff + w * 256), 4,
                                                 R.srow + (uint32_t)(R.kt * 4), 0, 0, 0);
    }
    ++R.step;
    const int kt = R.kt + 1;
    const bool last = kt == R.k1;
    R.kt = kt;
    if (last) rows_open<EL, MODE, NB>(p, tb, wh, R);
}

template <int EL, int MODE, int NB>
__global__ __launch_bounds__(kRowsThreads, 2)
void grouped_mm_rows_kernel(MmP p) {
    using Geo = RowsGeom<EL, NB>;
    constexpr int BT = Geo::BT, NST = Geo::NST;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* const tab = (int*)(smem + NST * Geo::Stage);        // [G + 1] passes before group g
    const MmTables tb{tab, nullptr, nullptr};

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    const int at = (p.N + kRowsA - 1) / kRowsA;
    if (w == 0) mm_passes(p, BT, at * p.parts, lane, tab);
    __syncthreads();
    const int n_items = __builtin_amdgcn_readfirstlane(tab[p.G]) * at * p.parts;
    const int grid = gridDim.x;
    const int slot = (grid % 8 == 0) ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
    if (slot >= n_items) return;
    const MmWhere wh{n_items, at, grid, slot, lane, w, 0};

    // fp8: the weight scales of a part's K-tiles, one per lane, loaded an item
    // ahead (a load in the K loop would be waited for in every K-tile)
    uint32_t fwv = 0, fwn = 0;
    auto load_fw = [&](const MmItem& c, int kt) __attribute__((always_inline)) {
        const float* ws = p.ws + ((size_t)c.g * p.nb + (c.a0 >> 7)) * p.kb;
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(make_rsrc(ws, (uint32_t)(p.kb * 4)), (kt + lane) * 4, 0, 0);
    };
    if constexpr (EL == kElFp8) {
        int part, k0, k1;
        const MmItem c = rows_item<EL, MODE, BT>(p, tb, wh, slot, part, k0, k1);
        fwn = load_fw(c, k0);
    }

    RowsReq<Geo::NQ> R;
    R.item = slot;
    R.step = 0;
    rows_open<EL, MODE, NB>(p, tb, wh, R);
    #pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) rows_request<EL, MODE, NB>(p, tb, wh, R, smem);

    int step = 0;
    for (int item = slot; item < n_items; item += grid) {
        int part, k0, k1;
        const MmItem c = rows_item<EL, MODE, BT>(p, tb, wh, item, part, k0, k1);
        if constexpr (EL == kElFp8) {
            fwv = fwn;
            asm volatile("" : "+v"(fwv));
            if (item + grid < n_items) {
                int npart, nk0, nk1;
                const MmItem n = rows_item<EL, MODE, BT>(p, tb, wh, item + grid, npart, nk0, nk1);
                fwn = load_fw(n, nk0);
            }
        }
        f32x4 acc[NB];
        #pragma unroll
        for (int u = 0; u < NB; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        #pragma unroll 1
        for (int kt = k0; kt < k1; ++kt, ++step) {
            // this K-tile has landed (newer ones stay in flight), and behind
            // the barrier the previous one has been read: its stage is free
            if (R.live) __builtin_amdgcn_s_waitcnt(waitcnt_imm(Geo::Loads * (NST - 2), 15));
            else __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
            bare_barrier();
            rows_request<EL, MODE, NB>(p, tb, wh, R, smem);
            const uint8_t* st = smem + (step % NST) * Geo::Stage;
            i32x4 fp[2], fq[2][NB];
            float fs[NB], fw = 0.f;
            #pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int ch = ((4 * s + q) ^ ((j >> 1) & 7)) * 16;
                if constexpr (MODE == kMmNK) {
                    fp[s] = *(const i32x4*)(st + (16 * w + j) * 128 + ch);
                } else {
                    const int o = (32 * s + 8 * q + (j >> 2)) * 128 + ((w ^ (j >> 2)) * 32) + (j & 3) * 8;
                    const u32x2_t l = read_tr16((const mm_lds_s16x4*)(st + o)), hh = read_tr16((const mm_lds_s16x4*)(st + o + 4 * 128));
                    fp[s] = i32x4{(int)l.x, (int)l.y, (int)hh.x, (int)hh.y};
                }
                #pragma unroll
                for (int u = 0; u < NB; ++u) fq[s][u] = *(const i32x4*)(st + Geo::QOff + (16 * u + j) * 128 + ch);
            }
            if constexpr (EL == kElFp8) {
                #pragma unroll
                for (int u = 0; u < NB; ++u)
                    fs[u] = *(const float*)(st + Geo::SOff + ((16 * u + j) / (BT / 4)) * 256 + ((16 * u + j) % (BT / 4)) * 4);
                // (used here, so that the wait for it is here: behind the
                // branch it would drain the requests of every K-tile)
                if (((kt - k0) & 63) == 0 && kt > k0) {
                    fwv = load_fw(c, kt);
                    asm volatile("" : "+v"(fwv));
                }
                fw = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)fwv, (kt - k0) & 63));
                #pragma unroll
                for (int u = 0; u < NB; ++u) {
                    const f32x4 d = mfma_fp8(fp[0], fp[1], fq[0][u], fq[1][u], f32x4{0.f, 0.f, 0.f, 0.f});
                    const float sc = fs[u] * fw;
                    #pragma unroll
                    for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(d[v], sc, acc[u][v]);
                }
            } else {
                #pragma unroll
                for (int s = 0; s < 2; ++s)
                    #pragma unroll
                    for (int u = 0; u < NB; ++u) acc[u] = mfma16x16x32<EL>(fp[s], fq[s][u], acc[u]);
            }
            // the reads of this stage end here, before the next barrier
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        }
        const int a = c.a0 + 16 * w + 4 * q;
        const int f16 = EL == kElFp8 ? p.out_f16 : EL == kElF16;
        #pragma unroll
        for (int u = 0; u < NB; ++u) {
            const int b = 16 * u + j;
            if (b < c.nrows && a < p.N) {
                const size_t row = (size_t)(c.r0 + b);
                if (p.parts > 1)
                    *(f32x4*)(p.partial + ((size_t)part * p.R_max + row) * p.N + a) = acc[u];
                else
                    *(u32x2_t*)((uint16_t*)p.out + row * p.out_ld + a) =
                        u32x2_t{pack16(acc[u][0], acc[u][1], f16), pack16(acc[u][2], acc[u][3], f16)};
            }
        }
    }
}

// The sum of a split product's parts, in their order, rounded once: 4 values
// per lane, for the rows that belong to a group.
__global__ __launch_bounds__(256)
void mm_join_kernel(MmP p) {
    int lo, hi, end;
    group_rows(p, 0, lo, hi);
    group_rows(p, p.G - 1, hi, end);
    const int n4 = p.N / 4;
    const int64_t total = (int64_t)p.R_max * n4, stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
        const int row = (int)(i / n4), a = (int)(i - (int64_t)row * n4) * 4;
        if (row < lo || row >= end) continue;
        const float* src = p.partial + (size_t)row * p.N + a;
        f32x4 v = *(const f32x4*)src;
        for (int s = 1; s < p.parts; ++s) {
            const f32x4 e = *(const f32x4*)(src + (size_t)s * p.R_max * p.N);
            v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]};
        }
        *(u32x2_t*)((uint16_t*)p.out + (size_t)row * p.out_ld + a) =
            u32x2_t{pack16(v[0], v[1], p.out_f16), pack16(v[2], v[3], p.out_f16)};
    }
}

template <int EL, int MODE, int NB>
int launch_rows(const MmP& p, hipStream_t stream) {
    using Geo = RowsGeom<EL, NB>;
    auto* k = &grouped_mm_rows_kernel<EL, MODE, NB>;
    static bool ready[64] = {false};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return (int)e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, kMmLds);
        if (e != hipSuccess) return (int)e;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    const int64_t items = (int64_t)mm_items(p, Geo::BT, kRowsA) * p.parts;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(items, 2 * device_cu_count()));
    k<<<grid, kRowsThreads, (size_t)(Geo::Stage * Geo::NST + (p.G + 1) * 4), stream>>>(p);
    if (p.parts == 1) return (int)hipGetLastError();
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const int64_t lanes = (int64_t)p.R_max * (p.N / 4);
    mm_join_kernel<<<(int)std::min<int64_t>((lanes + 255) / 256, 4 * device_cu_count()), 256, 0, stream>>>(p);
    return (int)hipGetLastError();
}

template <int EL, int MODE>
int launch_few(const MmP& p, int rows, hipStream_t stream) {
    return rows > 32 ? launch_rows<EL, MODE, 4>(p, stream) : launch_rows<EL, MODE, 2>(p, stream);
}

}  // namespace

int moe_launch_mm_rows(const void* params, int el, int kind, int rows, hipStream_t stream) {
    const MmP& p = *(const MmP*)params;
    if (el == kElFp8) return launch_few<kElFp8, kMmNK>(p, rows, stream);
    if (el == kElF16) return kind ? launch_few<kElF16, kMmKN>(p, rows, stream) : launch_few<kElF16, kMmNK>(p, rows, stream);
    return kind ? launch_few<kElBf16, kMmKN>(p, rows, stream) : launch_few<kElBf16, kMmNK>(p, rows, stream);
}

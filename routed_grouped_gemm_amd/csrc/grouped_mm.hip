// Grouped products of 16-bit and block-scaled FP8 operands, ragged by expert:
//
//   mm, W [N, K]   y[r][n]  = sum_k x[r][k] W_g[n][k]
//   mm, W [K, N]   y[r][n]  = sum_k x[r][k] W_g[k][n]       (gradient of the rows)
//   wgrad          dW_g[n][k] = sum_{r in g} dy[r][n] x[r][k]
//   fp8            y[r][n]  = sum_b xs[r][b] ws_g[n/128][b] sum_{k in block b} xq[r][k] wq_g[n][k]
//
// One kernel body: a workgroup of 8 waves computes D[a][b] over tiles of 256
// values of the contiguous output axis a (n, or k for wgrad) and BT of the
// other axis b (rows, or n for wgrad). Wave w owns a-quarter w % 4 and b-half
// w / 4: 4 x NB tiles of the 16x16 matrix instruction. The a side is the
// instruction's A operand, so a lane ends up with 4 consecutive a values of
// one b: its stores are 8 or 16 bytes.
//
// Each operand is staged in LDS by buffer loads that write LDS directly, in
// K-tiles of 64 16-bit or 128 FP8 elements (128 bytes), in one of two forms:
//  - reduction axis contiguous in memory: [row][128 bytes], 16-byte chunks
//    XOR-swizzled by row so that the operand reads (16 rows, one chunk each)
//    hit distinct banks;
//  - reduction axis slow in memory (W [K, N]; both operands of wgrad):
//    [k][256 values], read through the transposing LDS load (16 lanes read
//    4 k x 16 values and receive 4 k of one value each), 32-byte chunks
//    XOR-swizzled by k so that a half wave's 8 rows hit distinct banks.
// Elements past an edge (rows past the group, the K tail, values past N) are
// zero: their offsets fall outside the resource.
//
// Two waves share a SIMD. They run half a step apart: while waves 4-7
// multiply, waves 0-3 read their fragments of the next K-tile from LDS, and
// the other way round, so the matrix cores and the LDS are both busy. One
// step of a wave is [requests for a later K-tile (waves 0-3), fragment reads]
// barrier [products] barrier; waves 4-7 start one barrier later. A K-tile's
// stage is rewritten only after the barrier behind which waves 4-7 have read
// it; waves 0-3 wait for their requests before the barrier that opens the
// step using them.
//
// Persistent grid; the requests run ahead across items, so the next item's
// first K-tiles are in flight during an item's epilogue.
#include <algorithm>

#include "grouped_mm.h"

namespace {

enum { kMmNK = 0, kMmKN = 1, kWgrad = 2, kWgrad8 = 3 };     // kWgrad8: x rows in E4M3 with block scales
constexpr bool is_wgrad(int mode) { return mode >= kWgrad; }

constexpr int kMmThreads = 512;
constexpr int kATile = 256;
constexpr int kPBytes = kATile * 128;       // one K-tile of the a operand

template <int EL, int NB>
struct MmGeom {
    static constexpr int BT = 32 * NB;                       // b values per workgroup tile
    static constexpr int QOff = kPBytes;
    static constexpr int SOff = kPBytes + BT * 128;          // fp8: row scales
    static constexpr int Stage = SOff + (EL == kElFp8 ? BT * 4 : 0);
    static constexpr int NST = Stage * 4 + 8320 <= 163840 ? 4 : (Stage * 3 + 8320 <= 163840 ? 3 : 2);
    static constexpr int Loads = 8 + NB + (EL == kElFp8 ? 1 : 0);   // per wave 0-3 and K-tile
    static constexpr int Lds(int G) { return Stage * NST + (G + 1) * 4; }
};

// chunk swizzle of a row in the contiguous form, and of a k in the slow form
MOE_DEV int kc_swz(int row) { return (row >> 1) & 7; }
MOE_DEV int tr_swz(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }

struct MmItem { int g, a0, b0, r0, nrows, nk; };

// the item's fields as scalars again (control flow that merely looks divergent
// would otherwise turn every descriptor load into a loop over lanes)
MOE_DEV MmItem mm_scalar(const MmItem& c) {
    return MmItem{__builtin_amdgcn_readfirstlane(c.g), __builtin_amdgcn_readfirstlane(c.a0),
                  __builtin_amdgcn_readfirstlane(c.b0), __builtin_amdgcn_readfirstlane(c.r0),
                  __builtin_amdgcn_readfirstlane(c.nrows), __builtin_amdgcn_readfirstlane(c.nk)};
}

// Where a workgroup is: its items and this lane.
struct MmWhere { int n_items, at, grid, lane, w; };

template <int EL, int MODE, int NB>
MOE_DEV MmItem mm_decode(const MmP& p, const int* pass_off, int at, int item) {
    constexpr int BT = 32 * NB, KT = EL == kElFp8 ? 128 : 64;
    MmItem c;
    int lo, hi, bt, l;
    if constexpr (is_wgrad(MODE)) {
        bt = (p.N + BT - 1) / BT;
        c.g = __builtin_amdgcn_readfirstlane(item / (at * bt));
        l = item - c.g * (at * bt);
    } else {
        int glo = 0, ghi = p.G;                              // largest g with pass_off[g] * at <= item
        while (ghi - glo > 1) {
            const int mid = (glo + ghi) >> 1;
            if (pass_off[mid] * at <= item) glo = mid; else ghi = mid;
        }
        c.g = __builtin_amdgcn_readfirstlane(glo);
        const int first = __builtin_amdgcn_readfirstlane(pass_off[c.g]);
        bt = __builtin_amdgcn_readfirstlane(pass_off[c.g + 1]) - first;
        l = item - first * at;
    }
    // bands of four b tiles, b fastest: the items that run together on one
    // XCD share operands in its L2
    const int band = l / (4 * at), h = min(4, bt - 4 * band), l2 = l - band * 4 * at;
    // (scalar registers: a descriptor built from them must not look divergent)
    const int ai = __builtin_amdgcn_readfirstlane(l2 / h);
    c.a0 = ai * kATile;
    c.b0 = (4 * __builtin_amdgcn_readfirstlane(band) + __builtin_amdgcn_readfirstlane(l2 - ai * h)) * BT;
    group_rows(p, c.g, lo, hi);
    c.r0 = __builtin_amdgcn_readfirstlane(lo);
    c.nrows = __builtin_amdgcn_readfirstlane(hi) - c.r0;
    if constexpr (is_wgrad(MODE)) {
        c.nk = (c.nrows + KT - 1) / KT;
    } else {
        c.r0 += c.b0;
        c.nrows = min(BT, c.nrows - c.b0);
        c.nk = (p.K + KT - 1) / KT;
    }
    return c;
}

// The request side of a workgroup (waves 0-3): the K-tile to request next.
template <int NB>
struct MmReq {
    int item, kt, step;                 // item: the one to open after this
    bool live;
    MmItem c;
    uint32_t row[NB];                   // contiguous form: byte offsets of this lane's rows of the b operand
    uint32_t srow;                      // fp8: byte offset of this lane's row of scales
    int psrc, qsrc;                     // wgrad: source rows of this wave's 16 k, one per lane % 16
};

// wgrad: sources of the K-tile about to be requested
template <int MODE, int NB>
MOE_DEV void mm_open_src(const MmP& p, const MmWhere& wh, MmReq<NB>& R) {
    if constexpr (is_wgrad(MODE)) {
        const int k = R.kt * 64 + 16 * wh.w + (wh.lane & 15);    // rows past the group: 0, never used
        if constexpr (MODE == kWgrad)
            R.psrc = __builtin_amdgcn_raw_buffer_load_b32(
                make_rsrc(p.x_src + R.c.r0, p.x_src ? (uint32_t)(R.c.nrows * 4) : 0u), k * 4, 0, 0);
        R.qsrc = __builtin_amdgcn_raw_buffer_load_b32(
            make_rsrc(p.dy_src + R.c.r0, p.dy_src ? (uint32_t)(R.c.nrows * 4) : 0u), k * 4, 0, 0);
    }
}

// the next item with K-tiles, or none
template <int EL, int MODE, int NB>
MOE_DEV void mm_open_item(const MmP& p, const int* pass_off, const MmWhere& wh, MmReq<NB>& R) {
    constexpr int BT = 32 * NB;
    int item = R.item;
    bool live = false;
    while (item < wh.n_items && !live) {
        R.c = mm_decode<EL, MODE, NB>(p, pass_off, wh.at, item);
        live = R.c.nk > 0;
        item += wh.grid;
    }
    R.item = item;
    R.live = live;
    if (!live) return;
    R.c = mm_scalar(R.c);
    if constexpr (!is_wgrad(MODE)) {
        // source rows without a branch: past the item (and without a source
        // array, whose resource is then empty) the loads return 0
        const rsrc_t rm = make_rsrc(p.x_src + R.c.r0, p.x_src ? (uint32_t)(R.c.nrows * 4) : 0u);
        #pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int row = (BT / 4) * wh.w + 8 * i + (wh.lane >> 3);
            const uint32_t s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, row * 4, 0, 0);
            R.row[i] = row < R.c.nrows && s < p.x_rows ? (p.x_src ? s : (uint32_t)row) * p.x_ld : kMmNoRow;
        }
        if constexpr (EL == kElFp8) {
            const int row = (BT / 4) * wh.w + wh.lane;
            const uint32_t s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, row * 4, 0, 0);
            R.srow = wh.lane < BT / 4 && row < R.c.nrows && s < p.x_rows ? (p.x_src ? s : (uint32_t)row) * (uint32_t)(p.kb * 4)
                                                                          : kMmNoRow;
        }
    }
}

// The lane number as a value the compiler cannot relate to the last K-tile's:
// offsets formed from it are recomputed (one or two instructions each) instead
// of being kept in registers across the products.
MOE_DEV int mm_fresh(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

// Slow form: K-tile rows [16 w, 16 w + 16) of an operand into dst. With a map
// the row of k is src (one per lane % 16) from the array's start, else row
// first + k. krem: rows left; columns [c0, c0 + 256) of ncols.
MOE_DEV void mm_stage_slow(uint8_t* dst, const uint8_t* base, uint32_t ld, uint32_t bytes, uint32_t rows, bool mapped,
                           int src, int first, int krem, int c0, int ncols, int w, int lane) {
    if (!mapped) {
        base += (size_t)first * ld + (size_t)c0 * 2;
        bytes = (uint32_t)(min(krem, 64) - 1) * ld + (uint32_t)(min(ncols - c0, 256) * 2);
    }
    const rsrc_t r = make_rsrc(base, bytes);
    lane = mm_fresh(lane);
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = 16 * w + 2 * i + (lane >> 5);
        const int col = (((lane & 31) >> 1) ^ tr_swz(k)) * 16 + (lane & 1) * 8;
        bool ok = k < krem && c0 + col < ncols;
        uint32_t o = (uint32_t)k * ld + (uint32_t)(col * 2);
        if (mapped) {
            const int s0 = __builtin_amdgcn_readlane(src, 2 * i), s1 = __builtin_amdgcn_readlane(src, 2 * i + 1);
            const int s = lane < 32 ? s0 : s1;
            ok = ok && (uint32_t)s < rows;
            o = (uint32_t)s * ld + (uint32_t)((c0 + col) * 2);
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void_t*)(dst + (16 * w + 2 * i) * 512), 16,
                                                 ok ? o : kMmInvalid, 0, 0, 0);
    }
}

// request one K-tile into its stage, then move on
template <int EL, int MODE, int NB>
MOE_DEV void mm_request(const MmP& p, const int* pass_off, const MmWhere& wh, MmReq<NB>& R, uint8_t* smem) {
    using Geo = MmGeom<EL, NB>;
    constexpr int EB = EL == kElFp8 ? 1 : 2, BT = 32 * NB;
    const int lane = mm_fresh(wh.lane), w = wh.w;
    const MmItem& c = R.c;
    uint8_t* st = smem + (R.step % Geo::NST) * Geo::Stage;
    const int kbyte = R.kt * 128;
    if constexpr (MODE == kMmNK) {
        const int rows = min(kATile, p.N - c.a0);
        const rsrc_t rw = make_rsrc(p.w + (size_t)c.g * p.w_group + (size_t)c.a0 * p.w_ld, (uint32_t)rows * p.w_ld);
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the swizzle of row 64 w + 8 i + lane / 8 depends on i's parity alone
            const int kb = kbyte + 16 * ((lane & 7) ^ ((lane >> 4) | (4 * (i & 1))));
            const uint32_t o = (uint32_t)(64 * w + (lane >> 3)) * p.w_ld + (uint32_t)kb;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw, (mm_lds_void_t*)(st + (64 * w + 8 * i) * 128), 16,
                kb < p.K * EB ? o + (uint32_t)(8 * i) * p.w_ld : kMmInvalid, 0, 0, 0);
        }
    } else if constexpr (MODE == kMmKN) {
        mm_stage_slow(st, p.w + (size_t)c.g * p.w_group, p.w_ld, 0, 0, false, 0, R.kt * 64, p.K - R.kt * 64, c.a0, p.N,
                      w, lane);
    } else {
        if constexpr (MODE == kWgrad)
            mm_stage_slow(st, p.x, p.x_ld, p.x_bytes, p.x_rows, p.x_src != nullptr, R.psrc, c.r0 + R.kt * 64, c.nrows - R.kt * 64,
                          c.a0, p.K, w, lane);
        mm_stage_slow(st + Geo::QOff, p.dy, p.dy_ld, p.dy_bytes, p.dy_rows, p.dy_src != nullptr, R.qsrc, c.r0 + R.kt * 64,
                      c.nrows - R.kt * 64, c.b0, p.N, w, lane);
    }
    if constexpr (!is_wgrad(MODE)) {
        // gathered rows are addressed from the array's start, a group's own rows from the tile's first
        const rsrc_t rx = make_rsrc(p.x_src ? p.x : p.x + (size_t)c.r0 * p.x_ld,
                                    p.x_src ? p.x_bytes : (uint32_t)(c.nrows - 1) * p.x_ld + (uint32_t)(p.K * EB));
        #pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int row = (BT / 4) * w + 8 * i + (lane >> 3);
            const int kb = kbyte + 16 * ((lane & 7) ^ kc_swz(row));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rx, (mm_lds_void_t*)(st + Geo::QOff + ((BT / 4) * w + 8 * i) * 128), 16,
                kb < p.K * EB ? R.row[i] + (uint32_t)kb : kMmInvalid, 0, 0, 0);
        }
        if constexpr (EL == kElFp8) {
            const rsrc_t rs = make_rsrc(p.x_src ? p.xs : p.xs + (size_t)c.r0 * p.kb,
                                        p.x_src ? p.xs_bytes : (uint32_t)(c.nrows * p.kb * 4));
            if (lane < BT / 4)          // only these lanes' 4 bytes are written
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rs, (mm_lds_void_t*)(st + Geo::SOff + (BT / 4) * w * 4), 4,
                    R.srow + (uint32_t)(R.kt * 4), 0, 0, 0);
        }
    }
    ++R.step;
    const int kt = R.kt + 1;
    const bool last = kt == c.nk;
    R.kt = last ? 0 : kt;
    if (last) mm_open_item<EL, MODE, NB>(p, pass_off, wh, R);
    if (R.live) mm_open_src<MODE>(p, wh, R);
}

// wgrad from 8-bit rows: the a operand passes through registers. Every wave
// takes 8 of a K-tile's 64 rows: lane l of piece i holds 8 codes of row
// 8 w + 2 i + l / 32. Codes are requested two K-tiles ahead and written to LDS
// as BF16 values (code * scale, rounded) one K-tile ahead.
struct MmKept {
    int item, kt, step;                 // step: of the K-tile held in q
    bool live, held;
    MmItem c;
    int src;                            // source rows of this wave's 8 k, one per lane % 8
    u32x2_t q[4];
    float s[4];
};

template <int NB>
MOE_DEV void kept_open(const MmP& p, const MmWhere& wh, MmKept& X) {
    int item = X.item;
    bool live = false;
    while (item < wh.n_items && !live) {
        X.c = mm_decode<kElBf16, kWgrad8, NB>(p, nullptr, wh.at, item);
        live = X.c.nk > 0;
        item += wh.grid;
    }
    X.item = item;
    X.live = live;
    X.c = mm_scalar(X.c);
}
MOE_DEV void kept_src(const MmP& p, const MmWhere& wh, MmKept& X) {
    const int k = X.kt * 64 + 8 * wh.w + (wh.lane & 7);
    X.src = __builtin_amdgcn_raw_buffer_load_b32(
        make_rsrc(p.x_src + X.c.r0, p.x_src ? (uint32_t)(X.c.nrows * 4) : 0u), k * 4, 0, 0);
}
template <int NB>
MOE_DEV void kept_load(const MmP& p, const MmWhere& wh, MmKept& X) {
    const int k0 = X.kt * 64, krem = X.c.nrows - k0, first = X.c.r0 + k0, rows = min(krem, 64);
    const bool mapped = p.x_src != nullptr;
    const rsrc_t rx = make_rsrc(mapped ? p.x : p.x + (size_t)first * p.x_ld,
                                mapped ? p.x_bytes : (uint32_t)(rows - 1) * p.x_ld + (uint32_t)p.K);
    const rsrc_t rs = make_rsrc(mapped ? p.xs : p.xs + (size_t)first * p.kb,
                                mapped ? p.xs_bytes : (uint32_t)(rows * p.kb * 4));
    const int col = X.c.a0 + (wh.lane & 31) * 8;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = 8 * wh.w + 2 * i + (wh.lane >> 5);
        int row = k;
        if (mapped) {
            const int s0 = __builtin_amdgcn_readlane(X.src, 2 * i), s1 = __builtin_amdgcn_readlane(X.src, 2 * i + 1);
            row = wh.lane < 32 ? s0 : s1;
        }
        const bool ok = k < krem && col < p.K && (!mapped || (uint32_t)row < p.x_rows);
        X.q[i] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
            rx, ok ? (uint32_t)row * p.x_ld + (uint32_t)col : kMmInvalid, 0, 0));
        X.s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rs, ok ? ((uint32_t)row * (uint32_t)p.kb + (uint32_t)(col >> 7)) * 4u : kMmInvalid, 0, 0));
    }
    X.held = true;
    const int kt = X.kt + 1;
    const bool last = kt == X.c.nk;
    X.kt = last ? 0 : kt;
    if (last) kept_open<NB>(p, wh, X);
    if (X.live) kept_src(p, wh, X);
}
MOE_DEV void kept_write(const MmWhere& wh, MmKept& X, uint8_t* st) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = 8 * wh.w + 2 * i + (wh.lane >> 5), c = wh.lane & 31;
        const uint32_t w[2] = {X.q[i].x, X.q[i].y};
        i32x4 o;
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
            const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
            o[2 * h] = (int)bf16x2(a[0] * X.s[i], a[1] * X.s[i]);
            o[2 * h + 1] = (int)bf16x2(b[0] * X.s[i], b[1] * X.s[i]);
        }
        *(i32x4*)(st + k * 512 + (((c >> 1) ^ tr_swz(k)) * 32) + (c & 1) * 16) = o;
    }
    X.held = false;
    ++X.step;
}

template <int EL, int MODE, int NB>
__global__ __launch_bounds__(kMmThreads, 1)
void grouped_mm_kernel(MmP p) {
    using Geo = MmGeom<EL, NB>;
    constexpr int BT = Geo::BT, NST = Geo::NST;
    constexpr bool P_TR = MODE != kMmNK, Q_TR = is_wgrad(MODE);
    static_assert(!Q_TR || BT == 256, "the slow form is laid out for 256 values");

    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* pass_off = (int*)(smem + NST * Geo::Stage);         // mm: [G + 1] passes before group g

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    const int wi = w & 3, ti = w >> 2;
    const bool lead = w < 4;                                 // waves 0-3 issue the requests

    const int na = is_wgrad(MODE) ? p.K : p.N;               // extent of the contiguous output axis
    const int at = (na + kATile - 1) / kATile;
    int n_items;
    if constexpr (is_wgrad(MODE)) {
        n_items = p.G * at * ((p.N + BT - 1) / BT);
    } else {
        if (w == 0) {
            int run = 0;
            for (int g0 = 0; g0 < p.G; g0 += 64) {
                int lo = 0, hi = 0;
                if (g0 + lane < p.G) group_rows(p, g0 + lane, lo, hi);
                const int n = (hi - lo + BT - 1) / BT;
                const int inc = wave_incl_scan(n);
                if (g0 + lane < p.G) pass_off[g0 + lane] = run + inc - n;
                run += __builtin_amdgcn_readlane(inc, 63);
            }
            if (lane == 0) pass_off[p.G] = run;
        }
        __syncthreads();
        n_items = __builtin_amdgcn_readfirstlane(pass_off[p.G]) * at;
    }
    const int grid = gridDim.x;
    const int slot = (grid % 8 == 0) ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
    if (slot >= n_items) return;

    const MmWhere wh{n_items, at, grid, lane, w};
    MmReq<NB> rq;                                            // waves 0-3
    rq.item = slot;

    // ---------------------------------------------------------- fragments
    // 16-bit: half h of a step is the K-tile's k-half; FP8 (whose instruction
    // takes the whole K-tile): half h is the wave's b tiles [h NB/2, (h+1) NB/2)
    constexpr int NS = EL == kElFp8 ? 2 : 1;                 // 16-byte pieces per fragment
    constexpr int NU = EL == kElFp8 && NB > 1 ? NB / 2 : NB; // b tiles per half
    constexpr int HALVES = EL == kElFp8 && NB == 1 ? 1 : 2;
    i32x4 fp[NS][4], fq[NS][NU];
    float fs[NU], fw = 0.f;
    auto read_slow = [&](const uint8_t* st, int s, int c) __attribute__((always_inline)) {
        i32x4 v;
        const int o = (32 * s + 8 * q + (j >> 2)) * 512 + ((c ^ ((j >> 2) | (q << 2))) * 32) + (j & 3) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_s16x4*)(st + o));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_s16x4*)(st + o + 4 * 512));
        const u32x2_t l = __builtin_bit_cast(u32x2_t, lo), h = __builtin_bit_cast(u32x2_t, hi);
        v[0] = (int)l.x; v[1] = (int)l.y; v[2] = (int)h.x; v[3] = (int)h.y;
        return v;
    };
    auto read_frags = [&](int step, int h, const MmItem& c, int kt) __attribute__((always_inline)) {
        const uint8_t* st = smem + (step % NST) * Geo::Stage;
        #pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int ks = EL == kElFp8 ? s : h;
            const int ch = ((4 * ks + q) ^ ((j >> 1) & 7)) * 16;
            if (EL != kElFp8 || h == 0) {
                #pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (P_TR) fp[s][t] = read_slow(st, ks, 4 * wi + t);
                    else fp[s][t] = *(const i32x4*)(st + (64 * wi + 16 * t + j) * 128 + ch);
                }
            }
            #pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int uu = EL == kElFp8 ? h * NU + u : u;
                if constexpr (Q_TR) fq[s][u] = read_slow(st + Geo::QOff, ks, NB * ti + uu);
                else fq[s][u] = *(const i32x4*)(st + Geo::QOff + (16 * NB * ti + 16 * uu + j) * 128 + ch);
            }
        }
        if constexpr (EL == kElFp8) {
            #pragma unroll
            for (int u = 0; u < NU; ++u)
                fs[u] = *(const float*)(st + Geo::SOff + (16 * NB * ti + 16 * (h * NU + u) + j) * 4);
            if (h == 0) fw = p.ws[((size_t)c.g * p.nb + min((c.a0 + 64 * wi) >> 7, p.nb - 1)) * p.kb + kt];
        }
    };

    f32x4 acc[NB][4];
    auto multiply = [&](auto half) __attribute__((always_inline)) {
        constexpr int h = decltype(half)::value;
        if constexpr (EL == kElFp8) {
            // the K-tile is one block of 128: its products go to cleared
            // registers and are added with the two scales' product, one b tile
            // behind: 4 additions in the shadow of each matrix instruction. The
            // empty asm statements order the two (b tile u's products before
            // and b tile u - 1's additions before u's); left alone the compiler
            // starts every product first and spills the accumulators.
            f32x4 d[2][4];
            float sc = 0.f;
            #pragma unroll
            for (int u = 0; u <= NU; ++u) {
                if (u < NU)
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        d[u & 1][t] = mfma_fp8(fp[0][t], fp[1][t], fq[0][u], fq[1][u], f32x4{0.f, 0.f, 0.f, 0.f});
                if (u > 0) {
                    f32x4* a = acc[h * NU + u - 1];
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        #pragma unroll
                        for (int v = 0; v < 4; ++v) a[t][v] = fmaf(d[(u - 1) & 1][t][v], sc, a[t][v]);
                    if (u < NU) {
                        #pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                        }
                    }
                    asm volatile("" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
                }
                if (u < NU) {
                    sc = fs[u] * fw;
                    const f32x4* e = d[u & 1];
                    asm volatile("" : "+v"(sc) : "v"(e[0]), "v"(e[1]), "v"(e[2]), "v"(e[3]));
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            #pragma unroll
            for (int u = 0; u < NB; ++u)
                #pragma unroll
                for (int t = 0; t < 4; ++t) acc[u][t] = mfma16x16x32<EL>(fp[0][t], fq[0][u], acc[u][t]);
        }
    };

    auto clear = [&]() __attribute__((always_inline)) {
        #pragma unroll
        for (int u = 0; u < NB; ++u)
            #pragma unroll
            for (int t = 0; t < 4; ++t) acc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    // sums stay in 32 bits until here: the one rounding to the output's type
    auto store = [&](const MmItem& c, auto f16_) __attribute__((always_inline)) {
        constexpr int f16 = decltype(f16_)::value;
        #pragma unroll
        for (int u = 0; u < NB; ++u) {
            const int b = 16 * NB * ti + 16 * u + j;
            #pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int a = c.a0 + 64 * wi + 16 * t + 4 * q;
                f32x4 v = acc[u][t];
                if constexpr (is_wgrad(MODE)) {
                    if (c.b0 + b < p.N && a < p.K) {
                        const size_t o = ((size_t)c.g * p.N + c.b0 + b) * p.K + a;
                        if (p.out_f32) {
                            f32x4* d = (f32x4*)((float*)p.out + o);
                            if (p.accumulate) { const f32x4 e = *d; v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]}; }
                            *d = v;
                        } else {
                            u32x2_t* d = (u32x2_t*)((uint16_t*)p.out + o);
                            if (p.accumulate) {
                                const u32x2_t e = *d;
                                v[0] += lo16(e.x, f16); v[1] += hi16(e.x, f16);
                                v[2] += lo16(e.y, f16); v[3] += hi16(e.y, f16);
                            }
                            *d = u32x2_t{pack16(v[0], v[1], f16), pack16(v[2], v[3], f16)};
                        }
                    }
                } else {
                    if (b < c.nrows && a < p.N)
                        *(u32x2_t*)((uint16_t*)p.out + (size_t)(c.r0 + b) * p.out_ld + a) =
                            u32x2_t{pack16(v[0], v[1], f16), pack16(v[2], v[3], f16)};
                }
            }
        }
    };

    // --------------------------------------------------------------- loop
    MmKept kept;
    if constexpr (MODE == kWgrad8) {
        kept.item = slot;
        kept.step = kept.kt = 0;
        kept.held = false;
        kept_open<NB>(p, wh, kept);
        if (kept.live) kept_src(p, wh, kept);
        if (kept.live) kept_load<NB>(p, wh, kept);
        if (kept.held) kept_write(wh, kept, smem);
        if (kept.live) kept_load<NB>(p, wh, kept);
    }
    if (lead) {
        rq.step = rq.kt = 0;
        mm_open_item<EL, MODE, NB>(p, pass_off, wh, rq);
        if (rq.live) mm_open_src<MODE>(p, wh, rq);
        #pragma unroll 1
        for (int i = 0; i < NST - 1; ++i)
            if (rq.live) mm_request<EL, MODE, NB>(p, pass_off, wh, rq, smem);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    bare_barrier();
    if (!lead) bare_barrier();
    int step = 0;
    for (int item = slot; item < n_items; item += grid) {
        const MmItem c = mm_decode<EL, MODE, NB>(p, pass_off, at, item);
        clear();
        #pragma unroll 1
        for (int kt = 0; kt < c.nk; ++kt, ++step) {
            if constexpr (MODE == kWgrad8) {
                if (kept.held) kept_write(wh, kept, smem + (kept.step % NST) * Geo::Stage);
                if (kept.live) kept_load<NB>(p, wh, kept);
            }
            if (lead && rq.live) mm_request<EL, MODE, NB>(p, pass_off, wh, rq, smem);
            static_for<HALVES>([&](auto half) __attribute__((always_inline)) {
                read_frags(step, decltype(half)::value, c, kt);
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
                bare_barrier();
                __builtin_amdgcn_s_setprio(1);
                multiply(half);
                __builtin_amdgcn_s_setprio(0);
                if (lead && decltype(half)::value == HALVES - 1) {      // the next step's K-tile has landed
                    if (rq.live) __builtin_amdgcn_s_waitcnt(waitcnt_imm(Geo::Loads * (NST - 2), 15));
                    else __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
                }
                bare_barrier();
            });
        }
        if (!is_wgrad(MODE) || c.nk > 0 || !p.accumulate) {
            if constexpr (EL == kElFp8) {
                if (p.out_f16) store(c, std::integral_constant<int, 1>{});
                else store(c, std::integral_constant<int, 0>{});
            } else {
                store(c, std::integral_constant<int, EL == kElF16>{});
            }
        }
    }
    if (lead) bare_barrier();
}

template <int EL, int MODE, int NB>
int launch_mm(const MmP& p, int max_items, hipStream_t stream) {
    using Geo = MmGeom<EL, NB>;
    const size_t lds = Geo::Lds(is_wgrad(MODE) ? 0 : p.G);
    auto* k = &grouped_mm_kernel<EL, MODE, NB>;
    static bool ready[64] = {false};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return (int)e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
        if (e != hipSuccess) return (int)e;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    const int grid = std::max(1, std::min(max_items, device_cu_count()));
    k<<<grid, kMmThreads, lds, stream>>>(p);
    return (int)hipGetLastError();
}

// launchers
template <int EL, int MODE>
int launch_mm_rows(const MmP& p, hipStream_t stream) {
    const int at = (p.N + kATile - 1) / kATile;
    auto items = [&](int bt) {
        return (int)std::min<int64_t>(((int64_t)p.R_max / bt + std::min(p.G, p.R_max)) * at, 1 << 30);
    };
    const int rows = (p.R_max + p.G - 1) / p.G;              // expected rows of a group
    if (rows > 128) return launch_mm<EL, MODE, 8>(p, items(256), stream);
    if (rows > 64) return launch_mm<EL, MODE, 4>(p, items(128), stream);
    if (rows > 32) return launch_mm<EL, MODE, 2>(p, items(64), stream);
    return launch_mm<EL, MODE, 1>(p, items(32), stream);
}

}  // namespace

size_t moe_mm_workspace_bytes(int kind, bool fp8, int R_max, int G, int N, int K) {
    (void)kind; (void)fp8; (void)R_max; (void)G; (void)N; (void)K;
    return 0;
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
        if (c.xs) return launch_mm<kElBf16, kWgrad8, 8>(p, items, stream);
        return f16 ? launch_mm<kElF16, kWgrad, 8>(p, items, stream) : launch_mm<kElBf16, kWgrad, 8>(p, items, stream);
    }
    p.w = (const uint8_t*)c.w;
    p.w_group = (size_t)c.N * c.K * eb;
    p.w_ld = (uint32_t)((c.kind == 1 ? c.N : c.K) * eb);
    if (c.fp8) {
        p.kb = (c.K + 127) / 128; p.nb = (c.N + 127) / 128;
        p.xs = c.xs; p.ws = c.wscale;
        if (c.x_src) p.xs_bytes = (uint32_t)((int64_t)c.x_rows * p.kb * 4);
        return launch_mm_rows<kElFp8, kMmNK>(p, stream);
    }
    if (c.kind == 0) return f16 ? launch_mm_rows<kElF16, kMmNK>(p, stream) : launch_mm_rows<kElBf16, kMmNK>(p, stream);
    return f16 ? launch_mm_rows<kElF16, kMmKN>(p, stream) : launch_mm_rows<kElBf16, kMmKN>(p, stream);
}

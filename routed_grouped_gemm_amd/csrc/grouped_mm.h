// Pieces shared by the grouped-product kernels (grouped_mm_tiled.h, the LDS-tiled
// kernel, and grouped_mm_rows.h, the weight-streaming kernel for few rows):
// element kinds, the parameter block and MFMA wrappers. Internal to libmoe.
#pragma once
#include "gemm_common.h"

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void mm_lds_void_t;
typedef __attribute__((address_space(3))) s16x4 mm_lds_s16x4;

enum { kElBf16 = 0, kElF16 = 1, kElFp8 = 2 };           // operand element kinds

// Byte offset that no bounded resource contains (their sizes stay below it).
constexpr uint32_t kMmInvalid = 0xFFFFFFF0u;
// Row offset past every gathered array (they stay below it, see the size
// checks) that remains one after adding an offset inside a row (< 2^22).
constexpr uint32_t kMmNoRow = 0xFFC00000u;

// One grouped product. mm: x rows times weights; wgrad: dy^T x per group.
struct MmP {
    const uint8_t* w; size_t w_group; uint32_t w_ld;     // weights: bytes per group, per row
    const uint8_t* x; uint32_t x_ld, x_bytes, x_rows;    // x rows: bytes per row; bytes and rows of the array (bounds)
    const int32_t* x_src;                                // null: row r of a group is row r of x
    const uint8_t* dy; uint32_t dy_ld, dy_bytes, dy_rows;   // wgrad
    const int32_t* dy_src;
    const int32_t* offsets;
    int G, N, K, R_max;
    uint8_t* out; size_t out_ld;                         // mm: elements per row
    int out_f16, out_f32, accumulate;
    const float* xs; uint32_t xs_bytes;                  // fp8: row scales [x_rows, kb]
    const float* ws;                                     // fp8: weight scales [G, nb, kb]
    int kb, nb;
    // work split along the reduction axis: K-tiles per part, parts (rows
    // kernel), and the fp32 partial sums (null: no splitting)
    int part, parts, max_slots;
    float* partial;
    // the epilogues (grouped_mm_act.h): activation, bias f32 [G, weight rows],
    // row weights, residual rows [R, N], pre-activation rows (written by the
    // forward epilogues, read by the backward one, whose h and dpre are dense)
    int act; float beta, limit;
    const float* bias; const float* row_w;
    const uint8_t* res; size_t res_ld;                       // elements per row
    uint8_t* pre; size_t pre_ld;
    uint8_t* h;
    float* dw_part; float* dw;                               // partial row sums [16- or 64-column parts][R_max]
    int gated;
    // the part of the output that a launch computes: `at` tiles of columns from
    // col0; of a single group all rows (row_part 0), those of whole passes of
    // row_tile rows (1) or the rest (2)
    int col0, at, row_part, row_tile, dw_slot0;
    size_t part_ld, part_rows;                               // its partial sums: values of a row, rows of a part
};

// Rows [lo, hi) of group g, held inside [0, R_max) whatever the offsets say.
MOE_DEV void group_rows(const MmP& p, int g, int& lo, int& hi) {
    lo = min(max(p.offsets[g], 0), p.R_max);
    hi = min(max(p.offsets[g + 1], lo), p.R_max);
}
// The rows of it that a launch of a product with an epilogue computes.
template <bool EPI>
MOE_DEV void part_rows(const MmP& p, int& lo, int& hi) {
    if constexpr (EPI) {
        const int rest = p.row_part ? (hi - lo) % p.row_tile : 0;
        if (p.row_part == 1) hi -= rest;
        if (p.row_part == 2) lo = hi - rest;
    }
}

// The row that is the first of a part's partial sums.
MOE_DEV int first_part_row(const MmP& p) {
    int lo = 0, hi;
    if (p.row_part != 2) return 0;
    group_rows(p, 0, lo, hi);
    part_rows<true>(p, lo, hi);
    return __builtin_amdgcn_readfirstlane(lo);
}

// The rows of one group for the whole wave, by scalar loads: waiting for a
// vector load would drain the requests in flight at every item.
MOE_DEV void group_rows_scalar(const MmP& p, int g, int& lo, int& hi) {
    typedef const __attribute__((address_space(4))) int32_t* const_i32;
    const const_i32 at = (const_i32)(uintptr_t)p.offsets + __builtin_amdgcn_readfirstlane(g);
    lo = min(max(at[0], 0), p.R_max);
    hi = min(max(at[1], lo), p.R_max);
}

// two floats -> two packed 16-bit values, round to nearest even
MOE_DEV uint32_t pack16(float a, float b, int f16) {
    if (f16) {
        const f16x2 v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    return bf16x2(a, b);
}
MOE_DEV float lo16(uint32_t v, int f16) {
    return f16 ? (float)__builtin_bit_cast(f16x2, v)[0] : bf16_to_f32(v & 0xFFFFu);
}
MOE_DEV float hi16(uint32_t v, int f16) {
    return f16 ? (float)__builtin_bit_cast(f16x2, v)[1] : bf16_to_f32(v >> 16);
}

// 16x16x32 product of 16-bit operands: lane l holds 8 values of row (A) /
// column (B) l % 16 at k = 8 (l / 16) .. + 7; result as the scaled form's,
// D[4 (l / 16) + v][l % 16].
template <int EL>
MOE_DEV f32x4 mfma16x16x32(const i32x4& a, const i32x4& b, f32x4 c) {
    if constexpr (EL == kElBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// 16x16x128 product of E4M3 operands without block scales (the two 16-byte
// halves of a lane's operand, see mfma16x16x128). The instruction does not sum
// its 128 products as an fp32 chain would: in a piece of them they are aligned
// to the largest, and one below about 2^-15 of it is dropped (the 32-deep FP8
// instruction, at half the rate, drops the same, so nothing is gained by it).
// Measured error beside the output's rounding, of the sum of |products|: 1e-5
// for Gaussian codes, 1.2e-4 for codes spread over the whole range of E4M3 (K =
// 128; 4e-5 at 1024). The sums over blocks are fp32.
MOE_DEV f32x4 mfma_fp8(const i32x4& alo, const i32x4& ahi, const i32x4& blo, const i32x4& bhi, f32x4 c) {
    const i32x8 a = __builtin_shufflevector(alo, ahi, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 b = __builtin_shufflevector(blo, bhi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, MFMA_FMT_FP8, MFMA_FMT_FP8, 0, 0, 0, 0);
}

// The transposing LDS load. Its argument is marked as sharing no memory with
// the loads that write LDS: the compiler would otherwise wait for all of them
// (vmcnt 0) before every one; the kernels order the two by their own waits and
// barriers.
MOE_DEV u32x2_t read_tr16(const mm_lds_s16x4* __restrict__ at) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<mm_lds_s16x4*>(at)));
}

// s_waitcnt immediate: vmcnt <= vm, lgkmcnt <= lgkm (15: no wait)
constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

// Workgroup barrier that neither drains outstanding memory requests nor lets
// the compiler move code across it.
MOE_DEV void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

enum { kMmNK = 0, kMmKN = 1, kWgrad = 2, kWgrad8 = 3 };     // kWgrad8: x rows in E4M3 with block scales
// wgrad modes also say at compile time which operand's rows are gathered (the
// offsets of gathered rows are formed for every K-tile, others once an item)
constexpr int kGatherX = 16, kGatherDy = 32;
constexpr int mm_kind(int mode) { return mode & 15; }
constexpr bool is_wgrad(int mode) { return mm_kind(mode) >= kWgrad; }

// Epilogue of a product: none; bias, activation, row weight and residual of a
// plain or a gated (W: gate rows, then up rows) product; the activation's
// gradient from the pre-activation (the product being that of its outputs').
enum { kEpiNone = 0, kEpiAct = 1, kEpiGated = 2, kEpiGrad = 3 };

constexpr int kMmThreads = 512;
constexpr int kMmLds = 163840;              // LDS of a compute unit
constexpr int kATile = 256;
constexpr int kPBytes = kATile * 128;       // one K-tile of the a operand
constexpr int kMmOut = 8 * 1024;            // stores pass through it
// output columns of a tile of the a operand (gated: 128 gate and 128 up rows)
constexpr int a_tile(int epi) { return epi == kEpiGated ? kATile / 2 : kATile; }

// chunk swizzle of a row in the contiguous form, and of a k in the slow form
MOE_DEV int kc_swz(int row) { return (row >> 1) & 7; }
MOE_DEV int tr_swz(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }
MOE_DEV int tr_swz_half(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

// rows [r0, r0 + nrows), nk K-tiles; slot: place of its partial sums, -1: the output itself
struct MmItem { int g, a0, b0, r0, nrows, nk, slot; };

// the item's fields as scalars again (control flow that merely looks divergent
// would otherwise turn every descriptor load into a loop over lanes)
MOE_DEV MmItem mm_scalar(const MmItem& c) {
    return MmItem{__builtin_amdgcn_readfirstlane(c.g), __builtin_amdgcn_readfirstlane(c.a0),
                  __builtin_amdgcn_readfirstlane(c.b0), __builtin_amdgcn_readfirstlane(c.r0),
                  __builtin_amdgcn_readfirstlane(c.nrows), __builtin_amdgcn_readfirstlane(c.nk),
                  __builtin_amdgcn_readfirstlane(c.slot)};
}

// pass_off[g] = passes of `bt` rows before group g, pass_off[G] their number,
// in LDS; one wave writes them (a barrier must follow). per: items of a pass.
// Rows are below 2^29 and a pass is 32 or more, so 64 groups' passes fit 32
// bits; the items of all do wherever y is an array that exists, but groups that
// overlap (offsets that do not ascend) can have more: then there are none.
template <bool EPI = false>
MOE_DEV void mm_passes(const MmP& p, int bt, int per, int lane, int* pass_off) {
    int64_t run = 0;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
        int lo = 0, hi = 0;
        if (g0 + lane < p.G) group_rows(p, g0 + lane, lo, hi);
        part_rows<EPI>(p, lo, hi);
        const int n = (hi - lo + bt - 1) / bt;
        const int inc = wave_incl_scan(n);
        if (g0 + lane < p.G) pass_off[g0 + lane] = (int)run + inc - n;
        run += __builtin_amdgcn_readlane(inc, 63);
    }
    if (lane == 0) pass_off[p.G] = (int)run;
    if (run * per > (1 << 30))
        for (int g = lane; g <= p.G; g += 64) pass_off[g] = 0;
}

// Where a workgroup is: its items and this lane. dealt: how wgrad's items are
// dealt out (mm_nth).
struct MmWhere { int n_items, at, grid, slot, lane, w, dealt; };

// largest index i in [0, n) with at[i] <= v (at[0] <= v, non-decreasing): 64
// entries at a time
MOE_DEV int last_at_most(const int* at, int n, int v) {
    int c = 0;
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + (int)(threadIdx.x & 63);
        const int here = __builtin_popcountll(__ballot(i < n && at[i] <= v));
        c += here;
        if (here < 64) break;
    }
    return __builtin_amdgcn_readfirstlane(c) - 1;
}

// Tables of a launch in LDS. mm: at [G + 1] passes of rows before group g.
// wgrad: groups in the order of their items, at [G + 1] units (parts of a
// group's K-tiles) before the i-th, order [G] the i-th group; slots [G] the
// first partial-sum slot of group g's tiles (-1: not split).
struct MmTables { const int* at; const uint16_t* order; const int* slots; };

// parts that group g's nk K-tiles are split into
MOE_DEV int wgrad_parts(const MmP& p, int nk) { return p.part > 0 ? max(1, (nk + p.part - 1) / p.part) : 1; }
MOE_DEV int group_ktiles(const MmP& p, int g) {
    int lo, hi;
    group_rows(p, g, lo, hi);
    return (hi - lo + 63) / 64;
}
// Number of the item that a workgroup takes in its round. wgrad's items come
// longest first and are dealt out backwards in some rounds: dealt 0, every
// other whole round; dealt 1, every round but the first.
MOE_DEV int wgrad_nth(int round, int n_items, int grid, int slot, int dealt) {
    const bool back = dealt ? round > 0 : (round & 1) && (round + 1) * grid <= n_items;
    return round * grid + (back ? grid - 1 - slot : slot);
}
template <int MODE>
MOE_DEV int mm_nth(int round, const MmWhere& wh) {
    if constexpr (is_wgrad(MODE)) return wgrad_nth(round, wh.n_items, wh.grid, wh.slot, wh.dealt);
    return round * wh.grid + wh.slot;
}

// work item number `item`: tiles of AT values of the a axis (at of them), BT of the b axis
template <int EL, int MODE, int BT, int AT = kATile, bool EPI = false>
MOE_DEV MmItem mm_decode(const MmP& p, const MmTables& tb, int at, int item) {
    constexpr int KT = EL == kElFp8 ? 128 : 64;
    MmItem c;
    int lo, hi, bt, l;
    c.slot = -1;
    if constexpr (is_wgrad(MODE)) {
        bt = (p.N + BT - 1) / BT;
        const int unit = __builtin_amdgcn_readfirstlane(item / (at * bt));
        l = item - unit * (at * bt);
        const int i = last_at_most(tb.at, p.G, unit);
        const int first = __builtin_amdgcn_readfirstlane(tb.at[i]), parts = __builtin_amdgcn_readfirstlane(tb.at[i + 1]) - first;
        const int part = unit - first;
        c.g = __builtin_amdgcn_readfirstlane(tb.order[i]);
        const int slot0 = __builtin_amdgcn_readfirstlane(tb.slots[c.g]);
        group_rows_scalar(p, c.g, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        const int rows = __builtin_amdgcn_readfirstlane(hi) - lo, nk = (rows + KT - 1) / KT;
        // the group's K-tiles in `parts` nearly equal runs
        const int each = __builtin_amdgcn_readfirstlane(nk / parts), more = nk - each * parts;
        const int k0 = part * each + min(part, more);
        c.nk = each + (part < more ? 1 : 0);
        c.r0 = lo + k0 * KT;
        c.nrows = min(rows - k0 * KT, c.nk * KT);
        if (slot0 >= 0) c.slot = slot0 + part * (at * bt) + l;
    } else {
        c.g = last_at_most(tb.at, p.G, item / at);           // (an empty group shares its first pass with the next)
        const int first = __builtin_amdgcn_readfirstlane(tb.at[c.g]);
        bt = __builtin_amdgcn_readfirstlane(tb.at[c.g + 1]) - first;
        l = item - first * at;
        group_rows_scalar(p, c.g, lo, hi);
        part_rows<EPI>(p, lo, hi);
    }
    // bands of four b tiles, b fastest: the items that run together on one
    // XCD share operands in its L2
    const int band = l / (4 * at), h = min(4, bt - 4 * band), l2 = l - band * 4 * at;
    // (scalar registers: a descriptor built from them must not look divergent)
    const int ai = __builtin_amdgcn_readfirstlane(l2 / h);
    c.a0 = ai * AT + (EPI ? p.col0 : 0);
    c.b0 = (4 * __builtin_amdgcn_readfirstlane(band) + __builtin_amdgcn_readfirstlane(l2 - ai * h)) * BT;
    if constexpr (!is_wgrad(MODE)) {
        c.r0 = __builtin_amdgcn_readfirstlane(lo) + c.b0;
        c.nrows = min(BT, __builtin_amdgcn_readfirstlane(hi) - c.r0);
        c.nk = (p.K + KT - 1) / KT;
    }
    return c;
}

// The lane number as a value the compiler cannot relate to the last K-tile's:
// offsets formed from it are recomputed (one or two instructions each) instead
// of being kept in registers across the products.
MOE_DEV int mm_fresh(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

// an upper bound on the work items of a product with tiles of bt rows
inline int mm_items(const MmP& p, int bt, int atile = kATile) {
    const int64_t passes = (int64_t)p.R_max / bt + (p.G < p.R_max ? p.G : p.R_max);
    const int64_t n = passes * ((p.N + atile - 1) / atile);
    return (int)(n < (1 << 30) ? n : (1 << 30));
}

}  // namespace

// Products of few rows per group (grouped_mm_rows.hip); p is an MmP, el its
// element kind, kind 0 for W [N, K] and 1 for W [K, N], rows its tile height.
int moe_launch_mm_rows(const void* p, int el, int kind, int rows, hipStream_t stream);

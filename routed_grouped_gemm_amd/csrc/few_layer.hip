// The routed layer for a few tokens (T <= 32) on 16-bit token rows and weights in
// 16 bits or in E4M3 with a scale per 128 x 128, in two launches:
//
//   few_w1  every workgroup routes and groups the tokens (a few thousand
//           cycles), then  h[r] = a(clamp(g)) clamp(u) w_r  for the rows r of the
//           experts that have tokens, [g | u] = x[src r] W1_g^T + b1_g
//   few_w2  out[t] = residual[t] + sum over t's rows r of (h[r] W2_g^T + w_r b2_g)
//
// Bound by the weights of the active experts, read once. In both kernels a
// workgroup of 16 waves, one on a compute unit, walks over 16 rows of weights at
// a time; the waves split the reduction axis: unit i (128 bytes of each of the 16
// rows) goes to wave i % 16 (few_w1: i % split, 16 / split runs of rows at once,
// so that a wave has some units before each barrier). A wave keeps four units in
// flight (128 KiB in a compute unit), or two or three where more than the weights
// is in registers, and requests whole lines, 8 lanes a row: with
// 4 lanes a row, the layout of the matrix instruction's operand, the same bytes
// took a quarter longer. The operand's layout is made by passing a unit through 2
// KiB of LDS a wave. The other operand, the token rows or h, is in LDS where it
// fits (all tokens, or the rows of a group at a time), else loaded with the
// weights. E4M3 codes become 16-bit values exactly; the scale of a unit's 128
// columns multiplies its fp32 sums.
//
// few_w1's 16 rows are 8 of the gate and the same 8 of the up projection, in
// the order 2 gate, 2 up, so that a lane ends with both halves of its outputs.
// Between the two, h is held in two parts of the operands' type, its value rounded and
// the rest (16 bits of it in BF16, 22 in FP16): rounded once, it was most of the
// outputs' error (2.3e-3 of them in the 2-norm in BF16, 1.6e-3 with two parts, which
// is the outputs' own rounding). few_w2's 16 columns of the 16x16 result are both
// parts of 8 rows of a group, or 16 rows with a product for each part (kCols8,
// kCols16). A unit's sums are added for the tokens that chose its expert (a choice, not a
// product with 0: another token's infinities stay out), so the sum over experts
// stays in fp32 registers and nothing has to be combined afterwards.
//
// Measured (a plain read of memory: 6.9 TB/s): one token on 6 of 64 experts of
// 2048 x 1408 in BF16 (104 MB) 30 us, of which the weights stream for 15 at 7
// TB/s; the rest is the start of two kernels. 16 tokens on 11 of 32 local experts of
// 7168 x 2048 in E4M3 (484 MB) 98 us, on 14 in BF16 (1.2 GB) 198 us, 6.2 TB/s.
// 32 tokens on 20 of them in BF16 (1.8 GB) 279 us, on 15 in E4M3 (661 MB) 144 us,
// 4.6 TB/s: few_w1 with two tiles of token rows and E4M3 weights has more in
// flight than 128 registers hold. 8 tokens on 7 experts of 4096 x 4096 in BF16
// 116 us, 6.1 TB/s. A shared expert costs more than its weights where its rows
// are many: 32 tokens on 23 of those experts, one of them shared, 365 us in BF16,
// 263 us on 22 in E4M3.
#include <algorithm>

#include "epilogue_act.h"
#include "grouped_mm.h"
#include "permute_block.h"

namespace {

constexpr int kFewWaves = 16;
constexpr int kFewThreads = 64 * kFewWaves;

struct FewP {
    const float* logits;
    int T, E, k, e0, E_loc, s, G, renorm;
    const uint8_t* x; uint32_t x_ld, x_bytes;                // bytes
    int H, I;
    uint64_t w1, w1s, w2, w2s, s1, s1s, s2, s2s;             // addresses of weights and scales: routed groups, the shared one
    int act; float beta, limit;
    const float* b1; const float* b2;
    const uint16_t* res; size_t ld_res;
    uint16_t* out; size_t ld_out;
    // workspace
    uint16_t* h;                                             // [R][2][I]: the two parts of a row
    float* row_w;                                            // [R]
    int32_t* active;                                         // groups with rows, rows used, then the groups
    int16_t* map;                                            // few_w2's columns (few_map)
    int split;                                               // few_w1: waves that share 16 weight rows
    int cb8, cb6, cb4, cb2; float per_grid;                  // items of a group with 8, 6, 4, 2 outputs for every `split` waves; 1 / grid
    int blocks, cols;                                        // few_w2: blocks of `cols` (at most 16) columns
};

// Units of a wave in flight (a slot of the ring each), the 16-byte pieces of a
// token row in a unit and its k. XL: token rows are in LDS, otherwise they are
// requested with the weights.
template <bool F8, int NT, bool XL>
struct FewGeom {
    static constexpr int NB = F8 ? 4 : 2;
    static constexpr int UK = F8 ? 128 : 64;
    static constexpr int Ring = XL ? (F8 && NT == 2 ? 3 : 4) : (NT == 1 ? 3 : 2);
};
template <bool F8, int NT, bool XL>
struct FewSlot {
    i32x4 a[2];
    i32x4 b[XL ? 1 : NT][XL ? 1 : FewGeom<F8, NT, XL>::NB];
    uint32_t sc[2];                                          // scales of this lane's results: gate, up
};
// What the 16 columns of few_w2's products are. Eight rows of a group and both parts
// of h: the first parts in columns 0 .. 7, the second in 8 .. 15, so that two parts
// cost the requests, registers and instructions of one. Or, where a group has more
// rows than 8, sixteen rows and a product for each part. The rows are those of the tokens in
// their order (column t: token t) where so many columns hold all tokens, else the
// group's, and the sums go from its columns to the tokens'.
enum { kCols8 = 0, kCols16 = 1 };
constexpr int few_cols_of(int form) { return form == kCols8 ? 8 : 16; }

// A slot of few_w2 for NT tiles of 16 tokens, with LP parts of h in LDS and the
// others requested with the weights.
template <bool F8, int NT, int FORM, int LP>
struct FewGeom2 {
    static constexpr int NB = F8 ? 4 : 2;
    static constexpr int UK = F8 ? 128 : 64;
    static constexpr int Sets = LP == 2 ? 0 : (FORM == kCols8 ? 1 : 2 - LP);   // pieces of how many parts a lane requests
    static constexpr int Regs = Sets * NB * 4;
    static constexpr int Ring = Regs <= 8 ? 4 : (Regs <= 16 && !(F8 && NT == 2 && FORM == kCols16) ? 3 : 2);
};
template <bool F8, int NT, int FORM, int LP>
struct FewSlot2 {
    using Geo = FewGeom2<F8, NT, FORM, LP>;
    i32x4 a[2];
    i32x4 b[Geo::Sets ? Geo::Sets : 1][Geo::NB];
    uint32_t sc;
    int col;                                                 // the column of this lane's token, or -1; 16 bits for each of two tiles
    int at;                                                  // place of the row's first piece in LDS
};

// h in two parts of the operands' type: the value rounded, and what that leaves
// out, rounded (in FP16 times 2^11, or the part of a small value would be below
// the type's range). 16 bits of it in BF16, 22 in FP16. A value past the type's
// range is infinite, its second part 0.
template <int F16>
MOE_DEV void few_parts(float v, uint16_t& hi, uint16_t& lo) {
    hi = (uint16_t)pack16(v, 0.f, F16);
    const float r = lo16(hi, F16);
    lo = (uint16_t)pack16(fabsf(r) < INFINITY ? (v - r) * (F16 ? 2048.f : 1.f) : 0.f, 0.f, F16);
}

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

// the products of one unit with one tile of 16 token rows (piece(i): piece i of this lane's token row)
template <int EL, bool F8, typename Piece>
MOE_DEV f32x4 few_unit(const i32x4 (&a)[2], Piece&& piece) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (F8) {
            d = mfma16x16x32<EL>(few_decode<EL>(a[h][0], a[h][1]), piece(2 * h), d);
            d = mfma16x16x32<EL>(few_decode<EL>(a[h][2], a[h][3]), piece(2 * h + 1), d);
        } else {
            d = mfma16x16x32<EL>(a[h], piece(h), d);
        }
    }
    return d;
}

// The sum of the products of both parts. Where the first part's is not finite it
// stands alone (an infinite weight times a second part of 0 is no number).
template <int EL>
MOE_DEV float few_both(float d, float e) {
    const float s = EL == kElF16 ? fmaf(e, 1.f / 2048.f, d) : d + e;
    return fabsf(d) < INFINITY ? s : d;
}
// The products of one unit with 16 rows and both parts of h, hi(i) and lo(i) their piece i.
template <int EL, bool F8, typename Hi, typename Lo>
MOE_DEV f32x4 few_unit2(const i32x4 (&a)[2], Hi&& hi, Lo&& lo) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f}, e = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        #pragma unroll
        for (int k = 0; k < (F8 ? 2 : 1); ++k) {
            const i32x4 w = F8 ? few_decode<EL>(a[h][2 * k], a[h][2 * k + 1]) : a[h];
            const int i = F8 ? 2 * h + k : h;
            d = mfma16x16x32<EL>(w, hi(i), d);
            e = mfma16x16x32<EL>(w, lo(i), e);
        }
    }
    #pragma unroll
    for (int v = 0; v < 4; ++v) d[v] = few_both<EL>(d[v], e[v]);
    return d;
}

// An address that is the same in the whole wave, as the compiler is to know too
// (a resource in vector registers is a loop over lanes at every request, which
// few_w1's weights and scales still have where its token rows are not in LDS).
MOE_DEV const uint8_t* few_uniform(uint64_t a) {
    return (const uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
                            (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32);
}
// Weights (or scales) of the groups, `bytes` a group and the shared one apart: scalars,
// taken from the parameters once (a choice between two of those becomes a load
// from a chosen address, and the parameters then live in scratch memory).
struct FewGroups {
    uint64_t at, shared;
    size_t bytes;
    int E_loc;
    MOE_DEV FewGroups(uint64_t a, uint64_t s, size_t n, int e)
        : at((uint64_t)few_uniform(a)), shared((uint64_t)few_uniform(s)), bytes(n), E_loc(__builtin_amdgcn_readfirstlane(e)) {}
    MOE_DEV const uint8_t* of(int g) const { return (const uint8_t*)(g < E_loc ? at + (uint64_t)g * bytes : shared); }
};
MOE_DEV i32x4 few_load(const rsrc_t& r, uint32_t o) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}
// weights: each byte is used once
MOE_DEV i32x4 few_load_w(const rsrc_t& r, uint32_t o) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 2));
}

// byte offset in a weight row of this lane's piece of unit u, and of piece i of
// a token row; past the row: kMmInvalid
template <bool F8>
MOE_DEV uint32_t few_koff_w(int u, int lane, int K) {
    const int b = u * 128 + 16 * (lane & 7);
    return b < (F8 ? K : 2 * K) ? (uint32_t)b : kMmInvalid;
}
// A unit of weights from the lanes that loaded it (8 lanes a row: whole lines)
// to those that multiply it (16 rows, 4 lanes each), through 2 KiB of LDS a wave,
// 16-byte pieces swizzled by row. A wave's LDS accesses are done in order.
MOE_DEV void few_swap(uint8_t* ex, int lane, const i32x4 (&in)[2], i32x4 (&out)[2]) {
    const int r = lane >> 3, j = lane & 15, q = lane >> 4;
    *(i32x4*)(ex + r * 128 + ((lane & 7) ^ kc_swz(r)) * 16) = in[0];
    *(i32x4*)(ex + (8 + r) * 128 + ((lane & 7) ^ kc_swz(8 + r)) * 16) = in[1];
    out[0] = *(const i32x4*)(ex + j * 128 + (q ^ kc_swz(j)) * 16);
    out[1] = *(const i32x4*)(ex + j * 128 + ((4 + q) ^ kc_swz(j)) * 16);
}
// (LDS rows are padded with zeros, so only loads from memory ask for the end)
template <bool F8>
MOE_DEV int few_kbyte_x(int u, int i, int q) { return F8 ? u * 256 + 128 * (i >> 1) + 32 * q + 16 * (i & 1) : u * 128 + 64 * i + 16 * q; }
template <bool F8>
MOE_DEV uint32_t few_koff_x(int u, int i, int q, int K) {
    const int b = few_kbyte_x<F8>(u, i, q);
    return b < 2 * K ? (uint32_t)b : kMmInvalid;
}
// the sum of two offsets, past every resource if one of them is
MOE_DEV uint32_t few_add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// What a workgroup knows of the routing, in LDS. Rows are the local assignments in
// the order of (token, choice), then the shared expert's tokens, so every
// workgroup numbers them alike; active groups are in the order of their first row.
struct FewTables {
    int* idx; float* w;                                      // [T k] choices and weights
    int *group, *cnt, *first;                                // [most] active groups, their rows, first member
    int* member;                                             // [R] rows by group (in any order inside one)
    int* token; float* row_w;                                // [R] of a row
    int *of, *num;                                           // [G] place among the active groups; rows so far
    int* wave;                                               // [3 x 16] sums of waves; [48] active, [49] rows, [50] rows of the longest
};
constexpr int kFewWaveInts = 52;
__host__ __device__ inline size_t few_table_ints(int T, int k, int G, int s) {
    const size_t R = (size_t)T * (k + s), most = (size_t)G < R ? G : R;
    return 2 * (size_t)T * k + 3 * most + 3 * R + 2 * (size_t)G + kFewWaveInts;
}
MOE_DEV FewTables few_tables(int* lds, int T, int k, int G, int s) {
    const int R = T * (k + s), most = min(G, R);
    FewTables t;
    t.idx = lds; lds += T * k;
    t.w = (float*)lds; lds += T * k;
    t.group = lds; lds += most;
    t.cnt = lds; lds += most;
    t.first = lds; lds += most;
    t.member = lds; lds += R;
    t.token = lds; lds += R;
    t.row_w = (float*)lds; lds += R;
    t.of = lds; lds += G;
    t.num = lds; lds += G;
    t.wave = lds;
    return t;
}
// few_w2's columns: rows of the group in its map (the columns' rows, then the column
// of each token, tokens t and t + 16 side by side), or -1. Tokens in their order: T
// entries, the rows of the tokens.
// A group of more than 16 rows is there twice, one after the other, so that its
// weights come from a cache the second time.
__host__ __device__ inline int few_map_width(int T) { return T > 16 ? 48 : (T > 8 ? 32 : T); }
// most groups of few_w2
__host__ __device__ inline int few_most(int T, int k, int G, int s) {
    const int R = T * (k + s), most = G < R ? G : R;
    return T > 16 ? most + R / 17 : most;
}
// the columns of a call, from the rows of its longest group
MOE_DEV int few_form(int most) { return most <= 8 ? kCols8 : kCols16; }
constexpr int kFewHead = 3;                                  // ints before the groups: their number, rows, form
// sum of the waves' values before this wave's, and of all
MOE_DEV int few_before(const int* wave, int w, int& all) {
    int run = 0;
    all = 0;
    #pragma unroll
    for (int i = 0; i < kFewWaves; ++i) {
        run += i < w ? wave[i] : 0;
        all += wave[i];
    }
    return run;
}

// The local group of routed assignment a, or -1. A token has one row in a group:
// where its logits hold a NaN (so its weights are NaN) the router can name an
// expert twice, and of those the first counts.
MOE_DEV int few_group_of(const FewP& p, const FewTables& t, int a) {
    const int e = t.idx[a] - p.e0;
    if ((uint32_t)e >= (uint32_t)p.E_loc) return -1;
    const float w = t.w[a];
    if (w != w)
        for (int i = a - a % p.k; i < a; ++i)
            if (t.idx[i] == t.idx[a]) return -1;
    return e;
}

// The grouping of up to 64 N assignments by one wave, without barriers (every
// instruction of a workgroup's 16 waves costs 16 cycles of a SIMD: the whole
// workgroup's way, below, takes 1.8 us): lane l of slot i has assignment 64 i + l; the
// lanes with the same group are found by a ballot per bit of its number.
template <int N>
MOE_DEV void few_group_wave(const FewP& p, const FewTables& t, int lane) {
    const int Tk = p.T * p.k, all = Tk + p.s * p.T;
    int g[N], tok[N], c[N], pos[N], ai[N], first[N];
    uint64_t eq[N][N], rows[N], lead[N];
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        const int a = 64 * i + lane;
        tok[i] = a < Tk ? a / p.k : a - Tk;
        g[i] = -1;
        if (a < Tk) {
            g[i] = few_group_of(p, t, a);
        } else if (a < all) {
            g[i] = p.E_loc;
        }
        rows[i] = __ballot(g[i] >= 0);
    }
    #pragma unroll
    for (int i = 0; i < N; ++i)
        #pragma unroll
        for (int j = 0; j < N; ++j) eq[i][j] = rows[j];
    for (int b = 0; b < group_bits(p.G); ++b)
        #pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t m = __ballot((g[j] >> b) & 1);
            #pragma unroll
            for (int i = 0; i < N; ++i) eq[i][j] &= ((g[i] >> b) & 1) ? m : ~m;
        }
    int before = 0, n_act = 0, n_rows = 0, most = 0;
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = pos[i] = 0;
        #pragma unroll
        for (int j = 0; j < N; ++j) {
            c[i] += __popcll(eq[i][j]);
            if (j < i) pos[i] += __popcll(eq[i][j]);
        }
        pos[i] += __popcll(eq[i][i] & lanemask_lt(lane));
        lead[i] = __ballot(g[i] >= 0 && pos[i] == 0);
        ai[i] = n_act + __popcll(lead[i] & lanemask_lt(lane));
        n_act += __popcll(lead[i]);
        const int mine = (lead[i] >> lane) & 1 ? c[i] : 0, inc = wave_incl_scan(mine);
        first[i] = before + inc - mine;
        before += __builtin_amdgcn_readlane(inc, 63);
        most = max(most, (int)wave_umax((uint32_t)mine));
    }
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        // the group's leader: the lowest lane of its first slot
        int f = 0;
        #pragma unroll
        for (int j = N - 1; j >= 0; --j) {
            const int v = __shfl(first[j], eq[i][j] ? __ffsll((unsigned long long)eq[i][j]) - 1 : 0, 64);
            f = eq[i][j] ? v : f;
        }
        const int row = n_rows + __popcll(rows[i] & lanemask_lt(lane));
        n_rows += __popcll(rows[i]);
        if (g[i] >= 0) {
            t.token[row] = tok[i];
            t.row_w[row] = 64 * i + lane < Tk ? t.w[64 * i + lane] : 1.f;
            t.member[f + pos[i]] = row;
            if (pos[i] == 0) {
                t.group[ai[i]] = g[i];
                t.cnt[ai[i]] = c[i];
                t.first[ai[i]] = f;
            }
        }
    }
    if (lane == 0) { t.wave[3 * kFewWaves] = n_act; t.wave[3 * kFewWaves + 1] = n_rows; t.wave[3 * kFewWaves + 2] = most; }
}

// A token whose logits are all -inf chooses nothing (its weights come out as NaN, like
// those of a token with a NaN or +inf, which keeps them): by the wave that routed it.
MOE_DEV void few_unrouted(const FewP& p, const FewTables& t, int tok, int lane) {
    if (tok >= p.T) return;
    const float w = t.w[tok * p.k];
    if (__builtin_amdgcn_readfirstlane(w == w ? 1 : 0)) return;
    bool other = false;
    for (int e = lane; e < p.E; e += 64) other |= !(p.logits[(size_t)tok * p.E + e] == -INFINITY);
    if (__ballot(other)) return;
    if (lane < p.k) t.idx[tok * p.k + lane] = -1;
}

// Routes the T tokens and groups their local assignments, by the whole
// workgroup; an assignment to a thread (T (k + s) <= 32 x 32).
MOE_DEV void few_route(const FewP& p, const FewTables& t) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < p.G; i += kFewThreads) {
        t.num[i] = 0;
        t.of[i] = kFewThreads;
    }
    const bool r = p.renorm != 0;
    if (p.E <= 64) route_block<kFewWaves, 32, 2>(p.logits, p.T, p.E, p.k, r, t.idx, t.w, nullptr, nullptr);
    else if (p.E <= 256) route_block<kFewWaves, 32, 8>(p.logits, p.T, p.E, p.k, r, t.idx, t.w, nullptr, nullptr);
    else if (p.E <= 512) route_block<kFewWaves, 64, 8>(p.logits, p.T, p.E, p.k, r, t.idx, t.w, nullptr, nullptr);
    else route_block<kFewWaves, 64, 32>(p.logits, p.T, p.E, p.k, r, t.idx, t.w, nullptr, nullptr);
    // (route_block's tokens of a wave: two side by side up to 256 experts, else one and 16 on)
    few_unrouted(p, t, p.E <= 256 ? 2 * w : w, lane);
    few_unrouted(p, t, p.E <= 256 ? 2 * w + 1 : w + kFewWaves, lane);
    __syncthreads();
    // thread a: assignment a of the routed ones, then the shared expert's tokens
    const int Tk = p.T * p.k, all = Tk + p.s * p.T, a = tid;
    if (all <= 128) {
        if (w == 0) {
            if (all <= 64) few_group_wave<1>(p, t, lane);
            else few_group_wave<2>(p, t, lane);
        }
        __syncthreads();
        return;
    }
    int g = -1, tok = 0, pos = 0;
    float wt = 1.f;
    if (a < Tk) {
        tok = a / p.k;
        wt = t.w[a];
        g = few_group_of(p, t, a);
        if (g >= 0) {
            pos = atomicAdd(t.num + g, 1);
            atomicMin(t.of + g, a);
        }
    } else if (a < all) {
        tok = pos = a - Tk;
        g = p.E_loc;
    }
    if (tid == 0 && p.s) {
        t.num[p.E_loc] = p.T;
        t.of[p.E_loc] = Tk;
    }
    __syncthreads();
    // a group's first row in order speaks for it (pos goes by the atomics' order)
    const bool leads = g >= 0 && t.of[g] == a;
    const uint64_t rows = __ballot(g >= 0), lead = __ballot(leads);
    if (lane == 0) { t.wave[w] = __popcll(rows); t.wave[kFewWaves + w] = __popcll(lead); }
    __syncthreads();
    int n_rows, n_act;
    const int row = few_before(t.wave, w, n_rows) + __popcll(rows & lanemask_lt(lane));
    const int ai = few_before(t.wave + kFewWaves, w, n_act) + __popcll(lead & lanemask_lt(lane));
    if (g >= 0) {
        t.token[row] = tok;
        t.row_w[row] = wt;
        if (leads) {
            t.group[ai] = g;
            t.of[g] = ai;
        }
    }
    __syncthreads();
    // first member of each active group: a scan of their rows, one group to a thread
    const int c = tid < n_act ? t.num[t.group[tid]] : 0, inc = wave_incl_scan(c);
    const int most = (int)wave_umax((uint32_t)c);
    if (lane == 63) t.wave[2 * kFewWaves + w] = inc;
    if (lane == 0) t.wave[w] = most;
    __syncthreads();
    if (tid < n_act) {
        int n;
        t.first[tid] = few_before(t.wave + 2 * kFewWaves, w, n) + inc - c;
        t.cnt[tid] = c;
    }
    if (tid < 64) {
        const int m = (int)wave_umax(lane < kFewWaves ? (uint32_t)t.wave[lane] : 0u);
        if (lane == 0) { t.wave[3 * kFewWaves] = n_act; t.wave[3 * kFewWaves + 1] = n_rows; t.wave[3 * kFewWaves + 2] = m; }
    }
    __syncthreads();
    if (g >= 0) t.member[t.first[t.of[g]] + pos] = row;
    __syncthreads();
}

// One 16-bit row into LDS, zeros up to `bytes` (a multiple of 1 KiB): piece c of
// a row by one wave, loads that write LDS directly.
MOE_DEV void few_stage(const rsrc_t& r, uint32_t row_off, int row_bytes, int c, uint8_t* dst, int lane) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int b = c * 1024 + lane * 16;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void_t*)(dst + c * 1024), 16,
                                             b < row_bytes ? row_off + (uint32_t)b : kMmInvalid, 0, 0, 0);
#endif
}

// Keeps the order of requests, where a wait counts the younger ones.
MOE_DEV void few_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// `steps` units in turns of the ring. The last turn is a whole one too (its units
// past the end are not there: nothing is loaded or stored for them), because with
// a way out between two slots the compiler sees paths on which slots are skipped,
// and waits for requests that are long to come.
template <int RING, typename Slot, typename Step>
MOE_DEV void few_turns(Slot (&ring)[RING], int steps, Step&& step) {
    #pragma unroll 1
    for (; steps > 0; steps -= RING)
        static_for<RING>([&](auto s) __attribute__((always_inline)) { step(ring[decltype(s)::value]); });
}

// ------------------------------------------------------------------ few_w1
// bytes of a token row in LDS: all units of all waves, and 64 so that rows start in other banks
template <bool F8>
__host__ __device__ inline int few_row_lds(int units, int split) { return ((units + split - 1) / split * split * (F8 ? 256 : 128) + 1023) / 1024 * 1024 + 64; }

// The items of `n_list` active groups (list: their places among the active ones;
// NULL: all). XL: token rows are read from LDS, all of them if ALL (staged by the
// caller), else each group's in turn.
template <int EL, bool F8, int NT, bool XL, bool ALL>
MOE_DEV void few_w1_body(const FewP& p, const FewTables& tb, const int* list, int n_list, float* part, uint8_t* swap, uint8_t* rows) {
    using Geo = FewGeom<F8, NT, XL>;
    constexpr int RING = Geo::Ring;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    // an item is `subs` times `ob` outputs of a group, each by `split` waves: 8, or
    // fewer where that fills the grid's last round better; a workgroup takes a
    // contiguous run of items, so few groups
    const int split = p.split, subs = kFewWaves / split, sub = w / split, wk = w - sub * split;
    int ob = 8, cb = __builtin_amdgcn_readfirstlane(p.cb8);
    float least = ceilf((float)(n_list * cb) * p.per_grid) * 9.f;
    auto consider = [&](int o, int c) __attribute__((always_inline)) {
        const int n = __builtin_amdgcn_readfirstlane(c);
        const float cost = ceilf((float)(n_list * n) * p.per_grid) * (float)(o + 1);
        if (cost < least) { least = cost; ob = o; cb = n; }
    };
    consider(6, p.cb6);
    consider(4, p.cb4);
    consider(2, p.cb2);
    ob = __builtin_amdgcn_readfirstlane(ob);
    cb = __builtin_amdgcn_readfirstlane(cb);
    const int wide = ob * subs;                              // outputs of an item
    const int n_items = n_list * cb, grid = gridDim.x, each = n_items / grid, more = n_items - each * grid;
    const int first = (int)blockIdx.x * each + min((int)blockIdx.x, more), end = first + each + ((int)blockIdx.x < more ? 1 : 0);
    if (first >= end) return;
    const int wrow = p.H * (F8 ? 1 : 2);                     // bytes of a weight row
    const int units = (p.H + Geo::UK - 1) / Geo::UK, upw = (units + split - 1) / split;
    const int nsb = (2 * p.I + 127) >> 7, ksb = (p.H + 127) >> 7;
    const FewGroups w_of(p.w1, p.w1s, (size_t)(2 * p.I) * (size_t)wrow, p.E_loc), s_of(p.s1, p.s1s, (size_t)(nsb * ksb) * 4, p.E_loc);
    const int stride = few_row_lds<F8>(units, split);
    auto place = [&](int i) __attribute__((always_inline)) { return list ? __builtin_amdgcn_readfirstlane(list[i]) : i; };
    const rsrc_t rx = make_rsrc(p.x, p.x_bytes);
    uint8_t* const ex = swap + w * 2048;

    // the loader: one unit after another through all items
    struct { int ai, c, left, i; bool live; const uint8_t *w, *s; uint32_t ro[2], sg, su, xo[NT]; } L;
    auto open = [&]() __attribute__((always_inline)) {
        L.i = 0;
        L.live = L.left > 0;
        const int ai = place(min(L.ai, n_list - 1)), c0 = L.c * wide + sub * ob;
        const int g = __builtin_amdgcn_readfirstlane(tb.group[ai]);
        L.w = w_of.of(g);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + (lane >> 3), o = 2 * (r >> 2) + (r & 1), col = c0 + o;
            const uint32_t at = (uint32_t)((r & 2 ? p.I : 0) + col) * (uint32_t)wrow;
            L.ro[h] = (o < ob) & (col < p.I) ? at : kMmNoRow;
        }
        if constexpr (F8) {                                  // (an even column and the next one are of one block)
            L.s = s_of.of(g);
            const int c = min(c0 + 2 * q, p.I - 2);
            L.sg = (uint32_t)((c >> 7) * ksb);
            L.su = (uint32_t)(((p.I + c) >> 7) * ksb);
        }
        if constexpr (!XL) {
            const int lo = tb.first[ai], n = tb.cnt[ai];
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                L.xo[t] = 16 * t + j < n ? (uint32_t)tb.token[tb.member[lo + min(16 * t + j, n - 1)]] * p.x_ld : kMmNoRow;
        }
    };
    auto load = [&](FewSlot<F8, NT, XL>& S) __attribute__((always_inline)) {
        const rsrc_t rw = make_rsrc(L.w, L.live ? (uint32_t)(2 * p.I) * (uint32_t)wrow : 0u);
        const int u = L.i * split + wk;
        #pragma unroll
        for (int h = 0; h < 2; ++h) S.a[h] = few_load_w(rw, few_add(L.ro[h], few_koff_w<F8>(u, lane, p.H)));
        if constexpr (!XL) {
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                #pragma unroll
                for (int i = 0; i < Geo::NB; ++i) S.b[t][i] = few_load(rx, few_add(L.xo[t], few_koff_x<F8>(u, i, q, p.H)));
        }
        if constexpr (F8) {
            const rsrc_t rs = make_rsrc(L.s, L.live ? (uint32_t)(nsb * ksb) * 4u : 0u);
            const uint32_t kb = (uint32_t)min(u, ksb - 1);
            S.sc[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (L.sg + kb) * 4u, 0, 0);
            S.sc[1] = __builtin_amdgcn_raw_buffer_load_b32(rs, (L.su + kb) * 4u, 0, 0);
        }
        if (++L.i == upw) {
            --L.left;
            if (++L.c == cb) { L.c = 0; ++L.ai; }
            open();
        }
    };
    // the group's token rows into LDS; a wait for the requests and a barrier must follow
    auto stage = [&](int i) __attribute__((always_inline)) {
        const int ai = place(i), lo = tb.first[ai], n = tb.cnt[ai], chunks = stride / 1024;
        for (int r = 0; r < n; ++r) {
            const int tok = __builtin_amdgcn_readfirstlane(tb.token[tb.member[lo + r]]);
            for (int c = w; c < chunks; c += kFewWaves) few_stage(rx, (uint32_t)tok * p.x_ld, 2 * p.H, c, rows + r * stride, lane);
        }
    };

    int ai = __builtin_amdgcn_readfirstlane(first / cb), c8 = first - ai * cb, i = 0, left = end - first, turn = 0;
    if constexpr (XL && !ALL) stage(ai);
    few_fence();
    L.ai = ai;
    L.c = c8;
    L.left = left;
    open();
    FewSlot<F8, NT, XL> ring[RING];
    static_for<RING>([&](auto s) __attribute__((always_inline)) { load(ring[decltype(s)::value]); });
    if constexpr (XL) {                                      // (the rows were requested before the ring's units)
        few_fence();
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(RING * (F8 ? 4 : 2), 15));
        bare_barrier();
    }
    const uint8_t* xrow[NT];
    int g, lo, n;
    auto rows_of = [&]() __attribute__((always_inline)) {    // (lanes past the group's rows read its last: not stored)
        const int a = place(ai);
        g = __builtin_amdgcn_readfirstlane(tb.group[a]);
        lo = __builtin_amdgcn_readfirstlane(tb.first[a]);
        n = __builtin_amdgcn_readfirstlane(tb.cnt[a]);
        #pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = min(16 * t + j, n - 1);
            xrow[t] = rows + (ALL ? tb.token[tb.member[lo + r]] : r) * stride;
        }
    };
    rows_of();
    f32x4 acc[NT];
    #pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](FewSlot<F8, NT, XL>& S) __attribute__((always_inline)) {
        const int u = i * split + wk;
        float sc[2] = {1.f, 1.f};
        if constexpr (F8) {
            // (0 for a unit past the row's end, whose sums are 0: the last block's may be infinite)
            sc[0] = u < units ? __uint_as_float(S.sc[0]) : 0.f;
            sc[1] = u < units ? __uint_as_float(S.sc[1]) : 0.f;
        }
        i32x4 a[2];
        few_swap(ex, lane, S.a, a);
        #pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 d = few_unit<EL, F8>(a, [&](int x) __attribute__((always_inline)) {
                if constexpr (XL) return *(const i32x4*)(xrow[t] + few_kbyte_x<F8>(u, x, q));
                else return S.b[t][x];
            });
            #pragma unroll
            for (int v = 0; v < 4; ++v) acc[t][v] = F8 ? fmaf(d[v], sc[v >> 1], acc[t][v]) : acc[t][v] + d[v];
        }
        load(S);
        if (++i < upw || left == 0) return;
        i = 0;
        // an item's end: the waves' sums through LDS, two buffers in turn: one barrier an item
        float* const mine = part + turn * (kFewWaves * NT * 256);
        turn ^= 1;
        #pragma unroll
        for (int t = 0; t < NT; ++t)
            #pragma unroll
            for (int v = 0; v < 4; ++v) mine[(w * NT + t) * 256 + v * 64 + lane] = acc[t][v];
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        bare_barrier();
        // thread (part of the item, tile, output of a pair, lane of the result): gate v, up v + 2
        const int e = threadIdx.x, m = e / (NT * 128), t = (e >> 7) & (NT - 1), v = (e >> 6) & 1, l = e & 63;
        const int r = 16 * t + (l & 15), o8 = 2 * (l >> 4) + v, c = wide * c8 + m * ob + o8;
        if (m < subs && o8 < ob && c < p.I && r < n) {
            const float* const src = mine + (m * split * NT + t) * 256 + v * 64 + l;
            float z = 0.f, y = 0.f;
            #pragma unroll 4
            for (int x = 0; x < split; ++x) {
                z += src[x * (NT * 256)];
                y += src[x * (NT * 256) + 128];
            }
            if (p.b1) {
                z += p.b1[(size_t)g * 2 * p.I + c];
                y += p.b1[(size_t)g * 2 * p.I + p.I + c];
            }
            z = epi_clamp(z, p.limit);
            float a = 0.f;
            with_act(p.act, [&](auto act) { a = epi_act<decltype(act)::value>(z, p.beta); });
            const int row = tb.member[lo + r];
            const float o = a * epi_clamp(y, p.limit) * tb.row_w[row];
            uint16_t hi, lo;
            few_parts<EL == kElF16>(o, hi, lo);
            uint16_t* const d = p.h + (size_t)row * 2 * p.I + c;
            d[0] = hi;
            d[p.I] = lo;
        }
        #pragma unroll
        for (int x = 0; x < NT; ++x) acc[x] = f32x4{0.f, 0.f, 0.f, 0.f};
        --left;
        if (++c8 == cb && left > 0) {                                // the next group (every wave is past its products)
            c8 = 0;
            ++ai;
            if constexpr (XL && !ALL) {
                stage(ai);
                few_fence();
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
                bare_barrier();
            }
            rows_of();
        }
    };
    few_turns(ring, left * upw, step);
}

// What few_w2 reads of the routing, by one workgroup.
MOE_DEV void few_map(const FewP& p, const FewTables& tb, int n_act, int R, int most) {
    const int tid = threadIdx.x, lane = tid & 63, form = few_form(most);
    for (int i = tid; i < R; i += kFewThreads) p.row_w[i] = tb.row_w[i];
    if (tid == 0) { p.active[0] = n_act; p.active[1] = R; p.active[2] = form; }
    if (p.T <= 8 || (p.T <= 16 && form == kCols16)) {        // the columns are the tokens (few_w2_body)
        for (int i = tid; i < n_act; i += kFewThreads) p.active[kFewHead + i] = tb.group[i];
        for (int i = tid; i < n_act * p.T; i += kFewThreads) {
            const int a = i / p.T, t = i - a * p.T;
            int row = -1;
            for (int m = tb.first[a]; m < tb.first[a] + tb.cnt[a]; ++m) row = tb.token[tb.member[m]] == t ? tb.member[m] : row;
            p.map[i] = (int16_t)row;
        }
        return;
    }
    int* const at = tb.num;                                  // [n_act] first place of a group among few_w2's
    int* const sorted = tb.idx;                              // [R <= 2 T k] members, in each group in the order of the rows
    if (tid < 64) {
        int more = 0;
        for (int a0 = 0; a0 < n_act; a0 += 64) {
            const uint64_t big = __ballot(a0 + lane < n_act && tb.cnt[min(a0 + lane, n_act - 1)] > 16);
            if (a0 + lane < n_act) at[a0 + lane] = a0 + lane + more + __popcll(big & lanemask_lt(lane));
            more += __popcll(big);
        }
        if (lane == 0) p.active[0] = n_act + more;
    }
    for (int i = tid; i < n_act * 32; i += kFewThreads) {
        const int a = i >> 5, m = i & 31, lo = tb.first[a], n = tb.cnt[a];
        if (m >= n) continue;
        const int row = tb.member[lo + m];
        int rank = 0;
        for (int x = 0; x < n; ++x) rank += tb.member[lo + x] < row ? 1 : 0;
        sorted[lo + rank] = row;
    }
    __syncthreads();
    const int width = few_map_width(p.T);
    for (int i = tid; i < n_act * width; i += kFewThreads) {
        const int a = i / width, e = i - a * width, lo = tb.first[a], n = tb.cnt[a];
        const int t = p.T > 16 ? 16 * (e & 1) + ((e - 16) >> 1) : e - 16;
        int mine = -1;                                       // of a token: its row's place in the group
        if (e >= 16)
            for (int x = 0; x < n; ++x) mine = tb.token[sorted[lo + x]] == t ? x : mine;
        for (int h = 0; 16 * h < n; ++h) {
            const int c = e < 16 ? (16 * h + e < n ? sorted[lo + 16 * h + e] : -1) : (mine >> 4 == h ? mine & 15 : -1);
            p.map[(at[a] + h) * width + e] = (int16_t)c;
            if (e == 0) p.active[kFewHead + at[a] + h] = tb.group[a];
        }
    }
    __syncthreads();                                         // (the choices' place is used again)
}

template <int EL, bool F8, bool TWO>
__global__ __launch_bounds__(kFewThreads, 4)
void few_w1_kernel(FewP p, int lds_rows) {
    constexpr int NTM = TWO ? 2 : 1;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* const part = (float*)smem;                        // [2][16 waves][NT][4][64]
    uint8_t* const swap = smem + 2 * kFewWaves * NTM * 1024; // [16 waves][2 KiB]
    uint8_t* const rows = swap + kFewWaves * 2048;           // [lds_rows]
    const FewTables tb = few_tables((int*)(rows + lds_rows), p.T, p.k, p.G, p.s);
    // the token rows, if all of them fit, are on their way while the tokens are routed
    const int stride = few_row_lds<F8>((p.H + (F8 ? 127 : 63)) / (F8 ? 128 : 64), p.split);
    const bool all = (int64_t)p.T * stride <= lds_rows;
    if (all) {
        const rsrc_t rx = make_rsrc(p.x, p.x_bytes);
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), chunks = stride / 1024;
        for (int t = 0; t < p.T; ++t)
            for (int c = w; c < chunks; c += kFewWaves)
                few_stage(rx, (uint32_t)t * p.x_ld, 2 * p.H, c, rows + t * stride, threadIdx.x & 63);
    }
    few_route(p, tb);
    const int n_act = __builtin_amdgcn_readfirstlane(tb.wave[3 * kFewWaves]), R = tb.wave[3 * kFewWaves + 1];
    const int most = __builtin_amdgcn_readfirstlane(tb.wave[3 * kFewWaves + 2]);
    if (blockIdx.x == gridDim.x - 1) few_map(p, tb, n_act, R, most);
    // groups whose rows fit LDS, then the others (one tile of 16 rows, or two as the longest group has)
    if (all) {
        if (TWO && most > 16) few_w1_body<EL, F8, NTM, true, true>(p, tb, nullptr, n_act, part, swap, rows);
        else few_w1_body<EL, F8, 1, true, true>(p, tb, nullptr, n_act, part, swap, rows);
        return;
    }
    const int cap = min(lds_rows / stride, 16);
    if (most <= cap) {
        few_w1_body<EL, F8, 1, true, false>(p, tb, nullptr, n_act, part, swap, rows);
        return;
    }
    int* const list = tb.idx;                                // (the choices are not needed any more)
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int n = 0;
        for (int big = 0; big < 2; ++big) {
            for (int a0 = 0; a0 < n_act; a0 += 64) {
                const bool in = a0 + lane < n_act && (tb.cnt[a0 + lane] > cap) == (big != 0);
                const uint64_t m = __ballot(in);
                if (in) list[n + __popcll(m & lanemask_lt(lane))] = a0 + lane;
                n += __popcll(m);
            }
            if (big == 0 && lane == 0) tb.wave[0] = n;
        }
    }
    __syncthreads();
    const int small = __builtin_amdgcn_readfirstlane(tb.wave[0]);
    few_w1_body<EL, F8, 1, true, false>(p, tb, list, small, part, swap, rows);
    __syncthreads();                                         // (the sums' places are used again)
    if (TWO && most > 16) few_w1_body<EL, F8, NTM, false, false>(p, tb, list + small, n_act - small, part, swap, rows);
    else few_w1_body<EL, F8, 1, false, false>(p, tb, list + small, n_act - small, part, swap, rows);
}

// ------------------------------------------------------------------ few_w2
// bytes in LDS of one part of a row of h, and of a row with n parts there (64 so that rows start in other banks)
template <bool F8>
MOE_DEV int few_h_part(int I) { return ((I + (F8 ? 127 : 63)) / (F8 ? 128 : 64) * (F8 ? 256 : 128) + 1023) / 1024 * 1024; }
template <bool F8>
MOE_DEV int few_h_row(int I, int n) { return n * few_h_part<F8>(I) + 64; }

// The waves' sums take the place of their exchanged units.
template <int EL, bool F8, int TC, int FORM, int LP>
MOE_DEV void few_w2_body(const FewP& p, const int* active, const int16_t* map, int n_act, int R, uint8_t* swap, uint8_t* rows) {
    constexpr int NT = TC == 32 ? 2 : 1;
    using Geo = FewGeom2<F8, NT, FORM, LP>;
    using Slot = FewSlot2<F8, NT, FORM, LP>;
    constexpr bool PACK = FORM == kCols8, TOKENS = few_cols_of(FORM) >= TC;
    const int width = TOKENS ? p.T : few_map_width(p.T);
    constexpr int RING = Geo::Ring;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    const int wrow = p.I * (F8 ? 1 : 2);
    const int upg = (p.I + Geo::UK - 1) / Geo::UK;           // units of a group
    const int units = n_act * upg;
    const int nsb = (p.H + 127) >> 7, ksb = (p.I + 127) >> 7;
    const FewGroups w_of(p.w2, p.w2s, (size_t)p.H * (size_t)wrow, p.E_loc), s_of(p.s2, p.s2s, (size_t)(nsb * ksb) * 4, p.E_loc);
    const int hpart = few_h_part<F8>(p.I), stride = few_h_row<F8>(p.I, LP);
    uint8_t* const ex = swap + w * 2048;
    float* const part = (float*)swap;                        // [16 waves][2][4][64]
    const int upw = max(1, (units + kFewWaves - 1) / kFewWaves);      // rounds of units of a block of columns
    const rsrc_t rh = make_rsrc(p.h, (uint32_t)((size_t)R * p.I * 4));

    struct { int block, i, ai, ku, sb; bool live; uint32_t ro[2]; } L;
    auto open = [&]() __attribute__((always_inline)) {
        L.i = 0;
        L.live = L.block < p.blocks;
        const int n0 = (L.live ? L.block : 0) * p.cols;
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + (lane >> 3);
            L.ro[h] = r < p.cols && n0 + r < p.H ? (uint32_t)(n0 + r) * (uint32_t)wrow : kMmNoRow;
        }
        // (columns 4 q .. 4 q + 3 are of one block of scales: blocks of E4M3 columns are multiples of 4)
        L.sb = (min(n0 + 4 * q, p.H - 1) >> 7) * ksb;
        L.ai = w / upg;
        L.ku = w - L.ai * upg;
    };
    auto load = [&](Slot& S) __attribute__((always_inline)) {
        const bool live = L.live && L.ai < n_act;
        const int g = live ? __builtin_amdgcn_readfirstlane(active[L.ai]) : 0;
        const rsrc_t rw = make_rsrc(w_of.of(g), live ? (uint32_t)p.H * (uint32_t)wrow : 0u);
        #pragma unroll
        for (int h = 0; h < 2; ++h) S.a[h] = few_load_w(rw, few_add(L.ro[h], few_koff_w<F8>(L.ku, lane, p.I)));
        const int c = PACK ? j & 7 : j, m0 = PACK ? j >> 3 : 0;                // this lane's row's column, its part of h
        const int row = live && (!TOKENS || c < p.T) ? map[L.ai * width + c] : -1;
        #pragma unroll
        for (int m = 0; m < Geo::Sets; ++m) {
            const uint32_t o = row >= 0 ? (uint32_t)(2 * row + m0 + LP + m) * (uint32_t)(p.I * 2) : kMmNoRow;
            #pragma unroll
            for (int i = 0; i < Geo::NB; ++i) S.b[m][i] = few_load(rh, few_add(o, few_koff_x<F8>(L.ku, i, q, p.I)));
        }
        if constexpr (LP > 0) S.at = max(row, 0) * stride + m0 * hpart + few_kbyte_x<F8>(L.ku, 0, q);
        const int16_t* const cols = map + L.ai * width + 16;
        if constexpr (TOKENS) S.col = row;                   // (its own column)
        else if constexpr (NT == 1) S.col = live ? cols[j] : -1;
        else S.col = live ? ((const int*)cols)[j] : -1;
        if constexpr (F8) {
            const rsrc_t rs = make_rsrc(s_of.of(g), live ? (uint32_t)(nsb * ksb) * 4u : 0u);
            S.sc = __builtin_amdgcn_raw_buffer_load_b32(rs, (L.sb + L.ku) * 4, 0, 0);
        }
        L.ku += kFewWaves;
        while (L.ku >= upg) { L.ku -= upg; ++L.ai; }
        L.ai = __builtin_amdgcn_readfirstlane(L.ai);
        L.ku = __builtin_amdgcn_readfirstlane(L.ku);
        if (++L.i == upw) {
            L.block += gridDim.x;
            open();
        }
    };

    if constexpr (LP > 0) {
        const int chunks = hpart / 1024;
        for (int c = w; c < R * LP * chunks; c += kFewWaves) {
            const int rm = c / chunks, r = rm / LP, m = rm - r * LP;
            few_stage(rh, (uint32_t)(2 * r + m) * (uint32_t)(p.I * 2), 2 * p.I, c - rm * chunks, rows + r * stride + m * hpart, lane);
        }
    }
    few_fence();
    L.block = blockIdx.x;
    open();
    Slot ring[RING];
    static_for<RING>([&](auto s) __attribute__((always_inline)) { load(ring[decltype(s)::value]); });
    if constexpr (LP > 0) {                                  // (the rows were requested before the ring's units)
        few_fence();
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(RING * ((F8 ? 3 : 2) + Geo::Sets * Geo::NB), 15));
        bare_barrier();
    }
    f32x4 acc[NT];
    #pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    int block = blockIdx.x, i = 0;
    auto step = [&](Slot& S) __attribute__((always_inline)) {
        i32x4 a[2];
        few_swap(ex, lane, S.a, a);
        // (the scale is used behind the slot's next requests, so it leaves the slot here:
        // otherwise those go to other registers, and the copies back at the end of a
        // turn wait for every request in flight)
        uint32_t sc = 0;
        if constexpr (F8) asm volatile("v_mov_b32 %0, %1" : "=v"(sc) : "v"(S.sc));
        const int own = S.col;
        auto piece = [&](auto m, int x) __attribute__((always_inline)) {
            constexpr int M = decltype(m)::value;
            if constexpr (M < LP) return *(const i32x4*)(rows + S.at + M * hpart + few_kbyte_x<F8>(0, x, 0));
            else return S.b[M - LP][x];
        };
        auto first = [&](int x) __attribute__((always_inline)) { return piece(std::integral_constant<int, 0>{}, x); };
        f32x4 d;
        if constexpr (PACK) {
            d = few_unit<EL, F8>(a, first);
            #pragma unroll
            for (int v = 0; v < 4; ++v)                      // the lane 8 columns on has the second part's
                d[v] = few_both<EL>(d[v], __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(d[v]), 0x128, 0xF, 0xF, true)));
        } else {
            d = few_unit2<EL, F8>(a, first, [&](int x) __attribute__((always_inline)) { return piece(std::integral_constant<int, 1>{}, x); });
        }
        #pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int col = NT == 1 ? own : (t ? own >> 16 : (int)(int16_t)own);
            const bool in = col >= 0;
            #pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float z = TOKENS ? d[v] : __shfl(d[v], (lane & 48) + (col & 15), 64);
                const float y = F8 ? fmaf(z, __uint_as_float(sc), acc[t][v]) : acc[t][v] + z;
                acc[t][v] = in ? y : acc[t][v];
            }
        }
        load(S);
        if (++i < upw || block >= p.blocks) return;
        i = 0;
        #pragma unroll
        for (int t = 0; t < NT; ++t)
            #pragma unroll
            for (int v = 0; v < 4; ++v) part[(2 * w + t) * 256 + v * 64 + lane] = acc[t][v];
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        bare_barrier();
        // thread (token, column): the waves' sums in their order
        const int e = threadIdx.x, t = e >> 4, c = e & 15, n = block * p.cols + c;
        if (e < NT * 256 && t < p.T && c < p.cols && n < p.H) {
            float o = 0.f;
            #pragma unroll
            for (int x = 0; x < kFewWaves; ++x) o += part[(2 * x + (t >> 4)) * 256 + (c & 3) * 64 + (c >> 2) * 16 + (t & 15)];
            if (p.b2) {
                #pragma unroll 4
                for (int a = 0; a < n_act; ++a) {
                    const int c = TOKENS ? t : map[a * width + 16 + (NT == 2 ? 2 * (t & 15) + (t >> 4) : t)], row = c >= 0 ? map[a * width + c] : -1;
                    const float y = fmaf(p.row_w[max(row, 0)], p.b2[(size_t)active[a] * p.H + n], o);
                    o = row >= 0 ? y : o;
                }
            }
            if (p.res) o += lo16(p.res[(size_t)t * p.ld_res + n], EL == kElF16);
            p.out[(size_t)t * p.ld_out + n] = (uint16_t)pack16(o, 0.f, EL == kElF16);
        }
        #pragma unroll
        for (int x = 0; x < NT; ++x) acc[x] = f32x4{0.f, 0.f, 0.f, 0.f};
        block += gridDim.x;
        // the sums have been read before the next units are exchanged
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        bare_barrier();
    };
    few_turns(ring, (p.blocks - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * upw, step);
}

// TC: 8, 16 or 32, at least the tokens
template <int EL, bool F8, int TC>
__global__ __launch_bounds__(kFewThreads, 4)
void few_w2_kernel(FewP p, int lds_rows, int most) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t* const swap = smem;                              // [16 waves][2 KiB]
    uint8_t* const rows = swap + kFewWaves * 2048;           // [lds_rows]
    int* const active = (int*)(rows + lds_rows);             // [kFewHead + most], then the map
    int16_t* const map = (int16_t*)(active + kFewHead + most);
    // all of the tables at once, whatever they hold past the active groups
    for (int i = threadIdx.x; i < most + kFewHead; i += kFewThreads) active[i] = p.active[i];
    for (int i = threadIdx.x; i < (most * few_map_width(p.T) + 1) / 2; i += kFewThreads) ((int*)map)[i] = ((const int*)p.map)[i];
    __syncthreads();
    const int n_act = __builtin_amdgcn_readfirstlane(active[0]), R = __builtin_amdgcn_readfirstlane(active[1]);
    const int64_t n = max(R, 1);
    const bool both = n * few_h_row<F8>(p.I, 2) <= lds_rows;
    const int* const groups = active + kFewHead;
    if (TC == 8 || __builtin_amdgcn_readfirstlane(active[2]) == kCols8) {
        if (both) few_w2_body<EL, F8, TC, kCols8, 2>(p, groups, map, n_act, R, swap, rows);
        else few_w2_body<EL, F8, TC, kCols8, 0>(p, groups, map, n_act, R, swap, rows);
        return;
    }
    if constexpr (TC > 8) {
        if (both) few_w2_body<EL, F8, TC, kCols16, 2>(p, groups, map, n_act, R, swap, rows);
        else if (n * few_h_row<F8>(p.I, 1) <= lds_rows) few_w2_body<EL, F8, TC, kCols16, 1>(p, groups, map, n_act, R, swap, rows);
        else few_w2_body<EL, F8, TC, kCols16, 0>(p, groups, map, n_act, R, swap, rows);
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

// LDS left for token rows: a compute unit's, less the sums and the tables
template <int EL, bool F8, int TC>
int launch_few(FewP& p, hipStream_t stream) {
    constexpr int NT = TC == 32 ? 2 : 1;
    static bool ready1[64] = {false}, ready2[64] = {false};
    auto* k1 = &few_w1_kernel<EL, F8, NT == 2>;
    auto* k2 = &few_w2_kernel<EL, F8, TC>;
    int e = few_ready(k1, ready1);
    if (e || (e = few_ready(k2, ready2))) return e;
    const int64_t rows = (int64_t)p.T * (p.k + p.s), most = std::min<int64_t>(p.G, rows);
    const int cus = device_cu_count(), most2 = few_most(p.T, p.k, p.G, p.s);
    const int64_t items = most * (p.I / 8);
    const int grid1 = (int)std::min<int64_t>(items, cus), grid2 = std::min(p.blocks, cus);
    const int64_t fix1 = (int64_t)2 * kFewWaves * NT * 1024 + kFewWaves * 2048 +
                         (int64_t)few_table_ints(p.T, p.k, p.G, p.s) * 4;
    const int64_t fix2 = (int64_t)kFewWaves * 2048 + (kFewHead + most2) * 4 + (most2 * few_map_width(p.T) + 1) / 2 * 4;
    const int rows1 = (int)((kMmLds - fix1) / 16 * 16), rows2 = (int)((kMmLds - fix2) / 16 * 16);
    // about four units of the reduction axis to a wave: a barrier and an epilogue
    // for every unit cost more than they are worth (16 tokens on 51 experts of 2048
    // x 1408 in E4M3, 16 units: 110 us with all 16 waves on a row, 103 with 4)
    const int units = (p.H + (F8 ? 127 : 63)) / (F8 ? 128 : 64), subs = units >= 48 ? 1 : (units >= 24 ? 2 : 4);
    p.split = kFewWaves / subs;
    p.cb8 = (p.I + 8 * subs - 1) / (8 * subs); p.cb6 = (p.I + 6 * subs - 1) / (6 * subs);
    p.cb4 = (p.I + 4 * subs - 1) / (4 * subs); p.cb2 = (p.I + 2 * subs - 1) / (2 * subs);
    p.per_grid = 1.0f / (float)grid1;
    k1<<<grid1, kFewThreads, (size_t)(fix1 + rows1), stream>>>(p, rows1);
    if ((e = (int)hipGetLastError())) return e;
    k2<<<grid2, kFewThreads, (size_t)(fix2 + rows2), stream>>>(p, rows2, most2);
    return (int)hipGetLastError();
}

template <int EL, bool F8>
int launch_tokens(FewP& p, hipStream_t stream) {
    if (p.T > 16) return launch_few<EL, F8, 32>(p, stream);
    return p.T > 8 ? launch_few<EL, F8, 16>(p, stream) : launch_few<EL, F8, 8>(p, stream);
}

// Columns of few_w2's blocks: up to 16, fewer where that fills the last round of
// workgroups better (a round costs its columns and about one more).
int few_cols(int H, bool eight) {
    const int cus = device_cu_count(), step = eight ? 4 : 1;
    int best = 16;
    int64_t least = 1ll << 60;
    for (int c = 16; c >= 4; c -= step) {
        const int64_t cost = ((H + c - 1) / c + cus - 1) / cus * (c + 1);
        if (cost < least) { least = cost; best = c; }
    }
    return best;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// byte offsets of the workspace's regions: h, row_w, active, map, end
void few_regions(int T, int k, int G, int s, int I, size_t (&at)[5]) {
    const size_t R = (size_t)T * (k + s), most = few_most(T, k, G, s);
    at[0] = 0;
    at[1] = at[0] + up16(R * I * 4);
    at[2] = at[1] + up16(R * 4);
    at[3] = at[2] + up16((most + kFewHead) * 4);
    at[4] = at[3] + up16(most * few_map_width(T) * 2 + 2);
}

}  // namespace

size_t moe_few_bytes(int T, int k, int G, int s, int I) {
    size_t at[5];
    few_regions(T, k, G, s, I, at);
    return at[4];
}

int moe_launch_few(const moe_few_args& a, void* ws, hipStream_t stream) {
    FewP p{};
    p.logits = a.logits;
    p.T = a.T; p.E = a.E_tot; p.k = a.k; p.e0 = a.e0; p.E_loc = a.E_loc; p.s = a.shared_w1 ? 1 : 0;
    p.G = p.E_loc + p.s; p.renorm = (a.flags & MOE_ROUTE_RENORM) != 0;
    p.x = (const uint8_t*)a.x; p.x_ld = (uint32_t)a.ldx * 2; p.x_bytes = (uint32_t)(a.T - 1) * p.x_ld + (uint32_t)a.H * 2;
    p.H = a.H; p.I = a.I;
    p.w1 = (uint64_t)a.w1; p.w1s = (uint64_t)a.shared_w1;
    p.w2 = (uint64_t)a.w2; p.w2s = (uint64_t)a.shared_w2;
    p.s1 = (uint64_t)a.w1_scales; p.s1s = (uint64_t)a.shared_w1_scales;
    p.s2 = (uint64_t)a.w2_scales; p.s2s = (uint64_t)a.shared_w2_scales;
    p.act = a.epi ? a.epi->act : MOE_ACT_SWIGLU; p.beta = a.epi ? a.epi->beta : 1.0f; p.limit = a.epi ? a.epi->limit : 0.0f;
    p.b1 = a.epi ? a.epi->bias : nullptr; p.b2 = a.bias2;
    p.res = (const uint16_t*)a.residual; p.ld_res = (size_t)a.ld_res;
    p.out = (uint16_t*)a.out; p.ld_out = (size_t)a.ld_out;
    p.cols = few_cols(a.H, a.w1_scales != nullptr); p.blocks = (a.H + p.cols - 1) / p.cols;
    size_t at[5];
    few_regions(p.T, p.k, p.G, p.s, p.I, at);
    uint8_t* b = (uint8_t*)ws;
    p.h = (uint16_t*)(b + at[0]); p.row_w = (float*)(b + at[1]); p.active = (int32_t*)(b + at[2]);
    p.map = (int16_t*)(b + at[3]);
    const bool f8 = a.w1_scales != nullptr;
    if (a.dtype == MOE_T_F16) return f8 ? launch_tokens<kElF16, true>(p, stream) : launch_tokens<kElF16, false>(p, stream);
    return f8 ? launch_tokens<kElBf16, true>(p, stream) : launch_tokens<kElBf16, false>(p, stream);
}

// Grouped products of 16-bit and block-scaled FP8 operands, ragged by expert:
//
//   mm, W [N, K]   y[r][n]  = sum_k x[r][k] W_g[n][k]
//   mm, W [K, N]   y[r][n]  = sum_k x[r][k] W_g[k][n]       (gradient of the rows)
//   wgrad          dW_g[n][k] = sum_{r in g} dy[r][n] x[r][k]
//   fp8            y[r][n]  = sum_b xs[r][b] ws_g[n/128][b] sum_{k in block b} xq[r][k] wq_g[n][k]
//
// One kernel body: a workgroup of 8 waves computes D[a][b] over tiles of 256
// values of the contiguous output axis a (n, or k for wgrad) and BT = 256 or
// 128 of the other axis b (rows, or n for wgrad). Wave w owns a-quarter w % 4
// and b-half w / 4: 4 x NB tiles of the 16x16 matrix instruction. The a side
// is the instruction's A operand, so a lane ends up with 4 consecutive a
// values of one b. (Groups of few rows: grouped_mm_rows.hip.)
//
// Each operand is staged in LDS by buffer loads that write LDS directly, in
// K-tiles of 64 16-bit or 128 FP8 elements (128 bytes), in one of two forms:
//  - reduction axis contiguous in memory: [row][128 bytes], 16-byte chunks
//    XOR-swizzled by row so that the operand reads (16 rows, one chunk each)
//    hit distinct banks;
//  - reduction axis slow in memory (W [K, N]; both operands of wgrad):
//    [k][256 or 128 values], read through the transposing LDS load (16 lanes
//    read 4 k x 16 values and receive 4 k of one value each), 32-byte chunks
//    XOR-swizzled by k so that the 4 rows hit distinct banks.
// Elements past an edge (rows past the group, the K tail, values past N) are
// zero: their offsets fall outside the resource.
//
// Two waves share a SIMD. They run half a step apart: while waves 4-7
// multiply, waves 0-3 read fragments from LDS, and the other way round, so the
// matrix cores and the LDS are both busy. A K-tile is two such turns: turn 0
// reads the wave's a fragments and the first half of its b fragments, turn 1
// the other half of the b fragments. So a stage's a operand and first b half
// are free for the K-tile NST later after turn 0, and a request is in flight
// for about a K-tile's products although LDS holds only two stages of the
// largest tile.
// Requests are issued between matrix instructions: the address unit takes 16
// cycles for each, and a wave that issues them in its reading turn delays the
// reads behind them and with them the other waves' products.
// A wave waits for its own requests (vmcnt, leaving the newer ones in flight)
// before the barrier that opens the turn reading them.
//
// Persistent grid; the requests run ahead across items, so the next item's
// first K-tiles are in flight during an item's epilogue.
//
// Measured, one group, BF16: 16384 x 4096 x 4096 413 us (1330 TFLOP/s) with W
// [N, K], 395 (1390) with W [K, N], FP8 250 (2200); weight gradients of 16384 x
// 2816 x 2048 in 8 equal groups 187 us (1010), from 8-bit rows 209. The matrix
// cores are busy half of the cycles (few, uneven items) to 62%, and the clock
// falls to 1.8 to 2.1 GHz under them; the LDS is active for about a quarter, bank
// conflicts come from the stores alone. FP8 has the same LDS traffic and matrix cycles per K-tile, and
// 4 additions with the block's scale per matrix instruction besides (and sums the
// 128 products of a block as the instruction does, see mfma_fp8).
#include <algorithm>

#include "grouped_mm.h"

namespace {

template <int EL, int NB>
struct MmGeom {
    static constexpr int BT = 32 * NB;                       // b values per workgroup tile
    static constexpr int NU = NB / 2;                        // b tiles of a wave per turn
    static constexpr int NQ = NB / 4;                        // requests of a wave per half of the b operand
    static constexpr int HRows = 2 * NB;                     // rows of a wave per half of the b operand
    static constexpr int QOff = kPBytes;
    static constexpr int SOff = kPBytes + BT * 128;          // fp8: row scales, 256 bytes per wave and half
    static constexpr int Stage = SOff + (EL == kElFp8 ? 4096 : 0);
    // beside the stages: 1 KiB a wave for its stores, and the tables
    static constexpr int NST = Stage * 3 + 2 * kMmOut <= kMmLds ? 3 : 2;
    static constexpr int Lds(int G, bool wgrad) { return Stage * NST + kMmOut + (G + 1) * 4 + (wgrad ? 6 * G : 0); }
};

// The requests of a wave: one K-tile after another through all items, an
// eighth of each operand half: 32 or 2 NB rows (contiguous form) or 8 k (slow
// form). Turn 1 moves on to a K-tile and requests its a operand and first b
// half, the next turn 0 its second b half. Row sources are loaded an item
// (wgrad: a K-tile) before their use: waiting for one would drain the requests
// in flight.
template <int NQ>
struct MmReq {
    int round, kt, step;                // round: the one to look at after n
    int at, nat;                        // numbers of c and n
    bool live, nlive;
    MmItem c, n;                        // the item requested now, and the next one
    uint32_t nrow[2][NQ];               // contiguous b operand: sources of this lane's rows of the next item
    uint32_t srow[2], nsrow[2];         // fp8: byte offset of this lane's row of scales; next item's source
    uint32_t psrc, qsrc, npsrc, nqsrc;  // wgrad: source rows of the next K-tile's k, one k per lane % 8
    uint32_t pc[2], qc[2];              // wgrad, gathered rows: byte offsets inside a row
    uint32_t po[4], qo[2][NQ];          // the next request's byte offsets,
    const uint8_t *pb, *qb, *sb;        // what they count from
    uint32_t pn, qn, sn;                // and the bytes that may be read there
};

// first of the rows that wave w takes of half `half` of the b tile
template <int NB>
MOE_DEV int q_first(int w, int half) { return (w >> 2) * (16 * NB) + half * (8 * NB) + (w & 3) * (2 * NB); }

// byte offset in a row's 128 bytes of the chunk that this lane takes of the
// rows of request i (the swizzle of row 8 m + lane / 8 depends on m's parity)
template <int NB>
MOE_DEV int q_chunk(int lane, int w, int half, int i) {
    return 16 * ((lane & 7) ^ ((lane >> 4) | (4 * (((q_first<NB>(w, half) >> 3) + i) & 1))));
}

// wgrad: sources of this wave's 8 k of K-tile kt of item c (past the group: not looked at)
template <int MODE>
MOE_DEV void mm_load_src(const MmP& p, const MmWhere& wh, const MmItem& c, int kt, uint32_t& ps, uint32_t& qs) {
    const int k = kt * 64 + 8 * wh.w + (wh.lane & 7);
    if constexpr (mm_kind(MODE) == kWgrad && (MODE & kGatherX) != 0)
        ps = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.x_src + c.r0, (uint32_t)(c.nrows * 4)), k * 4, 0, 0);
    if constexpr ((MODE & kGatherDy) != 0)
        qs = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.dy_src + c.r0, (uint32_t)(c.nrows * 4)), k * 4, 0, 0);
}

// find the next item with K-tiles and load its row sources
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void mm_look(const MmP& p, const MmTables& tb, const MmWhere& wh, MmReq<NQ>& R) {
    int round = R.round;
    bool live = false;
    for (int item; !live && (item = mm_nth<MODE>(round, wh)) < wh.n_items; ++round) {
        R.n = mm_scalar(mm_decode<EL, MODE, 32 * NB>(p, tb, wh.at, item));
        R.nat = item;
        live = R.n.nk > 0;
    }
    R.round = round;
    R.nlive = live;
    if (!live) return;
    if constexpr (is_wgrad(MODE)) {
        mm_load_src<MODE>(p, wh, R.n, 0, R.npsrc, R.nqsrc);
    } else {
        // without a branch: past the item (and without a source array, whose
        // resource is then empty) the loads return 0
        const rsrc_t rm = make_rsrc(p.x_src + R.n.r0, p.x_src ? (uint32_t)(R.n.nrows * 4) : 0u);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int first = q_first<NB>(wh.w, h);
            #pragma unroll
            for (int i = 0; i < NQ; ++i)
                R.nrow[h][i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, (first + 8 * i + (wh.lane >> 3)) * 4, 0, 0);
            if constexpr (EL == kElFp8)
                R.nsrow[h] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rm, (first + wh.lane) * 4, 0, 0);
        }
    }
}
// make the next item the one requested, and look for the one after
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void mm_take(const MmP& p, const MmTables& tb, const MmWhere& wh, MmReq<NQ>& R) {
    R.live = R.nlive;
    if (!R.live) return;
    R.c = R.n;
    R.at = R.nat;
    if constexpr (is_wgrad(MODE)) {
        R.psrc = R.npsrc;
        R.qsrc = R.nqsrc;
    } else {
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int first = q_first<NB>(wh.w, h);
            #pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int row = first + 8 * i + (wh.lane >> 3);
                const uint32_t s = R.nrow[h][i];
                R.qo[h][i] = (row < R.c.nrows && s < p.x_rows ? (p.x_src ? s : (uint32_t)row) * p.x_ld : kMmNoRow) +
                             (uint32_t)q_chunk<NB>(wh.lane, wh.w, h, i);
            }
            if constexpr (EL == kElFp8) {
                const int row = first + wh.lane;
                const uint32_t s = R.nsrow[h];
                R.srow[h] = wh.lane < 2 * NB && row < R.c.nrows && s < p.x_rows
                                ? (p.x_src ? s : (uint32_t)row) * (uint32_t)(p.kb * 4) : kMmNoRow;
            }
        }
    }
    mm_look<EL, MODE, NB>(p, tb, wh, R);
}

// bounds a request to 64 rows of the slow form
MOE_DEV void mm_slow_bounds(const uint8_t*& base, uint32_t& bytes, uint32_t ld, int first, int krem, int c0, int ncols) {
    base += (size_t)first * ld + (size_t)c0 * 2;
    // (a scalar again: the clamp becomes a vector instruction, and a
    // descriptor in vector registers a loop over lanes at every request)
    const int rows = __builtin_amdgcn_readfirstlane(max(min(krem, 64), 1));
    bytes = (uint32_t)(rows - 1) * ld + (uint32_t)(min(ncols - c0, 256) * 2);
}

// Offsets of the next request (all past the resource once the items have
// ended: such a request reads nothing and clears a stage nothing reads).
// Slow form, RPI rows of LPR lanes each per request: k = 8 w + RPI i + lane / LPR.
template <int COLS>
MOE_DEV int mm_slow_col(int i, int half, int w, int lane) {
    constexpr int RPI = 512 / COLS, LPR = 64 / RPI;
    const int k = 8 * w + RPI * i + lane / LPR, p32 = (lane % LPR) >> 1;
    if constexpr (COLS == 256) return (p32 ^ tr_swz(k)) * 16 + (lane & 1) * 8;
    const int ch = p32 ^ tr_swz_half(k);
    return (ch >> 2) * 128 + half * 64 + (ch & 3) * 16 + (lane & 1) * 8;
}
template <int COLS, int N>
MOE_DEV void mm_slow_offsets(uint32_t (&o)[N], bool live, uint32_t ld, int krem, int c0, int ncols, int half, int w, int lane) {
    constexpr int RPI = 512 / COLS, LPR = 64 / RPI;
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = 8 * w + RPI * i + lane / LPR, col = mm_slow_col<COLS>(i, half, w, lane);
        o[i] = live && k < krem && c0 + col < ncols ? (uint32_t)k * ld + (uint32_t)(col * 2) : kMmInvalid;
    }
}
// The same of gathered rows, every K-tile anew: so little of it as the products
// of the other waves hide. The part inside a row stays for an item; it is the
// same for requests i and i + 2 (COLS 256) or all (COLS 128, one per half).
// Columns past the end and rows past the group or the array are all ones, which
// the saturating sum keeps.
template <int COLS>
MOE_DEV void mm_gather_cols(uint32_t (&c)[2], int c0, int ncols, int w, int lane) {
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = COLS == 256 ? mm_slow_col<COLS>(i, 0, w, lane) : mm_slow_col<COLS>(0, i, w, lane);
        c[i] = c0 + col < ncols ? (uint32_t)((c0 + col) * 2) : 0xFFFFFFFFu;
    }
}
// byte offset of the row of this lane in request i, from one source row per lane % 8
template <int COLS>
MOE_DEV uint32_t mm_gather_row(uint32_t so, int i, int lane) {
    // (readlanes and masks: an LDS permute would wait behind the fragment
    // reads, and a choice between readlanes becomes a branch)
    constexpr int RPI = 512 / COLS;
    const uint32_t r0 = (uint32_t)__builtin_amdgcn_readlane((int)so, RPI * i), r1 = (uint32_t)__builtin_amdgcn_readlane((int)so, RPI * i + 1);
    if constexpr (COLS == 256) return r0 ^ ((r0 ^ r1) & (uint32_t)((int)((uint32_t)lane << 26) >> 31));
    const uint32_t r2 = (uint32_t)__builtin_amdgcn_readlane((int)so, RPI * i + 2), r3 = (uint32_t)__builtin_amdgcn_readlane((int)so, RPI * i + 3);
    const uint32_t odd = (uint32_t)((int)((uint32_t)lane << 27) >> 31), high = (uint32_t)((int)((uint32_t)lane << 26) >> 31);
    const uint32_t a = r0 ^ ((r0 ^ r1) & odd), b = r2 ^ ((r2 ^ r3) & odd);
    return a ^ ((a ^ b) & high);
}
MOE_DEV uint32_t mm_gather_so(uint32_t src, uint32_t rows, uint32_t ld, int krem, int w, int lane) {
    const uint32_t o = src * ld;
    return (src < rows) & (8 * w + (lane & 7) < krem) ? o : 0xFFFFFFFFu;
}
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void mm_offsets(const MmP& p, const MmWhere& wh, MmReq<NQ>& R, bool edge, bool for_p, bool for_q) {
    constexpr int EB = EL == kElFp8 ? 1 : 2;
    const int lane = mm_fresh(wh.lane), w = wh.w;
    const MmItem& c = R.c;
    if (for_p) {
        if constexpr (MODE == kMmNK) {
            R.pb = p.w + (size_t)c.g * p.w_group + (size_t)c.a0 * p.w_ld + (size_t)(R.kt * 128);
            R.pn = (uint32_t)min(kATile, p.N - c.a0) * p.w_ld - (uint32_t)(R.kt * 128);
            // requests i and i + 2 differ by 16 rows (added when issued); the
            // swizzle of row 32 w + 8 i + lane / 8 depends on i's parity alone
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kb = 16 * ((lane & 7) ^ ((lane >> 4) | (4 * h)));
                R.po[h] = R.live && R.kt * 128 + kb < p.K * EB
                              ? (uint32_t)(32 * w + 8 * h + (lane >> 3)) * p.w_ld + (uint32_t)kb : 0x80000000u;
            }
        } else if constexpr (MODE == kMmKN) {
            R.pb = p.w + (size_t)c.g * p.w_group;
            mm_slow_bounds(R.pb, R.pn, p.w_ld, R.kt * 64, p.K - R.kt * 64, c.a0, p.N);
            mm_slow_offsets<256>(R.po, R.live, p.w_ld, p.K - R.kt * 64, c.a0, p.N, 0, w, lane);
        } else if constexpr (mm_kind(MODE) == kWgrad && (MODE & kGatherX) != 0) {
            if (edge) {
                R.pb = p.x;
                R.pn = R.live ? p.x_bytes : 0u;
                mm_gather_cols<256>(R.pc, c.a0, p.K, w, lane);
            }
            const uint32_t so = mm_gather_so(R.psrc, p.x_rows, p.x_ld, c.nrows - R.kt * 64, w, lane);
            #pragma unroll
            for (int i = 0; i < 4; ++i) R.po[i] = __builtin_elementwise_add_sat(mm_gather_row<256>(so, i, lane), R.pc[i & 1]);
        } else if constexpr (mm_kind(MODE) == kWgrad) {
            R.pb = p.x;
            mm_slow_bounds(R.pb, R.pn, p.x_ld, c.r0 + R.kt * 64, c.nrows - R.kt * 64, c.a0, p.K);
            mm_slow_offsets<256>(R.po, R.live, p.x_ld, c.nrows - R.kt * 64, c.a0, p.K, 0, w, lane);
        }
    }
    if (!for_q) return;
    if constexpr (is_wgrad(MODE) && (MODE & kGatherDy) != 0) {
        if (edge) {
            R.qb = p.dy;
            R.qn = R.live ? p.dy_bytes : 0u;
            mm_gather_cols<128>(R.qc, c.b0, p.N, w, lane);
        }
        const uint32_t so = mm_gather_so(R.qsrc, p.dy_rows, p.dy_ld, c.nrows - R.kt * 64, w, lane);
        #pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const uint32_t row = mm_gather_row<128>(so, i, lane);
            #pragma unroll
            for (int h = 0; h < 2; ++h) R.qo[h][i] = __builtin_elementwise_add_sat(row, R.qc[h]);
        }
    } else if constexpr (is_wgrad(MODE)) {
        R.qb = p.dy;
        mm_slow_bounds(R.qb, R.qn, p.dy_ld, c.r0 + R.kt * 64, c.nrows - R.kt * 64, c.b0, p.N);
        #pragma unroll
        for (int h = 0; h < 2; ++h)
            mm_slow_offsets<128>(R.qo[h], R.live, p.dy_ld, c.nrows - R.kt * 64, c.b0, p.N, h, w, lane);
    } else {
        // gathered rows are addressed from the array's start, a group's own rows from the tile's first
        R.qb = (p.x_src ? p.x : p.x + (size_t)c.r0 * p.x_ld) + (size_t)(R.kt * 128);
        R.qn = (p.x_src ? p.x_bytes : (uint32_t)(c.nrows - 1) * p.x_ld + (uint32_t)(p.K * EB)) - (uint32_t)(R.kt * 128);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            #pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const uint32_t o = R.qo[h][i];
                R.qo[h][i] = R.live && R.kt * 128 + q_chunk<NB>(lane, w, h, i) < p.K * EB ? o : kMmInvalid;
            }
        }
        if constexpr (EL == kElFp8) {
            R.sb = (const uint8_t*)(p.x_src ? p.xs : p.xs + (size_t)c.r0 * p.kb) + R.kt * 4;
            R.sn = R.live ? (p.x_src ? p.xs_bytes : (uint32_t)(c.nrows * p.kb * 4)) - (uint32_t)(R.kt * 4) : 0u;
        }
    }
}

// Step past the K-tile just requested. Inside an item the offsets stay and
// what they count from moves on (scalar additions); they are formed anew for
// an item's first and last K-tile, and for every one of gathered wgrad rows.
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void mm_advance(const MmP& p, const MmTables& tb, const MmWhere& wh, MmReq<NQ>& R) {
    ++R.step;
    if (!R.live) return;
    const int kt = R.kt + 1;
    const bool last = kt == R.c.nk;
    R.kt = last ? 0 : kt;
    if (last) mm_take<EL, MODE, NB>(p, tb, wh, R);
    const bool edge = last || kt == R.c.nk - 1;
    const bool anew_p = edge || (mm_kind(MODE) == kWgrad && (MODE & kGatherX) != 0), anew_q = edge || (MODE & kGatherDy) != 0;
    if (anew_p || anew_q) mm_offsets<EL, MODE, NB>(p, wh, R, edge, anew_p, anew_q);
    if (!anew_p) {
        if constexpr (MODE == kMmNK) { R.pb += 128; R.pn -= 128; }
        else if constexpr (MODE == kMmKN) R.pb += (size_t)p.w_ld * 64;
        else if constexpr (mm_kind(MODE) == kWgrad) R.pb += (size_t)p.x_ld * 64;
    }
    if (!anew_q) {
        if constexpr (is_wgrad(MODE)) R.qb += (size_t)p.dy_ld * 64;
        else { R.qb += 128; R.qn -= 128; }
        if constexpr (EL == kElFp8) { R.sb += 4; R.sn -= 4; }
    }
    if constexpr (is_wgrad(MODE)) {
        if (R.live && R.kt + 1 < R.c.nk) mm_load_src<MODE>(p, wh, R.c, R.kt + 1, R.psrc, R.qsrc);
    }
}
template <int EL, int MODE, int NB, int NQ>
MOE_DEV void mm_start(const MmP& p, const MmTables& tb, const MmWhere& wh, MmReq<NQ>& R) {
    R.round = R.step = R.kt = 0;
    R.c = MmItem{0, 0, 0, 0, 1, 1, -1};
    R.at = -1;
    mm_look<EL, MODE, NB>(p, tb, wh, R);
    mm_take<EL, MODE, NB>(p, tb, wh, R);
    mm_offsets<EL, MODE, NB>(p, wh, R, true, true, true);
    if constexpr (is_wgrad(MODE)) {
        if (R.live && R.c.nk > 1) mm_load_src<MODE>(p, wh, R.c, 1, R.psrc, R.qsrc);
    }
}

// Request number I of the 4 of the a operand.
template <int EL, int MODE, int NB, int I>
MOE_DEV void mm_request_p(const MmP& p, const MmWhere& wh, const MmReq<NB / 4>& R, uint8_t* smem) {
#if defined(__HIP_DEVICE_COMPILE__)          // the host pass has no buffer resources
    using Geo = MmGeom<EL, NB>;
    uint8_t* st = smem + (R.step % Geo::NST) * Geo::Stage;
    const rsrc_t r = make_rsrc(R.pb, R.pn);
    if constexpr (MODE == kMmNK)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void_t*)(st + (32 * wh.w + 8 * I) * 128), 16,
                                                 R.po[I & 1] + (uint32_t)(8 * (I & 2)) * p.w_ld, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void_t*)(st + (8 * wh.w + 2 * I) * 512), 16, R.po[I], 0, 0, 0);
#endif
}
// Request number I of the NQ of one half of the b operand.
template <int EL, int MODE, int NB, int HALF, int I>
MOE_DEV void mm_request_q(const MmWhere& wh, const MmReq<NB / 4>& R, uint8_t* smem) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Geo = MmGeom<EL, NB>;
    uint8_t* st = smem + (R.step % Geo::NST) * Geo::Stage + Geo::QOff;
    const rsrc_t r = make_rsrc(R.qb, R.qn);
    if constexpr (is_wgrad(MODE))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (mm_lds_void_t*)(st + HALF * (kPBytes / 2) + (8 * wh.w + 4 * I) * 256), 16, R.qo[HALF][I], 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void_t*)(st + (q_first<NB>(wh.w, HALF) + 8 * I) * 128), 16,
                                                 R.qo[HALF][I], 0, 0, 0);
#endif
}
// fp8: the scales of this wave's rows of one half (the first 2 NB lanes; the
// others clear the rest of the wave's 256 bytes)
template <int EL, int NB, int HALF>
MOE_DEV void mm_request_s(const MmWhere& wh, const MmReq<NB / 4>& R, uint8_t* smem) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Geo = MmGeom<EL, NB>;
    uint8_t* st = smem + (R.step % Geo::NST) * Geo::Stage;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(R.sb, R.sn),
                                             (mm_lds_void_t*)(st + Geo::SOff + HALF * 2048 + wh.w * 256), 4, R.srow[HALF],
                                             0, 0, 0);
#endif
}
// Requests of turn H: the a operand (turn 1), half 1 - H of the b operand, its scales.
constexpr int mm_turn_p(int mode, int turn) { return turn == 1 && mm_kind(mode) != kWgrad8 ? 4 : 0; }
constexpr int mm_turn_requests(int el, int mode, int nb, int turn) {
    return mm_turn_p(mode, turn) + nb / 4 + (el == kElFp8 ? 1 : 0);
}
// numbers [I0, I1) of them
template <int EL, int MODE, int NB, int H, int I0, int I1, int NQ>
MOE_DEV void mm_requests(const MmP& p, const MmWhere& wh, const MmReq<NQ>& R, uint8_t* smem) {
    if constexpr (I0 < I1) {
        constexpr int NP = mm_turn_p(MODE, H);
        if constexpr (I0 < NP) mm_request_p<EL, MODE, NB, I0>(p, wh, R, smem);
        else if constexpr (I0 < NP + NQ) mm_request_q<EL, MODE, NB, 1 - H, I0 - NP>(wh, R, smem);
        else mm_request_s<EL, NB, 1 - H>(wh, R, smem);
        mm_requests<EL, MODE, NB, H, I0 + 1, I1>(p, wh, R, smem);
    }
}

// wgrad from 8-bit rows: the a operand passes through registers. Every wave
// takes 8 of a K-tile's 64 rows: lane l of piece i holds 8 codes of row
// 8 w + 2 i + l / 32. Codes are requested two K-tiles ahead between the products
// of turn 1 and written to LDS as BF16 values (code * scale, rounded) between
// those of the next turn 0: a wave that did so in its reading turn would hold
// up the other waves' products (8 groups of 16384 x 2816 x 2048: 298 -> 210 us).
struct MmKept {
    int round, kt;                      // K-tile to request next
    bool live;
    MmItem c;
    uint32_t src;                       // source rows of this wave's 8 k, one per lane % 8
    u32x2_t q[4];
    float s[4];
};

template <int MODE, int NB>
MOE_DEV void kept_open(const MmP& p, const MmTables& tb, const MmWhere& wh, MmKept& X) {
    int round = X.round;
    bool live = false;
    MmItem c = X.c;
    for (int item; !live && (item = mm_nth<MODE>(round, wh)) < wh.n_items; ++round) {
        c = mm_decode<kElBf16, MODE, 32 * NB>(p, tb, wh.at, item);
        live = c.nk > 0;
    }
    X.round = round;
    X.live = live;
    X.c = mm_scalar(c);
}
template <int MODE>
MOE_DEV void kept_src(const MmP& p, const MmWhere& wh, MmKept& X) {
    if constexpr ((MODE & kGatherX) != 0) {
        const int k = X.kt * 64 + 8 * wh.w + (wh.lane & 7);
        X.src = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.x_src + X.c.r0, (uint32_t)(X.c.nrows * 4)), k * 4, 0, 0);
    }
}
// request the K-tile's codes and scales (nothing once the items have ended)
template <int MODE>
MOE_DEV void kept_load(const MmP& p, const MmWhere& wh, MmKept& X) {
    const int lane = mm_fresh(wh.lane), w = wh.w;
    const int k0 = X.kt * 64, krem = X.c.nrows - k0, first = X.c.r0 + k0;
    const int col = X.c.a0 + (lane & 31) * 8;
    if constexpr ((MODE & kGatherX) != 0) {
        const rsrc_t rx = make_rsrc(p.x, X.live ? p.x_bytes : 0u), rs = make_rsrc(p.xs, X.live ? p.xs_bytes : 0u);
        const uint32_t cq = col < p.K ? (uint32_t)col : 0xFFFFFFFFu, cs = (uint32_t)(col >> 7) * 4u;
        const uint32_t oq = mm_gather_so(X.src, p.x_rows, p.x_ld, krem, w, lane);
        const uint32_t os = mm_gather_so(X.src, p.x_rows, (uint32_t)p.kb * 4u, krem, w, lane);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            X.q[i] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                rx, __builtin_elementwise_add_sat(mm_gather_row<256>(oq, i, lane), cq), 0, 0));
            // (columns past the end read some scale of the row: their codes are zero)
            X.s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                rs, __builtin_elementwise_add_sat(mm_gather_row<256>(os, i, lane), cs), 0, 0));
        }
    } else {
        // rows past the group are past the resource
        const int rows = __builtin_amdgcn_readfirstlane(max(min(krem, 64), 1));
        const rsrc_t rx = make_rsrc(p.x + (size_t)first * p.x_ld, X.live ? (uint32_t)(rows - 1) * p.x_ld + (uint32_t)p.K : 0u);
        const rsrc_t rs = make_rsrc(p.xs + (size_t)first * p.kb, X.live ? (uint32_t)(rows * p.kb * 4) : 0u);
        const uint32_t k = (uint32_t)(8 * w + (lane >> 5));
        // (opaque: with a visible choice the compiler makes two loads of each,
        // the second waiting for the first)
        uint32_t oq = col < p.K ? k * p.x_ld + (uint32_t)col : 0x80000000u;
        const uint32_t os = (k * (uint32_t)p.kb + (uint32_t)(col >> 7)) * 4u;
        asm("" : "+v"(oq));
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            X.q[i] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rx, oq + (uint32_t)(2 * i) * p.x_ld, 0, 0));
            X.s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, os + (uint32_t)(2 * i) * (uint32_t)p.kb * 4u, 0, 0));
        }
    }
}
// step past the K-tile just requested
template <int MODE, int NB>
MOE_DEV void kept_next(const MmP& p, const MmTables& tb, const MmWhere& wh, MmKept& X) {
    if (!X.live) return;
    const int kt = X.kt + 1;
    const bool last = kt == X.c.nk;
    X.kt = last ? 0 : kt;
    if (last) kept_open<MODE, NB>(p, tb, wh, X);
    if (X.live) kept_src<MODE>(p, wh, X);
}
MOE_DEV void kept_write(const MmWhere& wh, const MmKept& X, uint8_t* st) {
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
}

// wgrad's tables (see MmTables), by the whole workgroup; a barrier must follow.
// Groups go by the length of their parts, longest first (up to 512 groups; with
// more, in their own order: a rank is found by comparing with every other).
MOE_DEV void wgrad_tables(const MmP& p, int tiles, int* at, uint16_t* order, int* slots, uint16_t* len) {
    const int tid = threadIdx.x, lane = tid & 63;
    for (int g = tid; g < p.G; g += kMmThreads) {
        const int nk = group_ktiles(p, g), n = wgrad_parts(p, nk);
        at[g] = (nk + n - 1) / n;                            // for now: the length of its parts
    }
    __syncthreads();
    for (int g = tid; g < p.G; g += kMmThreads) {
        int rank = g;
        if (p.G <= kMmThreads) {
            rank = 0;
            for (int i = 0; i < p.G; ++i) rank += at[i] > at[g] || (at[i] == at[g] && i < g) ? 1 : 0;
        }
        order[rank] = (uint16_t)g;
        len[rank] = (uint16_t)min(at[g], 65000);
    }
    __syncthreads();
    if (tid >= 64) return;
    int units = 0, slot = 0;
    for (int i0 = 0; i0 < p.G; i0 += 64) {
        const int i = i0 + lane;
        const int n = i < p.G ? wgrad_parts(p, group_ktiles(p, order[i])) : 0;
        const int m = i < p.G ? wgrad_parts(p, group_ktiles(p, i)) : 0, sl = m > 1 ? m * tiles : 0;
        const int inc = wave_incl_scan(n), sinc = wave_incl_scan(sl);
        if (i < p.G) {
            at[i] = units + inc - n;
            slots[i] = sl > 0 ? slot + sinc - sl : -1;
        }
        units += __builtin_amdgcn_readlane(inc, 63);
        slot += __builtin_amdgcn_readlane(sinc, 63);
    }
    if (lane == 0) at[p.G] = units;
    if (slot > p.max_slots) {                                // only where groups overlap: nothing is split
        for (int i = lane; i <= p.G; i += 64) {
            at[i] = i;
            if (i < p.G) slots[i] = -1;
        }
    }
}

// Which way of dealing out the items (mm_nth) ends earlier, by the whole
// workgroup: half of the threads add up each way's K-tiles for one workgroup
// of the grid, an item counted as 4 more. len: K-tiles of a part of each group
// (in the order of their items). E.g. 16384 rows in 8 uneven groups, 2816 x
// 2048: 246 -> 226 us.
MOE_DEV int wgrad_dealt(const MmP& p, const int* at, const uint16_t* len, int tiles, int n_items, int grid, int* scratch) {
    const int dealt = threadIdx.x >> 8;
    int longest = 0;
    for (int slot = threadIdx.x & 255; slot < grid; slot += 256) {
        int sum = 0;
        for (int round = 0, item; (item = wgrad_nth(round, n_items, grid, slot, dealt)) < n_items; ++round) {
            const int unit = item / tiles;
            int lo = 0, hi = p.G - 1;                        // the last group with at[group] <= unit
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (at[mid] <= unit) lo = mid;
                else hi = mid - 1;
            }
            sum += len[lo] + 4;
        }
        longest = max(longest, sum);
    }
    longest = (int)wave_umax((uint32_t)longest);
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = longest;
    __syncthreads();
    const int a = max(max(scratch[0], scratch[1]), max(scratch[2], scratch[3]));
    const int b = max(max(scratch[4], scratch[5]), max(scratch[6], scratch[7]));
    return __builtin_amdgcn_readfirstlane(b < a ? 1 : 0);
}

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

template <int EL, int MODE, int NB>
__global__ __launch_bounds__(kMmThreads, 1)
void grouped_mm_kernel(MmP p) {
    using Geo = MmGeom<EL, NB>;
    constexpr int BT = Geo::BT, NST = Geo::NST;
    constexpr bool P_TR = MODE != kMmNK, Q_TR = is_wgrad(MODE);
    static_assert(!Q_TR || BT == 256, "the slow form is laid out for 256 values");

    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* const tab = (int*)(smem + NST * Geo::Stage + kMmOut);
    uint16_t* const order = (uint16_t*)(tab + 2 * p.G + 1);
    const MmTables tb{tab, order, tab + p.G + 1};

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, j = lane & 15;
    const int wi = w & 3, ti = w >> 2;
    const bool lead = w < 4;                                 // the half that multiplies first, half a step ahead

    const int na = is_wgrad(MODE) ? p.K : p.N;               // extent of the contiguous output axis
    const int at = (na + kATile - 1) / kATile;
    int n_items;
    if constexpr (is_wgrad(MODE)) {
        wgrad_tables(p, at * ((p.N + BT - 1) / BT), tab, order, tab + p.G + 1, (uint16_t*)(smem + NST * Geo::Stage));
        __syncthreads();
        n_items = __builtin_amdgcn_readfirstlane(tab[p.G]) * at * ((p.N + BT - 1) / BT);
    } else {
        if (w == 0) mm_passes(p, BT, at, lane, tab);
        __syncthreads();
        n_items = __builtin_amdgcn_readfirstlane(tab[p.G]) * at;
    }
    const int grid = gridDim.x;
    const int slot = (grid % 8 == 0) ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
    if (slot >= n_items) return;

    int dealt = 0;
    if constexpr (is_wgrad(MODE)) {
        if (n_items > grid && n_items <= 16 * grid)            // (with more rounds the last one matters less)
            dealt = wgrad_dealt(p, tab, (const uint16_t*)(smem + NST * Geo::Stage), at * ((p.N + BT - 1) / BT), n_items, grid,
                                (int*)smem);
        __syncthreads();                                     // (before anything is staged there)
    }
    const MmWhere wh{n_items, at, grid, slot, lane, w, dealt};

    // ---------------------------------------------------------- fragments
    constexpr int NU = Geo::NU, NQ = Geo::NQ;
    i32x4 fp[2][4], fq[2][NU];
    float fs[NU], fw = 0.f;
    uint32_t fwv = 0, fwn = 0;          // fp8: weight scales of this item's and the next item's K-tiles
    auto load_fw = [&](const MmItem& c, int kt) __attribute__((always_inline)) {
        const float* ws = p.ws + ((size_t)c.g * p.nb + min((c.a0 + 64 * wi) >> 7, p.nb - 1)) * p.kb;
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(make_rsrc(ws, (uint32_t)(p.kb * 4)), (kt + lane) * 4, 0, 0);
    };
    // 8 k of one value (k = 32 s + 8 q ..) from rows of `rb` bytes: at o + k's row
    auto read_slow = [&](const uint8_t* st, int o, int rb) __attribute__((always_inline)) {
        i32x4 v;
        const u32x2_t l = read_tr16((const mm_lds_s16x4*)(st + o)), h = read_tr16((const mm_lds_s16x4*)(st + o + 4 * rb));
        v[0] = (int)l.x; v[1] = (int)l.y; v[2] = (int)h.x; v[3] = (int)h.y;
        return v;
    };
    auto read_frags = [&](int step, int turn, const MmItem& c, int kt) __attribute__((always_inline)) {
        const uint8_t* st = smem + (step % NST) * Geo::Stage;
        #pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int ch = ((4 * s + q) ^ ((j >> 1) & 7)) * 16;
            const int k = 32 * s + 8 * q + (j >> 2);
            if (turn == 0) {
                #pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (P_TR)
                        fp[s][t] = read_slow(st, k * 512 + ((4 * wi + t) ^ ((j >> 2) | (q << 2))) * 32 + (j & 3) * 8, 512);
                    else
                        fp[s][t] = *(const i32x4*)(st + (64 * wi + 16 * t + j) * 128 + ch);
                }
            }
            #pragma unroll
            for (int u = 0; u < NU; ++u) {
                if constexpr (Q_TR)
                    fq[s][u] = read_slow(st + Geo::QOff + turn * (kPBytes / 2),
                                         k * 256 + ((4 * ti + u) ^ ((j >> 2) | ((q & 1) << 2))) * 32 + (j & 3) * 8, 256);
                else
                    fq[s][u] = *(const i32x4*)(st + Geo::QOff + (16 * NB * ti + 16 * (turn * NU + u) + j) * 128 + ch);
            }
        }
        if constexpr (EL == kElFp8) {
            #pragma unroll
            for (int u = 0; u < NU; ++u)
                fs[u] = *(const float*)(st + Geo::SOff + turn * 2048 +
                                        (ti * 4 + (16 * u + j) / Geo::HRows) * 256 + ((16 * u + j) % Geo::HRows) * 4);
            if (turn == 0) {
                // a block row's scales, 64 K-tiles to a register: one per lane
                // (used here, so that the wait for it is here: behind the
                // branch it would drain the requests of every K-tile)
                if ((kt & 63) == 0 && kt > 0) {
                    fwv = load_fw(c, kt);
                    asm volatile("" : "+v"(fwv));
                }
                fw = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)fwv, kt & 63));
            }
        }
    };

    f32x4 acc[NB][4];
    MmReq<NQ> R;

    f32x4 d[4];                         // fp8: products not yet added, and their scales
    float sc = 0.f;

    MmKept kept;
    int step = 0;

    // the products of one turn, with the turn's requests between them
    auto multiply = [&](auto turn) __attribute__((always_inline)) {
        constexpr int h = decltype(turn)::value;
        constexpr int NR = mm_turn_requests(EL, MODE, NB, h);
        if constexpr (EL == kElFp8) {
            // the K-tile is one block of 128: its products go to cleared
            // registers and are added with the two scales' product, four
            // instructions behind: 4 additions in the shadow of each matrix
            // instruction, the registers then being the next one's; a turn's
            // last b tile in the next turn (or after the item's last). The
            // empty asm statements order the two (the additions of the b tile
            // before, b tile u's products); left alone the compiler starts
            // every product first and spills the accumulators.
            static_for<NU>([&](auto uu) __attribute__((always_inline)) {
                constexpr int u = decltype(uu)::value, before = u > 0 ? h * NU + u - 1 : (1 - h) * NU + NU - 1;
                f32x4* a = acc[before];
                #pragma unroll
                for (int t = 0; t < 4; ++t) {
                    #pragma unroll
                    for (int v = 0; v < 4; ++v) a[t][v] = fmaf(d[t][v], sc, a[t][v]);
                    d[t] = mfma_fp8(fp[0][t], fp[1][t], fq[0][u], fq[1][u], f32x4{0.f, 0.f, 0.f, 0.f});
                }
                mm_requests<EL, MODE, NB, h, (NR * u) / NU, (NR * (u + 1)) / NU>(p, wh, R, smem);
                #pragma unroll
                for (int t = 0; t < 4; ++t) {
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                }
                asm volatile("" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
                sc = fs[u] * fw;
                asm volatile("" : "+v"(sc) : "v"(d[0]), "v"(d[1]), "v"(d[2]), "v"(d[3]));
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            constexpr bool kKept = mm_kind(MODE) == kWgrad8;
            mm_requests<EL, MODE, NB, h, 0, NR>(p, wh, R, smem);
            if constexpr (kKept && h == 0) kept_write(wh, kept, smem + ((step + 1) % NST) * Geo::Stage);
            if constexpr (kKept && h == 1) kept_load<MODE>(p, wh, kept);
            #pragma unroll
            for (int s = 0; s < 2; ++s)
                #pragma unroll
                for (int u = 0; u < NU; ++u)
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[h * NU + u][t] = mfma16x16x32<EL>(fp[s][t], fq[s][u], acc[h * NU + u][t]);
            if constexpr (kKept && h == 0) {
                #pragma unroll
                for (int i = 0; i < 4; ++i) {                // a piece's conversions and its write
                    if (i < NR) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                    #pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                    }
                    __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                }
            } else {
                constexpr int NM = NR + (kKept ? 8 : 0);     // requests in all
                #pragma unroll
                for (int i = 0; i < NM; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 8 * NU / (NM + 1), 0);
                    __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                }
            }
        }
    };

    auto clear = [&]() __attribute__((always_inline)) {
        #pragma unroll
        for (int u = 0; u < NB; ++u)
            #pragma unroll
            for (int t = 0; t < 4; ++t) acc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (EL == kElFp8) {
            sc = 0.f;
            #pragma unroll
            for (int t = 0; t < 4; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
    // Sums stay in 32 bits until here: the one rounding to the output's type.
    // The values pass through LDS, 16 rows x 64 bytes at a time (two tiles in 16
    // bits or one in 32), so that 4 neighbouring lanes store 64 bytes of a row:
    // stored as they come out of the products, 16 neighbouring lanes hold 16
    // rows, and an item of any length took 3.6 us longer. A wave's LDS accesses
    // are done in order, so one piece of LDS serves all its passes without waits.
    // Every lane stores, past an edge outside the resource (dropped), so a wave
    // always issues 2 NB (4 NB) stores and the next K-tile's waits can leave them
    // in flight.
    // (the variants are compiled apart: with a run-time choice inside, the waits
    // of the adding variant's loads end up before every store of the others)
    auto store = [&](const MmItem& c, auto f16_, auto f32_, auto add_) __attribute__((always_inline)) {
        constexpr int f16 = decltype(f16_)::value, es = decltype(f32_)::value ? 4 : 2;
        constexpr bool add = decltype(add_)::value;
        // a part of a split group goes to its tile of partial sums
        const bool partial = is_wgrad(MODE) && c.slot >= 0;
        const size_t ld = partial ? kATile : (is_wgrad(MODE) ? (size_t)p.K : p.out_ld);
        const size_t row0 = is_wgrad(MODE) ? (size_t)c.g * p.N + c.b0 : (size_t)c.r0;
        const int rows = partial ? BT : (is_wgrad(MODE) ? min(BT, p.N - c.b0) : c.nrows);
        const int cols = partial ? kATile : min(kATile, na - c.a0);
        uint8_t* base = partial ? (uint8_t*)(p.partial + (size_t)c.slot * (kATile * BT)) : p.out + (row0 * ld + c.a0) * es;
        const rsrc_t r = make_rsrc(base, (uint32_t)(((size_t)(rows - 1) * ld + cols) * es));
        // rows past the tile's are past the resource by themselves; values past
        // the operand's end (a partial tile only) are sent there
        constexpr bool pair = es == 2 && !add;
        const int fresh = mm_fresh(lane), wr = fresh & 15, wq = fresh >> 4, rr = fresh >> 2, rc = fresh & 3;
        uint8_t* const out = smem + NST * Geo::Stage + w * (kMmOut / 8);
        uint8_t* const put = out + wr * 64;                  // 16-byte chunks swizzled by row / 4
        const uint8_t* const got = out + rr * 64 + (rc ^ ((rr >> 2) & 3)) * 16;
        const int a0 = 64 * wi + (pair ? 8 : 4) * rc;
        uint32_t o = (uint32_t)((16 * NB * ti + rr) * (int)ld + a0) * (uint32_t)es;
        #pragma unroll
        for (int u = 0; u < NB; ++u) {
            #pragma unroll
            for (int t = 0; t < 4; t += pair ? 2 : 1) {
                const uint32_t ot = a0 + 16 * t < cols ? o + (uint32_t)(16 * t * es) : kMmInvalid;
                if constexpr (pair) {
                    #pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f32x4& v = acc[u][t + k];
                        *(u32x2_t*)(put + ((2 * k + (wq >> 1)) ^ ((wr >> 2) & 3)) * 16 + (wq & 1) * 8) =
                            u32x2_t{pack16(v[0], v[1], f16), pack16(v[2], v[3], f16)};
                    }
                    __builtin_amdgcn_raw_buffer_store_b128(*(const i32x4*)got, r, ot, 0, 0);
                    continue;
                }
                *(f32x4*)(put + (wq ^ ((wr >> 2) & 3)) * 16) = acc[u][t];
                f32x4 v = *(const f32x4*)got;
                if constexpr (es == 4) {
                    if constexpr (add) {
                        const f32x4 e = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, ot, 0, 0));
                        v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]};
                    }
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), r, ot, 0, 0);
                } else {
                    if constexpr (add) {
                        const u32x2_t e = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, ot, 0, 0));
                        v[0] += lo16(e.x, f16); v[1] += hi16(e.x, f16);
                        v[2] += lo16(e.y, f16); v[3] += hi16(e.y, f16);
                    }
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{pack16(v[0], v[1], f16), pack16(v[2], v[3], f16)}, r, ot, 0, 0);
                }
            }
            o += (uint32_t)(16 * (int)ld * es);
            asm volatile("" : "+v"(o));                      // one row of tiles at a time: no offsets kept for all
        }
    };

    // --------------------------------------------------------------- loop
    if constexpr (mm_kind(MODE) == kWgrad8) {
        kept.round = kept.kt = 0;
        kept.src = 0;
        kept.c = MmItem{0, 0, 0, 0, 1, 1, -1};
        kept_open<MODE, NB>(p, tb, wh, kept);
        if (kept.live) kept_src<MODE>(p, wh, kept);
        kept_load<MODE>(p, wh, kept);
        kept_write(wh, kept, smem);
        kept_next<MODE, NB>(p, tb, wh, kept);
        kept_load<MODE>(p, wh, kept);
    }
    mm_start<EL, MODE, NB>(p, tb, wh, R);
    #pragma unroll 1
    for (int i = 0; i < NST; ++i) {     // the last one's second b half follows in the first turn
        mm_requests<EL, MODE, NB, 1, 0, mm_turn_requests(EL, MODE, NB, 1)>(p, wh, R, smem);
        if (i < NST - 1) {
            mm_requests<EL, MODE, NB, 0, 0, mm_turn_requests(EL, MODE, NB, 0)>(p, wh, R, smem);
            mm_advance<EL, MODE, NB>(p, tb, wh, R);
        }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    bare_barrier();
    if (!lead) bare_barrier();

    // Turn 1 requests K-tile NST ahead, turn 0 the second b half of NST - 1
    // ahead, both between the products. Waits: the newer requests left in flight when the
    // ones that the next turn reads have landed. Waves 0-3 wait after their
    // products, waves 4-7 (half a turn later, before this turn's requests) after
    // their reads. Requests not counted (row sources, stores) only make a wait
    // longer; once a stream has ended its requests still count. In the first
    // NST - 1 K-tiles after an item's stores the requests waited for are older
    // than the stores, which then count as newer.
    constexpr int KEPT = mm_kind(MODE) == kWgrad8 ? 8 : 0;            // requests of the 8-bit rows in turn 1
    constexpr int L1 = mm_turn_requests(EL, MODE, NB, 1), L2 = mm_turn_requests(EL, MODE, NB, 0);
    constexpr int STORES = is_wgrad(MODE) ? 4 * NB : 2 * NB;
    int stored = 0;                                          // K-tiles whose waits leave the last stores in flight
    auto wait_for = [&](auto n) __attribute__((always_inline)) {
        constexpr int N = decltype(n)::value;
        static_assert(N + STORES < 64, "vmcnt");
        if (stored > 0) __builtin_amdgcn_s_waitcnt(waitcnt_imm(N + STORES, 15));
        else __builtin_amdgcn_s_waitcnt(waitcnt_imm(N, 15));
    };
    if constexpr (EL == kElFp8) fwn = load_fw(mm_scalar(mm_decode<EL, MODE, 32 * NB>(p, tb, at, slot)), 0);
    for (int round = 0, item; (item = mm_nth<MODE>(round, wh)) < n_items; ++round) {
        // the item is the one being requested, unless items are very short
        const MmItem c = R.live && R.at == item ? R.c : mm_scalar(mm_decode<EL, MODE, 32 * NB>(p, tb, at, item));
        if constexpr (EL == kElFp8) {   // the next item's scales are loaded an item ahead
            fwv = fwn;
            asm volatile("" : "+v"(fwv));
            if (item + grid < n_items) fwn = load_fw(mm_scalar(mm_decode<EL, MODE, 32 * NB>(p, tb, at, item + grid)), 0);
        }
        clear();
        #pragma unroll 1
        for (int kt = 0; kt < c.nk; ++kt, ++step) {
            static_for<2>([&](auto turn) __attribute__((always_inline)) {
                constexpr int h = decltype(turn)::value;
                read_frags(step, h, c, kt);
                if constexpr (mm_kind(MODE) == kWgrad8 && h == 0) kept_next<MODE, NB>(p, tb, wh, kept);
                if constexpr (h == 1) mm_advance<EL, MODE, NB>(p, tb, wh, R);
                // the reads end before this wave's products and so a turn before
                // the stage is requested again
                if (!lead) wait_for(std::integral_constant<int, h ? (NST - 2) * (L1 + KEPT) + (NST - 1) * L2
                                                                  : (NST - 1) * (L1 + KEPT) + (NST - 2) * L2>{});
                bare_barrier();
                __builtin_amdgcn_s_setprio(1);
                multiply(turn);
                __builtin_amdgcn_s_setprio(0);
                if (lead) wait_for(std::integral_constant<int, (NST - 1) * (L1 + KEPT + L2)>{});
                // (writes to LDS are done before the barrier)
                if constexpr (mm_kind(MODE) == kWgrad8 && h == 0) __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
                bare_barrier();
            });
            --stored;
        }
        if constexpr (EL == kElFp8) {
            #pragma unroll
            for (int t = 0; t < 4; ++t)
                #pragma unroll
                for (int v = 0; v < 4; ++v) acc[NB - 1][t][v] = fmaf(d[t][v], sc, acc[NB - 1][t][v]);
        }
        // (an item without K-tiles stores between two others' stores: not
        // counted, nor the fewer stores of a weight gradient in 16 bits)
        stored = is_wgrad(MODE) && (p.accumulate || c.nk == 0 || (c.slot < 0 && !p.out_f32)) ? 0 : NST - 1;
        if (!is_wgrad(MODE) || c.nk > 0 || !p.accumulate) {
            constexpr std::integral_constant<int, EL == kElF16> same{};
            constexpr std::true_type yes{};
            constexpr std::false_type no{};
            if constexpr (EL == kElFp8) {
                if (p.out_f16) store(c, std::integral_constant<int, 1>{}, no, no);
                else store(c, same, no, no);
            } else if constexpr (is_wgrad(MODE)) {
                if (c.slot >= 0 || (p.out_f32 && !p.accumulate)) store(c, same, yes, no);
                else if (p.out_f32) store(c, same, yes, yes);
                else if (p.accumulate) store(c, same, no, yes);
                else store(c, same, no, no);
            } else {
                store(c, same, no, no);
            }
        }
    }
    if (lead) bare_barrier();
}

template <int EL, int MODE, int NB>
int launch_mm(const MmP& p, int max_items, hipStream_t stream) {
    using Geo = MmGeom<EL, NB>;
    const size_t lds = Geo::Lds(p.G, is_wgrad(MODE));
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

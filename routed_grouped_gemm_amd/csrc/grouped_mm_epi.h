// Epilogues of the 16-bit grouped products, on a workgroup's accumulators as
// the matrix instructions leave them: lane l of a wave holds, for each tile (u,
// t), 4 consecutive columns 4 (l / 16) .. of row l % 16. Internal to libmoe.
//
//   forward    z = acc + b;  y = residual + w_r a(clamp z), or for a gated product
//              y = residual + w_r a(clamp g) clamp u;  z itself on request
//   gradient   acc = dh:  dg = dh w clamp(u) a'(clamp g) [|g| <= limit],
//              du = dh w a(clamp g) [|u| <= limit],  h = w a(clamp g) clamp u,
//              and the row's sum of dh a clamp u over the wave's 64 columns
//
// Everything is fp32 up to the one rounding of each output. 16-bit rows are
// loaded and stored 64 bytes of a row at a time by 4 neighbouring lanes and
// exchanged with the accumulators' layout through 1 KiB of LDS a wave (16 rows x
// 32 columns; a wave's LDS accesses are done in order, so it needs no waits).
#pragma once
#include "epilogue_act.h"
#include "grouped_mm.h"

namespace {

// one wave's exchange place: 16 rows of four 16-byte chunks, swizzled by row / 4
struct EpiSwap {
    uint8_t* put[2];                                         // two tiles' 4 columns of this lane's row
    uint8_t* got;                                            // 8 columns of row lane / 4
    MOE_DEV EpiSwap(uint8_t* piece, int lane) {
        const int r = lane & 15, q = lane >> 4, rr = lane >> 2, rc = lane & 3;
        #pragma unroll
        for (int k = 0; k < 2; ++k) put[k] = piece + r * 64 + ((2 * k + (q >> 1)) ^ ((r >> 2) & 3)) * 16 + (q & 1) * 8;
        got = piece + rr * 64 + (rc ^ ((rr >> 2) & 3)) * 16;
    }
    MOE_DEV i32x4 gather(u32x2_t a, u32x2_t b) const {
        *(u32x2_t*)put[0] = a;
        *(u32x2_t*)put[1] = b;
        return *(const i32x4*)got;
    }
    MOE_DEV void spread(const i32x4& v, u32x2_t& a, u32x2_t& b) const {
        *(i32x4*)got = v;
        a = *(const u32x2_t*)put[0];
        b = *(const u32x2_t*)put[1];
    }
};

// A tile's rows of a 16-bit array, seen by the lanes that load and store it, one
// row of tiles after another.
struct EpiRows {
    rsrc_t r;
    uint32_t o, step;                                        // byte offset of this lane's row and 8 columns, bytes of 16 rows
    int a, cols;
    MOE_DEV EpiRows(const void* base, size_t ld, const MmItem& c, size_t col0, int row, int col, int ncols) {
        r = make_rsrc((const uint8_t*)base + ((size_t)c.r0 * ld + col0) * 2, (uint32_t)(((size_t)(c.nrows - 1) * ld + ncols) * 2));
        o = (uint32_t)row * (uint32_t)(ld * 2) + (uint32_t)col * 2;
        step = (uint32_t)(ld * 32);
        a = col;
        cols = ncols;
    }
    // columns past the tile's, 16 t on from this lane's, are sent past the resource (rows past it are there by themselves)
    MOE_DEV uint32_t at(int t) const { return a + 16 * t < cols ? o + (uint32_t)(32 * t) : kMmInvalid; }
    MOE_DEV i32x4 load(int t) const { return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at(t), 0, 0)); }
    MOE_DEV void store(int t, const i32x4& v) const { __builtin_amdgcn_raw_buffer_store_b128(v, r, at(t), 0, 0); }
    // (opaque: otherwise the offsets of all rows are kept in registers)
    MOE_DEV void next() {
        o += step;
        asm volatile("" : "+v"(o));
    }
};
// Ends a row of tiles: nothing of the next is moved before it, or the registers
// would not hold what is started early.
MOE_DEV void epi_row_end() { __builtin_amdgcn_sched_barrier(0); }

template <int F16>
MOE_DEV u32x2_t epi_pack(const f32x4& v) { return u32x2_t{pack16(v[0], v[1], F16), pack16(v[2], v[3], F16)}; }
template <int F16>
MOE_DEV f32x4 epi_unpack(const u32x2_t& v) { return f32x4{lo16(v.x, F16), hi16(v.x, F16), lo16(v.y, F16), hi16(v.y, F16)}; }

template <int EL, int NB, int EPI>
MOE_DEV void epi_forward(const MmP& p, const MmItem& c, int wi, int ti, int lane, uint8_t* piece, f32x4 (&acc)[NB][4]) {
    constexpr bool GATED = EPI == kEpiGated;
    constexpr int F16 = EL == kElF16, NT = GATED ? 2 : 4;
    const int q = lane >> 4, j = lane & 15;
    const int colw = (GATED ? 32 : 64) * wi, row0 = 16 * NB * ti, lrow = row0 + (lane >> 2), lcol = colw + 8 * (lane & 3);
    const int cols = min(a_tile(EPI), p.N - c.a0);
    const EpiSwap swap(piece, lane);
    f32x4 bias[4];
    #pragma unroll
    for (int t = 0; t < 4; ++t) bias[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (p.bias) {
        const float* b = p.bias + (size_t)c.g * (GATED ? 2 * p.N : p.N) + c.a0;
        #pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int up = GATED && t >= 2 ? 1 : 0, col = colw + 16 * (up ? t - 2 : t) + 4 * q;
            bias[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                make_rsrc(b + (size_t)up * p.N, (uint32_t)(cols * 4)), col < cols ? (uint32_t)(col * 4) : kMmInvalid, 0, 0));
        }
    }
    float w[NB];
    #pragma unroll
    for (int u = 0; u < NB; ++u) w[u] = 1.f;
    if (p.row_w) {
        const rsrc_t rw = make_rsrc(p.row_w + c.r0, (uint32_t)(c.nrows * 4));
        #pragma unroll
        for (int u = 0; u < NB; ++u) w[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, (row0 + 16 * u + j) * 4, 0, 0));
    }
    // (the variants are compiled apart: a run-time choice around loads or
    // stores makes the waits of all as long as the longest)
    auto rows = [&](auto keep_, auto res_) __attribute__((always_inline)) {
        constexpr bool KEEP = decltype(keep_)::value, RES = decltype(res_)::value;
        constexpr int AHEAD = 2;                             // rows of tiles whose residual is on its way
        EpiRows out(p.out, p.out_ld, c, (size_t)c.a0, lrow, lcol, cols);
        EpiRows pg(KEEP ? p.pre : p.out, KEEP ? p.pre_ld : p.out_ld, c, (size_t)c.a0, lrow, lcol, cols);
        EpiRows pu(KEEP ? p.pre : p.out, KEEP ? p.pre_ld : p.out_ld, c, (size_t)c.a0 + (KEEP && GATED ? p.N : 0), lrow, lcol, cols);
        EpiRows res(RES ? p.res : p.out, RES ? p.res_ld : p.out_ld, c, (size_t)c.a0, lrow, lcol, cols);
        i32x4 rv[AHEAD + 1][NT / 2];
        auto request = [&](int to) __attribute__((always_inline)) {
            #pragma unroll
            for (int t = 0; t < NT; t += 2) rv[to][t / 2] = res.load(t);
            res.next();
        };
        if constexpr (RES) {
            #pragma unroll
            for (int u = 0; u < AHEAD; ++u) request(u);
        }
        static_for<NB>([&](auto uu) __attribute__((always_inline)) {
            constexpr int u = decltype(uu)::value;
            if constexpr (RES && u + AHEAD < NB) request((u + AHEAD) % (AHEAD + 1));
            f32x4 (&z)[4] = acc[u];
            #pragma unroll
            for (int t = 0; t < 4; ++t)
                #pragma unroll
                for (int i = 0; i < 4; ++i) z[t][i] += bias[t][i];
            if constexpr (KEEP) {
                pg.store(0, swap.gather(epi_pack<F16>(z[0]), epi_pack<F16>(z[1])));
                const i32x4 v = swap.gather(epi_pack<F16>(z[2]), epi_pack<F16>(z[3]));
                if constexpr (GATED) pu.store(0, v);
                else pg.store(2, v);
                pg.next();
                pu.next();
            }
            if (p.limit > 0.f) {
                #pragma unroll
                for (int t = 0; t < 4; ++t)
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) z[t][i] = epi_clamp(z[t][i], p.limit);
            }
            with_act(p.act, [&](auto act) __attribute__((always_inline)) {
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = epi_act<decltype(act)::value>(z[t][i], p.beta);
                        z[t][i] = (GATED ? a * z[(t + 2) & 3][i] : a) * w[u];
                    }
            });
            #pragma unroll
            for (int t = 0; t < NT; t += 2) {
                if constexpr (RES) {
                    u32x2_t a, b;
                    swap.spread(rv[u % (AHEAD + 1)][t / 2], a, b);
                    const f32x4 ra = epi_unpack<F16>(a), rb = epi_unpack<F16>(b);
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) { z[t][i] += ra[i]; z[t + 1][i] += rb[i]; }
                }
                out.store(t, swap.gather(epi_pack<F16>(z[t]), epi_pack<F16>(z[t + 1])));
            }
            out.next();
            epi_row_end();
        });
    };
    if (p.pre) {
        if (p.res) rows(std::true_type{}, std::true_type{});
        else rows(std::true_type{}, std::false_type{});
    } else if (p.res) {
        rows(std::false_type{}, std::true_type{});
    } else {
        rows(std::false_type{}, std::false_type{});
    }
}

// The gradients at one (gate, up) pair; returns the term of the row's sum.
template <int ACT, bool GATED>
MOE_DEV float epi_grad_one(float dh, float w, float g, float u, float beta, float limit, float& dg, float& du, float& h) {
    const float gc = epi_clamp(g, limit), uc = GATED ? epi_clamp(u, limit) : 1.f;
    float a, da;
    epi_act_grad<ACT>(gc, beta, a, da);
    const float d = dh * w;
    dg = GATED ? d * uc * da * epi_inside(g, limit) : d * da * epi_inside(g, limit);
    du = GATED ? d * a * epi_inside(u, limit) : 0.f;
    const float au = GATED ? a * uc : a;
    h = au * w;
    return dh * au;
}

template <int EL, int NB>
MOE_DEV void epi_grad(const MmP& p, const MmItem& c, int wi, int ti, int lane, uint8_t* piece, f32x4 (&acc)[NB][4]) {
    constexpr int F16 = EL == kElF16;
    const int q = lane >> 4, j = lane & 15;
    const int row0 = 16 * NB * ti, lrow = row0 + (lane >> 2), lcol = 64 * wi + 8 * (lane & 3);
    const int cols = min(kATile, p.N - c.a0);
    const EpiSwap swap(piece, lane);
    float w[NB];
    #pragma unroll
    for (int u = 0; u < NB; ++u) w[u] = 1.f;
    if (p.row_w) {
        const rsrc_t rw = make_rsrc(p.row_w + c.r0, (uint32_t)(c.nrows * 4));
        #pragma unroll
        for (int u = 0; u < NB; ++u) w[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, (row0 + 16 * u + j) * 4, 0, 0));
    }
    auto all = [&](auto act, auto gated) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        constexpr bool GATED = decltype(gated)::value;
        constexpr int AHEAD = 2;                             // pairs of tiles whose pre-activations are on their way
        const size_t wide = GATED ? 2 * (size_t)p.N : (size_t)p.N;
        EpiRows pg(p.pre, p.pre_ld, c, (size_t)c.a0, lrow, lcol, cols);
        EpiRows pu(p.pre, p.pre_ld, c, (size_t)c.a0 + (GATED ? p.N : 0), lrow, lcol, cols);
        EpiRows og(p.out, wide, c, (size_t)c.a0, lrow, lcol, cols);
        EpiRows ou(p.out, wide, c, (size_t)c.a0 + (GATED ? p.N : 0), lrow, lcol, cols);
        EpiRows oh(p.h ? p.h : p.out, (size_t)p.N, c, (size_t)c.a0, lrow, lcol, cols);
        i32x4 vg[AHEAD + 1], vu[AHEAD + 1];
        auto request = [&](auto nn) __attribute__((always_inline)) {
            constexpr int n = decltype(nn)::value, to = n % (AHEAD + 1), t = n % 2 * 2;
            vg[to] = pg.load(t);
            if constexpr (GATED) vu[to] = pu.load(t);
            if constexpr (t == 2) {
                pg.next();
                pu.next();
            }
        };
        static_for<AHEAD>(request);
        float sum = 0.f;
        static_for<2 * NB>([&](auto nn) __attribute__((always_inline)) {
            constexpr int n = decltype(nn)::value, u = n / 2, t = n % 2 * 2, from = n % (AHEAD + 1);
            if constexpr (n + AHEAD < 2 * NB) request(std::integral_constant<int, n + AHEAD>{});
            u32x2_t ga, gb, ua{}, ub{};
            swap.spread(vg[from], ga, gb);
            if constexpr (GATED) swap.spread(vu[from], ua, ub);
            u32x2_t dg[2], du[2], h[2];
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4 g = epi_unpack<F16>(k ? gb : ga), up = epi_unpack<F16>(k ? ub : ua);
                f32x4 vdg, vdu, vh;
                float part = 0.f;
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b, o;
                    part += epi_grad_one<ACT, GATED>(acc[u][t + k][i], w[u], g[i], up[i], p.beta, p.limit, a, b, o);
                    vdg[i] = a; vdu[i] = b; vh[i] = o;
                }
                dg[k] = epi_pack<F16>(vdg);
                if constexpr (GATED) du[k] = epi_pack<F16>(vdu);
                h[k] = epi_pack<F16>(vh);
                // (past the end an infinity of dy times the absent weights is NaN: left out)
                sum += 64 * wi + 16 * (t + k) + 4 * q < cols ? part : 0.f;
            }
            og.store(t, swap.gather(dg[0], dg[1]));
            if constexpr (GATED) ou.store(t, swap.gather(du[0], du[1]));
            if (p.h) oh.store(t, swap.gather(h[0], h[1]));
            if constexpr (t == 2) {
                og.next();
                ou.next();
                oh.next();
                sum += __shfl_xor(sum, 16, 64);
                sum += __shfl_xor(sum, 32, 64);
                const int row = row0 + 16 * u + j;
                if (p.dw_part && lane < 16 && row < c.nrows)
                    p.dw_part[(size_t)(c.a0 / kATile * 4 + wi) * p.R_max + c.r0 + row] = sum;
                sum = 0.f;
            }
            epi_row_end();
        });
    };
    with_act(p.act, [&](auto act) __attribute__((always_inline)) {
        if (p.gated) all(act, std::true_type{});
        else all(act, std::false_type{});
    });
}

}  // namespace

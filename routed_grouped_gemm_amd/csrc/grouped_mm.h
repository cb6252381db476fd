// Pieces shared by the grouped-product kernels (grouped_mm.hip, the LDS-tiled
// kernel, and grouped_mm_rows.hip, the weight-streaming kernel for few rows):
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
};

// Rows [lo, hi) of group g, held inside [0, R_max) whatever the offsets say.
MOE_DEV void group_rows(const MmP& p, int g, int& lo, int& hi) {
    lo = min(max(p.offsets[g], 0), p.R_max);
    hi = min(max(p.offsets[g + 1], lo), p.R_max);
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
// halves of a lane's operand, see mfma16x16x128)
MOE_DEV f32x4 mfma_fp8(const i32x4& alo, const i32x4& ahi, const i32x4& blo, const i32x4& bhi, f32x4 c) {
    const i32x8 a = __builtin_shufflevector(alo, ahi, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 b = __builtin_shufflevector(blo, bhi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, MFMA_FMT_FP8, MFMA_FMT_FP8, 0, 0, 0, 0);
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

}  // namespace

// Argument checks shared by the C entries of the grouped products (mm_api.cpp,
// mm_act_api.cpp). Host code, internal to libmoe.
#pragma once
#include <math.h>

#include "moe_internal.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

inline int32_t hip_status(int e) { return e == 0 ? MOE_OK : MOE_ERR_HIP; }

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// bound on an array that gathered rows are read from: 32-bit byte offsets, the
// last 4 MiB of which mark rows that are not there
constexpr int64_t kGatherBytes = (1ll << 32) - (1ll << 22);

// largest leading dimension: 256 rows of a tile stay below 2 GiB
constexpr int32_t kMaxLd = 1 << 22;

// bound on the rows of a call: row counts rounded up to a tile and the byte
// sizes of source arrays stay inside signed 32 bits
constexpr int32_t kMaxRows = MOE_MM_MAX_ROWS;

inline int32_t check_dims(int32_t R_max, int32_t N, int32_t K, int32_t G, int kmult) {
    if (R_max < 0 || R_max > kMaxRows || G < 1 || G > MOE_MAX_EXPERTS + 1) return MOE_ERR_SHAPE;
    if (N < 8 || N % 8 || N > MOE_MM_MAX_DIM || K < kmult || K % kmult || K > MOE_MM_MAX_DIM) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// A row operand: [rows, cols] elements of eb bytes with leading dimension ld,
// read whole rows at a time through `src` or directly by the R_max rows.
inline int32_t check_rows(const void* p, int32_t rows, int32_t cols, int32_t ld, int eb, const int32_t* src, int32_t R_max) {
    if (rows < 0 || ld < cols || ((int64_t)ld * eb) % 16 || ld > kMaxLd) return MOE_ERR_SHAPE;
    if (!src && rows < R_max) return MOE_ERR_SHAPE;
    if (src && R_max > 0 && rows < 1) return MOE_ERR_SHAPE;
    if (src && (int64_t)rows * ld * eb >= kGatherBytes) return MOE_ERR_SHAPE;
    if (R_max > 0 && !p) return MOE_ERR_NULL;
    if (!aligned(p, 16)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// partial sums are stored and loaded 16 bytes at a time
inline int32_t check_ws(size_t need, const void* ws, size_t ws_bytes) {
    if (ws_bytes < need || (need && !ws)) return MOE_ERR_WORKSPACE;
    return need && !aligned(ws, 16) ? MOE_ERR_SHAPE : MOE_OK;
}

inline bool t16(int32_t dtype) { return dtype == MOE_T_BF16 || dtype == MOE_T_F16; }

}  // namespace

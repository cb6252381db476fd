// FP8 with a scale for each block of 128, and the gated activation that keeps
// its input in that form.
//
// Quantising: s = 2^E with the smallest E >= -126 such that amax <= 448 * 2^E
// (amax over the block's finite values; s = 1 for a block of zeros), q = the
// E4M3 value nearest x / s. The division is by a power of two, so every code
// is exactly rounded whatever the instruction order. A lane holds 8 elements
// and 16 lanes (one DPP row) a block, so the amax costs four DPP steps and no
// LDS.
//
// All kernels here are bound by HBM: they read and write each byte once, 16
// bytes (8 for codes) per lane and request. Measured (a large copy: 5.2 TB/s):
// rows of 8192 x 7168 BF16 31 us, 5.7 TB/s; weights of 8 x 4096 x 7168 BF16 138 us
// (705 MB, 5.1 TB/s), FP32 of half the groups 109 us (5.4); the activation of
// 49152 x 1408 107 us (558 MB, 5.2 TB/s), without codes 77 to 82 (415 MB, 5.1 to
// 5.4), its backward of 24576 x 2048 FP16 95 us (506 MB, 5.3). With a few rows
// the call is host time, about 14 us.
#include <algorithm>

#include "grouped_mm.h"

namespace {

constexpr int kBqThreads = 256;

struct F8 { float v[8]; };

// 8 consecutive elements of the given type at p (16-byte aligned)
template <int T>
MOE_DEV F8 load8(const void* p) {
    F8 r;
    if constexpr (T == MOE_T_F32) {
        const f32x4 a = ((const f32x4*)p)[0], b = ((const f32x4*)p)[1];
        #pragma unroll
        for (int i = 0; i < 4; ++i) { r.v[i] = a[i]; r.v[4 + i] = b[i]; }
    } else {
        const i32x4 a = *(const i32x4*)p;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[2 * i] = lo16((uint32_t)a[i], T == MOE_T_F16);
            r.v[2 * i + 1] = hi16((uint32_t)a[i], T == MOE_T_F16);
        }
    }
    return r;
}
template <int T>
MOE_DEV void store8(void* p, const float (&v)[8]) {
    i32x4 o;
    #pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)pack16(v[2 * i], v[2 * i + 1], T == MOE_T_F16);
    *(i32x4*)p = o;
}

// bits of the largest |finite value| (fp32 pattern); odd: a NaN or infinity is among them
MOE_DEV uint32_t amax8(const F8& x, bool& odd) {
    uint32_t m = 0, f = 0;
    #pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x.v[i]) & 0x7FFFFFFFu);
    odd = m >= 0x7F800000u;
    if (odd) {
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = __float_as_uint(x.v[i]) & 0x7FFFFFFFu;
            f = max(f, u < 0x7F800000u ? u : 0u);
        }
        m = f;
    }
    return m;
}
// biased exponent of the block's scale
MOE_DEV uint32_t block_code(uint32_t amax) {
    if (amax == 0u) return 127u;
    const int c = (int)((amax + (0x7FFFFFu - 0x600000u)) >> 23) - 8;
    return (uint32_t)max(c, 1);
}
MOE_DEV float code_scale(uint32_t code) { return __uint_as_float(code << 23); }
// 8 codes of x / 2^(code - 127)
MOE_DEV u32x2_t codes8(const F8& x, uint32_t code, bool odd) {
    const float inv = __uint_as_float((254u - code) << 23);
    u32x2_t r;
    r.x = e4m3x4(x.v[0] * inv, x.v[1] * inv, x.v[2] * inv, x.v[3] * inv);
    r.y = e4m3x4(x.v[4] * inv, x.v[5] * inv, x.v[6] * inv, x.v[7] * inv);
    if (odd) {
        uint32_t w[2] = {r.x, r.y};
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = __float_as_uint(x.v[i]);
            if ((u & 0x7FFFFFFFu) >= 0x7F800000u) {
                const uint32_t sh = 8 * (i & 3);
                w[i >> 2] = (w[i >> 2] & ~(0xFFu << sh)) | ((((u >> 24) & 0x80u) | 0x7Fu) << sh);
            }
        }
        r = u32x2_t{w[0], w[1]};
    }
    return r;
}
// 8 codes -> values times the scale
MOE_DEV F8 decode8(const u32x2_t& c, float s) {
    F8 r;
    const uint32_t w[2] = {c.x, c.y};
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        r.v[4 * i] = a[0] * s; r.v[4 * i + 1] = a[1] * s; r.v[4 * i + 2] = b[0] * s; r.v[4 * i + 3] = b[1] * s;
    }
    return r;
}

MOE_DEV int used_rows(const int32_t* n_rows, int rows) { return n_rows ? min(max(*n_rows, 0), rows) : rows; }

// rows x ceil(K / 128) blocks, 16 lanes each
template <int T>
__global__ __launch_bounds__(kBqThreads)
void quantize_block_kernel(const uint8_t* __restrict__ x, int rows, int K, size_t ld_bytes,
                           const int32_t* __restrict__ n_rows, uint8_t* __restrict__ q, float* __restrict__ s) {
    constexpr int EB = T == MOE_T_F32 ? 4 : 2;
    rows = used_rows(n_rows, rows);
    const int nb = (K + 127) >> 7, per = nb * 16;
    const int64_t total = (int64_t)rows * per, stride = (int64_t)gridDim.x * kBqThreads;
    // whole 16-lane blocks enter and leave the loop together (total % 16 == 0)
    for (int64_t i = (int64_t)blockIdx.x * kBqThreads + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per);
        const bool in = c * 8 < K;
        F8 v{};
        if (in) v = load8<T>(x + row * ld_bytes + (size_t)c * 8 * EB);
        bool odd;
        const uint32_t code = block_code(row16_umax(amax8(v, odd)));
        if (in) *(u32x2_t*)(q + row * K + c * 8) = codes8(v, code, odd);
        if ((c & 15) == 0) s[row * nb + (c >> 4)] = code_scale(code);
    }
}

// one workgroup per 128 x 128 block of a [G, N, K] array: 8 pieces of 8
// elements per lane, the amax joined through LDS
template <int T>
__global__ __launch_bounds__(kBqThreads)
void quantize_weights_kernel(const uint8_t* __restrict__ w, int N, int K, uint8_t* __restrict__ q,
                             float* __restrict__ s) {
    constexpr int EB = T == MOE_T_F32 ? 4 : 2;
    __shared__ uint32_t part[kBqThreads / 64];
    const int kb = blockIdx.x, nb = blockIdx.y, g = blockIdx.z;
    const int lane = threadIdx.x & 63, c = kb * 128 + (threadIdx.x & 15) * 8;
    F8 v[8];
    bool odd[8];
    uint32_t m = 0;
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = nb * 128 + 16 * i + (threadIdx.x >> 4);
        v[i] = F8{};
        if (n < N && c < K) v[i] = load8<T>(w + (((size_t)g * N + n) * K + c) * EB);
        m = max(m, amax8(v[i], odd[i]));
    }
    m = wave_umax(m);
    if (lane == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
    const uint32_t code = block_code(m);
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = nb * 128 + 16 * i + (threadIdx.x >> 4);
        if (n < N && c < K) *(u32x2_t*)(q + ((size_t)g * N + n) * K + c) = codes8(v[i], code, odd[i]);
    }
    if (threadIdx.x == 0) s[((size_t)g * gridDim.y + nb) * gridDim.x + kb] = code_scale(code);
}

struct GluP {
    const uint8_t* in; size_t ld_bytes;
    const uint8_t* q_in; const float* s_in;
    const float* row_w; const int32_t* n_rows;
    int rows, I, act;
    float beta, limit;
    uint8_t* h; uint8_t* q; float* s; uint8_t* dpre; float* dw;
};

// clamp to +-lim (lim > 0); a NaN stays one
MOE_DEV float clamp_to(float v, float lim) {
    if (!(lim > 0.f)) return v;
    return v < -lim ? -lim : (v > lim ? lim : v);
}

// The activations of moe_device.h with a NaN gate kept by the squared ReLU too
// (a maximum with 0 turns it into 0, and a diverged step would look sound).
MOE_DEV float gate_value(float z, int act, float beta) {
    return act == MOE_ACT_SRELU && z != z ? z : act_value(z, act, beta);
}
MOE_DEV void gate_and_grad(float z, int act, float beta, float& a, float& da) {
    act_and_grad(z, act, beta, a, da);
    if (act == MOE_ACT_SRELU && z != z) a = da = z;
}

// h = a(clamp(g)) clamp(u) w and the block codes of g and u: a lane holds 8
// of each, 16 lanes a block of each half
template <int T>
__global__ __launch_bounds__(kBqThreads)
void glu_forward_kernel(GluP p) {
    const int rows = used_rows(p.n_rows, p.rows);
    const int I = p.I, nb = (I + 127) >> 7, per = nb * 16;
    const int64_t total = (int64_t)rows * per, stride = (int64_t)gridDim.x * kBqThreads;
    for (int64_t i = (int64_t)blockIdx.x * kBqThreads + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per);
        const bool in = c * 8 < I;
        F8 g{}, u{};
        if (in) {
            const uint8_t* src = p.in + row * p.ld_bytes + (size_t)c * 16;
            g = load8<T>(src);
            u = load8<T>(src + (size_t)I * 2);
        }
        const float w = p.row_w ? p.row_w[row] : 1.0f;
        if (p.q) {
            bool og, ou;
            const uint32_t cg = block_code(row16_umax(amax8(g, og)));
            const uint32_t cu = block_code(row16_umax(amax8(u, ou)));
            if (in) {
                uint8_t* d = p.q + row * 2 * I + c * 8;
                *(u32x2_t*)d = codes8(g, cg, og);
                *(u32x2_t*)(d + I) = codes8(u, cu, ou);
            }
            if ((c & 15) == 0) {
                float* d = p.s + row * 2 * nb + (c >> 4);
                d[0] = code_scale(cg);
                d[nb] = code_scale(cu);
            }
        }
        if (in) {
            float h[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k)
                h[k] = gate_value(clamp_to(g.v[k], p.limit), p.act, p.beta) * clamp_to(u.v[k], p.limit) * w;
            store8<T>(p.h + (row * I + c * 8) * 2, h);
        }
    }
}

// One wave per row: the row's dw is one wave's sum, in a fixed order.
template <int T>
__global__ __launch_bounds__(kBqThreads)
void glu_backward_kernel(GluP p) {
    const int rows = used_rows(p.n_rows, p.rows);
    const int I = p.I, nb = (I + 127) >> 7, lane = threadIdx.x & 63;
    const int wave = blockIdx.x * (kBqThreads / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = gridDim.x * (kBqThreads / 64);
    for (int64_t row = wave; row < rows; row += waves) {
        const float w = p.row_w ? p.row_w[row] : 1.0f;
        float sum = 0.f;
        for (int c = lane * 8; c < I; c += 512) {
            const uint8_t* qr = p.q_in + row * 2 * I + c;
            const float* sr = p.s_in + row * 2 * nb + (c >> 7);
            const F8 g = decode8(*(const u32x2_t*)qr, sr[0]);
            const F8 u = decode8(*(const u32x2_t*)(qr + I), sr[nb]);
            const F8 d = load8<T>(p.in + row * p.ld_bytes + (size_t)c * 2);
            float dg[8], du[8], h[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float lim = p.limit;
                const float mg = !(lim > 0.f) || fabsf(g.v[k]) <= lim ? 1.f : 0.f;
                const float mu = !(lim > 0.f) || fabsf(u.v[k]) <= lim ? 1.f : 0.f;
                const float gc = clamp_to(g.v[k], lim), uc = clamp_to(u.v[k], lim);
                float a, da;
                gate_and_grad(gc, p.act, p.beta, a, da);
                const float dw = d.v[k] * w;
                dg[k] = dw * uc * da * mg;
                du[k] = dw * a * mu;
                h[k] = a * uc * w;
                sum += d.v[k] * a * uc;
            }
            uint8_t* o = p.dpre + (row * 2 * I + c) * 2;
            store8<T>(o, dg);
            store8<T>(o + (size_t)I * 2, du);
            if (p.h) store8<T>(p.h + (row * I + c) * 2, h);
        }
        if (p.dw) {
            sum = wave_sum(sum);
            if (lane == 0) p.dw[row] = sum;
        }
    }
}

int grid_for(int64_t lanes) {
    return (int)std::min<int64_t>((lanes + kBqThreads - 1) / kBqThreads, (int64_t)device_cu_count() * 32);
}

}  // namespace

int moe_launch_quantize_block(const void* x, int dtype, int rows, int K, int ld, const int32_t* n_rows, uint8_t* q,
                              float* s, hipStream_t stream) {
    const int grid = grid_for((int64_t)rows * ((K + 127) / 128) * 16);
    const uint8_t* b = (const uint8_t*)x;
    if (dtype == MOE_T_BF16)
        quantize_block_kernel<MOE_T_BF16><<<grid, kBqThreads, 0, stream>>>(b, rows, K, (size_t)ld * 2, n_rows, q, s);
    else if (dtype == MOE_T_F16)
        quantize_block_kernel<MOE_T_F16><<<grid, kBqThreads, 0, stream>>>(b, rows, K, (size_t)ld * 2, n_rows, q, s);
    else
        quantize_block_kernel<MOE_T_F32><<<grid, kBqThreads, 0, stream>>>(b, rows, K, (size_t)ld * 4, n_rows, q, s);
    return (int)hipGetLastError();
}

int moe_launch_quantize_block_weights(const void* w, int dtype, int G, int N, int K, uint8_t* q, float* s,
                                      hipStream_t stream) {
    const dim3 grid((K + 127) / 128, (N + 127) / 128, G);
    const uint8_t* b = (const uint8_t*)w;
    if (dtype == MOE_T_BF16) quantize_weights_kernel<MOE_T_BF16><<<grid, kBqThreads, 0, stream>>>(b, N, K, q, s);
    else if (dtype == MOE_T_F16) quantize_weights_kernel<MOE_T_F16><<<grid, kBqThreads, 0, stream>>>(b, N, K, q, s);
    else quantize_weights_kernel<MOE_T_F32><<<grid, kBqThreads, 0, stream>>>(b, N, K, q, s);
    return (int)hipGetLastError();
}

static GluP glu_params(const GluCall& c) {
    GluP p{};
    p.in = (const uint8_t*)c.in; p.ld_bytes = (size_t)c.ld * 2;
    p.q_in = c.q_in; p.s_in = c.s_in; p.row_w = c.row_w; p.n_rows = c.n_rows;
    p.rows = c.rows; p.I = c.I; p.act = c.act; p.beta = c.beta; p.limit = c.limit;
    p.h = (uint8_t*)c.h; p.q = c.q; p.s = c.s; p.dpre = (uint8_t*)c.dpre; p.dw = c.dw;
    return p;
}

int moe_launch_glu_forward(const GluCall& c, hipStream_t stream) {
    const GluP p = glu_params(c);
    const int grid = grid_for((int64_t)c.rows * ((c.I + 127) / 128) * 16);
    if (c.dtype == MOE_T_BF16) glu_forward_kernel<MOE_T_BF16><<<grid, kBqThreads, 0, stream>>>(p);
    else glu_forward_kernel<MOE_T_F16><<<grid, kBqThreads, 0, stream>>>(p);
    return (int)hipGetLastError();
}

int moe_launch_glu_backward(const GluCall& c, hipStream_t stream) {
    const GluP p = glu_params(c);
    const int grid = grid_for((int64_t)c.rows * 64);
    if (c.dtype == MOE_T_BF16) glu_backward_kernel<MOE_T_BF16><<<grid, kBqThreads, 0, stream>>>(p);
    else glu_backward_kernel<MOE_T_F16><<<grid, kBqThreads, 0, stream>>>(p);
    return (int)hipGetLastError();
}

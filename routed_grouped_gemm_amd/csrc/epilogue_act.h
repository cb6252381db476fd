// Activations of the product epilogues (grouped_mm_epi.h, few_layer.hip): the
// gated unit a(clamp(g)) clamp(u) and the plain a(clamp(z)), and their
// derivatives. Internal to libmoe.
#pragma once
#include "moe_device.h"

namespace {

// clamp to +-lim (lim > 0); a NaN stays one
MOE_DEV float epi_clamp(float v, float lim) {
    if (!(lim > 0.f)) return v;
    return v < -lim ? -lim : (v > lim ? lim : v);
}
MOE_DEV float epi_inside(float v, float lim) { return !(lim > 0.f) || fabsf(v) <= lim ? 1.f : 0.f; }

// Phi(z), the normal distribution, and e = exp(-z^2 / 2). For x = |z| / sqrt 2,
// erfc(x) exp(x^2) is t times a polynomial in t = 1 / (1 + 0.45 x): degree 7,
// fitted to the least largest relative error (4e-7). With fp32's roundings, that of
// the exponent growing with z^2, it is 7e-7 down to z = -2, 1e-6 to -4, 3e-6 to -8 and
// 8e-6 to -13, so Phi keeps its relative precision where it is small (1 + erf loses it: at z =
// -4 an error of 1e-3 of the value, past FP16's half step) at a few instructions
// more than the exponential.
MOE_DEV float epi_phi(float z, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.318198055f, 1.0f));
    float s = 0.0347582772f;
    s = fmaf(s, t, -0.125720039f);
    s = fmaf(s, t, 0.114143476f);
    s = fmaf(s, t, 0.0111250253f);
    s = fmaf(s, t, 0.0991159827f);
    s = fmaf(s, t, 0.112589903f);
    s = fmaf(s, t, 0.127047703f);
    s = fmaf(s, t, 0.126939863f);
    e = __expf(-0.5f * z * z);
    const float tail = s * t * e;                            // Phi(-|z|); the halving is in the polynomial
    return z < 0.f ? tail : 1.0f - tail;
}

// Swish (z sigmoid(beta z)), exact GELU, squared ReLU (a NaN stays one), or z
template <int ACT>
MOE_DEV float epi_act(float z, float beta) {
    if constexpr (ACT == MOE_ACT_GEGLU) {
        float e;
        return z * epi_phi(z, e);
    }
    if constexpr (ACT == MOE_ACT_SRELU) return z < 0.f ? 0.f : z * z;
    if constexpr (ACT == MOE_ACT_NONE) return z;
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-beta * z));
}
template <int ACT>
MOE_DEV void epi_act_grad(float z, float beta, float& a, float& da) {
    if constexpr (ACT == MOE_ACT_GEGLU) {
        float e;
        const float phi = epi_phi(z, e);
        a = z * phi;
        da = phi + z * (0.39894228040143268f * e);
    } else if constexpr (ACT == MOE_ACT_SRELU) {
        a = z < 0.f ? 0.f : z * z;
        da = z < 0.f ? 0.f : 2.0f * z;
    } else if constexpr (ACT == MOE_ACT_NONE) {
        a = z;
        da = 1.f;
    } else {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-beta * z));
        a = z * s;
        da = s + beta * a * (1.0f - s);
    }
}

// f(std::integral_constant<int, act>) of a run-time activation
template <typename F>
MOE_DEV void with_act(int act, F&& f) {
    if (act == MOE_ACT_SWIGLU) f(std::integral_constant<int, MOE_ACT_SWIGLU>{});
    else if (act == MOE_ACT_GEGLU) f(std::integral_constant<int, MOE_ACT_GEGLU>{});
    else if (act == MOE_ACT_SRELU) f(std::integral_constant<int, MOE_ACT_SRELU>{});
    else f(std::integral_constant<int, MOE_ACT_NONE>{});
}

}  // namespace

// Device-side helpers of the dense half of the layer: its activations and the values of
// 8-bit checkpoints. Apart from the grouped GEMMs' headers, whose text names the sources
// that the committed traffic counters were taken on.
#pragma once

#include "dense_launch.hpp"
#include "gemm_common.hpp"
#include "mx_common.hpp"

namespace moe {

// Phi(x), the standard normal distribution, and exp(-x^2 / 2). Its lower tail is
// Phi(-a) = exp(-a^2 / 2) t q(t) for a >= 0, t = 1 / (1 + 0.345 a), with q a degree-8
// polynomial fitted in relative error (4e-8 at most over a <= 14 with these coefficients,
// before the fp32 evaluation's own; weighted least squares on erfcx). One exponential serves the tail and the density,
// there is no branch, and no 1 + erf(x) cancels for negative x, so the tail keeps its
// relative precision (the grouped GEMMs' GeGLU keeps the erf form and its results).
__device__ __forceinline__ void normal_cdf(float x, float& cdf, float& e) {
    const float a = fabsf(x);
    e = __expf(-0.5f * a * a);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.345f, a, 1.f));
    float r = -0.0283819679f;
    r = fmaf(r, t, 0.145282f);
    r = fmaf(r, t, -0.27117312f);
    r = fmaf(r, t, 0.187196702f);
    r = fmaf(r, t, -0.0376016684f);
    r = fmaf(r, t, 0.11179959f);
    r = fmaf(r, t, 0.117238291f);
    r = fmaf(r, t, 0.138020888f);
    r = fmaf(r, t, 0.137619287f);
    const float tail = e * (t * r);
    cdf = x < 0.f ? tail : 1.f - tail;
}

// Activations of the dense linear layer: ACT 2 squared ReLU, 3 identity, 4 SiLU, 5
// GELU; the gate activation of a gated layer (ACT 0, 1) is SiLU or GELU. And with the
// derivative. A NaN stays one (no maximum with 0, which would take the 0).
template <int ACT>
__device__ __forceinline__ float dense_act(float x) {
    if constexpr (ACT == 2) {
        const float r = x < 0.f ? 0.f : x;
        return r * r;
    } else if constexpr (ACT == 3) {
        return x;
    } else if constexpr (ACT == 0 || ACT == 4) {
        return x * sigmoid_f(x);
    } else {
        float cdf, e;
        normal_cdf(x, cdf, e);
        return x * cdf;
    }
}
template <int ACT>
__device__ __forceinline__ void dense_act_grad(float x, float& f, float& df) {
    if constexpr (ACT == 2) {
        const float r = x < 0.f ? 0.f : x;
        f = r * r;
        df = 2.f * r;
    } else if constexpr (ACT == 3) {
        f = x;
        df = 1.f;
    } else if constexpr (ACT == 0 || ACT == 4) {
        glu_gate_grad<0>(x, f, df);
    } else {
        float cdf, e;
        normal_cdf(x, cdf, e);
        f = x * cdf;
        df = fmaf(x, 0.39894228040143268f * e, cdf);
    }
}

// 2^(s - 127); code 0 is the subnormal 2^-127, code 255 NaN
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}

// 4 E4M3 codes (low byte first) times a scale
__device__ __forceinline__ void e4m3x4_value(uint32_t w, float sc, float* v) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = a.x * sc, v[1] = a.y * sc, v[2] = b.x * sc, v[3] = b.y * sc;
}

}  // namespace moe

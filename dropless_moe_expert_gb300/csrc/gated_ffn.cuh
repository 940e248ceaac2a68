// Activations of the gated feed-forward and their derivatives, in fp32.
//
// silu(g) = g s(g) with the logistic function s, gelu_tanh(g) = g s(z) with
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3), because (1 + tanh(z / 2)) / 2 = s(z);
// gelu(g) = g Phi(g) with the normal distribution function, relu(g) = max(g, 0).
// Each is within a few 2^-22 of its value, far below the bf16 rounding of what it feeds.
#pragma once

#include <cuda_runtime.h>
#include <type_traits>

namespace moe {
namespace ff {

enum Act { SILU = 0, GELU = 1, GELU_TANH = 2, RELU = 3 };

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// Phi(g) of the normal distribution, and e = exp(-g^2 / 2).  The smaller tail is
// e t Q(t) with t = 1 / (1 + 0.3 |g| / sqrt 2): Q, a polynomial of degree 8, was fitted
// to exp(x^2) erfc(x) / (2 t) at x = |g| / sqrt 2, from 0 to 10, least relative error
// at most 2e-8 (in fp32 about 5e-7 near 0; the rounding of g^2 / 2 counts beyond).
__device__ __forceinline__ float normal_cdf(float g, float &e) {
    const float t = __fdividef(1.0f, __fmaf_rn(0.21213203435596426f, fabsf(g), 1.0f));
    e = __expf(-0.5f * g * g);
    float q = -0.06476146727800369f;
    q = __fmaf_rn(q, t, 0.24278171360492706f);
    q = __fmaf_rn(q, t, -0.2561393082141876f);
    q = __fmaf_rn(q, t, 0.2738603949546814f);
    q = __fmaf_rn(q, t, -0.047325700521469116f);
    q = __fmaf_rn(q, t, 0.10746320337057114f);
    q = __fmaf_rn(q, t, 0.07416953146457672f);
    q = __fmaf_rn(q, t, 0.08535762131214142f);
    q = __fmaf_rn(q, t, 0.0845940038561821f);
    const float tail = e * (q * t);
    return g > 0.0f ? 1.0f - tail : tail;
}

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == SILU) {
        return g * logistic(g);
    } else if constexpr (ACT == GELU_TANH) {
        return g * logistic(g * __fmaf_rn(kTanhScale * kTanhCubic, g * g, kTanhScale));
    } else if constexpr (ACT == GELU) {
        float e;
        return g * normal_cdf(g, e);
    } else {
        return g < 0.0f ? 0.0f : g;  // a NaN stays one
    }
}

// The activation and its derivative.  A factor that has run to zero ends a
// term, also where the other one is infinite.
template <int ACT>
__device__ __forceinline__ float activate(float g, float &slope) {
    if constexpr (ACT == SILU || ACT == GELU_TANH) {
        const float g2 = g * g;
        const float z = ACT == SILU ? g : g * __fmaf_rn(kTanhScale * kTanhCubic, g2, kTanhScale);
        const float dz = ACT == SILU ? 1.0f : __fmaf_rn(3.0f * kTanhScale * kTanhCubic, g2, kTanhScale);
        const float s = logistic(z), v = s * (1.0f - s);
        slope = v == 0.0f ? s : __fmaf_rn(g * v, dz, s);
        return g * s;
    } else if constexpr (ACT == GELU) {
        float e;
        const float cdf = normal_cdf(g, e);
        slope = e == 0.0f ? cdf : __fmaf_rn(g * e, 0.3989422804014327f, cdf);  // 1 / sqrt(2 pi)
        return g * cdf;
    } else {
        slope = g > 0.0f ? 1.0f : g != g ? g : 0.0f;
        return g < 0.0f ? 0.0f : g;
    }
}

// body(std::integral_constant<int, ACT>) for the activation given at run time;
// the branch is the same for a whole launch.
template <typename Body>
__device__ __forceinline__ void with_activation(int act, Body body) {
    switch (act) {
        case SILU: return body(std::integral_constant<int, SILU>{});
        case GELU: return body(std::integral_constant<int, GELU>{});
        case GELU_TANH: return body(std::integral_constant<int, GELU_TANH>{});
        default: return body(std::integral_constant<int, RELU>{});
    }
}

}  // namespace ff
}  // namespace moe

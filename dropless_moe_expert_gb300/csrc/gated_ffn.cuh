// Activations of the gated feed-forward and their derivatives, in fp32.
//
// silu(g) = g s(g) with the logistic function s, gelu_tanh(g) = g s(z) with
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3), because (1 + tanh(z / 2)) / 2 = s(z);
// gelu(g) = g Phi(g) with the normal distribution function, relu(g) = max(g, 0).
// Each is within a few 2^-22 of its value, far below the bf16 rounding of what it feeds.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>

namespace moe {
namespace ff {

enum Act { SILU = 0, GELU = 1, GELU_TANH = 2, RELU = 3 };

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == SILU) {
        return g * logistic(g);
    } else if constexpr (ACT == GELU_TANH) {
        return g * logistic(g * __fmaf_rn(kTanhScale * kTanhCubic, g * g, kTanhScale));
    } else if constexpr (ACT == GELU) {
        return g * normcdff(g);
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
        const float cdf = normcdff(g), e = __expf(-0.5f * g * g);
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

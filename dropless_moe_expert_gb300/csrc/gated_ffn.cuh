// Activations of the gated feed-forward and their derivatives, in fp32.
//
// silu(g) = g s(g) with the logistic function s, gelu_tanh(g) = g s(z) with
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3), because (1 + tanh(z / 2)) / 2 = s(z);
// gelu(g) = g Phi(g) with the normal distribution function, relu(g) = max(g, 0).
// Each is within a few 2^-22 of the magnitudes of its terms (and 2^-22 of the
// exponent that they take), far below the bf16 rounding of what it feeds: of its
// value too, but for a derivative whose terms cancel (silu's near g = -1.28)
// and a factor below 2^-126, which is 0.
//
// Two values at a time: what an epilogue warp issues is what bounds the tiles
// with few slices of K, and packed fp32 instructions are half as many.
#pragma once

#include <cuda_runtime.h>
#include <type_traits>

#include "vec8.cuh"

namespace moe {
namespace ff {

enum Act { SILU = 0, GELU = 1, GELU_TANH = 2, RELU = 3 };

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 exp2_approx(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_approx(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
// t, or `otherwise` where the factor v has run to zero (whatever the others are)
__device__ __forceinline__ float2 unless_zero(float2 v, float2 t, float2 otherwise) {
    return make_float2(v.x == 0.0f ? otherwise.x : t.x, v.y == 0.0f ? otherwise.y : t.y);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// s(z)
__device__ __forceinline__ float2 logistic(float2 z) {
    return rcp_approx(add2(both(1.0f), exp2_approx(mul2(both(-kLog2e), z))));
}

// Phi(g) of the normal distribution, and e = exp(-g^2 / 2).  The smaller tail is
// e t Q(t) with t = 1 / (1 + 0.3 |g| / sqrt 2): Q, a polynomial of degree 8, was fitted
// to exp(x^2) erfc(x) / (2 t) at x = |g| / sqrt 2, from 0 to 10, for a small relative error:
// 3.4e-8 at most, at x = 10 (in fp32 about 5e-7 near 0; the rounding of g^2 / 2 counts beyond).
__device__ __forceinline__ float2 normal_cdf(float2 g, float2 &e) {
    const float2 a = make_float2(fabsf(g.x), fabsf(g.y));
    const float2 t = rcp_approx(fma2(both(0.21213203435596426f), a, both(1.0f)));
    e = exp2_approx(mul2(both(-0.5f * kLog2e), mul2(g, g)));
    float2 q = both(-0.06476146727800369f);
    q = fma2(q, t, both(0.24278171360492706f));
    q = fma2(q, t, both(-0.2561393082141876f));
    q = fma2(q, t, both(0.2738603949546814f));
    q = fma2(q, t, both(-0.047325700521469116f));
    q = fma2(q, t, both(0.10746320337057114f));
    q = fma2(q, t, both(0.07416953146457672f));
    q = fma2(q, t, both(0.08535762131214142f));
    q = fma2(q, t, both(0.0845940038561821f));
    const float2 tail = mul2(e, mul2(q, t));
    return make_float2(g.x > 0.0f ? 1.0f - tail.x : tail.x, g.y > 0.0f ? 1.0f - tail.y : tail.y);
}

template <int ACT>
__device__ __forceinline__ float2 activate(float2 g) {
    if constexpr (ACT == SILU) {
        return mul2(g, logistic(g));
    } else if constexpr (ACT == GELU_TANH) {
        return mul2(g, logistic(mul2(g, fma2(both(kTanhScale * kTanhCubic), mul2(g, g), both(kTanhScale)))));
    } else if constexpr (ACT == GELU) {
        float2 e;
        return mul2(g, normal_cdf(g, e));
    } else {
        return make_float2(g.x < 0.0f ? 0.0f : g.x, g.y < 0.0f ? 0.0f : g.y);  // a NaN stays one
    }
}
template <int ACT>
__device__ __forceinline__ float activate(float g) {
    return activate<ACT>(both(g)).x;
}

// The activation and its derivative.  A factor that has run to zero ends a
// term, also where the other one is infinite.
template <int ACT>
__device__ __forceinline__ float2 activate(float2 g, float2 &slope) {
    if constexpr (ACT == SILU || ACT == GELU_TANH) {
        const float2 g2 = mul2(g, g);
        const float2 z = ACT == SILU ? g : mul2(g, fma2(both(kTanhScale * kTanhCubic), g2, both(kTanhScale)));
        const float2 s = logistic(z), v = mul2(s, fma2(both(-1.0f), s, both(1.0f))), gv = mul2(g, v);
        const float2 dz = fma2(both(3.0f * kTanhScale * kTanhCubic), g2, both(kTanhScale));
        slope = unless_zero(v, ACT == SILU ? add2(gv, s) : fma2(gv, dz, s), s);
        return mul2(g, s);
    } else if constexpr (ACT == GELU) {
        float2 e;
        const float2 cdf = normal_cdf(g, e);
        slope = unless_zero(e, fma2(mul2(g, e), both(0.3989422804014327f), cdf), cdf);  // 1 / sqrt(2 pi)
        return mul2(g, cdf);
    } else {
        slope = make_float2(g.x > 0.0f ? 1.0f : g.x != g.x ? g.x : 0.0f, g.y > 0.0f ? 1.0f : g.y != g.y ? g.y : 0.0f);
        return activate<ACT>(g);
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

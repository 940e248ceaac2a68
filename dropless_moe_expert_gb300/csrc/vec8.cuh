// Eight consecutive elements of a bf16 or fp32 row as fp32 registers: one
// (bf16) or two (fp32) 16-byte accesses per thread.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ void bf16x8_to_f32(const uint4 &u, float *o) {
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(p[i] << 16);
        o[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float *v) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// Two fp32 lanes per instruction (each lane rounds as the scalar operation does).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// `i` counts vectors of eight elements; the row starts on a 16-byte boundary.
__device__ __forceinline__ void load8(const uint16_t *row, int i, float *o) {
    bf16x8_to_f32(reinterpret_cast<const uint4 *>(row)[i], o);
}
__device__ __forceinline__ void load8(const float *row, int i, float *o) {
    const float4 a = reinterpret_cast<const float4 *>(row)[2 * i], b = reinterpret_cast<const float4 *>(row)[2 * i + 1];
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *row, int i, const float *v) {
    reinterpret_cast<uint4 *>(row)[i] = f32_to_bf16x8(v);
}
__device__ __forceinline__ void store8(float *row, int i, const float *v) {
    reinterpret_cast<float4 *>(row)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(row)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The same as one 32-byte access; `row` on a 32-byte boundary.
__device__ __forceinline__ void store8_wide(float *row, int i, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + 8 * static_cast<int64_t>(i)),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

}  // namespace moe

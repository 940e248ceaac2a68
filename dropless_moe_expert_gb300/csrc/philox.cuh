// Random words from a counter: Philox4x32-10 of Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011).  Ten rounds of two
// 32 x 32-bit products; nothing is held between calls, so the backward draws
// what the forward drew from the same key and counter.
#pragma once

#include <stdint.h>

namespace moe {

// N counters at once: they share the rounds' keys.
template <int N>
__device__ __forceinline__ void philox4x32_10(uint2 key, uint4 (&c)[N]) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c[j].x, q = static_cast<uint64_t>(0xCD9E8D57u) * c[j].z;
            c[j] = make_uint4(static_cast<uint32_t>(q >> 32) ^ c[j].y ^ key.x, static_cast<uint32_t>(q),
                              static_cast<uint32_t>(p >> 32) ^ c[j].w ^ key.y, static_cast<uint32_t>(p));
        }
        key.x += 0x9E3779B9u, key.y += 0xBB67AE85u;
    }
}

// Dropout of elements in blocks of eight: one 16-bit draw per element, from the
// four words of the counter (block, call), low halves first.  16 bits: half the
// generator's work of 32, and the share that is dropped, a multiple of 2^-16, is
// what the kept elements are scaled by, so the expectation is exact.
//
// What is kept is told to the arithmetic by predicates, not by factors or
// selects: a dropped element leaves a sum as it was, whatever its value, and
// no instruction is spent on zeroing it.
struct Dropout {
    uint2 key, call;
    uint32_t bar;  // the least draw that is kept, in the upper half
    __device__ __forceinline__ Dropout(const uint64_t *rng, uint32_t drop)
        : key(make_uint2(static_cast<uint32_t>(rng[0]), static_cast<uint32_t>(rng[0] >> 32))),
          call(make_uint2(static_cast<uint32_t>(rng[1]), static_cast<uint32_t>(rng[1] >> 32))), bar(drop << 16) {}
    // The words of N blocks, `step` apart.
    template <int N>
    __device__ __forceinline__ void words(uint64_t block, uint32_t step, uint4 (&w)[N]) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t b = block + j * step;
            w[j] = make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32), call.x, call.y);
        }
        philox4x32_10(key, w);
    }
};
// A draw in the upper half of a word (what lies below it does not matter: bar's lower half is zero).
__device__ __forceinline__ uint32_t draw(const uint4 &w, int element) {
    const uint32_t v = element < 2 ? w.x : element < 4 ? w.y : element < 6 ? w.z : w.w;
    return element & 1 ? v : v << 16;
}
// s += a b where the draw is kept.
__device__ __forceinline__ void fma_kept(float &s, float a, float b, uint32_t draw, uint32_t bar) {
    asm("{\n\t.reg .pred p;\n\t"
        "setp.ge.u32 p, %3, %4;\n\t"
        "@p fma.rn.f32 %0, %1, %2, %0;\n\t}"
        : "+f"(s)
        : "f"(a), "f"(b), "r"(draw), "r"(bar));
}
// Sets `bit` of the mask where the draw is kept.
__device__ __forceinline__ void mark_kept(uint32_t &mask, uint32_t bit, uint32_t draw, uint32_t bar) {
    asm("{\n\t.reg .pred p;\n\t"
        "setp.ge.u32 p, %1, %2;\n\t"
        "@p or.b32 %0, %0, %3;\n\t}"
        : "+r"(mask)
        : "r"(draw), "r"(bar), "r"(bit));
}
// s += a b and t += c d where `bit` of the mask is set.
__device__ __forceinline__ void fma_masked(float &s, float a, float b, float &t, float c, float d, uint32_t mask,
                                           uint32_t bit) {
    asm("{\n\t.reg .pred p;\n\t.reg .b32 m;\n\t"
        "and.b32 m, %6, %7;\n\t"
        "setp.ne.u32 p, m, 0;\n\t"
        "@p fma.rn.f32 %0, %2, %3, %0;\n\t"
        "@p fma.rn.f32 %1, %4, %5, %1;\n\t}"
        : "+f"(s), "+f"(t)
        : "f"(a), "f"(b), "f"(c), "f"(d), "r"(mask), "r"(bit));
}

}  // namespace moe

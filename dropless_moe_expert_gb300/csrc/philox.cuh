// Random words from a counter: Philox4x32-10 of Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011).  Ten rounds of two
// 32 x 32-bit products; nothing is held between calls, so the backward draws
// what the forward drew from the same key and counter.
#pragma once

#include <stdint.h>

namespace moe {

__device__ __forceinline__ uint4 philox4x32_10(uint2 key, uint4 c) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c.x, q = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
        c = make_uint4(static_cast<uint32_t>(q >> 32) ^ c.y ^ key.x, static_cast<uint32_t>(q),
                       static_cast<uint32_t>(p >> 32) ^ c.w ^ key.y, static_cast<uint32_t>(p));
        key.x += 0x9E3779B9u, key.y += 0xBB67AE85u;
    }
    return c;
}

// Dropout of elements in blocks of eight: one 16-bit draw per element, from the
// four words of the counter (block, call), low halves first.  16 bits: half the
// generator's work of 32, and the share that is dropped, a multiple of 2^-16, is
// what the kept elements are scaled by, so the expectation is exact.
struct Dropout {
    uint2 key, call;
    uint32_t bar;  // the least draw that is kept, in the upper half
    __device__ __forceinline__ Dropout(const uint64_t *rng, uint32_t drop)
        : key(make_uint2(static_cast<uint32_t>(rng[0]), static_cast<uint32_t>(rng[0] >> 32))),
          call(make_uint2(static_cast<uint32_t>(rng[1]), static_cast<uint32_t>(rng[1] >> 32))), bar(drop << 16) {}
    // Bit i: whether element i of the block is kept.
    __device__ __forceinline__ uint32_t kept(uint64_t block) const {
        const uint4 w = philox4x32_10(
            key, make_uint4(static_cast<uint32_t>(block), static_cast<uint32_t>(block >> 32), call.x, call.y));
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m |= (v[i] << 16 >= bar ? 1u : 0u) << (2 * i);
            m |= (v[i] >= bar ? 1u : 0u) << (2 * i + 1);
        }
        return m;
    }
};
// The i-th pair of a block's elements, zero where they are not kept, whatever they are.
__device__ __forceinline__ float2 only(uint32_t kept, int i, float2 v) {
    return make_float2(kept >> (2 * i) & 1 ? v.x : 0.0f, kept >> (2 * i + 1) & 1 ? v.y : 0.0f);
}

}  // namespace moe

// The global norm of a step's gradients, and clipping by it, over many
// tensors of both types, with nothing read back to the host:
//   N = sqrt(sum over all tensors of |g|^2),  c = min(1, max_norm / (N + 1e-6)),  out = c g
// A NaN in any gradient makes N and c NaN; an infinity makes N infinite and c
// zero (so that entry becomes NaN): N tells the caller to skip the step.
//
// Two launches for every GROUP tensors each: the sums of squares, one fp32
// value per CTA in a fixed order of addition; then each CTA adds those values
// (in fp64, the same in every CTA) and scales its part.  The tensors'
// addresses and sizes travel as kernel arguments, so the calls can be
// captured in a graph and need no table in device memory.
#include "kernels.h"
#include "vec8.cuh"

#include <algorithm>

namespace moe {
namespace gc {

constexpr int GROUP = 512;       // tensors per launch (20 bytes each of the 32 KB of kernel arguments)
constexpr int CHUNK = 16384;     // elements that a CTA takes at a time
constexpr int THREADS = 512;
constexpr int CTAS = 304;
constexpr unsigned FULL = 0xffffffffu;

struct Table {
    const void *g[GROUP];
    void *out[GROUP];
    int64_t size[GROUP];
    int32_t first[GROUP + 1];  // the tensor's first chunk
    uint8_t bf16[GROUP];
    int n;
};

__device__ __forceinline__ int tensor_of(const Table &t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float value(const float *p) { return *p; }
__device__ __forceinline__ float value(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
}

// Elements [0, n) of g through f(index, vector of eight) and f(index, one):
// vectors from the first 16-byte boundary on.
template <typename E, typename F8, typename F1>
__device__ __forceinline__ void walk(const E *g, int n, F8 eight, F1 one) {
    const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(g) & 15)) % 16 / sizeof(E)));
    const int nvec = (n - head) / 8;
    for (int i = threadIdx.x; i < head; i += THREADS) one(i);
#pragma unroll 4
    for (int v = threadIdx.x; v < nvec; v += THREADS) eight(head + 8 * v);
    for (int i = head + 8 * nvec + threadIdx.x; i < n; i += THREADS) one(i);
}

template <typename E>
__device__ __forceinline__ float squares(const E *g, int n) {
    float s = 0.0f;
    walk(g, n,
         [&](int i) {
             float v[8];
             load8(g + i, 0, v);
#pragma unroll
             for (int q = 0; q < 8; ++q) s = __fmaf_rn(v[q], v[q], s);
         },
         [&](int i) { s = __fmaf_rn(value(g + i), value(g + i), s); });
    return s;
}

template <typename E>
__device__ __forceinline__ void scale(const E *g, E *out, int n, float c) {
    const bool together = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    walk(g, n,
         [&](int i) {
             float v[8];
             load8(g + i, 0, v);
#pragma unroll
             for (int q = 0; q < 8; ++q) v[q] *= c;
             if (together) {
                 store8(out + i, 0, v);
             } else {
#pragma unroll
                 for (int q = 0; q < 8; ++q) put(out + i + q, v[q]);
             }
         },
         [&](int i) { put(out + i, c * value(g + i)); });
}

__global__ void __launch_bounds__(THREADS) grad_squares_kernel(const __grid_constant__ Table t, float *__restrict__ part) {
    __shared__ float red[THREADS / 32];
    float s = 0.0f;
    for (int c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t at = static_cast<int64_t>(c - t.first[i]) * CHUNK;
        const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK), t.size[i] - at));
        s += t.bf16[i] ? squares(static_cast<const uint16_t *>(t.g[i]) + at, n)
                       : squares(static_cast<const float *>(t.g[i]) + at, n);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float a = 0.0f;
        for (int w = 0; w < THREADS / 32; ++w) a += red[w];
        part[blockIdx.x] = a;
    }
}

// The norm from all partial sums, in every thread of the block.
__device__ __forceinline__ float total_norm(const float *part, int parts) {
    __shared__ double red[THREADS / 32];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += THREADS) s += part[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) s += red[w];
    return static_cast<float>(sqrt(s));
}

__global__ void __launch_bounds__(THREADS)
grad_norm_kernel(const float *__restrict__ part, int parts, float *__restrict__ norm_out) {
    const float norm = total_norm(part, parts);
    if (threadIdx.x == 0) *norm_out = norm;
}

__global__ void __launch_bounds__(THREADS)
grad_scale_kernel(const __grid_constant__ Table t, const float *__restrict__ part, int parts, float max_norm,
                  float *__restrict__ norm_out) {
    const float norm = total_norm(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    float c = max_norm / (norm + 1e-6f);
    if (c > 1.0f) c = 1.0f;  // a NaN stays
    for (int q = blockIdx.x; q < t.first[t.n]; q += gridDim.x) {
        const int i = tensor_of(t, q);
        if (c == 1.0f && t.out[i] == t.g[i]) continue;  // in place and nothing to clip
        const int64_t at = static_cast<int64_t>(q - t.first[i]) * CHUNK;
        const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK), t.size[i] - at));
        if (t.bf16[i])
            scale(static_cast<const uint16_t *>(t.g[i]) + at, static_cast<uint16_t *>(t.out[i]) + at, n, c);
        else
            scale(static_cast<const float *>(t.g[i]) + at, static_cast<float *>(t.out[i]) + at, n, c);
    }
}

int groups(int n) { return std::max(1, (n + GROUP - 1) / GROUP); }

}  // namespace gc

size_t grad_clip_part_bytes(int n) { return static_cast<size_t>(gc::groups(n)) * gc::CTAS * sizeof(float); }

cudaError_t launch_grad_clip(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *kinds,
                             int n, bool clip, float max_norm, float *norm_out, float *part, int *launches,
                             cudaStream_t stream) {
    const int groups = gc::groups(n);
    const int parts = groups * gc::CTAS;
    gc::Table t;
    auto fill = [&](int first) {
        t.n = std::min(gc::GROUP, n - first);
        t.first[0] = 0;
        for (int i = 0; i < t.n; ++i) {
            t.g[i] = grads[first + i];
            t.out[i] = outs ? outs[first + i] : const_cast<void *>(grads[first + i]);
            t.size[i] = sizes[first + i];
            t.bf16[i] = kinds[first + i] == 1;
            t.first[i + 1] = t.first[i] + static_cast<int32_t>((sizes[first + i] + gc::CHUNK - 1) / gc::CHUNK);
        }
    };
    *launches = 0;
    for (int g = 0; g < groups; ++g) {
        fill(g * gc::GROUP);
        gc::grad_squares_kernel<<<gc::CTAS, gc::THREADS, 0, stream>>>(t, part + g * gc::CTAS);
        ++*launches;
    }
    if (!clip) {
        gc::grad_norm_kernel<<<1, gc::THREADS, 0, stream>>>(part, parts, norm_out);
        ++*launches;
        return cudaGetLastError();
    }
    for (int g = groups - 1; g >= 0; --g) {
        if (groups > 1) fill(g * gc::GROUP);
        gc::grad_scale_kernel<<<gc::CTAS, gc::THREADS, 0, stream>>>(t, part, parts, max_norm, norm_out);
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace moe

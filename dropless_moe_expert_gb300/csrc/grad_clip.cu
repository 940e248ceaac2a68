// The global norm of a step's gradients, and clipping by it, over many
// tensors of both types, with nothing read back to the host:
//   N = sqrt(sum over all tensors of |g|^2),  c = min(1, max_norm / (N + 1e-6)),  out = c g
// A NaN in any gradient makes N and c NaN; an infinity makes N infinite and c
// zero (so that entry becomes NaN): N tells the caller to skip the step.
//
// Two launches for every GROUP tensors each: the sums of squares, one fp32
// value per CTA in a fixed order of addition; then each CTA adds those values
// (in fp64, one warp: the fp64 units are few) and scales its part.  A thread
// adds the fp32 sums of its chunks in fp64, one addition a chunk: in fp32 equal
// terms round the same way each time, and 8.6e9 of them were off by up to 199
// units of 2^-24.  The
// tensors' addresses and sizes travel as kernel arguments, so the calls can be
// captured in a graph and need no table in device memory.
//
// Memory bounds both: a CTA takes 64 KB at a time, eight 16-byte loads of each
// thread in flight, and two CTAs share an SM.  The CTAs take chunks in turn
// (runs of neighbouring chunks per CTA: 84 us for 81 M bf16 values, in turn 80),
// and the second pass takes them backwards, so that it begins with what the
// first left in L2 (forwards: 82).  A layer's 605 M fp32 gradients take 1.09 ms,
// 6.7 TB/s over two reads and a write.
#include "kernels.h"
#include "ptx.cuh"
#include "vec8.cuh"

#include <algorithm>

namespace moe {
namespace gc {

constexpr int GROUP = 512;  // tensors per launch (29 bytes each of the 32 KB of kernel arguments)
constexpr int THREADS = 512;
constexpr int LOADS = 8;
constexpr int CHUNK_BYTES = THREADS * LOADS * 16;  // that a CTA takes at a time
constexpr int CTAS = 304;                          // two per SM
constexpr unsigned FULL = 0xffffffffu;

struct Table {
    const void *g[GROUP];
    void *out[GROUP];
    int64_t size[GROUP];
    int32_t first[GROUP + 1];  // the tensor's first chunk
    uint8_t bf16[GROUP];
    // The tensors of each CTA's first and last chunk: looked up in the table,
    // whose every cold read costs a constant-cache miss, they took two thirds
    // of a launch over small tensors.
    uint16_t begin[CTAS], end[CTAS];
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

// The thread's part of a chunk of n elements: one element before the first
// 16-byte boundary, LOADS vectors, one element behind the last whole vector.
template <typename E>
struct Part {
    static constexpr int V = 16 / sizeof(E);  // elements of a vector
    const E *g;
    int head, nvec, tail;
    float h, t;
    uint4 u[LOADS];
    __device__ __forceinline__ Part(const E *from, int n) : g(from) {
        head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(g) & 15)) % 16 / sizeof(E)));
        nvec = (n - head) / V;
        tail = n - head - nvec * V;
        const int tid = threadIdx.x;
        h = tid < head ? value(g + tid) : 0.0f;
        t = tid < tail ? value(g + head + nvec * V + tid) : 0.0f;
        const uint4 *p = reinterpret_cast<const uint4 *>(g + head);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            u[i] = tid + i * THREADS < nvec ? p[tid + i * THREADS] : make_uint4(0u, 0u, 0u, 0u);
    }
};

__device__ __forceinline__ float2 squares(const uint4 &u, const float *, float2 s) {
    s = fma2(make_float2(__uint_as_float(u.x), __uint_as_float(u.y)),
             make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), s);
    return fma2(make_float2(__uint_as_float(u.z), __uint_as_float(u.w)),
                make_float2(__uint_as_float(u.z), __uint_as_float(u.w)), s);
}
__device__ __forceinline__ float2 squares(const uint4 &u, const uint16_t *, float2 s) {
    float2 v[4];
    bf16x8_to_f32(u, &v[0].x);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(v[i], v[i], s);
    return s;
}
__device__ __forceinline__ uint4 scaled(const uint4 &u, const float *, float c) {
    return make_uint4(__float_as_uint(c * __uint_as_float(u.x)), __float_as_uint(c * __uint_as_float(u.y)),
                      __float_as_uint(c * __uint_as_float(u.z)), __float_as_uint(c * __uint_as_float(u.w)));
}
__device__ __forceinline__ uint4 scaled(const uint4 &u, const uint16_t *, float c) {
    float v[8];
    bf16x8_to_f32(u, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= c;
    return f32_to_bf16x8(v);
}

template <typename E>
__device__ __forceinline__ float sum_squares(const E *g, int n) {
    const Part<E> p(g, n);
    float2 s = make_float2(p.h * p.h, p.t * p.t);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) s = squares(p.u[i], g, s);
    return s.x + s.y;
}

template <typename E>
__device__ __forceinline__ void scale(const E *g, E *out, int n, float c) {
    const Part<E> p(g, n);
    const int tid = threadIdx.x;
    if (tid < p.head) put(out + tid, c * p.h);
    if (tid < p.tail) put(out + p.head + p.nvec * p.V + tid, c * p.t);
    E *to = out + p.head;
    const bool whole = (reinterpret_cast<uintptr_t>(to) & 15) == 0;  // the output's vectors are aligned too
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int v = tid + i * THREADS;
        if (v >= p.nvec) break;
        const uint4 o = scaled(p.u[i], g, c);
        if (whole) {
            reinterpret_cast<uint4 *>(to)[v] = o;
        } else {
            const E *e = reinterpret_cast<const E *>(&o);
#pragma unroll
            for (int q = 0; q < p.V; ++q) to[v * p.V + q] = e[q];
        }
    }
}

// Chunk `c`, of tensor i: where it begins and its elements.
template <typename E>
__device__ __forceinline__ int chunk_of(const Table &t, int i, int c, int64_t *at) {
    *at = static_cast<int64_t>(c - t.first[i]) * (CHUNK_BYTES / sizeof(E));
    return static_cast<int>(min(static_cast<int64_t>(CHUNK_BYTES / sizeof(E)), t.size[i] - *at));
}

__global__ void __launch_bounds__(THREADS, 2) grad_squares_kernel(const __grid_constant__ Table t, float *__restrict__ part) {
    __shared__ float red[THREADS / 32];
    double total = 0.0;  // of this thread
    int64_t at;
    for (int c = blockIdx.x, i = t.begin[blockIdx.x]; c < t.first[t.n]; c += gridDim.x) {
        if (c >= t.first[i + 1]) i = tensor_of(t, c);
        if (t.bf16[i]) {
            const int n = chunk_of<uint16_t>(t, i, c, &at);
            total += sum_squares(static_cast<const uint16_t *>(t.g[i]) + at, n);
        } else {
            const int n = chunk_of<float>(t, i, c, &at);
            total += sum_squares(static_cast<const float *>(t.g[i]) + at, n);
        }
    }
    float s = static_cast<float>(total);
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

// The norm from all partial sums; one warp.
__device__ __forceinline__ float total_norm(const float *part, int parts) {
    double s = 0.0;
    for (int i = threadIdx.x & 31; i < parts; i += 32 * 10) {
        float v[10];
#pragma unroll
        for (int q = 0; q < 10; ++q) v[q] = i + 32 * q < parts ? part[i + 32 * q] : 0.0f;
#pragma unroll
        for (int w = 5; w; w /= 2) {  // 10 -> 5 -> 4 -> 2 -> 1
#pragma unroll
            for (int q = 0; q < w; ++q) v[q] += v[q + w];
            if (w == 5) v[0] += v[4];
        }
        s += v[0];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    // s may pass what fp32 holds where its root does not; an fp64 root every time took 0.3 us of a call
    return s < 1e38 ? sqrtf(static_cast<float>(s)) : static_cast<float>(sqrt(s));
}

__global__ void __launch_bounds__(32)
grad_norm_kernel(const float *__restrict__ part, int parts, float *__restrict__ norm_out) {
    grid_dependency_wait();  // launched early: the partial sums
    const float norm = total_norm(part, parts);
    if (threadIdx.x == 0) *norm_out = norm;
}

__global__ void __launch_bounds__(THREADS, 2)
grad_scale_kernel(const __grid_constant__ Table t, const float *__restrict__ part, int parts, float max_norm,
                  float *__restrict__ norm_out) {
    __shared__ float factor;
    const int chunks = t.first[t.n], begin = blockIdx.x, step = gridDim.x;
    const int last = begin < chunks ? begin + (chunks - 1 - begin) / step * step : -1;
    int i = t.end[blockIdx.x];
    grid_dependency_wait();  // launched early: the partial sums
    if (threadIdx.x < 32) {
        const float norm = total_norm(part, parts);
        if (threadIdx.x == 0) {
            if (blockIdx.x == 0) *norm_out = norm;
            const float c = max_norm / (norm + 1e-6f);
            factor = c > 1.0f ? 1.0f : c;  // a NaN stays
        }
    }
    __syncthreads();
    const float f = factor;
    int64_t at;
    for (int c = last; c >= begin; c -= step) {
        if (c < t.first[i]) i = tensor_of(t, c);
        if (f == 1.0f && t.out[i] == t.g[i]) continue;  // in place and nothing to clip
        if (t.bf16[i]) {
            const int n = chunk_of<uint16_t>(t, i, c, &at);
            scale(static_cast<const uint16_t *>(t.g[i]) + at, static_cast<uint16_t *>(t.out[i]) + at, n, f);
        } else {
            const int n = chunk_of<float>(t, i, c, &at);
            scale(static_cast<const float *>(t.g[i]) + at, static_cast<float *>(t.out[i]) + at, n, f);
        }
    }
}

int groups(int n) { return std::max(1, (n + GROUP - 1) / GROUP); }

}  // namespace gc

size_t grad_clip_part_bytes(int n) { return static_cast<size_t>(gc::groups(n)) * gc::CTAS * sizeof(float); }

cudaError_t launch_grad_clip(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *kinds,
                             int n, bool clip, float max_norm, float *norm_out, float *part, int *launches,
                             cudaStream_t stream) {
    const int groups = gc::groups(n);
    gc::Table t;
    // the group's table; returns its CTAs
    auto fill = [&](int first) {
        t.n = std::min(gc::GROUP, n - first);
        t.first[0] = 0;
        for (int i = 0; i < t.n; ++i) {
            const bool bf16 = kinds[first + i] == 1;
            const int64_t chunk = gc::CHUNK_BYTES / (bf16 ? 2 : 4);
            t.g[i] = grads[first + i];
            t.out[i] = outs ? outs[first + i] : const_cast<void *>(grads[first + i]);
            t.size[i] = sizes[first + i];
            t.bf16[i] = bf16;
            t.first[i + 1] = t.first[i] + static_cast<int32_t>((sizes[first + i] + chunk - 1) / chunk);
        }
        const int chunks = t.first[t.n], ctas = std::max(1, std::min(gc::CTAS, chunks));
        for (int b = 0, i = 0; b < ctas; ++b) {
            while (i + 1 < t.n && b >= t.first[i + 1]) ++i;
            t.begin[b] = static_cast<uint16_t>(i);
        }
        // the last chunks of the CTAs are the last `ctas` chunks
        for (int q = 0, i = t.n - 1; q < ctas; ++q) {
            const int c = chunks - 1 - q;
            while (i > 0 && c < t.first[i]) --i;
            t.end[c >= 0 ? c % ctas : 0] = static_cast<uint16_t>(std::max(i, 0));
        }
        return ctas;
    };
    *launches = 0;
    int parts = 0, ctas = 0;
    for (int g = 0; g < groups; ++g) {
        ctas = fill(g * gc::GROUP);
        gc::grad_squares_kernel<<<ctas, gc::THREADS, 0, stream>>>(t, part + parts);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        parts += ctas;
        ++*launches;
    }
    if (!clip) {
        ++*launches;
        return launch_dependent(gc::grad_norm_kernel, 1, 32, stream, static_cast<const float *>(part), parts, norm_out);
    }
    for (int g = groups - 1; g >= 0; --g) {
        if (groups > 1) ctas = fill(g * gc::GROUP);
        const cudaError_t e = launch_dependent(gc::grad_scale_kernel, ctas, gc::THREADS, stream, t,
                                               static_cast<const float *>(part), parts, max_norm, norm_out);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    return cudaSuccess;
}

}  // namespace moe

// What stands between two layers, in one pass over the rows: the norm of a
// layer's output y, its gate, the residual's scale and sum, and the norm that
// the next layer reads.  fp32 throughout, rounded once where a row is stored:
//   u  = y rp gp,  rp = 1 / sqrt(mean(y^2) + eps)      (u = y without gamma_post)
//   r' = a r + g u                                     (r' = r without y; g: [d], [T] or 1)
//   n  = r' rq gq, rq = 1 / sqrt(mean(r'^2) + eps)     (none without gamma_pre)
// The norm of r' takes the 32-bit r', before r_out is rounded.
//
// Backward, for the gradients dr' and dn; h = dn gq, r' as it was stored:
//   D   = dr' + rq (h - r' rq^2 mean(h r'))            (D = dr' without gamma_pre)
//   dr  = a D,   dgq = sum_t dn r' rq
//   k   = g D gp,  dy = rp (k - y rp^2 mean(k y))      (dy = g D without gamma_post)
//   dgp = sum_t g D y rp,   dg = u D summed over the axis that g is shared along
// The sums over t run in a fixed order: each CTA over its own rows, then the
// CTAs' partial sums in their order.
#include "kernels.h"
#include "vec8.cuh"

#include <algorithm>

namespace moe {
namespace nr {

constexpr unsigned FULL = 0xffffffffu;
constexpr int FWD_THREADS = 256;
constexpr int BWD_THREADS = 512;
constexpr int BWD_MAX_CTAS = 304;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// Sum over the block, the same in every thread; `red` holds a float per warp.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    __syncthreads();  // the last sum's readers are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += red[w];
    return s;
}

template <typename R>
__global__ void __launch_bounds__(FWD_THREADS)
norm_residual_kernel(NormResidualArgs a, const R *r, R *r_out, uint16_t *__restrict__ n, float *__restrict__ rstd_post,
                     float *__restrict__ rstd_pre) {
    extern __shared__ float s_row[];  // r' in 32 bits
    __shared__ float red[FWD_THREADS / 32];
    const int t = blockIdx.x;
    const size_t at = static_cast<size_t>(t) * a.d;
    const int nvec = a.d / 8;
    float rp = 1.0f;
    if (a.gamma_post) {
        float ss = 0.0f;
        for (int v = threadIdx.x; v < nvec; v += FWD_THREADS) {
            float y[8];
            load8(a.y + at, v, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(y[i], y[i], ss);
        }
        rp = 1.0f / sqrtf(block_sum<FWD_THREADS>(ss, red) / a.d + a.eps);
        if (threadIdx.x == 0) rstd_post[t] = rp;
    }
    const float gt = a.gate && a.gate_per_token ? a.gate[t] : 1.0f;
    float ss = 0.0f;
    for (int v = threadIdx.x; v < nvec; v += FWD_THREADS) {
        float x[8];
        load8(r + at, v, x);
        if (a.y) {
            float y[8], w[8];
            load8(a.y + at, v, y);
            if (a.gamma_post) {
                load8(a.gamma_post, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * rp * w[i];
            }
            if (a.gate && !a.gate_per_token) {
                load8(a.gate, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(a.res_scale, x[i], gt * y[i]);
            store8(r_out + at, v, x);
        }
        if (a.gamma_pre) {
            store8(s_row, v, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], ss);
        }
    }
    if (!a.gamma_pre) return;
    const float rq = 1.0f / sqrtf(block_sum<FWD_THREADS>(ss, red) / a.d + a.eps);
    if (threadIdx.x == 0) rstd_pre[t] = rq;
    for (int v = threadIdx.x; v < nvec; v += FWD_THREADS) {
        float x[8], w[8];
        load8(s_row, v, x);  // what this thread stored
        load8(a.gamma_pre, v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * rq * w[i];
        store8(n + at, v, x);
    }
}

// Each CTA takes rows blockIdx.x, + gridDim.x, ..; a thread owns VPT vectors
// of eight columns and keeps their two sums over the rows (of dn r' rq, and
// of y rp D, from which both dgp and a shared gate's dg follow).
template <typename R, int VPT>
__global__ void __launch_bounds__(BWD_THREADS)
norm_residual_bwd_kernel(NormResidualArgs a, const R *__restrict__ r_out, const R *dr_out,
                         const uint16_t *__restrict__ dn, const float *__restrict__ rstd_post,
                         const float *__restrict__ rstd_pre, R *dr, uint16_t *__restrict__ dy,
                         float *__restrict__ dgate, float *__restrict__ part) {
    __shared__ float red[BWD_THREADS / 32];
    const int nvec = a.d / 8;
    float accq[VPT][8], accp[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) accq[j][i] = accp[j][i] = 0.0f;

    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t at = static_cast<size_t>(t) * a.d;
        const float rp = a.gamma_post ? rstd_post[t] : 1.0f;
        const float rq = a.gamma_pre ? rstd_pre[t] : 0.0f;
        const float gt = a.gate && a.gate_per_token ? a.gate[t] : 1.0f;
        float m1 = 0.0f;
        if (a.gamma_pre) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = threadIdx.x + j * BWD_THREADS;
                if (v >= nvec) break;
                float x[8], g[8], w[8];
                load8(r_out + at, v, x);
                load8(dn + at, v, g);
                load8(a.gamma_pre, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m1 = __fmaf_rn(g[i] * w[i], x[i], m1);
                    accq[j][i] = __fmaf_rn(g[i] * rq, x[i], accq[j][i]);
                }
            }
            m1 = block_sum<BWD_THREADS>(m1, red) / a.d * rq * rq;
        }
        float m2 = 0.0f, dg = 0.0f;
        float D[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * BWD_THREADS;
            if (v >= nvec) break;
            if (dr_out) {
                load8(dr_out + at, v, D[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) D[j][i] = 0.0f;
            }
            if (a.gamma_pre) {
                float x[8], g[8], w[8];
                load8(r_out + at, v, x);
                load8(dn + at, v, g);
                load8(a.gamma_pre, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) D[j][i] = __fmaf_rn(rq, g[i] * w[i] - x[i] * m1, D[j][i]);
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.y ? a.res_scale * D[j][i] : D[j][i];
            store8(dr + at, v, o);
            if (!a.y) continue;
            float y[8], w[8], c[8];
            load8(a.y + at, v, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = c[i] = 1.0f;
            if (a.gamma_post) load8(a.gamma_post, v, w);
            if (a.gate && !a.gate_per_token) load8(a.gate, v, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = y[i] * D[j][i] * rp;
                accp[j][i] = __fmaf_rn(gt, q, accp[j][i]);
                dg = __fmaf_rn(q, w[i], dg);
                D[j][i] *= gt * c[i] * w[i];  // k
                m2 = __fmaf_rn(D[j][i], y[i], m2);
            }
        }
        if (!a.y) continue;
        if (a.gate && a.gate_per_token) {
            dg = block_sum<BWD_THREADS>(dg, red);
            if (threadIdx.x == 0) dgate[t] = dg;
        }
        if (a.gamma_post) m2 = block_sum<BWD_THREADS>(m2, red) / a.d * rp * rp;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * BWD_THREADS;
            if (v >= nvec) break;
            if (a.gamma_post) {
                float y[8];
                load8(a.y + at, v, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) D[j][i] = rp * (D[j][i] - y[i] * m2);
            }
            store8(dy + at, v, D[j]);
        }
    }
    float *mine = part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = threadIdx.x + j * BWD_THREADS;
        if (v >= nvec) break;
        store8(mine, v, accq[j]);
        store8(mine + a.d, v, accp[j]);
    }
}

// The CTAs' partial sums in their order; a thread per column.
__global__ void __launch_bounds__(128)
norm_residual_bwd_columns_kernel(NormResidualArgs a, const float *__restrict__ part, int ctas,
                                 float *__restrict__ dgamma_pre, float *__restrict__ dgamma_post,
                                 float *__restrict__ dgate) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= a.d) return;
    float q = 0.0f, p = 0.0f;
    for (int b = 0; b < ctas; ++b) {
        q += part[static_cast<size_t>(b) * 2 * a.d + c];
        p += part[static_cast<size_t>(b) * 2 * a.d + a.d + c];
    }
    if (a.gamma_pre) dgamma_pre[c] = q;
    const bool shared = a.gate && !a.gate_per_token;
    if (a.gamma_post) dgamma_post[c] = shared ? a.gate[c] * p : p;
    if (shared) dgate[c] = a.gamma_post ? a.gamma_post[c] * p : p;
}

int bwd_ctas(int T) { return std::min(T, BWD_MAX_CTAS); }

}  // namespace nr

cudaError_t launch_norm_residual(const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n, float *rstd_post,
                                 float *rstd_pre, cudaStream_t stream) {
    const size_t smem = a.gamma_pre ? static_cast<size_t>(a.d) * 4 : 0;
    auto go = [&](auto kernel, auto *src, auto *dst) {
        if (smem > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxD * 4);
            if (e != cudaSuccess) return e;
        }
        kernel<<<a.T, nr::FWD_THREADS, smem, stream>>>(a, src, dst, n, rstd_post, rstd_pre);
        return cudaGetLastError();
    };
    if (a.res_f32)
        return go(nr::norm_residual_kernel<float>, static_cast<const float *>(r), static_cast<float *>(r_out));
    return go(nr::norm_residual_kernel<uint16_t>, static_cast<const uint16_t *>(r), static_cast<uint16_t *>(r_out));
}

size_t norm_residual_bwd_part_bytes(int T, int d) { return static_cast<size_t>(nr::bwd_ctas(T)) * 2 * d * 4; }

cudaError_t launch_norm_residual_bwd(const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                                     int *launches, cudaStream_t stream) {
    const int ctas = nr::bwd_ctas(a.T);
    auto go = [&](auto kernel, auto *r) {
        using R = std::remove_pointer_t<decltype(r)>;
        kernel<<<ctas, nr::BWD_THREADS, 0, stream>>>(a, static_cast<const R *>(g.r_out), static_cast<const R *>(g.dr_out),
                                                     g.dn, g.rstd_post, g.rstd_pre, static_cast<R *>(g.dr), g.dy,
                                                     g.dgate, part);
        return cudaGetLastError();
    };
    auto by_width = [&](auto *r) {
        using R = std::remove_pointer_t<decltype(r)>;
        if (a.d <= nr::BWD_THREADS * 8) return go(nr::norm_residual_bwd_kernel<R, 1>, r);
        if (a.d <= nr::BWD_THREADS * 16) return go(nr::norm_residual_bwd_kernel<R, 2>, r);
        return go(nr::norm_residual_bwd_kernel<R, 4>, r);
    };
    *launches = 1;
    cudaError_t err = a.res_f32 ? by_width(static_cast<float *>(nullptr)) : by_width(static_cast<uint16_t *>(nullptr));
    if (err != cudaSuccess || !(a.gamma_pre || a.gamma_post || (a.gate && !a.gate_per_token))) return err;
    *launches = 2;
    nr::norm_residual_bwd_columns_kernel<<<(a.d + 127) / 128, 128, 0, stream>>>(a, part, ctas, g.dgamma_pre,
                                                                                g.dgamma_post, g.dgate);
    return cudaGetLastError();
}

}  // namespace moe

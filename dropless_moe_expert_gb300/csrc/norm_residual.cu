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
#include "ptx.cuh"
#include "vec8.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace nr {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SMS = 152;
constexpr int FWD_MAX_THREADS = 1024;  // 64 registers each
constexpr int BWD_MAX_THREADS = 512;   // 128 registers each
constexpr int RING_BYTES = 208 * 1024; // the largest ring of a CTA

// Rows in flight: 4 while a thread owns one vector, 2 and 1 for the wider rows, which fill shared memory.
__host__ __device__ constexpr int ring_stages(int vpt) { return 4 / vpt; }

// A row lies in shared memory in pieces of 32 vectors of eight elements, one
// vector per lane of the warp that copies and reads the piece.  fp32: the
// 16-byte halves of the vectors in two planes, so that a warp copies 512
// consecutive bytes and reads them without bank conflicts; the 64 bytes between the
// planes keep the copies apart too.
template <typename T>
__host__ __device__ constexpr int piece_bytes() { return sizeof(T) == 4 ? 1088 : 512; }

template <typename T>
__device__ __forceinline__ void fetch(uint8_t *dst, const T *row, int nvec, int piece, int lane) {
    dst += piece * piece_bytes<T>();
    if constexpr (sizeof(T) == 2) {
        const int v = piece * 32 + lane;
        if (v < nvec) cp_async_16(dst + lane * 16, row + 8 * v);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = piece * 64 + q * 32 + lane;
            if (c < 2 * nvec) cp_async_16(dst + (lane & 1) * 576 + (q * 16 + (lane >> 1)) * 16, row + 4 * c);
        }
    }
}

template <typename T>
__device__ __forceinline__ void read8(const uint8_t *src, int piece, int lane, float *o) {
    src += piece * piece_bytes<T>() + lane * 16;
    if constexpr (sizeof(T) == 2) {
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src), o);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 576);
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// Sum over the block, the same in every thread.  `red` (a float per warp) is
// one of two that calls take in turn: a call's barrier then also separates the
// last reads of the other one from its next writes.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f);
}

// The same for four values at once: each exchange of the first two halves the
// values that a lane carries, so a warp takes 6 exchanges instead of 20.
__device__ __forceinline__ void block_sum4(float (&v)[4], float (*red)[32]) {
    const int lane = threadIdx.x & 31;
    const int warps = blockDim.x >> 5;
    const bool up = lane & 16, odd = lane & 8;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(FULL, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(FULL, up ? v[1] : v[3], 16);
    float s = (odd ? b : a) + __shfl_xor_sync(FULL, odd ? a : b, 8);
    const int mine = lane >> 3;  // the value whose sum this lane's group of eight ends with
#pragma unroll
    for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    if ((lane & 7) == 0) red[mine][threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = lane & 7; w < warps; w += 8) s += red[mine][w];
#pragma unroll
    for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(FULL, s, 8 * i);
}

// Weight of eight columns of y (gamma_post times a channel gate) and of n.
__device__ __forceinline__ void weights(const NormResidualArgs &a, int v, bool ok, float *c, float *w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = w[i] = 1.0f;
    if (!ok) return;
    if (a.gamma_post) load8(a.gamma_post, v, c);
    if (a.gate && !a.gate_per_token) {
        float g[8];
        load8(a.gate, v, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] *= g[i];
    }
    if (a.gamma_pre) load8(a.gamma_pre, v, w);
}

// CTAs take rows blockIdx.x, + gridDim.x, ..; a thread owns VPT vectors of
// eight columns.  Its rows come ahead of their use through a ring of STAGES
// rows in shared memory (each warp copies what it reads, so no barrier is
// needed for them).
template <typename R, int VPT>
__global__ void __launch_bounds__(FWD_MAX_THREADS)
norm_residual_kernel(NormResidualArgs a, const R *r, R *r_out, uint16_t *__restrict__ n, float *__restrict__ rstd_post,
                     float *__restrict__ rstd_pre) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nvec = a.d / 8;
    const int y_bytes = VPT * warps * piece_bytes<uint16_t>();
    const int stage = y_bytes + VPT * warps * piece_bytes<R>();
    constexpr int STAGES = ring_stages(VPT);
    constexpr bool HOLD = VPT == 1;  // the weights stay in registers
    float c[8], w[8];
    if (HOLD) weights(a, warp * 32 + lane, warp * 32 + lane < nvec, c, w);

    auto issue = [&](int64_t t, int slot) {
        if (t < a.T) {
            uint8_t *at = ring + slot * stage;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int piece = warp + j * warps;
                if (a.y) fetch(at, a.y + t * a.d, nvec, piece, lane);
                fetch(at + y_bytes, r + t * a.d, nvec, piece, lane);
            }
        }
        cp_async_commit();
    };
    const int64_t step = gridDim.x;
    for (int s = 0; s < STAGES - 1; ++s) issue(blockIdx.x + s * step, s);
    const bool token_gate = a.gate && a.gate_per_token;
    float gt = token_gate ? a.gate[blockIdx.x] : 1.0f;
    int slot = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step) {
        const float gt_next = token_gate && t + step < a.T ? a.gate[t + step] : 1.0f;
        __syncwarp();  // the slot that is filled next has been read
        issue(t + (STAGES - 1) * step, slot + STAGES - 1 >= STAGES ? slot - 1 : slot + STAGES - 1);
        cp_async_wait_group<STAGES - 1>();
        __syncwarp();
        const uint8_t *at = ring + slot * stage;
        float x[VPT][8], rp = 1.0f;
        if (a.gamma_post) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int piece = warp + j * warps;
                if (piece * 32 + lane >= nvec) break;
                float y[8];
                read8<uint16_t>(at, piece, lane, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __fmaf_rn(y[i], y[i], ss);
            }
            rp = 1.0f / sqrtf(block_sum(ss, red[turn]) / a.d + a.eps);
            turn ^= 1;
            if (threadIdx.x == 0) rstd_post[t] = rp;
        }
        const float f = rp * gt;
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps, v = piece * 32 + lane;
            if (v >= nvec) break;
            read8<R>(at + y_bytes, piece, lane, x[j]);
            if (a.y) {
                float y[8];
                read8<uint16_t>(at, piece, lane, y);
                if (!HOLD) weights(a, v, true, c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = __fmaf_rn(a.res_scale, x[j][i], f * (y[i] * c[i]));
                store8(r_out + t * a.d, v, x[j]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[j][i], x[j][i], ss);
        }
        if (a.gamma_pre) {
            const float rq = 1.0f / sqrtf(block_sum(ss, red[turn]) / a.d + a.eps);
            turn ^= 1;
            if (threadIdx.x == 0) rstd_pre[t] = rq;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = (warp + j * warps) * 32 + lane;
                if (v >= nvec) break;
                if (!HOLD) load8(a.gamma_pre, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * rq * w[i];
                store8(n + t * a.d, v, x[j]);
            }
        }
        gt = gt_next;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
}

// Rows as above.  One reduction gives both means of a row: with m1 = rq^2
// mean(h r') and c the weight of y without a token gate g,
//   sum(k y) = g (sum(c y dr') + rq (sum(c y h) - m1 sum(c y r'))),
// and the token gate's gradient is the same bracket times rp.  Each thread
// keeps its columns' two sums over the rows (of dn r' rq, and of g y rp D,
// from which both dgp and a channel gate's dg follow).
template <typename R, int VPT>
__global__ void __launch_bounds__(BWD_MAX_THREADS)
norm_residual_bwd_kernel(NormResidualArgs a, const R *__restrict__ r_out, const R *dr_out,
                         const uint16_t *__restrict__ dn, const float *__restrict__ rstd_post,
                         const float *__restrict__ rstd_pre, R *dr, uint16_t *__restrict__ dy,
                         float *__restrict__ dgate, float *__restrict__ part) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nvec = a.d / 8;
    const int b_bytes = VPT * warps * piece_bytes<uint16_t>(), r_bytes = VPT * warps * piece_bytes<R>();
    const int at_y = 0, at_dn = b_bytes, at_x = 2 * b_bytes, at_dr = at_x + r_bytes, stage = at_dr + r_bytes;
    constexpr int STAGES = ring_stages(VPT);
    constexpr bool HOLD = VPT <= 2;
    float c[VPT][8], w[VPT][8], accq[VPT][8], accp[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = (warp + j * warps) * 32 + lane;
        if (HOLD) weights(a, v, v < nvec, c[j], w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) accq[j][i] = accp[j][i] = 0.0f;
    }

    auto issue = [&](int64_t t, int slot) {
        if (t < a.T) {
            uint8_t *at = ring + slot * stage;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int piece = warp + j * warps;
                if (a.y) fetch(at + at_y, a.y + t * a.d, nvec, piece, lane);
                if (dr_out) fetch(at + at_dr, dr_out + t * a.d, nvec, piece, lane);
                if (a.gamma_pre) {
                    fetch(at + at_dn, dn + t * a.d, nvec, piece, lane);
                    fetch(at + at_x, r_out + t * a.d, nvec, piece, lane);
                }
            }
        }
        cp_async_commit();
    };
    // the row's three factors, one row ahead
    struct Row {
        float rp, rq, gt;
    };
    auto factors = [&](int64_t t) {
        Row f{1.0f, 0.0f, 1.0f};
        if (t < a.T) {
            if (a.gamma_post) f.rp = rstd_post[t];
            if (a.gamma_pre) f.rq = rstd_pre[t];
            if (a.gate && a.gate_per_token) f.gt = a.gate[t];
        }
        return f;
    };
    const int64_t step = gridDim.x;
    for (int s = 0; s < STAGES - 1; ++s) issue(blockIdx.x + s * step, s);
    Row f = factors(blockIdx.x);
    int slot = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step) {
        const Row next = factors(t + step);
        __syncwarp();
        issue(t + (STAGES - 1) * step, slot + STAGES - 1 >= STAGES ? slot - 1 : slot + STAGES - 1);
        cp_async_wait_group<STAGES - 1>();
        __syncwarp();
        const uint8_t *at = ring + slot * stage;
        // sums of h r', c y dr', c y h, c y r'
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps, v = piece * 32 + lane;
            if (v >= nvec) break;
            if (!HOLD) weights(a, v, true, c[j], w[j]);
            float cy[8];
            if (a.y) {
                read8<uint16_t>(at + at_y, piece, lane, cy);
#pragma unroll
                for (int i = 0; i < 8; ++i) cy[i] *= c[j][i];
                if (dr_out) {
                    float g[8];
                    read8<R>(at + at_dr, piece, lane, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[1] = __fmaf_rn(cy[i], g[i], s[1]);
                }
            }
            if (a.gamma_pre) {
                float x[8], g[8];
                read8<R>(at + at_x, piece, lane, x);
                read8<uint16_t>(at + at_dn, piece, lane, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float h = g[i] * w[j][i];
                    s[0] = __fmaf_rn(h, x[i], s[0]);
                    accq[j][i] = __fmaf_rn(g[i] * f.rq, x[i], accq[j][i]);
                    if (a.y) {
                        s[2] = __fmaf_rn(cy[i], h, s[2]);
                        s[3] = __fmaf_rn(cy[i], x[i], s[3]);
                    }
                }
            }
        }
        block_sum4(s, red[turn]);
        turn ^= 1;
        const float m1 = s[0] / a.d * f.rq * f.rq;
        const float ky = s[1] + f.rq * (s[2] - m1 * s[3]);
        const float m2 = f.gt * ky / a.d * f.rp * f.rp;
        if (a.gate && a.gate_per_token && threadIdx.x == 0) dgate[t] = f.rp * ky;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps, v = piece * 32 + lane;
            if (v >= nvec) break;
            if (!HOLD) weights(a, v, true, c[j], w[j]);
            float D[8];
            if (dr_out) {
                read8<R>(at + at_dr, piece, lane, D);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) D[i] = 0.0f;
            }
            if (a.gamma_pre) {
                float x[8], g[8];
                read8<R>(at + at_x, piece, lane, x);
                read8<uint16_t>(at + at_dn, piece, lane, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) D[i] = __fmaf_rn(f.rq, g[i] * w[j][i] - x[i] * m1, D[i]);
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.res_scale * D[i];  // 1 without y
            store8(dr + t * a.d, v, o);
            if (!a.y) continue;
            float y[8];
            read8<uint16_t>(at + at_y, piece, lane, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                D[i] *= f.gt;
                accp[j][i] = __fmaf_rn(y[i] * f.rp, D[i], accp[j][i]);
                o[i] = D[i] * c[j][i];  // k
                if (a.gamma_post) o[i] = f.rp * (o[i] - y[i] * m2);
            }
            store8(dy + t * a.d, v, o);
        }
        f = next;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    float *mine = part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = (warp + j * warps) * 32 + lane;
        if (v >= nvec) break;
        store8(mine, v, accq[j]);
        store8(mine + a.d, v, accp[j]);
    }
}

// The CTAs' partial sums: 32 columns per block, each in eight runs of CTAs in
// their order, then the runs in theirs.
__global__ void __launch_bounds__(256)
norm_residual_bwd_columns_kernel(NormResidualArgs a, const float *__restrict__ part, int ctas,
                                 float *__restrict__ dgamma_pre, float *__restrict__ dgamma_post,
                                 float *__restrict__ dgate) {
    __shared__ float s_q[8][32], s_p[8][32];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // d is a multiple of 32
    const int each = (ctas + 7) / 8;
    float q = 0.0f, p = 0.0f;
#pragma unroll 8
    for (int b = run * each; b < min(ctas, (run + 1) * each); ++b) {
        q += part[static_cast<size_t>(b) * 2 * a.d + col];
        p += part[static_cast<size_t>(b) * 2 * a.d + a.d + col];
    }
    s_q[run][lane] = q;
    s_p[run][lane] = p;
    __syncthreads();
    if (run != 0) return;
    for (int i = 1; i < 8; ++i) q += s_q[i][lane], p += s_p[i][lane];
    if (a.gamma_pre) dgamma_pre[col] = q;
    const bool channel = a.gate && !a.gate_per_token;
    if (a.gamma_post) dgamma_post[col] = channel ? a.gate[col] * p : p;
    if (channel) dgate[col] = a.gamma_post ? a.gamma_post[col] * p : p;
}

// Threads of a CTA, its vectors per thread, the CTAs and the ring for rows of d elements.
struct Shape {
    int vpt, threads, ctas;
    size_t smem;
};
Shape shape(int T, int d, int max_threads, int bf16_rows, int res_rows, bool res_f32) {
    Shape s;
    const int nvec = d / 8;
    s.vpt = 1;
    while (nvec > s.vpt * max_threads) s.vpt *= 2;
    s.threads = (nvec + 32 * s.vpt - 1) / (32 * s.vpt) * 32;
    s.ctas = std::min(T, SMS * std::min(16, max_threads / s.threads));
    s.smem = static_cast<size_t>(ring_stages(s.vpt)) * s.vpt * (s.threads / 32) *
             (bf16_rows * piece_bytes<uint16_t>() +
              res_rows * (res_f32 ? piece_bytes<float>() : piece_bytes<uint16_t>()));
    return s;
}
Shape bwd_shape(int T, int d, bool res_f32) { return shape(T, d, BWD_MAX_THREADS, 2, 2, res_f32); }

// Raises the kernel's limit of dynamic shared memory, once per device.
template <typename Kernel>
cudaError_t allow_ring(Kernel kernel, std::atomic<uint64_t> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

template <typename R, int VPT>
cudaError_t forward(const Shape &s, const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n,
                    float *rstd_post, float *rstd_pre, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(norm_residual_kernel<R, VPT>, done);
    if (e != cudaSuccess) return e;
    norm_residual_kernel<R, VPT><<<s.ctas, s.threads, s.smem, stream>>>(
        a, static_cast<const R *>(r), static_cast<R *>(r_out), n, rstd_post, rstd_pre);
    return cudaGetLastError();
}

template <typename R, int VPT>
cudaError_t backward(const Shape &s, const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                     cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(norm_residual_bwd_kernel<R, VPT>, done);
    if (e != cudaSuccess) return e;
    norm_residual_bwd_kernel<R, VPT><<<s.ctas, s.threads, s.smem, stream>>>(
        a, static_cast<const R *>(g.r_out), static_cast<const R *>(g.dr_out), g.dn, g.rstd_post, g.rstd_pre,
        static_cast<R *>(g.dr), g.dy, g.dgate, part);
    return cudaGetLastError();
}

}  // namespace nr

cudaError_t launch_norm_residual(const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n, float *rstd_post,
                                 float *rstd_pre, cudaStream_t stream) {
    const nr::Shape s = nr::shape(a.T, a.d, nr::FWD_MAX_THREADS, 1, 1, a.res_f32);
    auto go = [&](auto type) {
        using R = decltype(type);
        return s.vpt == 1 ? nr::forward<R, 1>(s, a, r, r_out, n, rstd_post, rstd_pre, stream)
                          : nr::forward<R, 2>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
    };
    return a.res_f32 ? go(float{}) : go(uint16_t{});
}

size_t norm_residual_bwd_part_bytes(int T, int d) {
    return static_cast<size_t>(nr::bwd_shape(T, d, false).ctas) * 2 * d * 4;
}

cudaError_t launch_norm_residual_bwd(const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                                     int *launches, cudaStream_t stream) {
    const nr::Shape s = nr::bwd_shape(a.T, a.d, a.res_f32);
    auto go = [&](auto type) {
        using R = decltype(type);
        if (s.vpt == 1) return nr::backward<R, 1>(s, a, g, part, stream);
        return s.vpt == 2 ? nr::backward<R, 2>(s, a, g, part, stream) : nr::backward<R, 4>(s, a, g, part, stream);
    };
    *launches = 1;
    const cudaError_t err = a.res_f32 ? go(float{}) : go(uint16_t{});
    if (err != cudaSuccess || !(a.gamma_pre || a.gamma_post || (a.gate && !a.gate_per_token))) return err;
    *launches = 2;
    nr::norm_residual_bwd_columns_kernel<<<a.d / 32, 256, 0, stream>>>(a, part, s.ctas, g.dgamma_pre, g.dgamma_post,
                                                                       g.dgate);
    return cudaGetLastError();
}

}  // namespace moe

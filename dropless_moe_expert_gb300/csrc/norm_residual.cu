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
#include <atomic>

namespace moe {
namespace nr {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SMS = 152;
constexpr int MAX_THREADS = 512;       // of an SM, 128 registers each (the narrow forward: twice as many, 64 each)
constexpr int RING_BYTES = 208 * 1024; // the rings of an SM's CTAs
constexpr int MAX_STAGES = 4;

// Which backward kernels read a row ahead: those whose ring always holds three rows.
template <typename R>
__host__ __device__ constexpr bool pipelined(int vpt) { return vpt == 1 || (vpt == 2 && sizeof(R) == 2); }

// With what the launch adds to the caller's arguments.
struct Args : NormResidualArgs {
    int stages;  // rows in the ring
    bool wide;   // the fp32 rows that are written begin on 32-byte boundaries
    int *status;       // of the bounded waits
    uint64_t wait_ns;
};


// A row lies in shared memory in pieces of 32 vectors of eight elements, one
// vector per lane of the warp that copies and reads the piece, in the order of
// global memory: with the 16-byte halves of fp32 vectors in two planes the reads
// had no bank conflicts, but the copies no longer went as whole sectors (backward
// of 4093 x 7168 fp32: 127 us, 103 in order).
template <typename T>
__host__ __device__ constexpr int piece_bytes() { return sizeof(T) == 4 ? 1024 : 512; }

// A lane's part of copying piece `piece`: where in the row, where in the piece, and which of its copies exist.
template <typename T>
struct Copy {
    static constexpr int N = sizeof(T) / 2;
    int from, to;
    bool on[N];
    __device__ __forceinline__ Copy(int piece, int lane, int nvec) {
        from = piece * 256 + lane * (16 / static_cast<int>(sizeof(T)));
        to = piece * piece_bytes<T>() + lane * 16;
#pragma unroll
        for (int q = 0; q < N; ++q) on[q] = from + q * 128 < 8 * nvec;
    }
    __device__ __forceinline__ void go(uint8_t *dst, const T *row) const {
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (on[q]) cp_async_16(dst + to + q * 512, row + from + q * 128);
    }
};

template <typename T>
__device__ __forceinline__ void read8(const uint8_t *src, int piece, int lane, float2 (&o)[4]) {
    src += piece * piece_bytes<T>() + lane * 8 * static_cast<int>(sizeof(T));
    if constexpr (sizeof(T) == 2) {
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src), &o[0].x);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 16);
        o[0] = make_float2(a.x, a.y), o[1] = make_float2(a.z, a.w);
        o[2] = make_float2(b.x, b.y), o[3] = make_float2(b.z, b.w);
    }
}

// Until the oldest of the ring's rows is there (one group of copies per row).
__device__ __forceinline__ void wait_oldest(int stages) {
    switch (stages) {
        case 1: cp_async_wait_group<0>(); break;
        case 2: cp_async_wait_group<1>(); break;
        case 3: cp_async_wait_group<2>(); break;
        default: cp_async_wait_group<3>();
    }
}

__device__ __forceinline__ void store(uint16_t *row, int v, const float2 (&x)[4], bool) { store8(row, v, &x[0].x); }
__device__ __forceinline__ void store(float *row, int v, const float2 (&x)[4], bool wide) {
    wide ? store8_wide(row, v, &x[0].x) : store8(row, v, &x[0].x);
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

// The same for four values, in two steps around the caller's
// barrier.  Each exchange of the first two halves the values that a lane
// carries, so a warp takes 6 exchanges instead of 20; then every thread adds
// the warps' sums.
__device__ __forceinline__ void post_sums4(const float (&v)[4], float4 *red) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(FULL, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(FULL, up ? v[1] : v[3], 16);
    float s = (odd ? b : a) + __shfl_xor_sync(FULL, odd ? a : b, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    if ((lane & 7) == 0) reinterpret_cast<float *>(red + (threadIdx.x >> 5))[lane >> 3] = s;
}
__device__ __forceinline__ float4 collect_sums4(const float4 *red) {
    float2 a = both(0.0f), b = a;
    const int warps = blockDim.x >> 5;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
        const float4 s = red[w];
        a = add2(a, make_float2(s.x, s.y));
        b = add2(b, make_float2(s.z, s.w));
    }
    return make_float4(a.x, a.y, b.x, b.y);
}

// Weights of eight columns (vector v of nvec): c of y (gamma_post times a
// channel gate) and w of n; 1 for those left out.
__device__ __forceinline__ void weights(const NormResidualArgs &a, int v, int nvec, float2 (&c)[4], float2 (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = w[i] = both(1.0f);
    if (v >= nvec) return;
    if (a.gamma_post) load8(a.gamma_post, v, &c[0].x);
    if (a.gate && !a.gate_per_token) {
        float2 g[4];
        load8(a.gate, v, &g[0].x);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = mul2(c[i], g[i]);
    }
    if (a.gamma_pre) load8(a.gamma_pre, v, &w[0].x);
}

// Row r of CTA blockIdx.x is blockIdx.x + r gridDim.x.  A thread owns VPT
// vectors of eight columns; each warp copies the pieces that it reads, so its
// rows come ahead of their use through a ring in shared memory without
// barriers.  A row's slot is refilled as soon as the row is in registers, so
// the ring's copies stay in flight through the row's sums and stores.
template <typename R, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 2 * MAX_THREADS : MAX_THREADS)
norm_residual_kernel(Args a, float inv_d, const R *r, R *r_out, uint16_t *__restrict__ n,
                     float *__restrict__ rstd_post, float *__restrict__ rstd_pre) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    const int stages = a.stages;
    constexpr bool HOLD = VPT <= 2;  // the weights stay in registers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nvec = a.d / 8;
    const bool has_y = a.y != nullptr, post = a.gamma_post != nullptr, pre = a.gamma_pre != nullptr;
    const int y_bytes = VPT * warps * piece_bytes<uint16_t>();
    const int stage = y_bytes + VPT * warps * piece_bytes<R>();
    float2 c[VPT][4], w[VPT][4];
    if (HOLD) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) weights(a, (warp + j * warps) * 32 + lane, nvec, c[j], w[j]);
    }
    auto issue = [&](int64_t t, int slot) {
        if (t < a.T) {
            uint8_t *at = ring + slot * stage;
            const int64_t from = t * a.d;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (has_y) Copy<uint16_t>(warp + j * warps, lane, nvec).go(at, a.y + from);
                Copy<R>(warp + j * warps, lane, nvec).go(at + y_bytes, r + from);
            }
        }
        cp_async_commit();
    };
    const int64_t step = gridDim.x;
    for (int s = 0; s < stages; ++s) issue(blockIdx.x + s * step, s);
    const bool token_gate = a.gate && a.gate_per_token;
    float gt = token_gate ? a.gate[blockIdx.x] : 1.0f;
    int slot = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step) {
        const float gt_next = token_gate && t + step < a.T ? a.gate[t + step] : 1.0f;
        wait_oldest(stages);
        __syncwarp();  // what the warp's other lanes copied
        const uint8_t *at = ring + slot * stage;
        float2 x[VPT][4], y[VPT][4];
        float2 ss = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][i] = y[j][i] = both(0.0f);
            if (piece * 32 + lane >= nvec) continue;
            read8<R>(at + y_bytes, piece, lane, x[j]);
            if (has_y) {
                read8<uint16_t>(at, piece, lane, y[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(y[j][i], y[j][i], ss);
            }
        }
        __syncwarp();
        issue(t + stages * step, slot);
        slot = slot + 1 == stages ? 0 : slot + 1;
        if (has_y) {
            float f = gt;
            if (post) {
                const float rp = rsqrtf(__fmaf_rn(block_sum(ss.x + ss.y, red[turn]), inv_d, a.eps));
                turn ^= 1;
                if (threadIdx.x == 0) rstd_post[t] = rp;
                f *= rp;
            }
            R *out = r_out + t * a.d;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = (warp + j * warps) * 32 + lane;
                if (!HOLD) weights(a, v, nvec, c[j], w[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[j][i] = fma2(mul2(both(f), c[j][i]), y[j][i], mul2(both(a.res_scale), x[j][i]));
                if (v < nvec) store(out, v, x[j], a.wide);
            }
        }
        if (pre) {
            ss = both(0.0f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(x[j][i], x[j][i], ss);
            const float rq = rsqrtf(__fmaf_rn(block_sum(ss.x + ss.y, red[turn]), inv_d, a.eps));
            turn ^= 1;
            if (threadIdx.x == 0) rstd_pre[t] = rq;
            uint16_t *out = n + t * a.d;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = (warp + j * warps) * 32 + lane;
                if (!HOLD && v < nvec) load8(a.gamma_pre, v, &w[j][0].x);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = mul2(x[j][i], mul2(both(rq), w[j][i]));
                if (v < nvec) store8(out, v, &x[j][0].x);
            }
        }
        gt = gt_next;
    }
}

// Rows and ring as above, but the row is read from its slot twice, before and
// after the sums, and each piece refilled once it has been read the second time.
// PIPE: the first reading of row r + 1 stands between the sums of row r and
// their use, so one barrier per row remains and nothing waits for the sums'
// exchanges (8192 x 4096 bf16: 84.6 us, 79.7 with it); it needs a third row in the ring, which
// fp32 rows do not leave room for.
// One reduction gives both means of a row: with z = r' rq, m1 = rq mean(h z)
// and c the weight of y without a token gate g,
//   D = dr' + rq h - m1 z,   sum(c y D) = sum(c y dr') + rq sum(c y h) - m1 sum(c y z),
// g times which is sum(k y), and rp times which is the token gate's gradient.
// Each thread keeps its columns' two sums over the rows (of dn z, and of
// g y rp D, from which both dgp and a channel gate's dg follow).
// FULL: y, dr' and gamma_pre are all there (fewer branches in the inner loops).
template <typename R, int VPT, bool FULL>
__global__ void __launch_bounds__(MAX_THREADS)
norm_residual_bwd_kernel(Args a, float inv_d, const R *__restrict__ r_out, const R *dr_out,
                         const uint16_t *__restrict__ dn, const float *__restrict__ rstd_post,
                         const float *__restrict__ rstd_pre, R *dr, uint16_t *__restrict__ dy,
                         float *__restrict__ dgate, float *__restrict__ part) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float4 red[2][MAX_THREADS / 32];
    __shared__ uint64_t posted;  // a phase per row, an arrival per warp
    __shared__ int abort;
    constexpr bool PIPE = pipelined<R>(VPT);
    const int stages = a.stages;
    constexpr bool HOLD = VPT <= 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nvec = a.d / 8;
    const bool has_y = FULL || a.y, has_dr = FULL || dr_out, pre = FULL || a.gamma_pre, post = a.gamma_post != nullptr;
    const int b_bytes = VPT * warps * piece_bytes<uint16_t>(), r_bytes = VPT * warps * piece_bytes<R>();
    const int at_dn = b_bytes, at_x = 2 * b_bytes, at_dr = at_x + r_bytes, stage = at_dr + r_bytes;
    float2 c[VPT][4], w[VPT][4], accq[VPT][4], accp[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (HOLD) weights(a, (warp + j * warps) * 32 + lane, nvec, c[j], w[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) accq[j][i] = accp[j][i] = both(0.0f);
    }
    auto issue = [&](int64_t t, int slot, int piece) {
        if (t < a.T) {
            uint8_t *at = ring + slot * stage;
            const int64_t from = t * a.d;
            const Copy<uint16_t> b(piece, lane, nvec);
            const Copy<R> x(piece, lane, nvec);
            if (has_y) b.go(at, a.y + from);
            if (has_dr) x.go(at + at_dr, dr_out + from);
            if (pre) {
                b.go(at + at_dn, dn + from);
                x.go(at + at_x, r_out + from);
            }
        }
    };
    struct Row {  // the row's factors, loaded a row ahead
        float rp, rq, gt;
    };
    auto factors = [&](int64_t t) {
        Row f{1.0f, 0.0f, 1.0f};
        if (t < a.T) {
            if (post) f.rp = rstd_post[t];
            if (pre) f.rq = rstd_pre[t];
            if (a.gate && a.gate_per_token) f.gt = a.gate[t];
        }
        return f;
    };
    const int64_t step = gridDim.x;
    for (int s = 0; s < stages; ++s) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) issue(blockIdx.x + s * step, s, warp + j * warps);
        cp_async_commit();
    }
    // The first reading of the row in slot `slot`: the four sums (of h z,
    // c y dr', c y h, c y z) of the warp go to `sums`.
    auto first_pass = [&](int slot, float rq, float4 *sums) {
        const uint8_t *at = ring + slot * stage;
        float2 s0 = both(0.0f), s1 = s0, s2 = s0, s3 = s0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps, v = piece * 32 + lane;
            if (v >= nvec) continue;
            if (!HOLD) weights(a, v, nvec, c[j], w[j]);
            float2 cy[4];
            if (has_y) {
                read8<uint16_t>(at, piece, lane, cy);
#pragma unroll
                for (int i = 0; i < 4; ++i) cy[i] = mul2(cy[i], c[j][i]);
                if (has_dr) {
                    float2 g[4];
                    read8<R>(at + at_dr, piece, lane, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s1 = fma2(cy[i], g[i], s1);
                }
            }
            if (pre) {
                float2 z[4], g[4];
                read8<R>(at + at_x, piece, lane, z);
                read8<uint16_t>(at + at_dn, piece, lane, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[i] = mul2(z[i], both(rq));
                    accq[j][i] = fma2(g[i], z[i], accq[j][i]);
                    g[i] = mul2(g[i], w[j][i]);  // h
                    s0 = fma2(g[i], z[i], s0);
                }
                if (has_y) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s2 = fma2(cy[i], g[i], s2);
                        s3 = fma2(cy[i], z[i], s3);
                    }
                }
            }
        }
        const float s[4] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, s3.x + s3.y};
        post_sums4(s, sums);
        if (PIPE) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&posted);
        }
    };
    // Until every warp has posted its sums of the row (the waits alternate in parity).
    int parity = 0;
    auto collect = [&](const float4 *sums) {
        if (PIPE) {
            mbar_wait(&posted, parity, &abort, a.status, a.wait_ns);
            parity ^= 1;
        } else {
            __syncthreads();
        }
        return collect_sums4(sums);
    };
    if (PIPE) {
        if (threadIdx.x == 0) {
            mbar_init(&posted, warps);
            abort = 0;
            fence_mbar_init();
        }
        __syncthreads();
    }
    Row f = factors(blockIdx.x), next = factors(blockIdx.x + step);
    int slot = 0, turn = 0;
    if (PIPE) {
        wait_oldest(stages);
        __syncwarp();  // what the warp's other lanes copied
        first_pass(0, f.rq, red[0]);
    }
    for (int64_t t = blockIdx.x; t < a.T; t += step) {
        const Row after = factors(t + 2 * step);
        const int ahead = slot + 1 == stages ? 0 : slot + 1;
        float4 s;
        if (PIPE) {
            s = collect(red[turn]);
            wait_oldest(stages - 1);  // the newest `stages - 2` rows may still be on their way
            __syncwarp();
            if (t + step < a.T) first_pass(ahead, next.rq, red[turn ^ 1]);
        } else {
            wait_oldest(stages);
            __syncwarp();
            first_pass(slot, f.rq, red[turn]);
            s = collect(red[turn]);
        }
        turn ^= 1;
        const uint8_t *at = ring + slot * stage;
        const float m1 = f.rq * s.x * inv_d;
        const float cyD = s.y + f.rq * s.z - m1 * s.w;
        const float m2 = post ? f.gt * cyD * inv_d * f.rp * f.rp * f.rp : 0.0f;
        if (a.gate && a.gate_per_token && threadIdx.x == 0) dgate[t] = f.rp * cyD;
        const float2 q = both(f.gt * f.rp), mz = both(-m1 * f.rq), my = both(-m2), rq = both(f.rq);
        R *to_r = dr + t * a.d;
        uint16_t *to_y = dy + t * a.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int piece = warp + j * warps, v = piece * 32 + lane;
            float2 D[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) D[i] = both(0.0f);
            if (v < nvec) {
                if (!HOLD) weights(a, v, nvec, c[j], w[j]);
                if (has_dr) read8<R>(at + at_dr, piece, lane, D);
                if (pre) {
                    float2 x[4], g[4];
                    read8<R>(at + at_x, piece, lane, x);
                    read8<uint16_t>(at + at_dn, piece, lane, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) D[i] = fma2(mz, x[i], fma2(mul2(rq, g[i]), w[j][i], D[i]));
                }
                if (has_y) read8<uint16_t>(at, piece, lane, y);
            }
            __syncwarp();
            issue(t + stages * step, slot, piece);
            if (v >= nvec) continue;
            float2 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = mul2(both(a.res_scale), D[i]);  // res_scale is 1 without y
            store(to_r, v, o, a.wide);
            if (!has_y) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                D[i] = mul2(D[i], q);
                accp[j][i] = fma2(y[i], D[i], accp[j][i]);
                o[i] = fma2(my, y[i], mul2(D[i], c[j][i]));
            }
            store8(to_y, v, &o[0].x);
        }
        cp_async_commit();
        slot = ahead;
        f = next;
        next = after;
    }
    float *mine = part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = (warp + j * warps) * 32 + lane;
        if (v >= nvec) break;
        store8(mine, v, &accq[j][0].x);
        store8(mine + a.d, v, &accp[j][0].x);
    }
}

// The CTAs' partial sums: 32 columns per block, each in 32 runs of CTAs in
// their order, then the runs in theirs (runs of 5 to 10 for the usual 152 or
// 304 CTAs: every load of a thread in flight at once).
constexpr int RUNS = 32;
__global__ void __launch_bounds__(32 * RUNS)
norm_residual_bwd_columns_kernel(NormResidualArgs a, const float *__restrict__ part, int ctas,
                                 float *__restrict__ dgamma_pre, float *__restrict__ dgamma_post,
                                 float *__restrict__ dgate) {
    __shared__ float sums[2][RUNS][33];
    grid_dependency_wait();  // launched early: the partial sums
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // d is a multiple of 32
    const int each = (ctas + RUNS - 1) / RUNS;
    float q = 0.0f, p = 0.0f;
#pragma unroll 10
    for (int b = run * each; b < min(ctas, (run + 1) * each); ++b) {
        q += part[static_cast<size_t>(b) * 2 * a.d + col];
        p += part[static_cast<size_t>(b) * 2 * a.d + a.d + col];
    }
    sums[0][run][lane] = q;
    sums[1][run][lane] = p;
    __syncthreads();
    // warp 0 adds the runs of the first sums, warp 1 those of the second
    if (run > 1) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) v += sums[run][i][lane];
    if (run == 0) {
        if (a.gamma_pre) dgamma_pre[col] = v;
        return;
    }
    const bool channel = a.gate && !a.gate_per_token;
    if (a.gamma_post) dgamma_post[col] = channel ? a.gate[col] * v : v;
    if (channel) dgate[col] = a.gamma_post ? a.gamma_post[col] * v : v;
}

// Threads of a CTA, its vectors per thread, the CTAs and the ring.
struct Shape {
    int vpt, threads, ctas, stages;
    size_t smem;
};
// `piece`: bytes of one piece of all the arrays that a row is read from;
// `threads`: of an SM.
Shape shape(int T, int d, int vpt, int piece, int threads) {
    Shape s;
    s.vpt = vpt;
    s.threads = (d / 8 + 32 * vpt - 1) / (32 * vpt) * 32;
    const int per_sm = std::min(16, threads / s.threads);
    s.ctas = std::min(T, SMS * per_sm);
    const int row = vpt * (s.threads / 32) * piece;
    s.stages = std::max(1, std::min(MAX_STAGES, RING_BYTES / per_sm / row));
    s.smem = static_cast<size_t>(s.stages) * row;
    return s;
}
// One vector per thread and twice the threads, but two vectors for bf16 rows
// of more than 4096 columns, and four beyond 8192 (us, one vector / two:
// 8192 x 4096 bf16 47.0 / 50.9, 4093 x 7168 fp32 58.8 / 65.9, bf16 45.5 / 43.0).
Shape fwd_shape(int T, int d, bool res_f32) {
    const int vpt = d > 16 * MAX_THREADS ? 4 : d > 8 * MAX_THREADS && !res_f32 ? 2 : 1;
    return shape(T, d, vpt, piece_bytes<uint16_t>() + (res_f32 ? piece_bytes<float>() : piece_bytes<uint16_t>()),
                 vpt == 1 ? 2 * MAX_THREADS : MAX_THREADS);
}
// Two vectors per thread: the per-row work of a warp is what bounds the
// backward (4096 columns, bf16: 80.1 us; one vector and twice the threads 94.9).
Shape bwd_shape(int T, int d, bool res_f32) {
    return shape(T, d, d <= 512 ? 1 : d <= 16 * MAX_THREADS ? 2 : 4,
                 2 * piece_bytes<uint16_t>() + 2 * (res_f32 ? piece_bytes<float>() : piece_bytes<uint16_t>()),
                 MAX_THREADS);
}

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
    const Args args{a, s.stages, reinterpret_cast<uintptr_t>(r_out) % 32 == 0, nullptr, 0};
    norm_residual_kernel<R, VPT><<<s.ctas, s.threads, s.smem, stream>>>(
        args, 1.0f / a.d, static_cast<const R *>(r), static_cast<R *>(r_out), n, rstd_post, rstd_pre);
    return cudaGetLastError();
}

template <typename R, int VPT, bool FULL>
cudaError_t backward(const Shape &s, const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                     cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(norm_residual_bwd_kernel<R, VPT, FULL>, done);
    if (e != cudaSuccess) return e;
    const Args args{a, s.stages, reinterpret_cast<uintptr_t>(g.dr) % 32 == 0, g.status, g.wait_ns};
    norm_residual_bwd_kernel<R, VPT, FULL><<<s.ctas, s.threads, s.smem, stream>>>(
        args, 1.0f / a.d, static_cast<const R *>(g.r_out), static_cast<const R *>(g.dr_out), g.dn, g.rstd_post,
        g.rstd_pre, static_cast<R *>(g.dr), g.dy, g.dgate, part);
    return cudaGetLastError();
}

}  // namespace nr

cudaError_t launch_norm_residual(const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n, float *rstd_post,
                                 float *rstd_pre, cudaStream_t stream) {
    const nr::Shape s = nr::fwd_shape(a.T, a.d, a.res_f32);
    auto go = [&](auto type) {
        using R = decltype(type);
        if (s.vpt == 1) return nr::forward<R, 1>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
        if constexpr (sizeof(R) == 2) {
            if (s.vpt == 2) return nr::forward<R, 2>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
        }
        return nr::forward<R, 4>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
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
        if (a.y && g.dr_out && a.gamma_pre) {
            if (s.vpt == 1) return nr::backward<R, 1, true>(s, a, g, part, stream);
            return s.vpt == 2 ? nr::backward<R, 2, true>(s, a, g, part, stream)
                              : nr::backward<R, 4, true>(s, a, g, part, stream);
        }
        if (s.vpt == 1) return nr::backward<R, 1, false>(s, a, g, part, stream);
        return s.vpt == 2 ? nr::backward<R, 2, false>(s, a, g, part, stream)
                          : nr::backward<R, 4, false>(s, a, g, part, stream);
    };
    *launches = 1;
    const cudaError_t err = a.res_f32 ? go(float{}) : go(uint16_t{});
    if (err != cudaSuccess || !(a.gamma_pre || a.gamma_post || (a.gate && !a.gate_per_token))) return err;
    *launches = 2;
    return launch_dependent(nr::norm_residual_bwd_columns_kernel, a.d / 32, 32 * nr::RUNS, stream,
                            static_cast<const NormResidualArgs &>(a), static_cast<const float *>(part), s.ctas,
                            g.dgamma_pre, g.dgamma_post, g.dgate);
}

}  // namespace moe

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
// With dropout (DROP) what is added is g u / (1 - p) where an element is kept and 0 where it is not:
//   r' = a r + m g u,   and D in all of the y side's gradients is m D,   m = 0 or 1 / (1 - p)
// drawn again in the backward from the same state, before the row's bytes are
// waited for.  It adds no bytes, about 10 integer instructions per element and, in
// the backward, two tests.  Measured, 8192 x 4096 bf16 with both norms: forward 53.3 us
// a call (43.5 without dropout), backward 89.3 (68.1); 4093 x 7168 with the stream in fp32
// and without gamma_post 54.9 and 95.0.  One round of the generator instead of ten
// would take 10 us off either; a mask held as bits in one register is better than the
// draws themselves (2048 x 12288: 104 us), and predicates are than masks of the
// operands' bits where rows are bf16 (63 and 59 us for the residual's sum alone).
// The sums over t run in a fixed order: each CTA over its own rows, then the
// CTAs' partial sums in their order.
//
// Memory bounds both.  Measured: forward of 8192 x 4096 bf16 43.5 us, 6.2 TB/s,
// where a plain copy of as many bytes takes 46.8; backward 68.1 us, 5.9 TB/s,
// 4 of it the column sums; the main kernel takes as long with its arithmetic left out;
// backward of 4093 x 7168 with the stream in fp32 84.5 us, 6.3 TB/s.
#include "kernels.h"
#include "philox.cuh"
#include "ptx.cuh"
#include "vec8.cuh"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace moe {
namespace nr {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SMS = 152;
// Threads of an SM with 128 or 80 registers each.
constexpr int MAX_THREADS = 512, MORE_THREADS = 768;
constexpr int sm_threads(int regs) { return regs == 128 ? MAX_THREADS : MORE_THREADS; }
constexpr int RING_BYTES = 208 * 1024; // the rings of an SM's CTAs
// Rows in the ring.  More of them ahead made the forward slower (8192 x 4096
// bf16, us: 46.5 with two rows, 50.4 with three, 52.5 with four); the backward,
// which reads a row twice, needs a third one to run ahead.
constexpr int FWD_STAGES = 2;
constexpr int BWD_STAGES = 4;

// Which backward kernels read a row ahead: of those whose ring always holds three rows, the one it makes faster.
// With dropout none does, as the draws take its registers (us: 8192 x 4096 bf16
// 99 ahead and in teams, 87 without and in pairs; 16384 x 1024 59 and 47).
template <typename R>
__host__ __device__ constexpr bool pipelined(int vpt, bool full) { return full && vpt == 2 && sizeof(R) == 2; }

// How the rows of a backward share the SMs.  TEAM: a CTA whose teams of warps
// take a row each.  Teams leave one row of partial sums per SM instead of one per
// row in flight (us, bf16: 65536 x 256 50.4 with a CTA per row, 43.8 with teams;
// 16384 x 640 43.4 and 40.0; 2048 x 1024 19.2 and 14.2; 8192 x 4096 72.0 and 70.5).
// PAIR: two CTAs of a row each.  For two rows whose kernel does not read ahead they
// are faster than teams, as they need not keep in step (8192 x 4096 fp32: 98.5, 112.6
// with teams).  ALONE: a row at a time.  HALVES: a row by a cluster of two CTAs,
// which send each other their warps' sums; for rows that a CTA has too few registers
// for (us: 2048 x 12288 bf16 121, four vectors per thread, and 70; 2048 x 16384 fp32
// 179 and 104), and where three halves fit an SM instead of one row (4096 x 5120
// bf16: 61.7 and 56.6; fp32, without reading ahead, 70.0 and 74.6; with two halves
// 4096 x 8192 72.1 and 78.2).
enum Split { ALONE, PAIR, TEAM, HALVES };

// With what the launch adds to the caller's arguments.
struct Args : NormResidualArgs {
    int stages;  // rows in a team's ring
    int teams;   // of a backward's CTA
    bool wide;   // the fp32 rows that are written begin on 32-byte boundaries
};


// A row is cut into pieces of 32 vectors of eight elements, one vector per lane.
template <typename T>
__host__ __device__ constexpr int piece_bytes() { return 256 * static_cast<int>(sizeof(T)); }

template <typename T>
__device__ __forceinline__ void read8(const uint8_t *src, float2 (&o)[4]) {
    if constexpr (sizeof(T) == 2) {
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src), &o[0].x);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 16);
        o[0] = make_float2(a.x, a.y), o[1] = make_float2(a.z, a.w);
        o[2] = make_float2(b.x, b.y), o[3] = make_float2(b.z, b.w);
    }
}

// A vector to column `col` of a row.
__device__ __forceinline__ void store(uint16_t *row, uint32_t col, const float2 (&x)[4], bool) {
    store8(row + col, 0, &x[0].x);
}
__device__ __forceinline__ void store(float *row, uint32_t col, const float2 (&x)[4], bool wide) {
    wide ? store8_wide(row + col, 0, &x[0].x) : store8(row + col, 0, &x[0].x);
}

// What a thread owns: VPT neighbouring pieces per warp, a vector of each.
template <int VPT>
struct Owned {
    uint32_t col;  // of the first vector (the j-th: + 256 j)
    bool on[VPT];  // whether the row has them
    int first, cols;  // the warp's columns
    __device__ __forceinline__ Owned(int warp, int lane, int nvec, int from = 0) {
        col = from + (warp * VPT * 32 + lane) * 8;
#pragma unroll
        for (int j = 0; j < VPT; ++j) on[j] = (warp * VPT + j) * 32 + lane < nvec;
        first = from + warp * VPT * 256;
        cols = max(0, min(VPT * 32, nvec - warp * VPT * 32)) * 8;
    }
};

// The barriers of a warp's slots in the ring: each counts the bytes of a row's copies.
struct Ring {
    uint64_t *full;
    int *abort, *status;
    uint64_t wait_ns;
    bool used;  // the warp has columns
    // Until the row in a slot is there.  After another wait ran out this one
    // still waits (as long again) for its own copies.
    __device__ __forceinline__ void wait(int slot, int phase) const {
        int again = 0;
        if (used && !mbar_wait(&full[slot], phase, abort, status, wait_ns))
            mbar_wait(&full[slot], phase, &again, status, wait_ns);
    }
};

// The warp has read a slot: its refill lands behind that.  (Without the fence a
// copy may overtake a read that is still on its way.)
__device__ __forceinline__ void read_before_copies() {
    fence_proxy_async_smem();
    __syncwarp();
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

// The same for four values, in two steps around the caller's barrier.  Each
// exchange of the first two halves the values that a lane carries, so a warp
// takes 6 exchanges instead of 20; then every thread adds the warps' sums.
// SEND: they also go to the peer of a cluster, each an arrival at its `bar`.
template <bool SEND = false>
__device__ __forceinline__ void post_sums4(const float (&v)[4], float4 *red, uint32_t peer = 0, uint64_t *bar = nullptr) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(FULL, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(FULL, up ? v[1] : v[3], 16);
    float s = (odd ? b : a) + __shfl_xor_sync(FULL, odd ? a : b, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    if ((lane & 7) == 0) {
        float *to = reinterpret_cast<float *>(red + (threadIdx.x >> 5)) + (lane >> 3);
        *to = s;
        if (SEND) send_to_peer(mapa_shared(smem_u32(to), peer), __float_as_int(s), mapa_shared(smem_u32(bar), peer));
    }
}
__device__ __forceinline__ float4 collect_sums4(const float4 *red, int warps) {
    float2 a = both(0.0f), b = a;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
        const float4 s = red[w];
        a = add2(a, make_float2(s.x, s.y));
        b = add2(b, make_float2(s.z, s.w));
    }
    return make_float4(a.x, a.y, b.x, b.y);
}

// Between the warps of one of a CTA's teams (of at most 8, where they have two warps or more).  Not on
// barrier 0: that is __syncthreads' own, where teams without further rows already wait for the others.
__device__ __forceinline__ void team_sync(int team, int warps) {
    __syncwarp();  // the barrier, and that of a cluster below, is for whole warps at once
    if (warps > 1) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(32 * warps) : "memory");
}

// Weights of the eight columns from `col` (where the row has them): c of y
// (gamma_post times a channel gate) and w of n; 1 for those left out.
__device__ __forceinline__ void weights(const NormResidualArgs &a, uint32_t col, bool on, float2 (&c)[4], float2 (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = w[i] = both(1.0f);
    if (!on) return;
    if (a.gamma_post) load8(a.gamma_post + col, 0, &c[0].x);
    if (a.gate && !a.gate_per_token) {
        float2 g[4];
        load8(a.gate + col, 0, &g[0].x);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = mul2(c[i], g[i]);
    }
    if (a.gamma_pre) load8(a.gamma_pre + col, 0, &w[0].x);
}

// The draws of a thread's vectors of row t, and as a mask, a byte per vector (of four
// at most); without dropout, nothing.
template <bool DROP, int VPT>
struct Draws {
    __device__ __forceinline__ explicit Draws(const NormResidualArgs &) {}
    __device__ __forceinline__ void row(int64_t, int, uint32_t) {}
    __device__ __forceinline__ uint32_t mask(int64_t, int, uint32_t) { return 0; }
};
template <int VPT>
struct Draws<true, VPT> : Dropout {
    uint4 w[VPT];
    __device__ __forceinline__ explicit Draws(const NormResidualArgs &a) : Dropout(a.rng, a.drop) {}
    __device__ __forceinline__ void row(int64_t t, int d, uint32_t col) {
        words(static_cast<uint64_t>(t * d + col) >> 3, 32, w);
    }
    __device__ __forceinline__ uint32_t mask(int64_t t, int d, uint32_t col) {
        row(t, d, col);
        uint32_t m[4] = {};  // four at once: each bit waits for the one before
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) mark_kept(m[i >> 1], 1u << (8 * j + i), draw(w[j], i), bar);
        return m[0] | m[1] | m[2] | m[3];
    }
};

// Row r of CTA blockIdx.x is blockIdx.x + r gridDim.x.  A thread owns VPT
// vectors of eight columns; each warp fetches the columns that it reads with
// bulk copies of its own, so its rows come ahead of their use through a ring in
// shared memory and wait for no other warp.  (With 16-byte copies by every lane
// the backward of 8192 x 4096 took 78.3 us, 72.1 with bulk copies: the lanes'
// requests, not the memory, were the limit.)  A row's slot is refilled as soon as
// the row is in registers, so the ring's copies stay in flight through the row's
// sums and stores.
template <typename R, int VPT, int REGS, bool DROP>
__global__ void __launch_bounds__(sm_threads(REGS))
norm_residual_kernel(Args a, float inv_d, const R *r, R *r_out, uint16_t *__restrict__ n,
                     float *__restrict__ rstd_post, float *__restrict__ rstd_pre) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ uint64_t landed[MORE_THREADS / 32][FWD_STAGES];
    __shared__ int abort;
    const int stages = a.stages;
    constexpr bool HOLD = VPT <= 2;  // the weights stay in registers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const bool has_y = a.y != nullptr, post = a.gamma_post != nullptr, pre = a.gamma_pre != nullptr;
    const Owned<VPT> own(warp, lane, a.d / 8);
    constexpr int AT_R = VPT * piece_bytes<uint16_t>(), PART = AT_R + VPT * piece_bytes<R>();
    const int stage = warps * PART;
    uint8_t *const mine = ring + warp * PART;
    float2 c[VPT][4], w[VPT][4];
    grid_dependency_wait_to_copy();  // launched early
    if (HOLD) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) weights(a, own.col + 256 * j, own.on[j], c[j], w[j]);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < warps; ++i)
            for (int q = 0; q < FWD_STAGES; ++q) mbar_init(&landed[i][q], 1);
        abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const Ring rows{landed[warp], &abort, a.status, a.wait_ns, own.cols > 0};
    auto issue = [&](int64_t t, int slot) {
        if (lane == 0 && t < a.T && own.cols > 0) {
            uint8_t *to = mine + slot * stage;
            const int64_t from = t * a.d + own.first;
            const uint32_t nb = own.cols * 2, nr = own.cols * static_cast<int>(sizeof(R));
            mbar_arrive_expect_tx(&rows.full[slot], (has_y ? nb : 0) + nr);
            if (has_y) bulk_load(to, a.y + from, nb, &rows.full[slot]);
            bulk_load(to + AT_R, r + from, nr, &rows.full[slot]);
        }
    };
    const int64_t step = gridDim.x;
    for (int s = 0; s < stages; ++s) issue(blockIdx.x + s * step, s);
    const bool token_gate = a.gate && a.gate_per_token;
    float gt = token_gate ? a.gate[blockIdx.x] : 1.0f;
    Draws<DROP, VPT> draws(a);
    if (DROP && blockIdx.x == 0 && threadIdx.x < 2) a.rng_out[threadIdx.x] = a.rng[threadIdx.x];
    int slot = 0, turn = 0, phase = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += step) {
        const float gt_next = token_gate && t + step < a.T ? a.gate[t + step] : 1.0f;
        draws.row(t, a.d, own.col);  // while the row is on its way
        rows.wait(slot, phase);
        const uint8_t *at = mine + slot * stage;
        float2 x[VPT][4], y[VPT][4];
        float2 ss = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][i] = y[j][i] = both(0.0f);
            if (!own.on[j]) continue;
            read8<R>(at + AT_R + j * piece_bytes<R>() + lane * (8 * sizeof(R)), x[j]);
            if (has_y) {
                read8<uint16_t>(at + j * 512 + lane * 16, y[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(y[j][i], y[j][i], ss);
            }
        }
        read_before_copies();
        issue(t + stages * step, slot);
        slot = slot + 1 == stages ? 0 : slot + 1;
        if (slot == 0) phase ^= 1;
        if (has_y) {
            float f = gt;
            if (post) {
                const float rp = rsqrtf(__fmaf_rn(block_sum(ss.x + ss.y, red[turn]), inv_d, a.eps));
                turn ^= 1;
                if (threadIdx.x == 0) rstd_post[t] = rp;
                f *= rp;
            }
            if (DROP) f *= a.keep_scale;
            R *out = r_out + t * a.d;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!HOLD) weights(a, own.col + 256 * j, own.on[j], c[j], w[j]);
                if constexpr (DROP) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 fc = mul2(both(f), c[j][i]);
                        x[j][i] = mul2(both(a.res_scale), x[j][i]);
                        fma_kept(x[j][i].x, fc.x, y[j][i].x, draw(draws.w[j], 2 * i), draws.bar);
                        fma_kept(x[j][i].y, fc.y, y[j][i].y, draw(draws.w[j], 2 * i + 1), draws.bar);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[j][i] = fma2(mul2(both(f), c[j][i]), y[j][i], mul2(both(a.res_scale), x[j][i]));
                }
                if (own.on[j]) store(out, own.col + 256 * j, x[j], a.wide);
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
                if (!own.on[j]) continue;
                if (!HOLD) load8(a.gamma_pre + own.col + 256 * j, 0, &w[j][0].x);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = mul2(x[j][i], mul2(both(rq), w[j][i]));
                store(out, own.col + 256 * j, x[j], true);
            }
        }
        gt = gt_next;
    }
}

// Rows and ring as above, but the row is read from its slot twice, before and
// after the sums, and the slot refilled after the second time.
// PIPE: the first reading of row r + 1 stands between the sums of row r and
// their use, so that no warp waits for the others' sums (8192 x 4096 bf16:
// 77.2 us, 72.3 with it, both with a CTA per row).  It needs a third row in the
// ring, which fp32 rows do not leave room for.
// One reduction gives both means of a row: with z = r' rq, m1 = rq mean(h z)
// and c the weight of y without a token gate g,
//   D = dr' + rq h - m1 z,   sum(c y D) = sum(c y dr') + rq sum(c y h) - m1 sum(c y z),
// g times which is sum(k y), and rp times which is the token gate's gradient.
// Each thread keeps its columns' two sums over the rows (of dn z, and of
// g y rp D, from which both dgp and a channel gate's dg follow).
// Y, PRE, DR: whether there is a y, a gamma_pre and a dr' (y or gamma_pre is,
// dn or dr' is).  A kernel of its own for each form has no branches in the inner
// loops, and a ring of the arrays that it reads only.  8192 x 4096 bf16 with one
// kernel for all that lack one: 66.3 us without y, 57.3 without gamma_pre; with
// their own 48.9 and 51.3.  A higher share of the SM's threads for these lighter
// forms was slower up to 4096 columns (us): 768 of 80 registers 53.1 and 56.5, 1024
// of 64 55.2 and 58.0.
template <typename R, int VPT, bool Y, bool PRE, bool DR, Split SPLIT, int REGS, bool DROP>
__global__ void __launch_bounds__(sm_threads(REGS))
norm_residual_bwd_kernel(Args a, float inv_d, const R *__restrict__ r_out, const R *dr_out,
                         const uint16_t *__restrict__ dn, const float *__restrict__ rstd_post,
                         const float *__restrict__ rstd_pre, R *dr, uint16_t *__restrict__ dy,
                         float *__restrict__ dgate, float *__restrict__ part) {
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr bool HALF = SPLIT == HALVES;
    __shared__ float4 red[HALF ? 3 : 2][32];
    __shared__ uint64_t landed[MORE_THREADS / 32][BWD_STAGES];
    // Of a team: a phase per row, an arrival per warp.  Of halves: two that rows take in turn, five arrivals
    // per warp (its own one, four sums from the peer's warp).  In turn, because a sum of the peer's next
    // row may come before the last one of this row; no sum of the row after that can, as it
    // waits for this CTA's own of the next row.  The same order of events frees the third set of `red`.
    __shared__ uint64_t posted[MAX_THREADS / 32];
    __shared__ int abort;
    constexpr bool PIPE = !DROP && pipelined<R>(VPT, Y && PRE), TEAMS = SPLIT == TEAM;
    // Whether the warps wait for the row's sums by an mbarrier, which lets the first ones through go on
    // (4093 x 7168 fp32: 90.0 us, 95.3 with __syncthreads).
    constexpr bool POSTS = PIPE || SPLIT == ALONE || SPLIT == HALVES;
    // Whether a slot is refilled after the row's last stores instead of before them: where the fence would
    // wait for the reads of an fp32 row beside the draws (us: 4093 x 7168 95.1, 97.9 before them; bf16 8192 x 4096
    // 91.4, 88.8).
    constexpr bool LATE = DROP && sizeof(R) == 4;
    const uint32_t rank = HALF ? blockIdx.x & 1 : 0, group = HALF ? blockIdx.x >> 1 : blockIdx.x;
    const uint32_t groups = HALF ? gridDim.x >> 1 : gridDim.x;
    const int stages = a.stages;
    const int teams = TEAMS ? a.teams : 1;
    const int lane = threadIdx.x & 31, all = blockDim.x >> 5, warps = all / teams;
    const int team = TEAMS ? (threadIdx.x >> 5) / warps : 0, warp = TEAMS ? (threadIdx.x >> 5) % warps : threadIdx.x >> 5;
    constexpr bool has_y = Y, pre = PRE;
    const bool post = a.gamma_post != nullptr;
    const Owned<VPT> own(warp, lane, HALF ? a.d / 16 : a.d / 8, rank * a.d / 2);
    // a warp's part of a row in the ring: its columns of y, dn, r' and dr'
    constexpr int B = VPT * piece_bytes<uint16_t>(), AT_DN = Y ? B : 0, AT_X = AT_DN + (PRE ? B : 0);
    constexpr int AT_DR = AT_X + (PRE ? VPT * piece_bytes<R>() : 0), PART = AT_DR + VPT * piece_bytes<R>();
    const int stage = warps * PART;
    uint8_t *const mine = ring + team * stages * stage + warp * PART;
    float2 c[VPT][4], w[VPT][4], accq[VPT][4], accp[VPT][4];
    grid_dependency_wait_to_copy();  // launched early
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        weights(a, own.col + 256 * j, own.on[j], c[j], w[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) accq[j][i] = accp[j][i] = both(0.0f);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < all; ++i)
            for (int q = 0; q < BWD_STAGES; ++q) mbar_init(&landed[i][q], 1);
        for (int i = 0; i < (HALF ? 2 : teams); ++i) mbar_init(&posted[i], HALF ? 5 * warps : warps);
        abort = 0;
        fence_mbar_init();
    }
    __syncwarp();
    HALF ? cluster_sync() : __syncthreads();
    const Ring rows{landed[threadIdx.x >> 5], &abort, a.status, a.wait_ns, own.cols > 0};
    const uint32_t rows_end = a.T;  // a row number a few rows past it still fits
    auto issue = [&](uint32_t t, int slot) {
        if (lane == 0 && t < rows_end && own.cols > 0) {
            uint8_t *to = mine + slot * stage;
            const int64_t from = static_cast<int64_t>(t) * a.d + own.first;
            const uint32_t nb = own.cols * 2, nr = own.cols * static_cast<int>(sizeof(R));
            uint64_t *full = rows.full;
            mbar_arrive_expect_tx(&full[slot], (has_y ? nb : 0) + (DR ? nr : 0) + (pre ? nb + nr : 0));
            if (has_y) bulk_load(to, a.y + from, nb, &full[slot]);
            if (DR) bulk_load(to + AT_DR, dr_out + from, nr, &full[slot]);
            if (pre) {
                bulk_load(to + AT_DN, dn + from, nb, &full[slot]);
                bulk_load(to + AT_X, r_out + from, nr, &full[slot]);
            }
        }
    };
    struct Row {  // the row's factors, loaded a row ahead
        float rp, rq, gt;
    };
    auto factors = [&](uint32_t t) {
        Row f{1.0f, 0.0f, 1.0f};
        if (t < rows_end) {
            if (post) f.rp = rstd_post[t];
            if (pre) f.rq = rstd_pre[t];
            if (a.gate && a.gate_per_token) f.gt = a.gate[t];
        }
        return f;
    };
    const uint32_t begin = group + team * groups, step = groups * teams;
    for (int s = 0; s < stages; ++s) issue(begin + s * step, s);
    // The first reading of the row in slot `slot`: the four sums (of h z,
    // c y dr', c y h, c y z) of the warp go to `sums`.
    // With dropout (`kept`: the row's mask) only the kept elements' products with
    // y enter, and s1 and s2 as the one sum that is needed of them, s1 + rq s2.
    Draws<DROP, VPT> draws(a);
    auto first_pass = [&](int slot, float rq, float4 *sums, uint32_t k, uint32_t kept) {
        const uint8_t *at16 = mine + slot * stage + lane * 16, *at_r = mine + slot * stage + lane * (8 * sizeof(R));
        float2 s0 = both(0.0f), s1 = s0, s2 = s0, s3 = s0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (!own.on[j]) continue;
            float2 cy[4];
            if (has_y) {
                read8<uint16_t>(at16 + j * 512, cy);
#pragma unroll
                for (int i = 0; i < 4; ++i) cy[i] = mul2(cy[i], c[j][i]);
                if (DR && !DROP) {
                    float2 g[4];
                    read8<R>(at_r + j * piece_bytes<R>() + AT_DR, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s1 = fma2(cy[i], g[i], s1);
                }
            }
            float2 e[4];
            if constexpr (DROP) {
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = both(0.0f);
                if (DR) read8<R>(at_r + j * piece_bytes<R>() + AT_DR, e);
            }
            if (pre) {
                float2 z[4], g[4];
                read8<R>(at_r + j * piece_bytes<R>() + AT_X, z);
                read8<uint16_t>(at16 + j * 512 + AT_DN, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[i] = mul2(z[i], both(rq));
                    accq[j][i] = fma2(g[i], z[i], accq[j][i]);
                    g[i] = mul2(g[i], w[j][i]);  // h
                    s0 = fma2(g[i], z[i], s0);
                    if constexpr (DROP) {
                        e[i] = fma2(both(rq), g[i], e[i]);
                        fma_masked(s1.x, cy[i].x, e[i].x, s3.x, cy[i].x, z[i].x, kept, 1u << (8 * j + 2 * i));
                        fma_masked(s1.y, cy[i].y, e[i].y, s3.y, cy[i].y, z[i].y, kept, 2u << (8 * j + 2 * i));
                    }
                }
                if (has_y && !DROP) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s2 = fma2(cy[i], g[i], s2);
                        s3 = fma2(cy[i], z[i], s3);
                    }
                }
            } else if constexpr (DROP) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float none = 0.0f;
                    fma_masked(s1.x, cy[i].x, e[i].x, none, 0.0f, 0.0f, kept, 1u << (8 * j + 2 * i));
                    fma_masked(s1.y, cy[i].y, e[i].y, none, 0.0f, 0.0f, kept, 2u << (8 * j + 2 * i));
                }
            }
        }
        const float s[4] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, s3.x + s3.y};
        post_sums4<HALF>(s, sums + rank * warps, rank ^ 1, &posted[k & 1]);
        if (POSTS) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&posted[HALF ? k & 1 : team]);
        }
    };
    // Until every warp of the team has posted its sums of the row (the k-th).
    auto collect = [&](const float4 *sums, uint32_t k) {
        if (POSTS) {
            mbar_wait<HALF>(&posted[HALF ? k & 1 : team], (HALF ? k >> 1 : k) & 1, &abort, a.status, a.wait_ns);
        } else {
            TEAMS ? team_sync(team, warps) : __syncthreads();
        }
        return collect_sums4(sums + team * warps, HALF ? 2 * warps : warps);
    };
    Row f = factors(begin), next = factors(begin + step);
    int slot = 0, turn = 0;
    int phase = 0;  // of the slot that first_pass reads next
    uint32_t k = 0, kept = 0;
    if (PIPE && begin < rows_end) {  // (never with dropout)
        rows.wait(0, 0);
        first_pass(0, f.rq, red[0], 0, 0);
    }
    for (uint32_t t = begin; t < rows_end; t += step) {
        const Row after = factors(t + 2 * step);
        const int ahead = slot + 1 == stages ? 0 : slot + 1, other = HALF ? (turn == 2 ? 0 : turn + 1) : turn ^ 1;
        float4 s;
        if (PIPE) {
            s = collect(red[turn], k);
            if (ahead == 0) phase ^= 1;
            if (t + step < rows_end) {
                rows.wait(ahead, phase);
                first_pass(ahead, next.rq, red[other], k + 1, 0);
            }
        } else {
            kept = draws.mask(t, a.d, own.col);  // while the row is on its way
            rows.wait(slot, phase);
            first_pass(slot, f.rq, red[turn], k, kept);
            s = collect(red[turn], k);
            if (ahead == 0) phase ^= 1;
        }
        turn = other;
        ++k;
        const uint8_t *at16 = mine + slot * stage + lane * 16, *at_r = mine + slot * stage + lane * (8 * sizeof(R));
        const float m1 = f.rq * s.x * inv_d;
        float cyD = s.y + f.rq * s.z - m1 * s.w;
        if (DROP) cyD *= a.keep_scale;
        const float m2 = post ? f.gt * cyD * inv_d * f.rp * f.rp * f.rp : 0.0f;
        if (a.gate && a.gate_per_token && warp == 0 && lane == 0 && rank == 0) dgate[t] = f.rp * cyD;
        const float2 q = both(DROP ? f.gt * f.rp * a.keep_scale : f.gt * f.rp), mz = both(-m1 * f.rq), my = both(-m2), rq = both(f.rq);
        R *to_r = dr + static_cast<int64_t>(t) * a.d;
        uint16_t *to_y = dy + static_cast<int64_t>(t) * a.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const uint32_t col = own.col + 256 * j;
            float2 D[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) D[i] = both(0.0f);
            if (own.on[j]) {
                if (DR) read8<R>(at_r + j * piece_bytes<R>() + AT_DR, D);
                if (pre) {
                    float2 x[4], g[4];
                    read8<R>(at_r + j * piece_bytes<R>() + AT_X, x);
                    read8<uint16_t>(at16 + j * 512 + AT_DN, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) D[i] = fma2(mz, x[i], fma2(mul2(rq, g[i]), w[j][i], D[i]));
                }
                if (has_y) read8<uint16_t>(at16 + j * 512, y);
            }
            if (!LATE && j == VPT - 1) {
                read_before_copies();
                issue(t + stages * step, slot);
            }
            if (!own.on[j]) continue;
            float2 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = mul2(both(a.res_scale), D[i]);  // res_scale is 1 without y
            store(to_r, col, o, a.wide);
            if constexpr (has_y) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    D[i] = mul2(D[i], q);
                    if constexpr (DROP) {
                        o[i] = post ? mul2(my, y[i]) : both(0.0f);
                        fma_masked(accp[j][i].x, y[i].x, D[i].x, o[i].x, c[j][i].x, D[i].x, kept, 1u << (8 * j + 2 * i));
                        fma_masked(accp[j][i].y, y[i].y, D[i].y, o[i].y, c[j][i].y, D[i].y, kept, 2u << (8 * j + 2 * i));
                    } else {
                        accp[j][i] = fma2(y[i], D[i], accp[j][i]);
                        o[i] = fma2(my, y[i], mul2(D[i], c[j][i]));
                    }
                }
                store(to_y, col, o, true);
            }
        }
        if (LATE) {
            read_before_copies();
            issue(t + stages * step, slot);
        }
        slot = ahead;
        f = next;
        next = after;
    }
    // the CTA's sums: the teams' ones in the rings, now empty, added in the teams' order
    float *out = part + static_cast<size_t>(group) * 2 * a.d, *held = reinterpret_cast<float *>(ring);
    float *sums = teams > 1 ? held + team * 2 * a.d : out;
    if (teams > 1) __syncthreads();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (!own.on[j]) break;
        store8(sums + own.col + 256 * j, 0, &accq[j][0].x);
        store8(sums + a.d + own.col + 256 * j, 0, &accp[j][0].x);
    }
    __syncwarp();
    if (HALF) cluster_sync();  // a CTA stays while the other one may still post to it
    if (teams == 1) return;
    __syncthreads();
    for (int i = threadIdx.x; i < a.d / 2; i += blockDim.x) {
        float4 v = reinterpret_cast<const float4 *>(held)[i];
        for (int k = 1; k < teams; ++k) {
            const float4 u = reinterpret_cast<const float4 *>(held + k * 2 * a.d)[i];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        reinterpret_cast<float4 *>(out)[i] = v;
    }
}

// The CTAs' partial sums: 32 columns per block, each in 32 runs of CTAs in
// their order, then the runs in theirs (runs of 5 or 10 for 152 or 304 CTAs:
// every load of a thread in flight at once).
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

// Threads of a CTA, its vectors per thread and registers, the CTAs and the ring.
struct Shape {
    int vpt, regs, threads, ctas, stages, teams = 1;
    Split split = ALONE;
    size_t smem;
    int per_sm() const { return sm_threads(regs) / threads; }
    // `piece`: bytes of one piece of all the arrays that a row is read from.
    Shape(int T, int d, int vpt_, int regs_, int most_stages, int piece) : vpt(vpt_), regs(regs_) {
        threads = (d / 8 + 32 * vpt - 1) / (32 * vpt) * 32;
        ctas = std::min(T, SMS * per_sm());
        const int row = vpt * (threads / 32) * piece;
        stages = std::max(1, std::min(most_stages, RING_BYTES / per_sm() / row));
        smem = static_cast<size_t>(stages) * row;
    }
};
// Rows that fit an SM with two vectors per thread.
constexpr int sm_rows(int d, int regs) { return sm_threads(regs) / ((d / 8 + 63) / 64 * 32); }

// Two vectors per thread: the work of a warp per row is what bounds these
// kernels next to memory (one vector and twice the threads, us: forward of
// 8192 x 4096 bf16 56.5, 46.5 with two; backward 86.7 and 72.3).  Fewer
// registers where they give an SM another row of more than 4096 columns (us
// bf16: 4096 x 5120 39.2 and 33.0, 2048 x 12288 61.0 and 39.3; narrower rows lose
// by them, 8192 x 4096 46.2 and 48.4), or short rows more of them (16384 x 128
// 12.5 and 10.6; fp32 rows of 1 KB and more lose, 65536 x 256 37.1 and 39.5).
template <typename R>
Shape fwd_shape(int T, int d) {
    const int piece = piece_bytes<uint16_t>() + piece_bytes<R>();
    if (d <= 256) return Shape(T, d, 1, d * sizeof(R) <= 512 ? 80 : 128, FWD_STAGES, piece);
    if (d > 4096 && sm_rows(d, 80) > sm_rows(d, 128)) return Shape(T, d, 2, 80, FWD_STAGES, piece);
    return Shape(T, d, d <= 8192 ? 2 : 4, 128, FWD_STAGES, piece);
}
// The same for a bf16 backward without y or gamma_pre (us: without y 4096 x 5120
// 45.4 and 39.3, 2048 x 10240 in halves 49.4 and 44.5); an fp32 one's ring gets too
// short (4096 x 5120 51.8 and 53.9, 2048 x 12288 in halves 62.7 and 80.8), and one
// with both needs its 128.  Teams are as many as rows spread over all SMs allow;
// the ring also holds their partial sums in the end.
template <typename R>
Shape bwd_shape(int T, int d, bool y, bool pre, bool drop) {
    const int piece = (y + pre) * piece_bytes<uint16_t>() + (1 + pre) * piece_bytes<R>();
    const bool fewer = sizeof(R) == 2 && !(y && pre) && d > 4096 && sm_rows(d, 80) > sm_rows(d, 128);
    const bool ahead = pipelined<R>(2, y && pre);
    if (!fewer && (d > 8192 || (d > 4096 && d <= 5120 && ahead))) {
        Shape s(T, d / 2, 2, 128, BWD_STAGES, piece);
        s.ctas = 2 * std::min(T, SMS / 2 * s.per_sm());
        s.split = HALVES;
        return s;
    }
    Shape s(T, d, d <= 256 ? 1 : 2, fewer ? 80 : 128, BWD_STAGES, piece);
    const int per_sm = s.per_sm();
    s.split = per_sm == 1 ? ALONE : per_sm == 2 && (!ahead || drop) ? PAIR : TEAM;
    if (s.split != TEAM) return s;
    s.teams = std::min(per_sm, (T + SMS - 1) / SMS);
    s.ctas = std::min(T, SMS);
    s.threads *= s.teams;
    s.smem = std::max(s.smem * s.teams, static_cast<size_t>(s.teams > 1 ? s.teams * 2 * d * 4 : 0));
    return s;
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

template <typename R, int VPT, int REGS, bool DROP>
cudaError_t forward(const Shape &s, const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n,
                    float *rstd_post, float *rstd_pre, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(norm_residual_kernel<R, VPT, REGS, DROP>, done);
    if (e != cudaSuccess) return e;
    const Args args{a, s.stages, s.teams, reinterpret_cast<uintptr_t>(r_out) % 32 == 0};
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s.ctas), cfg.blockDim = dim3(s.threads), cfg.dynamicSmemBytes = s.smem, cfg.stream = stream;
    cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_residual_kernel<R, VPT, REGS, DROP>, args, 1.0f / a.d,
                              static_cast<const R *>(r), static_cast<R *>(r_out), n, rstd_post, rstd_pre);
}

template <typename R, int VPT, bool Y, bool PRE, bool DR, Split SPLIT, int REGS, bool DROP>
cudaError_t backward(const Shape &s, const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                     cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(norm_residual_bwd_kernel<R, VPT, Y, PRE, DR, SPLIT, REGS, DROP>, done);
    if (e != cudaSuccess) return e;
    const Args args{a, s.stages, s.teams, reinterpret_cast<uintptr_t>(g.dr) % 32 == 0};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s.ctas), cfg.blockDim = dim3(s.threads), cfg.dynamicSmemBytes = s.smem, cfg.stream = stream;
    cfg.attrs = attr, cfg.numAttrs = SPLIT == HALVES ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, norm_residual_bwd_kernel<R, VPT, Y, PRE, DR, SPLIT, REGS, DROP>, args, 1.0f / a.d,
                              static_cast<const R *>(g.r_out), static_cast<const R *>(g.dr_out),
                              static_cast<const uint16_t *>(g.dn), static_cast<const float *>(g.rstd_post),
                              static_cast<const float *>(g.rstd_pre), static_cast<R *>(g.dr), g.dy, g.dgate, part);
}

}  // namespace nr

cudaError_t launch_norm_residual(const NormResidualArgs &a, const void *r, void *r_out, uint16_t *n, float *rstd_post,
                                 float *rstd_pre, cudaStream_t stream) {
    auto go = [&](auto type, auto dropout) {
        using R = decltype(type);
        constexpr bool DROP = decltype(dropout)::value;
        const nr::Shape s = nr::fwd_shape<R>(a.T, a.d);
        if (s.vpt == 1) return nr::forward<R, 1, 80, DROP>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
        if (s.regs == 80) return nr::forward<R, 2, 80, DROP>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
        if (s.vpt == 2) return nr::forward<R, 2, 128, DROP>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
        return nr::forward<R, 4, 128, DROP>(s, a, r, r_out, n, rstd_post, rstd_pre, stream);
    };
    if (a.rng) return a.res_f32 ? go(float{}, std::true_type{}) : go(uint16_t{}, std::true_type{});
    return a.res_f32 ? go(float{}, std::false_type{}) : go(uint16_t{}, std::false_type{});
}

size_t norm_residual_bwd_part_bytes(int T, int d) {
    int ctas = 0;  // the most of any form
    for (const bool y : {false, true})
        for (const bool pre : {!y, true})
            for (const bool drop : {false, true})
                ctas = std::max({ctas, nr::bwd_shape<float>(T, d, y, pre, drop).ctas,
                                 nr::bwd_shape<uint16_t>(T, d, y, pre, drop).ctas});
    return static_cast<size_t>(ctas) * 2 * d * 4;
}

cudaError_t launch_norm_residual_bwd(const NormResidualArgs &a, const NormResidualGradArgs &g, float *part,
                                     int *launches, cudaStream_t stream) {
    int parts = 0;
    auto go = [&](auto type, auto dropout) {
        using R = decltype(type);
        const nr::Shape s = nr::bwd_shape<R>(a.T, a.d, a.y, a.gamma_pre, a.rng);
        parts = s.split == nr::HALVES ? s.ctas / 2 : s.ctas;
        auto form = [&](auto y, auto pre, auto dr) {
            constexpr bool Y = decltype(y)::value, PRE = decltype(pre)::value, DR = decltype(dr)::value;
            constexpr bool DROP = Y && decltype(dropout)::value;
            if (s.vpt == 1) return nr::backward<R, 1, Y, PRE, DR, nr::TEAM, 128, DROP>(s, a, g, part, stream);
            if (s.split == nr::HALVES) return nr::backward<R, 2, Y, PRE, DR, nr::HALVES, 128, DROP>(s, a, g, part, stream);
            if constexpr (sizeof(R) == 2 && !(Y && PRE)) {
                if (s.regs == 80 && s.split == nr::PAIR)
                    return nr::backward<R, 2, Y, PRE, DR, nr::PAIR, 80, DROP>(s, a, g, part, stream);
                if (s.regs == 80) return nr::backward<R, 2, Y, PRE, DR, nr::ALONE, 80, DROP>(s, a, g, part, stream);
            }
            if (s.split == nr::TEAM) return nr::backward<R, 2, Y, PRE, DR, nr::TEAM, 128, DROP>(s, a, g, part, stream);
            if constexpr (DROP || !nr::pipelined<R>(2, Y && PRE))
                if (s.split == nr::PAIR) return nr::backward<R, 2, Y, PRE, DR, nr::PAIR, 128, DROP>(s, a, g, part, stream);
            return nr::backward<R, 2, Y, PRE, DR, nr::ALONE, 128, DROP>(s, a, g, part, stream);
        };
        constexpr std::true_type with{};
        constexpr std::false_type without{};
        if (!a.gamma_pre) return form(with, without, with);  // dr_out is what it has instead of dn
        if (!a.y) return g.dr_out ? form(without, with, with) : form(without, with, without);
        return g.dr_out ? form(with, with, with) : form(with, with, without);
    };
    *launches = 1;
    const cudaError_t err = a.rng ? (a.res_f32 ? go(float{}, std::true_type{}) : go(uint16_t{}, std::true_type{}))
                                  : (a.res_f32 ? go(float{}, std::false_type{}) : go(uint16_t{}, std::false_type{}));
    if (err != cudaSuccess || !(a.gamma_pre || a.gamma_post || (a.gate && !a.gate_per_token))) return err;
    *launches = 2;
    return launch_dependent(nr::norm_residual_bwd_columns_kernel, a.d / 32, 32 * nr::RUNS, stream,
                            static_cast<const NormResidualArgs &>(a), static_cast<const float *>(part), parts,
                            g.dgamma_pre, g.dgamma_post, g.dgate);
}

}  // namespace moe

// The gated feed-forward of all tokens (a shared expert, a dense layer), and its backward:
//   a = x W1^T = [g | u],  h = act(g) u,  y = h W2^T + add
//   dh = dy W2,  da = [dh u act'(g) | dh act(g)],  dx = da W1 + add,  dW1 = da^T x,  dW2 = dy^T h
// with x, y, dx, add [T, d], W1 [2f, d] (gate rows, then up rows), W2 [d, f], a [T, 2f], all bf16.
// Sums are fp32 in tensor memory.  h and da are rounded to bf16 once, as they
// are operands of the next product; dh and, in the forward, a are not rounded
// before the activation.  Backward reads a as the forward stored it.
//
// One persistent kernel makes all five products, on CTA pairs: a 256 x 256
// tile of the result per pair through cta_group::2 MMAs, each CTA loading its
// 128 rows of A and half of the columns of B per 64-wide slice of K (32 KB),
// two accumulators in TMEM so that a tile's epilogue runs beside the next
// tile's products.  The sizes are known on the host, so tensor maps cut every
// matrix to its own size: loads past it read zeros, stores past it do nothing,
// and no size has to fill a tile.
//   epilogue GATED   h (and a) from a tile whose B rows are 128 gate and 128 up rows
//            PLAIN   the product, plus a matrix (ADD); fp32 for weight gradients on request
//            DACT    da and h from the tile of dh and the tiles of g and u
// Warps: 0 TMA loads, 1 MMAs and TMEM, 2 to 5 epilogue.  Every wait is bounded.
#include <algorithm>
#include <type_traits>

#include "gated_ffn.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tmap.h"

namespace moe {
namespace ff {

using gg::pack_bf16x2;

enum Epi { GATED, PLAIN, ADD, DACT };

constexpr int BK = 64;          // a slice of K: 128 bytes, one swizzle line
constexpr int UMMA_K = 16;
constexpr int TILE_M = 256, TILE_N = 256;
constexpr int BAND = 8;         // row blocks that sweep the column blocks together
constexpr int THREADS = 192;
constexpr int BOX = 64 * 64 * 2;  // an MN-major box: 64 rows of K x 64 columns
constexpr int STAGE = 4 * BOX;    // of a CTA: 128 rows of A, 128 columns of B
constexpr int CHUNK = 32;         // the epilogue takes 32 rows x 32 columns per warp at a time
constexpr int BUF = CHUNK * CHUNK * 2;

// An epilogue warp's buffers in shared memory: `sets` of `boxes` 32 x 32 boxes,
// of which the first `in` are filled by TMA before a chunk is computed.
struct Buffers {
    int sets, boxes, in, bytes;
};
template <Epi EPI, typename Out>
__host__ __device__ constexpr Buffers buffers() {
    return EPI == DACT ? Buffers{2, 3, 2, BUF} : EPI == ADD ? Buffers{3, 1, 1, BUF}
                                               : Buffers{2, 1, 0, CHUNK * CHUNK * static_cast<int>(sizeof(Out))};
}

template <Epi EPI, typename Out>
struct Layout {
    static constexpr Buffers B = buffers<EPI, Out>();
    static constexpr int WARP_BYTES = B.sets * B.boxes * B.bytes;
    static constexpr int STAGES = EPI == DACT ? 5 : 6;
    static constexpr int OFF_EPI = STAGES * STAGE;
    static constexpr int OFF_BARS = OFF_EPI + 4 * WARP_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 5 + 4 * B.sets;  // full, empty, tfull[2], tempty[2], drain, landed[4][sets]
    static constexpr int OFF_TMEM = OFF_BARS + NUM_BARS * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 4;
    static constexpr int BYTES = OFF_ABORT + 4 + 1024;  // slack for 1024-byte alignment
    static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

struct Params {
    int M, N, K;   // of the result and the sum; GATED: N = f
    int MT, NT;    // tiles
    int act;
    bool keep;     // GATED: store a
    int *status;
    uint64_t timeout_ns;
};
// a, b: operands.  GATED: out h, more g and u of `a`.  ADD: in.  DACT: in, in2 g and u, out h, more dg and du.
struct Maps {
    CUtensorMap a, b, out, more[2], in, in2;
};

struct Tile {
    int m0, n0;
};
template <Epi EPI>
__device__ __forceinline__ Tile decode(const Params &p, int tile) {
    const int band = tile / (BAND * p.NT), within = tile - band * BAND * p.NT;
    const int height = min(BAND, p.MT - band * BAND), n = within / height;
    return Tile{(band * BAND + within - n * height) * TILE_M, n * (EPI == GATED ? TILE_N / 2 : TILE_N)};
}

// One lane's 32 values into its row of a 32 x 32 bf16 box (64-byte swizzle), and back.
__device__ __forceinline__ void write_row(uint8_t *box, int lane, const uint32_t (&packed)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4 *>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
}
__device__ __forceinline__ void read_row(const uint8_t *box, int lane, uint32_t (&packed)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = *reinterpret_cast<const uint4 *>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
        packed[4 * j] = v.x, packed[4 * j + 1] = v.y, packed[4 * j + 2] = v.z, packed[4 * j + 3] = v.w;
    }
}
// The same for a 32 x 32 fp32 box (128-byte swizzle).
__device__ __forceinline__ void write_row(uint8_t *box, int lane, const uint32_t (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ float low(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// An epilogue warp: its 32 rows of a CTA's 128, and its buffers.
template <Epi EPI, typename Out>
struct Warp {
    using L = Layout<EPI, Out>;
    const Params &p;
    const Maps &maps;
    uint8_t *bufs;
    uint64_t *landed;
    volatile int *abort;
    int lane, row_of_tile;   // the first of its rows within a tile
    int pair, npairs;
    uint32_t turn = 0;       // chunks stored (without inputs: boxes stored)
    // the next chunk whose inputs are to be loaded
    int next_tile, next_c = 0;
    uint32_t asked = 0;

    // Without inputs: a box of packed values out through the next buffer.
    template <typename Values>
    __device__ __forceinline__ void put(const CUtensorMap *tm, const Values &v, int col, int row) {
        uint8_t *box = bufs + (turn & 1) * L::B.bytes;
        if (lane == 0) bulk_wait_read<1>();  // the store from two boxes ago has read it
        __syncwarp();
        write_row(box, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d_evict_first(tm, box, col, row, l2_policy_evict_first());
            bulk_commit();
        }
        ++turn;
    }

    // With inputs: asks for those of the next chunk (every lane follows the order, lane 0 loads).
    __device__ __forceinline__ void ask() {
        const int total = p.MT * p.NT;
        for (; next_tile < total; next_tile += npairs, next_c = 0) {
            const Tile t = decode<EPI>(p, next_tile);
            const int row = t.m0 + row_of_tile, col = t.n0 + next_c;
            if (row >= p.M || next_c >= TILE_N || col >= p.N) continue;
            if (lane == 0) {
                const int set = asked % L::B.sets;
                uint8_t *box = bufs + set * L::B.boxes * L::B.bytes;
                bulk_wait_read<L::B.sets - 2>();  // the stores of the chunk that used the set have read it
                mbar_arrive_expect_tx(&landed[set], L::B.in * L::B.bytes);
                tma_load_2d(box, &maps.in, &landed[set], col, row);
                if (EPI == DACT) tma_load_2d(box + L::B.bytes, &maps.in2, &landed[set], col, row);
            }
            ++asked;
            next_c += CHUNK;
            return;
        }
    }
    __device__ __forceinline__ bool inputs(uint32_t chunk) {
        return mbar_wait(&landed[chunk % L::B.sets], (chunk / L::B.sets) & 1, abort, p.status, p.timeout_ns);
    }
    // Before the warp leaves: its own copies have landed.
    __device__ __forceinline__ void finish() {
        volatile int no_abort = 0;
        for (uint32_t c = turn; L::B.in && c < asked; ++c)
            mbar_wait(&landed[c % L::B.sets], (c / L::B.sets) & 1, &no_abort, p.status, p.timeout_ns);
        if (lane == 0) bulk_wait_all();
    }

    // The warp's part of a tile, its accumulator (lane quarter) at tbase.
    __device__ __forceinline__ bool tile(const Tile &t, uint32_t tbase) {
        const int row = t.m0 + row_of_tile;
        if (row >= p.M) return true;  // the same for the warp
        if constexpr (EPI == GATED) {
#pragma unroll 1
            for (int c = 0; c < TILE_N / 2 && t.n0 + c < p.N; c += CHUNK) {
                uint32_t g[32], u[32], packed[16];
                tmem_ld_32x32b_x32(tbase + c, g);
                tmem_ld_32x32b_x32(tbase + TILE_N / 2 + c, u);
                tmem_ld_wait();
                with_activation(p.act, [&](auto act) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[i] = pack_bf16x2(
                            activate<act.value>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                            activate<act.value>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
                });
                put(&maps.out, packed, t.n0 + c, row);
                if (p.keep) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[i] = pack_bf16x2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
                    put(&maps.more[0], packed, t.n0 + c, row);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[i] = pack_bf16x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                    put(&maps.more[1], packed, t.n0 + c, row);
                }
            }
        } else if constexpr (EPI == PLAIN && sizeof(Out) == 4) {
#pragma unroll 1
            for (int c = 0; c < TILE_N && t.n0 + c < p.N; c += CHUNK) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tbase + c, v);
                tmem_ld_wait();
                put(&maps.out, v, t.n0 + c, row);
            }
        } else if constexpr (EPI == PLAIN) {
#pragma unroll 1
            for (int c = 0; c < TILE_N && t.n0 + c < p.N; c += 2 * CHUNK) {
                uint32_t v[2][32], packed[16];
                tmem_ld_32x32b_x32(tbase + c, v[0]);
                tmem_ld_32x32b_x32(tbase + c + CHUNK, v[1]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (t.n0 + c + k * CHUNK >= p.N) break;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[i] = pack_bf16x2(__uint_as_float(v[k][2 * i]), __uint_as_float(v[k][2 * i + 1]));
                    put(&maps.out, packed, t.n0 + c + k * CHUNK, row);
                }
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < TILE_N && t.n0 + c < p.N; c += CHUNK) {
                ask();  // for the chunk after this one
                uint32_t v[32], e[16];
                tmem_ld_32x32b_x32(tbase + c, v);
                tmem_ld_wait();
                if (!inputs(turn)) return false;
                uint8_t *box = bufs + (turn % L::B.sets) * L::B.boxes * L::B.bytes;
                read_row(box, lane, e);
                if constexpr (EPI == ADD) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        e[i] = pack_bf16x2(__uint_as_float(v[2 * i]) + low(e[i]),
                                           __uint_as_float(v[2 * i + 1]) + high(e[i]));
                    write_row(box, lane, e);
                } else {
                    uint32_t u[16], h[16];
                    read_row(box + L::B.bytes, lane, u);
                    with_activation(p.act, [&](auto act) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float slope[2];
                            const float a0 = activate<act.value>(low(e[i]), slope[0]);
                            const float a1 = activate<act.value>(high(e[i]), slope[1]);
                            const float d0 = __uint_as_float(v[2 * i]), d1 = __uint_as_float(v[2 * i + 1]);
                            const float u0 = low(u[i]), u1 = high(u[i]);
                            h[i] = pack_bf16x2(a0 * u0, a1 * u1);
                            e[i] = pack_bf16x2(d0 * u0 * slope[0], d1 * u1 * slope[1]);
                            u[i] = pack_bf16x2(d0 * a0, d1 * a1);
                        }
                    });
                    write_row(box, lane, e);
                    write_row(box + L::B.bytes, lane, u);
                    write_row(box + 2 * L::B.bytes, lane, h);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    const int col = t.n0 + c;
                    tma_store_2d_evict_first(EPI == ADD ? &maps.out : &maps.more[0], box, col, row,
                                             l2_policy_evict_first());
                    if (EPI == DACT) {
                        tma_store_2d_evict_first(&maps.more[1], box + L::B.bytes, col, row, l2_policy_evict_first());
                        tma_store_2d_evict_first(&maps.out, box + 2 * L::B.bytes, col, row, l2_policy_evict_first());
                    }
                    bulk_commit();
                }
                ++turn;
            }
        }
        return true;
    }
};

template <Epi EPI, bool A_MN, bool B_MN, typename Out>
__global__ void __launch_bounds__(THREADS, 1) ffn_gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
    using L = Layout<EPI, Out>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::OFF_BARS);  // used in CTA 0 only
    uint64_t *empty = full + STAGES;                                    // both CTAs
    uint64_t *tfull = empty + STAGES;                                   // both CTAs
    uint64_t *tempty = tfull + 2;                                       // CTA 0: 4 warps x 2 CTAs arrive
    uint64_t *drain = tempty + 2;
    uint64_t *landed = drain + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::OFF_TMEM);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0 issues the MMAs
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int half = 128 * static_cast<int>(rank);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 8);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < 4 * L::B.sets; ++i) mbar_init(&landed[i], 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
    }
    __syncthreads();
    // both CTAs' barriers exist before anything crosses the pair, and before
    // the collective allocation
    cluster_sync();
    if (warp == 1) {
        tmem_alloc_pair(s_tmem, 2 * TILE_N);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem;
    const int total = p.MT * p.NT, KB = (p.K + BK - 1) / BK;

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);  // both CTAs' copies signal CTA 0's barriers
            int armed[STAGES];
#pragma unroll
            for (int i = 0; i < STAGES; ++i) armed[i] = -1;
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < total; tile += npairs) {
                const Tile t = decode<EPI>(p, tile);
                const int a0 = t.m0 + half;
                // GATED: CTA 0 loads the gate rows, CTA 1 the up rows (those of a last
                // block past their half of W1 give columns that are not stored)
                const int b0 = EPI == GATED ? t.n0 + static_cast<int>(rank) * p.N : t.n0 + half;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait<true>(&empty[stage], phase ^ 1u, s_abort, p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + stage * STAGE, *sb = sa + 2 * BOX;
                    const uint32_t bar = full0 + 8u * stage;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * STAGE);
                    if (A_MN) {
                        tma_load_2d_pair(sa, &maps.a, bar, a0, kb * BK);
                        tma_load_2d_pair(sa + BOX, &maps.a, bar, a0 + 64, kb * BK);
                    } else {
                        tma_load_2d_pair(sa, &maps.a, bar, kb * BK, a0);
                    }
                    if (B_MN) {
                        tma_load_2d_pair(sb, &maps.b, bar, b0, kb * BK);
                        tma_load_2d_pair(sb + BOX, &maps.b, bar, b0 + 64, kb * BK);
                    } else {
                        tma_load_2d_pair(sb, &maps.b, bar, kb * BK, b0);
                    }
                    armed[stage] = static_cast<int>(phase);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
            if (!ok) {
                volatile int no_abort = 0;
                if (rank == 0) {
                    for (int i = 0; i < STAGES; ++i)
                        if (armed[i] >= 0)
                            mbar_wait<true>(&full[i], static_cast<uint32_t>(armed[i]), &no_abort, p.status,
                                            p.timeout_ns);
                } else {
                    // this CTA's copies signal CTA 0's barriers: give them time to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(TILE_M, TILE_N, A_MN, B_MN);
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true, issued = false;
            for (int tile = pair; ok && tile < total; tile += npairs) {
                if (!mbar_wait<true>(&tempty[acc], acc_phase ^ 1u, s_abort, p.status, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * TILE_N;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait<true>(&full[stage], phase, s_abort, p.status, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * STAGE);
                    const uint64_t adesc = A_MN ? smem_desc_mnmajor_sw128(sa, BOX) : smem_desc_kmajor_sw128(sa);
                    const uint64_t bdesc =
                        B_MN ? smem_desc_mnmajor_sw128(sa + 2 * BOX, BOX) : smem_desc_kmajor_sw128(sa + 2 * BOX);
#pragma unroll
                    for (int j = 0; j < BK / UMMA_K; ++j)
                        umma_bf16_pair(d_tmem, adesc + (A_MN ? 128 : 2) * j, bdesc + (B_MN ? 128 : 2) * j, idesc,
                                       (kb | j) != 0);
                    issued = true;
                    umma_commit_pair_multicast(&empty[stage], 0x3);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                umma_commit_pair_multicast(&tfull[acc], 0x3);
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok && issued) {
                volatile int no_abort = 0;
                umma_commit_pair_multicast(drain, 0x1);
                mbar_wait<true>(drain, 0, &no_abort, p.status, p.timeout_ns);
            }
        }
    } else {
        const int q = warp & 3;  // the lane quarter that a warp may read
        Warp<EPI, Out> w{p, maps, smem + L::OFF_EPI + (warp - 2) * L::WARP_BYTES, landed + (warp - 2) * L::B.sets, s_abort,
                         lane, half + 32 * q, pair, npairs, 0, pair};
        if (L::B.in) w.ask();
        const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
        uint32_t acc = 0, acc_phase = 0;
        for (int tile = pair; tile < total; tile += npairs) {
            if (!mbar_wait<true>(&tfull[acc], acc_phase, s_abort, p.status, p.timeout_ns)) break;
            tc_fence_after();
            if (!w.tile(decode<EPI>(p, tile), tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE_N)) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_cta(tempty0 + 8u * acc);
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
        w.finish();
    }

    tc_fence_before();
    __syncthreads();
    // neither CTA leaves (or frees TMEM) while its peer may still touch its
    // shared memory or tensor memory
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * TILE_N);
    }
}

// ======================================================================
// Few tokens: the weights are the 128 rows of an MMA and the tokens its
// columns (16 to 128), so that a weight is read once and no row is masked; the
// result lies transposed in TMEM, a lane per weight row.  A cluster of CTAs
// shares a block of rows, each a run of K's slices, so that weights stream into
// most SMs whatever their shape; the CTAs then send each other their partial
// sums, each getting those of a share of the tokens, and add them in the
// order of the CTAs (the same bits on every call).
// GATED: two MMAs per step, the block's gate rows and its up rows.
// ======================================================================
constexpr int FEW_ROWS = 128;
constexpr int FEW_THREADS = 128;
constexpr int FEW_A = 2 * FEW_ROWS * BK * 2;  // weights of a stage: a slice of gate and up rows, or two slices
constexpr int FEW_MAX_TOKENS = 128, FEW_MAX_STAGES = 6;

struct FewParams {
    int T, N, K;   // tokens, result columns (weight rows), length of the sum
    int tokens;    // of a block, a multiple of 16
    int stages, split;
    int tmem_cols;
    int act;
    __nv_bfloat16 *out, *preact;  // [T, N]; GATED, nullable: [T, 2N]
    const __nv_bfloat16 *add;     // nullable, not GATED: [T, N]
    bool behind;                  // launched before the kernel that writes B has ended
    int *status;
    uint64_t timeout_ns;
};
struct FewMaps {
    CUtensorMap w, x;
};

template <bool GATE>
__global__ void __launch_bounds__(FEW_THREADS) ffn_few_kernel(const __grid_constant__ FewMaps maps, const FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[FEW_MAX_STAGES], empty[FEW_MAX_STAGES], done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    volatile int *abort = &s_abort;
    constexpr int SLICES = GATE ? 1 : 2;  // of K in a stage
    const int warp = threadIdx.x >> 5;
    const int rank = static_cast<int>(blockIdx.x) % p.split, row0 = static_cast<int>(blockIdx.x) / p.split * FEW_ROWS;
    const int t0 = static_cast<int>(blockIdx.y) * p.tokens;
    const int box = p.tokens * BK * 2, stage_bytes = FEW_A + SLICES * box;
    const int KB = (p.K + SLICES * BK - 1) / (SLICES * BK);
    const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / p.split);
    const int kbs = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / p.split) - kb0;  // 1 or more

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        s_abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
    }
    if (warp == 1) {
        tmem_alloc(&s_tmem, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // the kernel behind this one (the product with W2) may start, up to where it needs h
    if (GATE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        auto weights = [&](int i, int stage) {
            uint8_t *sa = smem + stage * stage_bytes;
            const int k = (kb0 + i) * SLICES * BK;
            mbar_arrive_expect_tx(&full[stage], stage_bytes);
            if (GATE) {
                tma_load_2d(sa, &maps.w, &full[stage], k, row0);
                tma_load_2d(sa + FEW_A / 2, &maps.w, &full[stage], k, p.N + row0);
            } else {
                tma_load_2d(sa, &maps.w, &full[stage], k, row0);
                tma_load_2d(sa + FEW_A / 2, &maps.w, &full[stage], k + BK, row0);
            }
        };
        auto activations = [&](int i, int stage) {
            uint8_t *sb = smem + stage * stage_bytes + FEW_A;
            const int k = (kb0 + i) * SLICES * BK;
            for (int s = 0; s < SLICES; ++s) tma_load_2d(sb + s * box, &maps.x, &full[stage], k + s * BK, t0);
        };
        // the weights of the first stages do not wait for the kernel before
        const int first = min(kbs, p.stages);
        for (int i = 0; i < first; ++i) weights(i, i);
        if (p.behind) {
            grid_dependency_wait();
            asm volatile("fence.proxy.async;" ::: "memory");  // its plain stores before these copies
        }
        for (int i = 0; i < first; ++i) activations(i, i);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int armed = first;
        for (int i = first; i < kbs; ++i) {
            if (!mbar_wait(&empty[stage], phase, abort, p.status, p.timeout_ns)) {
                ok = false;
                break;
            }
            weights(i, stage);
            activations(i, stage);
            ++armed;
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        }
        if (!ok) {
            volatile int no_abort = 0;  // the copies in flight: the last ones of each stage
            for (int i = max(0, armed - p.stages); i < armed; ++i)
                mbar_wait(&full[i % p.stages], (i / p.stages) & 1, &no_abort, p.status, p.timeout_ns);
        }
    } else if (threadIdx.x == 32) {
        const uint32_t idesc = idesc_bf16_f32(FEW_ROWS, p.tokens);
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; i < kbs; ++i) {
            if (!mbar_wait(&full[stage], phase, abort, p.status, p.timeout_ns)) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * stage_bytes), sb = sa + FEW_A;
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // GATE: gate and up rows; else the two slices
                const uint64_t adesc = smem_desc_kmajor_sw128(sa + s * (FEW_A / 2));
                const uint64_t bdesc = smem_desc_kmajor_sw128(sb + (GATE ? 0 : s * box));
#pragma unroll
                for (int j = 0; j < BK / UMMA_K; ++j)
                    umma_bf16(tmem + (GATE ? s * p.tokens : 0), adesc + 2 * j, bdesc + 2 * j, idesc,
                              GATE ? (i | j) != 0 : (i | s | j) != 0);
            }
            umma_commit(&empty[stage]);
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        }
        umma_commit(&done);
    }
    __syncwarp();
    // every thread waits for the MMAs (after a wait that ran out: for those that were issued)
    volatile int no_abort = 0;
    mbar_wait(&done, 0, &no_abort, p.status, 2 * p.timeout_ns);
    __syncwarp();  // what follows is for whole warps at once
    tc_fence_after();
    const uint32_t tbase = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int row = row0 + static_cast<int>(threadIdx.x);  // the lane's weight row is the result's column
    auto store = [&](int t, float a, float u) {
        if (t >= p.T || row >= p.N) return;
        const size_t at = static_cast<size_t>(t) * p.N + row;
        if constexpr (GATE) {
            float act;
            with_activation(p.act, [&](auto k) { act = activate<k.value>(a); });
            p.out[at] = __float2bfloat16_rn(act * u);
            if (p.preact) {
                p.preact[2 * static_cast<size_t>(t) * p.N + row] = __float2bfloat16_rn(a);
                p.preact[(2 * static_cast<size_t>(t) + 1) * p.N + row] = __float2bfloat16_rn(u);
            }
        } else {
            p.out[at] = __float2bfloat16_rn(p.add ? a + __bfloat162float(p.add[at]) : a);
        }
    };
    if (p.split == 1) {
        if (!GATE && p.behind) grid_dependency_wait();  // before plain loads and stores of this thread
        for (int c = 0; c < p.tokens; c += 16) {
            if (t0 + c >= p.T) break;
            uint32_t a[16], u[16];
            tmem_ld_32x32b_x16(tbase + c, a);
            if (GATE) tmem_ld_32x32b_x16(tbase + p.tokens + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) store(t0 + c + i, __uint_as_float(a[i]), GATE ? __uint_as_float(u[i]) : 0.0f);
        }
    } else {
        // [source CTA][token of this CTA's share][gate, up][row], over the ring
        constexpr int PARTS = GATE ? 2 : 1;
        const int share = p.tokens / p.split;
        float *sums = reinterpret_cast<float *>(smem);
        cluster_sync();  // no CTA's ring is in use any more
        for (int c = 0; c < p.tokens; c += 16) {
            if (t0 + c >= p.T) break;
            uint32_t v[PARTS][16];
            tmem_ld_32x32b_x16(tbase + c, v[0]);
            if (GATE) tmem_ld_32x32b_x16(tbase + p.tokens + c, v[PARTS - 1]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int owner = (c + i) / share, mine = (c + i) % share;
#pragma unroll
                for (int k = 0; k < PARTS; ++k) {
                    const int at = ((rank * share + mine) * PARTS + k) * FEW_ROWS + static_cast<int>(threadIdx.x);
                    const uint32_t to = mapa_shared(smem_u32(sums + at), owner);
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v[k][i]) : "memory");
                }
            }
        }
        cluster_sync();  // every CTA's sums are there
        __syncwarp();
        if (!GATE && p.behind) grid_dependency_wait();
        for (int mine = 0; mine < share; ++mine) {
            const int t = t0 + rank * share + mine;
            if (t >= p.T) break;
            float v[PARTS] = {};
            for (int s = 0; s < p.split; ++s)
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
                    v[k] += sums[((s * share + mine) * PARTS + k) * FEW_ROWS + threadIdx.x];
            store(t, v[0], v[PARTS - 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
}

// ------------------------------------------------------------------ host side
namespace {

// bf16 [rows, cols] with rows `ld` elements apart.
bool map2d(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows, int box_cols,
           CUtensorMapSwizzle swizzle) {
    auto fn = tmap_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An operand: K-major boxes of 128 rows, or MN-major ones of 64 x 64.
bool operand(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, bool mn) {
    return map2d(m, base, rows, cols, cols, mn ? 64 : 128, BK, CU_TENSOR_MAP_SWIZZLE_128B);
}
// A matrix that the epilogue reads or writes in 32 x 32 boxes.
bool boxes(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld) {
    return map2d(m, base, rows, cols, ld, CHUNK, CHUNK, CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaLaunchConfig_t pair_config(int grid, int smem, cudaStream_t stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(THREADS), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = 2, attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = 1;
    return cfg;
}

template <Epi EPI, bool A_MN, bool B_MN, typename Out>
cudaError_t set_up(int *pairs) {
    auto kernel = ffn_gemm_kernel<EPI, A_MN, B_MN, Out>;
    constexpr int smem = Layout<EPI, Out>::BYTES;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = pair_config(2, smem, nullptr, &attr);
    int n = 0;
    const cudaError_t q = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (q != cudaSuccess) return q;
    *pairs = std::min(*pairs, n);
    return cudaSuccess;
}

template <Epi EPI, bool A_MN, bool B_MN, typename Out = uint16_t>
cudaError_t gemm(const Maps &maps, Params p, const GemmLaunch &lc, cudaStream_t stream) {
    constexpr int n = EPI == GATED ? TILE_N / 2 : TILE_N;
    p.MT = (p.M + TILE_M - 1) / TILE_M, p.NT = (p.N + n - 1) / n;
    cudaLaunchAttribute attr;
    const int64_t tiles = static_cast<int64_t>(p.MT) * p.NT;
    const int grid = 2 * static_cast<int>(std::min<int64_t>(tiles, lc.ffn_pairs));
    cudaLaunchConfig_t cfg = pair_config(grid, Layout<EPI, Out>::BYTES, stream, &attr);
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, A_MN, B_MN, Out>, maps, p);
}

constexpr int FEW_SMEM = 224 * 1024;

// How a product of few tokens is cut.
struct FewShape {
    int tokens, blocks, rows, split, stages, smem;
    FewShape(int T, int N, int K, bool gate, int sms) {
        blocks = (T + FEW_MAX_TOKENS - 1) / FEW_MAX_TOKENS;
        tokens = ((T + blocks - 1) / blocks + 15) / 16 * 16;
        rows = (N + FEW_ROWS - 1) / FEW_ROWS;
        const int slices = gate ? 1 : 2, KB = (K + slices * BK - 1) / (slices * BK);
        const int stage = FEW_A + slices * tokens * BK * 2;
        const int per_sm = tokens <= 16 ? 2 : 1;
        const int room = (FEW_SMEM / per_sm - 2048) / stage;
        split = 1;
        while (split < 8 && 2 * split * rows * blocks <= per_sm * sms && KB >= 4 * split) split *= 2;
        stages = std::min({room, FEW_MAX_STAGES, (KB + split - 1) / split});
        // the ring also holds the partial sums
        const int sums = split > 1 ? tokens * FEW_ROWS * 4 * (gate ? 2 : 1) : 0;
        smem = std::max(stages * stage, sums) + 1024;
    }
};

// `behind`: launched while the kernel before it, which writes x, still runs.
template <bool GATE>
cudaError_t few(const uint16_t *w, const uint16_t *x, int T, int N, int K, FewParams p, bool behind,
                const GemmLaunch &lc, cudaStream_t stream) {
    const FewShape s(T, N, K, GATE, lc.num_sms);
    FewMaps maps;
    if (!operand(&maps.w, w, GATE ? 2 * static_cast<int64_t>(N) : N, K, false) ||
        !map2d(&maps.x, x, T, K, K, s.tokens, BK, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.T = T, p.N = N, p.K = K, p.tokens = s.tokens, p.stages = s.stages, p.split = s.split, p.behind = behind;
    p.tmem_cols = 32;
    while (p.tmem_cols < s.tokens * (GATE ? 2 : 1)) p.tmem_cols *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s.split, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s.rows * s.split, s.blocks), cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = s.smem, cfg.stream = stream;
    cfg.attrs = attr, cfg.numAttrs = behind ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ffn_few_kernel<GATE>, maps, p);
}

// Where the tiles of CTA pairs are too few to keep the SMs busy.
bool use_few(int T, int N, bool gate, int pairs) {
    const int n = gate ? TILE_N / 2 : TILE_N;
    const int64_t tiles = static_cast<int64_t>((T + TILE_M - 1) / TILE_M) * ((N + n - 1) / n);
    return T <= FEW_MAX_TOKENS || 2 * tiles <= pairs;
}

}  // namespace
}  // namespace ff

cudaError_t ffn_setup(GemmLaunch *cfg) {
    using namespace ff;
    int pairs = cfg->num_sms / 2;
    cudaError_t e;
    if ((e = set_up<GATED, false, false, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<PLAIN, false, false, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<ADD, false, false, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<DACT, false, true, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<PLAIN, false, true, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<ADD, false, true, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<PLAIN, true, true, uint16_t>(&pairs)) != cudaSuccess ||
        (e = set_up<PLAIN, true, true, float>(&pairs)) != cudaSuccess)
        return e;
    for (const void *k : {reinterpret_cast<const void *>(ffn_few_kernel<true>),
                          reinterpret_cast<const void *>(ffn_few_kernel<false>)})
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM)) != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cfg->ffn_pairs = pairs;
    return cudaSuccess;
}

cudaError_t launch_ffn(const FfnArgs &a, const GemmLaunch &lc, cudaStream_t stream) {
    using namespace ff;
    const bool few_up = use_few(a.T, a.f, true, lc.ffn_pairs), few_down = use_few(a.T, a.d, false, lc.ffn_pairs);
    FewParams fp = {};
    fp.act = a.act, fp.status = a.status, fp.timeout_ns = a.timeout_ns;
    Params p = {};
    p.act = a.act, p.status = a.status, p.timeout_ns = a.timeout_ns;
    cudaError_t e;
    if (few_up) {
        fp.out = reinterpret_cast<__nv_bfloat16 *>(a.h), fp.preact = reinterpret_cast<__nv_bfloat16 *>(a.preact);
        e = few<true>(a.W1, a.x, a.T, a.f, a.d, fp, false, lc, stream);
    } else {
        Maps m = {};
        p.M = a.T, p.N = a.f, p.K = a.d, p.keep = a.preact != nullptr;
        if (!operand(&m.a, a.x, a.T, a.d, false) || !operand(&m.b, a.W1, 2 * static_cast<int64_t>(a.f), a.d, false) ||
            !boxes(&m.out, a.h, a.T, a.f, a.f) ||
            (a.preact && (!boxes(&m.more[0], a.preact, a.T, a.f, 2 * static_cast<int64_t>(a.f)) ||
                          !boxes(&m.more[1], a.preact + a.f, a.T, a.f, 2 * static_cast<int64_t>(a.f)))))
            return cudaErrorInvalidValue;
        e = gemm<GATED, false, false>(m, p, lc, stream);
    }
    if (e != cudaSuccess) return e;
    if (few_down) {
        fp.out = reinterpret_cast<__nv_bfloat16 *>(a.y), fp.preact = nullptr;
        fp.add = reinterpret_cast<const __nv_bfloat16 *>(a.add);
        return few<false>(a.W2, a.h, a.T, a.d, a.f, fp, few_up, lc, stream);
    }
    Maps m = {};
    p.M = a.T, p.N = a.d, p.K = a.f;
    if (!operand(&m.a, a.h, a.T, a.f, false) || !operand(&m.b, a.W2, a.d, a.f, false) ||
        !boxes(&m.out, a.y, a.T, a.d, a.d) || (a.add && !boxes(&m.in, a.add, a.T, a.d, a.d)))
        return cudaErrorInvalidValue;
    return a.add ? gemm<ADD, false, false>(m, p, lc, stream) : gemm<PLAIN, false, false>(m, p, lc, stream);
}

cudaError_t launch_ffn_bwd(const FfnGradArgs &a, const GemmLaunch &lc, int *launches, cudaStream_t stream) {
    using namespace ff;
    const int64_t f = a.f;
    Params p = {};
    p.act = a.act, p.status = a.status, p.timeout_ns = a.timeout_ns;
    *launches = 0;
    // da and h, from dh = dy W2 (W2 read as stored)
    {
        Maps m = {};
        p.M = a.T, p.N = a.f, p.K = a.d;
        if (!operand(&m.a, a.dy, a.T, a.d, false) || !operand(&m.b, a.W2, a.d, f, true) ||
            !boxes(&m.in, a.preact, a.T, f, 2 * f) || !boxes(&m.in2, a.preact + f, a.T, f, 2 * f) ||
            !boxes(&m.more[0], a.da, a.T, f, 2 * f) || !boxes(&m.more[1], a.da + f, a.T, f, 2 * f) ||
            !boxes(&m.out, a.h, a.T, f, f))
            return cudaErrorInvalidValue;
        const cudaError_t e = gemm<DACT, false, true>(m, p, lc, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    // dW [rows, cols] = left [T, rows]^T right [T, cols]
    auto wgrad = [&](const uint16_t *left, int64_t rows, const uint16_t *right, int64_t cols, void *out) {
        Maps m = {};
        p.M = static_cast<int>(rows), p.N = static_cast<int>(cols), p.K = a.T;
        if (!operand(&m.a, left, a.T, rows, true) || !operand(&m.b, right, a.T, cols, true)) return cudaErrorInvalidValue;
        ++*launches;
        if (a.weights_f32)
            return make_tmap_2d(&m.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, out, rows, cols, CHUNK, CHUNK,
                                CU_TENSOR_MAP_SWIZZLE_128B)
                       ? gemm<PLAIN, true, true, float>(m, p, lc, stream)
                       : cudaErrorInvalidValue;
        return boxes(&m.out, out, rows, cols, cols) ? gemm<PLAIN, true, true>(m, p, lc, stream) : cudaErrorInvalidValue;
    };
    if (a.dW2) {
        const cudaError_t e = wgrad(a.dy, a.d, a.h, f, a.dW2);
        if (e != cudaSuccess) return e;
    }
    if (a.dW1) {
        const cudaError_t e = wgrad(a.da, 2 * f, a.x, a.d, a.dW1);
        if (e != cudaSuccess) return e;
    }
    if (!a.dx) return cudaSuccess;
    Maps m = {};
    p.M = a.T, p.N = a.d, p.K = 2 * a.f;
    if (!operand(&m.a, a.da, a.T, 2 * f, false) || !operand(&m.b, a.W1, 2 * f, a.d, true) ||
        !boxes(&m.out, a.dx, a.T, a.d, a.d) || (a.add && !boxes(&m.in, a.add, a.T, a.d, a.d)))
        return cudaErrorInvalidValue;
    ++*launches;
    return a.add ? gemm<ADD, false, true>(m, p, lc, stream) : gemm<PLAIN, false, true>(m, p, lc, stream);
}

}  // namespace moe

// The gated feed-forward of all tokens (a shared expert, a dense layer), and its backward:
//   a = x W1^T = [g | u],  h = act(g) u,  y = h W2^T + add
//   dh = dy W2,  da = [dh u act'(g) | dh act(g)],  dx = da W1 + add,  dW1 = da^T x,  dW2 = dy^T h
// with x, y, dx, add [T, d], W1 [2f, d] (gate rows, then up rows), W2 [d, f], a [T, 2f], all bf16.
// Sums are fp32 in tensor memory.  h and da are rounded to bf16 once, as they
// are operands of the next product; dh and, in the forward, a are not rounded
// before the activation.  Backward reads a as the forward stored it.
//
// Three kernels make the five products; which one, goes by models of their times at the
// sizes (Ways, prefer_few, launch_ffn_bwd): ffn_tiny_kernel and ffn_few_kernel for few tokens,
// below, and for the rest one persistent kernel on CTA pairs: a 256 x 256 tile (or
// half of one, where tiles are few) of the result per pair through cta_group::2 MMAs, each CTA loading its
// 128 rows of A and half of the columns of B per 64-wide slice of K (32 KB),
// two accumulators in TMEM so that a tile's epilogue runs beside the next
// tile's products.  The sizes are known on the host, so tensor maps cut every
// matrix to its own size: loads past it read zeros, stores past it do nothing,
// and no size has to fill a tile.
//   epilogue GATED   h (and a) from a tile whose B rows are 128 gate and 128 up rows
//            PLAIN   the product, plus a matrix (ADD)
//            DACT    da and h from the tile of dh and the tiles of g and u
//            GRADS   dx, dW1 and dW2 from one list of tiles; the weights' in fp32 on request
// Warps: 0 TMA loads, 1 MMAs and TMEM, the others epilogue.  Every wait is bounded.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gated_ffn.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tmap.h"

namespace moe {
namespace ff {

using gg::pack_bf16x2;

enum Epi { GATED, PLAIN, ADD, DACT, GRADS };

constexpr int BK = 64;          // a slice of K: 128 bytes, one swizzle line
constexpr int UMMA_K = 16;
constexpr int TILE_M = 256, TILE_N = 256;
constexpr int BAND = 8;         // row blocks that sweep the column blocks together
// Epilogue warps: of GATED eight, two per lane quarter with half of a tile's columns
// each, as the last tile's epilogue is waited for (1003 x 2056 x 1368: 30.9 us with
// four, 30.0); DACT's buffers would leave eight a shorter ring (as measured when its
// outputs still took their inputs' place and that backward 64 us: 66.5, 4096 x 7168 x 2048 400
// and 411), or no input ahead (level: two warps per scheduler then take twice as long for a chunk).
__host__ __device__ constexpr int epi_warps(Epi epi) { return epi == GATED ? 8 : 4; }
__host__ __device__ constexpr int threads_of(Epi epi) { return 64 + 32 * epi_warps(epi); }
constexpr int BOX = 64 * 64 * 2;  // an MN-major box: 64 rows of K x 64 columns
constexpr int STAGE = 4 * BOX;    // of a CTA: 128 rows of A, 128 columns of B
constexpr int CHUNK = 32;         // the epilogue takes 32 rows x 32 columns per warp at a time
constexpr int BUF = CHUNK * CHUNK * 2;

// An epilogue warp's buffers in shared memory.  A chunk without inputs takes
// one of two boxes in turn.  TMA fills the `in` boxes of one of `sets` sets before a chunk
// with inputs is computed; the output takes their place, but for DACT, whose three outputs
// have boxes of their own: a chunk's inputs can so be asked for two chunks ahead, and
// none waits for stores (a chunk 1.6 us with outputs over inputs, 1.2).
struct Buffers {
    int sets, in, bytes;
};
template <Epi EPI, typename Out>
__host__ __device__ constexpr Buffers buffers() {
    constexpr int plain = 2 * CHUNK * CHUNK * static_cast<int>(sizeof(Out));
    return EPI == DACT                  ? Buffers{2, 2, (2 * 2 + 3) * BUF}
           : EPI == ADD || EPI == GRADS ? Buffers{3, 1, 3 * BUF > plain ? 3 * BUF : plain}
                                        : Buffers{2, 0, plain};
}

template <Epi EPI, typename Out>
struct Layout {
    static constexpr Buffers B = buffers<EPI, Out>();
    static constexpr int WARPS = epi_warps(EPI);
    static constexpr int STAGES = EPI == DACT ? 5 : 6;
    static constexpr int QUEUE = EPI == GRADS ? gg::queue_slots(STAGES) : 0;
    static constexpr int OFF_EPI = STAGES * STAGE;
    static constexpr int OFF_BARS = OFF_EPI + WARPS * B.bytes;
    // full, empty, tfull[2], tempty[2], drain, landed[WARPS][sets], queued[QUEUE]
    static constexpr int NUM_BARS = 2 * STAGES + 5 + WARPS * B.sets + QUEUE;
    static constexpr int OFF_QUEUE = OFF_BARS + NUM_BARS * 8;
    static constexpr int OFF_TMEM = OFF_QUEUE + QUEUE * 4;
    static constexpr int OFF_ABORT = OFF_TMEM + 4;
    static constexpr int BYTES = OFF_ABORT + 4 + 1024;  // slack for 1024-byte alignment
    static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

// One product: a result of M x N (GATED: N = f) and a sum of length K, in MT x NT
// tiles, band by band; those from `halves` on are cut into two of half the width,
// which come in the list in their place.
struct Product {
    int M, N, K, MT, NT;
    int halves, first, tiles;   // `first`: of this product in the list of tiles
};
constexpr int PRODUCTS = 3;     // GRADS: dx, dW1, dW2, in the order that the host gives
struct Params {
    Product product[PRODUCTS];
    int products, tiles;
    int kind[PRODUCTS];         // GRADS: which of KIND_*
    bool add;                   // GRADS: dx has a matrix to be added
    int act;
    bool keep;                  // GATED: store a
    int *tickets;               // GRADS, nullable: of the order of tiles (gg::Params::sched)
    int *status;
    uint64_t timeout_ns;
};
constexpr int KIND_DX = 0, KIND_WEIGHTS = 1;
// a, b: operands (half_b: b with boxes for half a tile, where b is K-major).
// GATED: out h, more g and u of `a`.  ADD: in.  DACT: in, in2 g and u, out h, more dg and du.
struct Maps {
    CUtensorMap a, b, half_b, out, more[2], in, in2;
};
struct GradMaps {
    CUtensorMap a[PRODUCTS], b[PRODUCTS], out[PRODUCTS], in;
};

struct Tile {
    int product, m0, n0, width;  // width: accumulator columns
};
template <Epi EPI>
__device__ __forceinline__ Tile decode(const Params &p, int tile) {
    Tile t;
    t.product = 0;
    if (EPI == GRADS)
        while (t.product + 1 < p.products && tile >= p.product[t.product + 1].first) ++t.product;
    const Product &q = p.product[t.product];
    int at = tile - q.first, sub = 0;
    t.width = TILE_N;
    if (at >= q.halves) {
        sub = (at - q.halves) & 1;
        at = q.halves + ((at - q.halves) >> 1);
        t.width = TILE_N / 2;
    }
    const int band = at / (BAND * q.NT), within = at - band * BAND * q.NT;
    const int height = min(BAND, q.MT - band * BAND), n = within / height;
    t.m0 = (band * BAND + within - n * height) * TILE_M;
    t.n0 = (2 * n + sub) * (EPI == GATED ? TILE_N / 4 : TILE_N / 2);
    return t;
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
// The i-th pair of a row's fp32 values; a pair of bf16, and back.
__device__ __forceinline__ float2 pair_of(const uint32_t (&v)[32], int i) {
    return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}
__device__ __forceinline__ float2 unpack(uint32_t p) {
    return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float2 v) { return pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ void pack(const uint32_t (&v)[32], uint32_t (&packed)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) packed[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// An epilogue warp: its 32 rows of a CTA's 128, and its buffers.
template <Epi EPI, typename Out>
struct Warp {
    using L = Layout<EPI, Out>;
    const Params &p;
    uint8_t *bufs;
    uint64_t *landed;
    volatile int *abort;
    int lane, row_of_tile;   // the first of its rows within a tile
    int part;                // of the columns: the first or the second half, where two warps share a lane quarter
    uint32_t boxes = 0;      // stored by put()
    uint32_t asked = 0, taken = 0;  // chunks whose inputs were asked for, and used

    // A box of values out through the next buffer.
    template <typename Values>
    __device__ __forceinline__ void put(const CUtensorMap *tm, const Values &v, int col, int row) {
        uint8_t *box = bufs + (boxes & 1) * sizeof(v) * 32;
        if (lane == 0) bulk_wait_read<1>();  // the store from two boxes ago has read it
        __syncwarp();
        write_row(box, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d_evict_first(tm, box, col, row, l2_policy_evict_first());
            bulk_commit();
        }
        ++boxes;
    }

    // Asks for the inputs of the next chunk.  FIRST: of a tile, whose buffers may be in other
    // use.  (DACT: the set's inputs have been read.)
    template <bool FIRST>
    __device__ __forceinline__ void ask(const CUtensorMap *in, const CUtensorMap *in2, int col, int row) {
        if (lane == 0) {
            const int set = asked % L::B.sets;
            uint8_t *box = bufs + set * L::B.in * BUF;
            // the store of the chunk that used the set has read it
            if (EPI != DACT) bulk_wait_read<FIRST ? 0 : L::B.sets - 2>();
            mbar_arrive_expect_tx(&landed[set], L::B.in * BUF);
            tma_load_2d(box, in, &landed[set], col, row);
            if (EPI == DACT) tma_load_2d(box + BUF, in2, &landed[set], col, row);
        }
        ++asked;
    }
    // Before the warp leaves: its own copies have landed.
    __device__ __forceinline__ void finish() {
        volatile int no_abort = 0;
        for (uint32_t c = taken; L::B.in && c != asked; ++c)
            mbar_wait(&landed[c % L::B.sets], (c / L::B.sets) & 1, &no_abort, p.status, p.timeout_ns);
        if (lane == 0) bulk_wait_all();
    }

    // 64 columns at a time of a product that is stored as it is
    __device__ __forceinline__ void plain(const CUtensorMap *out, const Product &q, const Tile &t, uint32_t tbase, int row) {
        // the boxes may hold inputs' chunks that are still being stored
        if (EPI == GRADS && lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < t.width && t.n0 + c < q.N; c += 2 * CHUNK) {
            uint32_t v[2][32];
            tmem_ld_32x32b_x32(tbase + c, v[0]);
            tmem_ld_32x32b_x32(tbase + c + CHUNK, v[1]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int col = t.n0 + c + k * CHUNK;
                if (col >= q.N) break;
                if constexpr (sizeof(Out) == 4) {
                    put(out, v[k], col, row);
                } else {
                    uint32_t packed[16];
                    pack(v[k], packed);
                    put(out, packed, col, row);
                }
            }
        }
    }

    // The first of the warp's columns of a tile that has `columns`, and the end of them.
    __device__ __forceinline__ int begin(int columns) const { return L::WARPS == 8 ? part * columns / 2 : 0; }
    __device__ __forceinline__ int end(int columns) const { return L::WARPS == 8 ? (part + 1) * columns / 2 : columns; }

    // h of a tile whose accumulator holds gate columns and then as many up columns
    __device__ __forceinline__ void gated(const Maps &maps, const Product &q, const Tile &t, uint32_t tbase, int row) {
#pragma unroll 1
        for (int c = begin(t.width / 2); c < end(t.width / 2) && t.n0 + c < q.N; c += CHUNK) {
            uint32_t g[32], u[32], packed[16];
            tmem_ld_32x32b_x32(tbase + c, g);
            tmem_ld_32x32b_x32(tbase + t.width / 2 + c, u);
            tmem_ld_wait();
            with_activation(p.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 16; ++i) packed[i] = pack(mul2(activate<act.value>(pair_of(g, i)), pair_of(u, i)));
            });
            put(&maps.out, packed, t.n0 + c, row);
            if (p.keep) {
                pack(g, packed);
                put(&maps.more[0], packed, t.n0 + c, row);
                pack(u, packed);
                put(&maps.more[1], packed, t.n0 + c, row);
            }
        }
    }

    // A chunk's inputs are on their way while the one (DACT: the two) before it are computed.
    __device__ __forceinline__ bool with_inputs(const CUtensorMap *in, const CUtensorMap *in2, const CUtensorMap *out,
                                                const CUtensorMap *out2, const CUtensorMap *out3, const Product &q,
                                                const Tile &t, uint32_t tbase, int row) {
#pragma unroll 1
        for (int c = begin(t.width); c < end(t.width) && t.n0 + c < q.N; c += CHUNK) {
            const int col = t.n0 + c;
            const auto ask_for = [&](int chunks) {  // the inputs that lie so many on
                if (c + chunks * CHUNK < end(t.width) && col + chunks * CHUNK < q.N)
                    ask<false>(in, in2, col + chunks * CHUNK, row);
            };
            if (EPI != DACT) ask_for(1);
            uint32_t v[32], e[16];
            tmem_ld_32x32b_x32(tbase + c, v);
            tmem_ld_wait();
            const uint32_t set = taken % L::B.sets;
            if (!mbar_wait(&landed[set], (taken / L::B.sets) & 1, abort, p.status, p.timeout_ns)) return false;
            ++taken;
            uint8_t *box = bufs + set * L::B.in * BUF;
            read_row(box, lane, e);
            if constexpr (EPI != DACT) {
#pragma unroll
                for (int i = 0; i < 16; ++i) e[i] = pack(add2(pair_of(v, i), unpack(e[i])));
                write_row(box, lane, e);
            } else {
                uint32_t u[16], h[16];
                read_row(box + BUF, lane, u);
                // the whole warp has read them: without the fence a copy could land before a
                // read that was still on its way (once in 2e6 chunks)
                fence_proxy_async_smem();
                __syncwarp();
                ask_for(2);
                with_activation(p.act, [&](auto act) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 slope;
                        const float2 a = activate<act.value>(unpack(e[i]), slope), up = unpack(u[i]), d = pair_of(v, i);
                        h[i] = pack(mul2(a, up));
                        e[i] = pack(mul2(mul2(d, up), slope));
                        u[i] = pack(mul2(d, a));
                    }
                });
                box = bufs + L::B.sets * L::B.in * BUF;
                if (lane == 0) bulk_wait_read<0>();  // the last chunk's stores have read the boxes
                __syncwarp();
                write_row(box, lane, e);
                write_row(box + BUF, lane, u);
                write_row(box + 2 * BUF, lane, h);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d_evict_first(out, box, col, row, l2_policy_evict_first());
                if (EPI == DACT) {
                    tma_store_2d_evict_first(out2, box + BUF, col, row, l2_policy_evict_first());
                    tma_store_2d_evict_first(out3, box + 2 * BUF, col, row, l2_policy_evict_first());
                }
                bulk_commit();
            }
        }
        return true;
    }
};

// M: Maps, or GradMaps for GRADS, whose products have operands of their own:
// dx an A that is K-major, the weights' gradients one that is MN-major; B is MN-major in all.
template <Epi EPI, bool A_MN, bool B_MN, typename Out, typename M>
__global__ void __launch_bounds__(threads_of(EPI), 1) ffn_gemm_kernel(const __grid_constant__ M maps, const Params p) {
    using L = Layout<EPI, Out>;
    constexpr int STAGES = L::STAGES, QUEUE = L::QUEUE;
    constexpr bool MANY = EPI == GRADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::OFF_BARS);  // used in CTA 0 only
    uint64_t *empty = full + STAGES;                                    // both CTAs
    uint64_t *tfull = empty + STAGES;                                   // both CTAs
    uint64_t *tempty = tfull + 2;                                       // CTA 0: the warps of both CTAs arrive
    uint64_t *drain = tempty + 2;
    uint64_t *landed = drain + 1;
    uint64_t *queued = landed + L::WARPS * L::B.sets;                          // both CTAs
    volatile int *queue = reinterpret_cast<volatile int *>(smem + L::OFF_QUEUE);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::OFF_TMEM);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0 issues the MMAs
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int half = 128 * static_cast<int>(rank);
    const bool drawn = MANY && p.tickets != nullptr;  // the order of tiles: by tickets, else in turn

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * L::WARPS);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < L::WARPS * L::B.sets; ++i) mbar_init(&landed[i], 1);
        for (int i = 0; i < QUEUE; ++i) mbar_init(&queued[i], 1);
        *s_abort = 0;
        fence_mbar_init();
    } else if (threadIdx.x == 32) {
        if constexpr (MANY) {
            for (int i = 0; i < p.products; ++i) {
                tma_prefetch_desc(&maps.a[i]);
                tma_prefetch_desc(&maps.b[i]);
                tma_prefetch_desc(&maps.out[i]);
            }
        } else {
            tma_prefetch_desc(&maps.a);
            tma_prefetch_desc(&maps.b);
            tma_prefetch_desc(&maps.out);
        }
    }
    // both CTAs' barriers exist before anything crosses the pair, and before
    // the collective allocation, which the loads need not wait for
    cluster_sync();
    uint32_t tmem_base = 0;
    if (warp != 0) {
        if (warp == 1) {
            tmem_alloc_pair(s_tmem, 2 * TILE_N);
            tmem_relinquish_pair();
        }
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(threads_of(EPI) - 32) : "memory");
        tc_fence_after();
        tmem_base = *s_tmem;
    }

    // The k-th tile of the pair (a negative one ends the list) for the roles that do not decide it.
    auto tile_of = [&](int k, int *tile) {
        if (!drawn) {
            *tile = pair + k * npairs < p.tiles ? pair + k * npairs : -1;
            return true;
        }
        if (!mbar_wait<true>(&queued[k % max(QUEUE, 1)], (k / max(QUEUE, 1)) & 1, s_abort, p.status, p.timeout_ns))
            return false;
        *tile = queue[k % max(QUEUE, 1)];
        return true;
    };
    auto slices = [&](const Tile &t) { return (p.product[t.product].K + BK - 1) / BK; };

    if (warp == 0) {
        if (lane == 0) {
            // (only now may the next kernel start: it goes by what was written before this one)
            grid_dependency_wait_to_copy();
            grid_dependency_launch();
            const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);  // both CTAs' copies signal CTA 0's barriers
            const uint32_t queue1 = mapa_shared(smem_u32(const_cast<int *>(queue)), 1);
            const uint32_t queued1 = mapa_shared(smem_u32(queued), 1);
            // CTA 0 draws the pair's tiles and tells both CTAs: the ticket of tile k + 1 at most
            // 24 slices before the loads of tile k end, so that a pair with a long tile keeps no
            // others from those that are free (777 x 1032 x 2056: 64 us with two tiles drawn
            // ahead, 48).  Not by a test in the loop over the slices: this thread's latency per
            // slice counts (4096 x 7168 x 2048: 428 us with it, 394).
            auto publish = [&](int k, int tile) {
                queue[k % max(QUEUE, 1)] = tile;
                mbar_arrive(&queued[k % max(QUEUE, 1)]);
                send_to_peer(queue1 + 4u * (k % max(QUEUE, 1)), tile, queued1 + 8u * (k % max(QUEUE, 1)));
            };
            int current = -1, next = -1;
            if (drawn && rank == 0) {
                current = atomicAdd(p.tickets, 1);
                if (current >= p.tiles) current = -1;
                publish(0, current);
            }
            int armed[STAGES];
#pragma unroll
            for (int i = 0; i < STAGES; ++i) armed[i] = -1;
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                int tile;
                if (drawn && rank == 0) {
                    tile = current;
                } else if (!tile_of(k, &tile)) {
                    ok = false;
                    break;
                }
                if (tile < 0) break;
                const Tile t = decode<EPI>(p, tile);
                const bool whole = t.width == TILE_N;
                const CUtensorMap *ma, *mb;
                bool a_mn = A_MN;
                if constexpr (MANY) {
                    ma = &maps.a[t.product], mb = &maps.b[t.product];
                    a_mn = p.kind[t.product] == KIND_WEIGHTS;
                } else {
                    ma = &maps.a, mb = whole || B_MN ? &maps.b : &maps.half_b;
                }
                const int a0 = t.m0 + half, KB = slices(t);
                // GATED: CTA 0 loads the gate rows, CTA 1 the up rows (those of a last
                // block past their half of W1 give columns that are not stored)
                const int b0 = EPI == GATED ? t.n0 + static_cast<int>(rank) * p.product[0].N
                                            : t.n0 + static_cast<int>(rank) * (t.width / 2);
                auto load = [&](int from, int to) {
                    for (int kb = from; kb < to; ++kb) {
                        if (!mbar_wait<true>(&empty[stage], phase ^ 1u, s_abort, p.status, p.timeout_ns)) {
                            ok = false;
                            return;
                        }
                        uint8_t *sa = smem + stage * STAGE, *sb = sa + 2 * BOX;
                        const uint32_t bar = full0 + 8u * stage;
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], whole ? 2 * STAGE : 2 * (STAGE - BOX));
                        if (a_mn) {
                            tma_load_2d_pair(sa, ma, bar, a0, kb * BK);
                            tma_load_2d_pair(sa + BOX, ma, bar, a0 + 64, kb * BK);
                        } else {
                            tma_load_2d_pair(sa, ma, bar, kb * BK, a0);
                        }
                        if (B_MN) {
                            tma_load_2d_pair(sb, mb, bar, b0, kb * BK);
                            if (whole) tma_load_2d_pair(sb + BOX, mb, bar, b0 + 64, kb * BK);
                        } else {
                            tma_load_2d_pair(sb, mb, bar, kb * BK, b0);
                        }
                        armed[stage] = static_cast<int>(phase);
                        if (++stage == STAGES) stage = 0, phase ^= 1u;
                    }
                };
                int at = 0;
                if (drawn && rank == 0) {
                    load(0, at = max(KB - 24, 0));
                    if (!ok) break;
                    next = atomicAdd(p.tickets, 1);
                    const int then = max(KB - 16, min(KB, 1));
                    load(at, then);
                    at = then;
                    if (!ok) break;
                    current = next < p.tiles ? next : -1;
                    publish(k + 1, current);
                }
                load(at, KB);
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
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true, issued = false;
            for (int k = 0; ok; ++k) {
                int tile;
                if (!tile_of(k, &tile)) {
                    ok = false;
                    break;
                }
                if (tile < 0) break;
                const Tile t = decode<EPI>(p, tile);
                const bool a_mn = MANY ? p.kind[t.product] == KIND_WEIGHTS : A_MN;
                const uint32_t idesc = idesc_bf16_f32(TILE_M, TILE_N, false, B_MN) - ((TILE_N - t.width) >> 3 << 17) +
                                       (a_mn ? 1u << 15 : 0u);
                const int KB = slices(t);
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
                    const uint64_t adesc = a_mn ? smem_desc_mnmajor_sw128(sa, BOX) : smem_desc_kmajor_sw128(sa);
                    const uint64_t bdesc =
                        B_MN ? smem_desc_mnmajor_sw128(sa + 2 * BOX, BOX) : smem_desc_kmajor_sw128(sa + 2 * BOX);
                    const uint32_t step = a_mn ? 128 : 2;
#pragma unroll
                    for (int j = 0; j < BK / UMMA_K; ++j)
                        umma_bf16_pair(d_tmem, adesc + step * j, bdesc + (B_MN ? 128 : 2) * j, idesc, (kb | j) != 0);
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
        Warp<EPI, Out> w{p, smem + L::OFF_EPI + (warp - 2) * L::B.bytes, landed + (warp - 2) * L::B.sets, s_abort, lane,
                         half + 32 * q, (warp - 2) >> 2};
        const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
        uint32_t acc = 0, acc_phase = 0;
        grid_dependency_wait_to_copy();  // its loads and stores are behind the kernel before, too
        for (int k = 0;; ++k) {
            int tile;
            if (!tile_of(k, &tile) || tile < 0) break;
            const Tile t = decode<EPI>(p, tile);
            const Product &pr = p.product[t.product];
            const int row = t.m0 + w.row_of_tile;
            const int columns = EPI == GATED ? t.width / 2 : t.width, col = t.n0 + w.begin(columns);
            const bool any = row < pr.M && col < pr.N;  // the same for the warp
            const bool inputs = EPI == DACT || EPI == ADD || (MANY && p.add && p.kind[t.product] == KIND_DX);
            if constexpr (L::B.in > 0)
                if (any && inputs) {
                    if constexpr (EPI == DACT) {
                        w.template ask<true>(&maps.in, &maps.in2, col, row);
                        if (col + CHUNK < pr.N) w.template ask<true>(&maps.in, &maps.in2, col + CHUNK, row);
                    } else {
                        w.template ask<true>(&maps.in, nullptr, col, row);
                    }
                }
            if (!mbar_wait<true>(&tfull[acc], acc_phase, s_abort, p.status, p.timeout_ns)) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE_N;
            bool ok = true;
            if (any) {
                if constexpr (EPI == GATED) {
                    w.gated(maps, pr, t, tbase, row);
                } else if constexpr (EPI == DACT) {
                    ok = w.with_inputs(&maps.in, &maps.in2, &maps.more[0], &maps.more[1], &maps.out, pr, t, tbase, row);
                } else if constexpr (EPI == ADD) {
                    ok = w.with_inputs(&maps.in, nullptr, &maps.out, nullptr, nullptr, pr, t, tbase, row);
                } else if constexpr (EPI == PLAIN) {
                    w.plain(&maps.out, pr, t, tbase, row);
                } else if (p.kind[t.product] == KIND_WEIGHTS) {
                    w.plain(&maps.out[t.product], pr, t, tbase, row);
                } else if (inputs) {
                    ok = w.with_inputs(&maps.in, nullptr, &maps.out[t.product], nullptr, nullptr, pr, t, tbase, row);
                } else {
                    Warp<PLAIN, uint16_t> dx{p, w.bufs, nullptr, s_abort, lane, w.row_of_tile, 0};
                    if (lane == 0) bulk_wait_read<0>();  // the boxes may still be being stored
                    __syncwarp();
                    dx.plain(&maps.out[t.product], pr, t, tbase, row);
                }
            }
            if (!ok) break;
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
    if (drawn && threadIdx.x == 0) {
        // the last CTA of the launch leaves the tickets as it found them
        __threadfence();
        if (atomicAdd(p.tickets + 1, 1) == static_cast<int>(gridDim.x) - 1) {
            atomicExch(p.tickets, 0);
            atomicExch(p.tickets + 1, 0);
            __threadfence();
        }
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
// GATED: two MMAs per step, the block's gate rows and its up rows.  The products of
// the backward take the weights as stored, with the rows of the result along
// memory: DACT (da and h from dh and a), and ADD for dx.
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
    __nv_bfloat16 *out;           // [T, N]
    __nv_bfloat16 *pair;          // [T, 2N]: GATED a (nullable), DACT da
    const __nv_bfloat16 *in;      // PLAIN and ADD what is added (nullable) [T, N], DACT a [T, 2N]
    int *status;
    uint64_t timeout_ns;
};
struct FewMaps {
    CUtensorMap w, x;
};

// EPI: GATED, PLAIN, DACT or ADD (PLAIN with the weights as dx reads them).
template <Epi EPI>
__global__ void __launch_bounds__(FEW_THREADS) ffn_few_kernel(const __grid_constant__ FewMaps maps, const FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[FEW_MAX_STAGES], empty[FEW_MAX_STAGES], done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    volatile int *abort = &s_abort;
    constexpr bool GATE = EPI == GATED, MN = EPI == DACT || EPI == ADD;  // MN: weights [K, N], else [N, K]
    constexpr int SLICES = GATE ? 1 : 2;  // of K in a stage
    constexpr int PARTS = GATE ? 2 : 1;   // sums per row and token: gate, up
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

    if (threadIdx.x == 0) {
        auto weights = [&](int i, int stage) {
            uint8_t *sa = smem + stage * stage_bytes;
            const int k = (kb0 + i) * SLICES * BK;
            mbar_arrive_expect_tx(&full[stage], stage_bytes);
            if (GATE) {
                tma_load_2d(sa, &maps.w, &full[stage], k, row0);
                tma_load_2d(sa + FEW_A / 2, &maps.w, &full[stage], k, p.N + row0);
            } else if (MN) {
                for (int i = 0; i < 4; ++i)
                    tma_load_2d(sa + i * BOX, &maps.w, &full[stage], row0 + (i & 1) * 64, k + (i >> 1) * BK);
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
        // the weights do not wait for the kernel before, where that is one of this operator's
        constexpr bool FIRST = EPI == GATED || EPI == DACT;
        if (FIRST)
            grid_dependency_wait_to_copy();
        else
            fence_proxy_async();  // what was stored before the kernel in front, which has waited for it
        const int first = min(kbs, p.stages);
        for (int i = 0; i < first; ++i) weights(i, i);
        if (!FIRST) grid_dependency_wait_to_copy();
        grid_dependency_launch();
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
        const uint32_t idesc = idesc_bf16_f32(FEW_ROWS, p.tokens, MN);
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; i < kbs; ++i) {
            if (!mbar_wait(&full[stage], phase, abort, p.status, p.timeout_ns)) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * stage_bytes), sb = sa + FEW_A;
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // GATE: gate and up rows; else the two slices
                const uint64_t adesc = MN ? smem_desc_mnmajor_sw128(sa + s * (FEW_A / 2), BOX)
                                          : smem_desc_kmajor_sw128(sa + s * (FEW_A / 2));
                const uint64_t bdesc = smem_desc_kmajor_sw128(sb + (GATE ? 0 : s * box));
#pragma unroll
                for (int j = 0; j < BK / UMMA_K; ++j)
                    umma_bf16(tmem + (GATE ? s * p.tokens : 0), adesc + (MN ? 128 : 2) * j, bdesc + 2 * j, idesc,
                              GATE ? (i | j) != 0 : (i | s | j) != 0);
            }
            umma_commit(&empty[stage]);
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        }
        umma_commit(&done);
    }
    __syncwarp();
    if (EPI == DACT && warp >= 2) {
        // what the results are made from besides the sums, into L2 meanwhile: the CTA's share of
        // the tokens, 128 bytes per lane
        grid_dependency_wait();
        const int share = p.tokens / p.split, first = t0 + rank * share, lane = threadIdx.x & 31;
        const int col = row0 + (lane & 1) * 64;
        for (int t = first + (warp - 2) * 8 + (lane >> 2); t < min(first + share, p.T); t += 16)
            if (col < p.N) l2_prefetch_line(p.in + 2 * static_cast<size_t>(t) * p.N + (lane & 2 ? p.N : 0) + col);
    }
    // every thread waits for the MMAs (after a wait that ran out: for those that were issued)
    volatile int no_abort = 0;
    mbar_wait(&done, 0, &no_abort, p.status, 2 * p.timeout_ns);
    __syncwarp();  // what follows is for whole warps at once
    tc_fence_after();
    const uint32_t tbase = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int row = row0 + static_cast<int>(threadIdx.x);  // the lane's weight row is the result's column
    // V tokens' sums (of GATED the gate's, u the up row's; of DACT dh) from token t on. What
    // is read for them is asked for before the first is used, and they are worked on side
    // by side: one by one, 128 tokens of DACT took 60 us.
    auto store = [&](int t, auto values, const float *a, const float *u) {
        constexpr int V = values.value;
        if (row >= p.N) return;
        const size_t N = p.N, at = static_cast<size_t>(t) * N + row;
        [[maybe_unused]] const size_t pair = at + static_cast<size_t>(t) * N;  // in [T, N], [T, 2N]
        const int n = min(V, p.T - t);
        if constexpr (GATE) {
            with_activation(p.act, [&](auto k) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 h = mul2(activate<k.value>(make_float2(a[i], a[i + 1])), make_float2(u[i], u[i + 1]));
                    if (i < n) p.out[at + N * i] = __float2bfloat16_rn(h.x);
                    if (i + 1 < n) p.out[at + N * i + N] = __float2bfloat16_rn(h.y);
                }
            });
            if (p.pair) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < n) {
                        p.pair[pair + 2 * N * i] = __float2bfloat16_rn(a[i]);
                        p.pair[pair + 2 * N * i + N] = __float2bfloat16_rn(u[i]);
                    }
            }
        } else if constexpr (EPI == DACT) {
            float g[V], up[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                g[i] = up[i] = 0.0f;
                if (i < n) {
                    g[i] = __bfloat162float(p.in[pair + 2 * N * i]);
                    up[i] = __bfloat162float(p.in[pair + 2 * N * i + N]);
                }
            }
            with_activation(p.act, [&](auto k) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 dh = make_float2(a[i], a[i + 1]), up2 = make_float2(up[i], up[i + 1]);
                    float2 slope;
                    const float2 act = activate<k.value>(make_float2(g[i], g[i + 1]), slope);
                    const float2 h = mul2(act, up2), dg = mul2(mul2(dh, up2), slope), du = mul2(dh, act);
                    if (i < n) {
                        p.out[at + N * i] = __float2bfloat16_rn(h.x);
                        p.pair[pair + 2 * N * i] = __float2bfloat16_rn(dg.x);
                        p.pair[pair + 2 * N * i + N] = __float2bfloat16_rn(du.x);
                    }
                    if (i + 1 < n) {
                        p.out[at + N * i + N] = __float2bfloat16_rn(h.y);
                        p.pair[pair + 2 * N * i + 2 * N] = __float2bfloat16_rn(dg.y);
                        p.pair[pair + 2 * N * i + 3 * N] = __float2bfloat16_rn(du.y);
                    }
                }
            });
        } else {
            float in[V];
#pragma unroll
            for (int i = 0; i < V; ++i) in[i] = p.in && i < n ? __bfloat162float(p.in[at + N * i]) : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) p.out[at + N * i] = __float2bfloat16_rn(p.in ? a[i] + in[i] : a[i]);
        }
    };
    if (p.split == 1) {
        grid_dependency_wait();  // before plain loads and stores of this thread
        for (int c = 0; c < p.tokens; c += 16) {
            if (t0 + c >= p.T) break;
            uint32_t v[PARTS][16];
            tmem_ld_32x32b_x16(tbase + c, v[0]);
            if (GATE) tmem_ld_32x32b_x16(tbase + p.tokens + c, v[PARTS - 1]);
            tmem_ld_wait();
            float sum[PARTS][16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[0][i] = __uint_as_float(v[0][i]), sum[PARTS - 1][i] = __uint_as_float(v[PARTS - 1][i]);
            store(t0 + c, std::integral_constant<int, 16>{}, sum[0], sum[PARTS - 1]);
        }
    } else {
        // The partial sums that this CTA gets, over its ring: of each CTA and part (gate,
        // up) a row of its share of the tokens, in groups of V that the lanes of
        // a warp write and read side by side.
        const int share = p.tokens / p.split;
        auto exchange = [&](auto vector) {
            using Vec = decltype(vector);
            constexpr int V = sizeof(Vec) / 4;
            const int groups = share / V;
            Vec *sums = reinterpret_cast<Vec *>(smem);
            cluster_sync();  // no CTA's ring is in use any more
            for (int c = 0; c < p.tokens; c += 16) {
                if (t0 + c >= p.T) break;
                uint32_t v[PARTS][16];
                tmem_ld_32x32b_x16(tbase + c, v[0]);
                if (GATE) tmem_ld_32x32b_x16(tbase + p.tokens + c, v[PARTS - 1]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += V) {
                    if (t0 + c + i >= p.T) break;
                    const int owner = (c + i) / share, group = ((c + i) % share) / V;
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        const uint32_t to =
                            mapa_shared(smem_u32(sums + ((rank * PARTS + k) * groups + group) * FEW_ROWS + threadIdx.x), owner);
                        if constexpr (V == 4)
                            asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[k][i]),
                                         "r"(v[k][i + 1]), "r"(v[k][i + 2]), "r"(v[k][i + 3])
                                         : "memory");
                        else
                            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(v[k][i]), "r"(v[k][i + 1])
                                         : "memory");
                    }
                }
            }
            __syncwarp();
            cluster_sync();  // every CTA's sums are there
            grid_dependency_wait();
            for (int g = 0; g < groups; ++g) {
                const int t = t0 + rank * share + g * V;
                if (t >= p.T) break;
                float v[PARTS][V] = {};
                for (int s = 0; s < p.split; ++s)
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        const Vec u = sums[((s * PARTS + k) * groups + g) * FEW_ROWS + threadIdx.x];
#pragma unroll
                        for (int i = 0; i < V; ++i) v[k][i] += reinterpret_cast<const float *>(&u)[i];
                    }
                store(t, std::integral_constant<int, V>{}, v[0], v[PARTS - 1]);
            }
        };
        if (share % 4 == 0)
            exchange(float4{});
        else
            exchange(float2{});
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
}

// ======================================================================
// Up to 64 tokens where that is faster: nothing but the weights' bytes counts, so they go straight
// to registers, each once.  A CTA has 16 weight rows (GATED: 8 gate rows and their 8 up
// rows), its warps every 8th 64 columns of them.  A quad of lanes reads 64 bytes of
// a row, 16 per lane, and multiplies them by mma.m16n8k16: which lane's elements stand for
// which k does not matter as long as the tokens' do for the same, so a lane's
// 8 consecutive elements of a weight row and of a token are two steps' operands as
// they are loaded.  A lane ends with the sums of a row (gate and up) for two
// tokens; the warps' are added in their order.
// ======================================================================
constexpr int TINY_WARPS = 8, TINY_SPLIT = 8;
// 64-column steps whose loads a warp has in flight, of 64 bytes of weights per lane each
__host__ __device__ constexpr int tiny_deep(int eights) { return eights == 1 ? 4 : eights <= 4 ? 2 : 1; }

// The first kernel's share of what the second one reads first, into L2: its CTAs ask
// for it as their own last loads come in, so that the memory is busy while one kernel
// ends and the next begins (us a call at one token without it, with 16 MB and with 32:
// 7168 x 2048 18.3, 17.5, 17.3; 4096 x 14336 54.4, 53.9, 53.3; 1024 x 4096 9.4, 8.9, 8.9).
constexpr int64_t AHEAD_BYTES = 32 << 20;
struct Ahead {
    const uint16_t *w;  // null: nothing
    int64_t bytes;      // a multiple of 16
    __device__ __forceinline__ void ask(int cta, int ctas) const {
        if (w == nullptr) return;
        const int64_t lines = bytes / 16, first = lines * cta / ctas, end = lines * (cta + 1) / ctas;
        for (int64_t at = first; at < end; at += 1024)
            l2_prefetch(reinterpret_cast<const uint8_t *>(w) + 16 * at, static_cast<uint32_t>(min(end - at, int64_t(1024))) * 16);
    }
};

struct TinyParams {
    const uint16_t *w, *x;  // [N or 2N, K], [T, K]
    int T, N, K;
    int act;
    __nv_bfloat16 *out, *preact;
    const __nv_bfloat16 *add;
    Ahead ahead;
    int split;  // CTAs of a cluster that share K
};

__device__ __forceinline__ uint4 load_once(const uint16_t *at, bool on) {
    uint4 v = make_uint4(0, 0, 0, 0);
    // volatile: these stay in front of the wait for the kernel before
    if (on)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(at));
    return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// EIGHTS: of tokens.
template <bool GATE, int EIGHTS>
__global__ void __launch_bounds__(32 * TINY_WARPS, 2) ffn_tiny_kernel(const TinyParams p) {
    constexpr int DEEP = tiny_deep(EIGHTS);
    __shared__ float4 sums[TINY_WARPS][EIGHTS][32], parts[TINY_SPLIT][EIGHTS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // the lane's two rows: of the gate and of the up weights, or 8 apart
    const int rank = static_cast<int>(blockIdx.x) % p.split, unit = static_cast<int>(blockIdx.x) / p.split;
    const int row = unit * (GATE ? 8 : 16) + g, row2 = GATE ? p.N + row : row + 8;
    const bool on = row < p.N, on2 = GATE ? on : row2 < p.N;
    const int64_t K = p.K;
    const uint16_t *w = p.w + row * K, *w2 = p.w + row2 * K, *x = p.x + g * K;
    if (GATE) {
        grid_dependency_wait();
        grid_dependency_launch();
    }
    if (p.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA runs
    float c[EIGHTS][4] = {};
    const int first_k = 64 * (rank * TINY_WARPS + warp), step = 64 * TINY_WARPS * p.split;
    for (int k0 = first_k; k0 < p.K; k0 += step * DEEP) {
        uint4 a[DEEP][2], b[DEEP][2];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + step * i + 32 * h + 8 * q;
                a[i][h] = load_once(w + k, on && k < p.K);
                b[i][h] = load_once(w2 + k, on2 && k < p.K);
            }
        if (!GATE && k0 == first_k) {  // W2's first loads did not wait for the kernel that writes h
            grid_dependency_wait();
            grid_dependency_launch();
        }
        uint4 t[DEEP][2][EIGHTS];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + step * i + 32 * h + 8 * q;
#pragma unroll
                for (int n = 0; n < EIGHTS; ++n) {
                    t[i][h][n] = make_uint4(0, 0, 0, 0);
                    if (8 * n + g < p.T && k < p.K) t[i][h][n] = *reinterpret_cast<const uint4 *>(x + 8 * n * K + k);
                }
            }
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 &u = a[i][h], &v = b[i][h];
#pragma unroll
                for (int n = 0; n < EIGHTS; ++n) {
                    mma_bf16(c[n], u.x, v.x, u.y, v.y, t[i][h][n].x, t[i][h][n].y);
                    mma_bf16(c[n], u.z, v.z, u.w, v.w, t[i][h][n].z, t[i][h][n].w);
                }
            }
    }
    if (GATE && threadIdx.x == 0) p.ahead.ask(blockIdx.x, gridDim.x);
#pragma unroll
    for (int n = 0; n < EIGHTS; ++n) sums[warp][n][lane] = make_float4(c[n][0], c[n][1], c[n][2], c[n][3]);
    __syncthreads();
    if (!GATE) grid_dependency_wait();  // (a warp without columns has not waited yet)
    // warp n: the n-th eight tokens
    auto add = [&](float4 &s, const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (warp < EIGHTS) {
        s = sums[0][warp][lane];
#pragma unroll
        for (int i = 1; i < TINY_WARPS; ++i) add(s, sums[i][warp][lane]);
    }
    if (p.split > 1) {  // the CTAs' sums, by the first one in their order
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (warp < EIGHTS) {
            const uint32_t to = mapa_shared(smem_u32(&parts[rank][warp][lane]), 0);
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(s.x), "f"(s.y), "f"(s.z), "f"(s.w)
                         : "memory");
        }
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
        if (warp < EIGHTS) {
            s = parts[0][warp][lane];
            for (int i = 1; i < p.split; ++i) add(s, parts[i][warp][lane]);
        }
    }
    if (warp >= EIGHTS) return;
    // s.x, s.y: of the first row for tokens 2q and 2q + 1; s.z, s.w: of the second
    const float first[2] = {s.x, s.y}, second[2] = {s.z, s.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t t = 8 * warp + 2 * q + i;
        if (t >= p.T) break;
        if constexpr (GATE) {
            if (!on) break;
            float act = 0.0f;
            with_activation(p.act, [&](auto k) { act = activate<k.value>(first[i]); });
            p.out[t * p.N + row] = __float2bfloat16_rn(act * second[i]);
            if (p.preact) {
                p.preact[2 * t * p.N + row] = __float2bfloat16_rn(first[i]);
                p.preact[(2 * t + 1) * p.N + row] = __float2bfloat16_rn(second[i]);
            }
        } else {
            const float add1 = p.add && on ? __bfloat162float(p.add[t * p.N + row]) : 0.0f;
            const float add2 = p.add && on2 ? __bfloat162float(p.add[t * p.N + row2]) : 0.0f;
            if (on) p.out[t * p.N + row] = __float2bfloat16_rn(first[i] + add1);
            if (on2) p.out[t * p.N + row2] = __float2bfloat16_rn(second[i] + add2);
        }
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
// A K-major B operand of tiles of half the width: 64 rows per CTA.
bool half_operand(CUtensorMap *m, const void *base, int64_t rows, int64_t cols) {
    return map2d(m, base, rows, cols, cols, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B);
}
// A matrix that the epilogue reads or writes in 32 x 32 boxes.
bool boxes(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld) {
    return map2d(m, base, rows, cols, ld, CHUNK, CHUNK, CU_TENSOR_MAP_SWIZZLE_64B);
}

// Every kernel here may start before the one in front of it in the stream has ended:
// it waits before it touches memory that another kernel writes or reads (W2 by
// its own kernel excepted, which starts only behind one that has waited).  Calls that
// follow one another so hide their launches (us a call, 7168 x 2048 at one token 20.0
// and 18.1; 2048 x 768 at 37 12.3 and 9.4; 1003 x 2056 x 1368 32.7 and 29.3).
cudaLaunchConfig_t pair_config(int grid, int threads, int smem, cudaStream_t stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr, cfg.numAttrs = 2;
    return cfg;
}

template <Epi EPI, bool A_MN, bool B_MN, typename Out, typename M = Maps>
cudaError_t set_up(int *pairs) {
    auto kernel = ffn_gemm_kernel<EPI, A_MN, B_MN, Out, M>;
    constexpr int smem = Layout<EPI, Out>::BYTES;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pair_config(2, threads_of(EPI), smem, nullptr, attr);
    int n = 0;
    const cudaError_t q = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (q != cudaSuccess) return q;
    *pairs = std::min(*pairs, n);
    return cudaSuccess;
}

// The tiles of a product that the list goes on with.
Product product(int M, int N, int K, bool gate, int first) {
    const int n = gate ? TILE_N / 2 : TILE_N;
    Product q{M, N, K, (M + TILE_M - 1) / TILE_M, (N + n - 1) / n, 0, first, 0};
    q.halves = q.tiles = q.MT * q.NT;
    return q;
}
// Those from the `whole`-th on in two halves each.
void cut(Product *q, int whole) {
    q->tiles = 2 * q->tiles - whole;
    q->halves = whole;
}

template <Epi EPI, bool A_MN, bool B_MN>
cudaError_t gemm(const Maps &maps, Params p, int M, int N, int K, const GemmLaunch &lc, cudaStream_t stream) {
    Product q = product(M, N, K, EPI == GATED, 0);
    // a last round that leaves half of the pairs without a tile takes tiles of half the width
    const int rest = q.tiles % lc.ffn_pairs;
    if (2 * rest <= lc.ffn_pairs) cut(&q, q.tiles - rest);
    p.product[0] = q, p.products = 1, p.tiles = q.tiles;
    cudaLaunchAttribute attr[2];
    const int grid = 2 * std::min(q.tiles, lc.ffn_pairs);
    cudaLaunchConfig_t cfg = pair_config(grid, threads_of(EPI), Layout<EPI, uint16_t>::BYTES, stream, attr);
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, A_MN, B_MN, uint16_t, Maps>, maps, p);
}

template <typename Out>
cudaError_t gradients(const GradMaps &maps, const Params &p, const GemmLaunch &lc, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    const int grid = 2 * std::min(p.tiles, lc.ffn_pairs);
    cudaLaunchConfig_t cfg = pair_config(grid, threads_of(GRADS), Layout<GRADS, Out>::BYTES, stream, attr);
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<GRADS, true, true, Out, GradMaps>, maps, p);
}

constexpr int FEW_SMEM = 224 * 1024;
// For da and h, beside the models below, in ns: what a token of a block takes longer in the
// kernel for few tokens (what it reads and stores besides the sums), and what a launch of
// pairs takes longer. By them the choice between the two is 0.1 us behind the better one
// on the mean and 2.4 at most, over 9 sizes at 16 to 1500 tokens.
constexpr double DACT_TOKEN_NS = 120, DACT_NS = 8000;

// How a product of few tokens is cut: the block of tokens and the split of K of
// the least time by a model of a CTA's steps, fitted to the times of 12 cuts of 14
// products (d, f from 512 to 14336) at 9 token counts each (the model's choice is
// 0.14 us behind the best of them on the mean, 2.6 at most).  In ns: 2700 until
// the first sums and after the last, the stages' bytes at 109 per SM and ns or
// 14000 together, 9 per token for the result, 55 where it is exchanged.
struct FewShape {
    int tokens, blocks, rows, split, stages, smem;
    double ns = 1e30;
    FewShape(int T, int N, int K, bool gate, const GemmLaunch &lc, double each = 0) {
        rows = (N + FEW_ROWS - 1) / FEW_ROWS;
        const int slices = gate ? 1 : 2, KB = (K + slices * BK - 1) / (slices * BK);
        for (int most = 16; most <= FEW_MAX_TOKENS; most *= 2) {
            const int nb = (T + most - 1) / most, nt = ((T + nb - 1) / nb + 15) / 16 * 16;
            const int stage = FEW_A + slices * nt * BK * 2;
            for (int i = 0, s = 1; i < 4 && s <= KB; ++i, s *= 2) {
                if (lc.few_clusters[i] < 1) break;
                const int per_sm = nt <= 16 ? 2 : 1;
                const double at_once = static_cast<double>(lc.few_clusters[i]) * per_sm;
                const double rounds = std::ceil(static_cast<double>(rows) * nb / at_once);
                const double bytes = static_cast<double>((KB + s - 1) / s) * stage;
                const double t = rounds * (2700 + bytes * std::max(1 / 109.0, at_once * s / 14000) +
                                           ((s == 1 ? 9.0 : 55.0) + each / s) * nt);
                if (t < ns) {
                    ns = t, tokens = nt, blocks = nb, split = s;
                    const int room = (FEW_SMEM / per_sm - 2048) / stage;
                    stages = std::min({room, FEW_MAX_STAGES, (KB + s - 1) / s});
                    // the ring also holds the partial sums
                    const int sums = s > 1 ? nt * FEW_ROWS * 4 * (gate ? 2 : 1) : 0;
                    smem = std::max(stages * stage, sums) + 1024;
                }
            }
            if (most >= T) break;
        }
    }
};

template <Epi EPI>
cudaError_t few(const uint16_t *w, const uint16_t *x, int T, int N, int K, FewParams p,
                const GemmLaunch &lc, cudaStream_t stream) {
    constexpr bool GATE = EPI == GATED, MN = EPI == DACT || EPI == ADD;
    const FewShape s(T, N, K, GATE, lc, EPI == DACT ? DACT_TOKEN_NS : 0);
    FewMaps maps;
    if (!(MN ? operand(&maps.w, w, K, N, true) : operand(&maps.w, w, GATE ? 2 * static_cast<int64_t>(N) : N, K, false)) ||
        !map2d(&maps.x, x, T, K, K, s.tokens, BK, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.T = T, p.N = N, p.K = K, p.tokens = s.tokens, p.stages = s.stages, p.split = s.split;
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
    cfg.attrs = attr, cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ffn_few_kernel<EPI>, maps, p);
}

// How a product of at most 64 tokens is cut without tiles.  K is shared by a cluster
// of CTAs where a CTA's bytes, at the 53 per ns of half an SM, would take longer than their
// share and the 1000 ns of adding up (us at one token: 1024 x 4096 11.4 behind by one
// CTA, 0 by four; 2048 x 768 5.4 by one, 6.4 by two).
struct TinyShape {
    int units, split = 1;
    TinyShape(int T, int N, int K, bool gate, int sms) {
        units = (N + (gate ? 7 : 15)) / (gate ? 8 : 16);
        const double ns = (32.0 + 2 * T) * K / 53;
        double best = ns;
        for (int s = 2; s <= TINY_SPLIT && units * s <= 2 * sms; s *= 2)
            if (ns / s + 1000 < best) best = ns / s + 1000, split = s;
    }
};
template <bool GATE>
cudaError_t tiny(TinyParams p, const GemmLaunch &lc, cudaStream_t stream) {
    const TinyShape s(p.T, p.N, p.K, GATE, lc.num_sms);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = s.split, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s.units * s.split), cfg.blockDim = dim3(32 * TINY_WARPS), cfg.stream = stream;
    cfg.attrs = attr, cfg.numAttrs = s.split > 1 ? 2 : 1;
    p.split = s.split;
    return p.T <= 8    ? cudaLaunchKernelEx(&cfg, ffn_tiny_kernel<GATE, 1>, p)
           : p.T <= 16 ? cudaLaunchKernelEx(&cfg, ffn_tiny_kernel<GATE, 2>, p)
           : p.T <= 32 ? cudaLaunchKernelEx(&cfg, ffn_tiny_kernel<GATE, 4>, p)
                       : cudaLaunchKernelEx(&cfg, ffn_tiny_kernel<GATE, 8>, p);
}

// Whether CTA pairs take longer than the kernel for few tokens, by their model beside
// FewShape's, in ns: 3200, and of each round 370 and 346 per slice of K (274 where
// the tiles are halved).  Fitted to 8 sizes at 37 to 1003 tokens, where it is 0.1 us
// behind the better choice on the mean (8 at most: 384 tokens, d = 4096, f = 14336).
bool prefer_few(int T, int N, int K, bool gate, double few_ns, int pairs) {
    const int n = gate ? TILE_N / 2 : TILE_N;
    const int64_t tiles = static_cast<int64_t>((T + TILE_M - 1) / TILE_M) * ((N + n - 1) / n);
    const int64_t rest = tiles % pairs;
    const double KB = (K + BK - 1) / BK, rounds = static_cast<double>(tiles / pairs);
    const double last = rest == 0 ? 0 : 2 * rest <= pairs ? 185 + 274 * KB : 370 + 346 * KB;
    return few_ns + 600 < 3200 + rounds * (370 + 346 * KB) + last;
}
// A bf16 matrix that a kernel takes as one.
__nv_bfloat16 *bf16(const uint16_t *t) { return reinterpret_cast<__nv_bfloat16 *>(const_cast<uint16_t *>(t)); }

struct Ways {
    bool tiny = false, few_up = false, few_down = false;
    Ways(int T, int d, int f, const GemmLaunch &lc) {
        if (T <= 16) {
            tiny = true;
            return;
        }
        // a product of so many tokens keeps the pairs busy whatever its other sizes
        if (T > 4096) return;
        const FewShape up(T, f, d, true, lc), down(T, d, f, false, lc);
        // Without tiles every row block reads all tokens again: the bytes of both products from L2
        // (6 df of weights, 3/8 df per token) at 12900 per ns, 11400 with over 32 tokens, and
        // 7900 ns, against the other's.  us with and without tiles: 2048 x 768, 37 tokens 13.7 and 9.7;
        // 7168 x 2048, 24 tokens 30.6 and 27.6, 48 tokens 30.6 and 38.9; 4096 x 14336, 17 tokens 65 and 86.
        // (One way for both products: behind one with tiles, one without took up to 50 us longer.)
        const double bytes = static_cast<double>(d) * f * (6 + 0.375 * T);
        if (T <= 64 && 7900 + bytes / (T <= 32 ? 12900 : 11400) < up.ns + down.ns + 1950) {
            tiny = true;
            return;
        }
        few_up = prefer_few(T, f, d, true, up.ns, lc.ffn_pairs);
        few_down = prefer_few(T, d, f, false, down.ns, lc.ffn_pairs);
    }
};

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
        (e = set_up<GRADS, true, true, uint16_t, GradMaps>(&pairs)) != cudaSuccess ||
        (e = set_up<GRADS, true, true, float, GradMaps>(&pairs)) != cudaSuccess)
        return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cfg->ffn_pairs = pairs;
    for (const void *k :
         {reinterpret_cast<const void *>(ffn_few_kernel<GATED>), reinterpret_cast<const void *>(ffn_few_kernel<PLAIN>),
          reinterpret_cast<const void *>(ffn_few_kernel<DACT>), reinterpret_cast<const void *>(ffn_few_kernel<ADD>)})
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess)
            return e;
    // clusters of 1, 2, 4 and 8 CTAs that are resident at once, one CTA per SM
    for (int i = 0; i < 4; ++i) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1 << i, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3(1 << i), c.blockDim = dim3(FEW_THREADS), c.dynamicSmemBytes = FEW_SMEM;
        c.attrs = &attr, c.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&cfg->few_clusters[i], ffn_few_kernel<GATED>, &c)) != cudaSuccess) return e;
    }
    return cfg->few_clusters[0] < 1 ? cudaErrorInvalidConfiguration : cudaSuccess;
}

cudaError_t launch_ffn(const FfnArgs &a, const GemmLaunch &lc, cudaStream_t stream) {
    using namespace ff;
    const Ways way(a.T, a.d, a.f, lc);
    const int64_t f = a.f;
    FewParams fp = {};
    fp.act = a.act, fp.status = a.status, fp.timeout_ns = a.timeout_ns;
    Params p = {};
    p.act = a.act, p.status = a.status, p.timeout_ns = a.timeout_ns;
    cudaError_t e;
    if (way.tiny) {
        const int64_t bytes = std::min<int64_t>(static_cast<int64_t>(a.d) * a.f * 2, AHEAD_BYTES);
        e = tiny<true>({a.W1, a.x, a.T, a.f, a.d, a.act, bf16(a.h), bf16(a.preact), nullptr, {a.W2, bytes}}, lc, stream);
    } else if (way.few_up) {
        fp.out = bf16(a.h), fp.pair = bf16(a.preact);
        e = few<GATED>(a.W1, a.x, a.T, a.f, a.d, fp, lc, stream);
    } else {
        Maps m = {};
        p.keep = a.preact != nullptr;
        if (!operand(&m.a, a.x, a.T, a.d, false) || !operand(&m.b, a.W1, 2 * f, a.d, false) ||
            !half_operand(&m.half_b, a.W1, 2 * f, a.d) || !boxes(&m.out, a.h, a.T, f, f) ||
            (a.preact && (!boxes(&m.more[0], a.preact, a.T, f, 2 * f) || !boxes(&m.more[1], a.preact + f, a.T, f, 2 * f))))
            return cudaErrorInvalidValue;
        e = gemm<GATED, false, false>(m, p, a.T, a.f, a.d, lc, stream);
    }
    if (e != cudaSuccess) return e;
    if (way.tiny)
        return tiny<false>({a.W2, a.h, a.T, a.d, a.f, a.act, bf16(a.y), nullptr, bf16(a.add), {}}, lc, stream);
    if (way.few_down) {
        fp.out = bf16(a.y), fp.pair = nullptr, fp.in = bf16(a.add);
        return few<PLAIN>(a.W2, a.h, a.T, a.d, a.f, fp, lc, stream);
    }
    Maps m = {};
    if (!operand(&m.a, a.h, a.T, f, false) || !operand(&m.b, a.W2, a.d, f, false) || !half_operand(&m.half_b, a.W2, a.d, f) ||
        !boxes(&m.out, a.y, a.T, a.d, a.d) || (a.add && !boxes(&m.in, a.add, a.T, a.d, a.d)))
        return cudaErrorInvalidValue;
    return a.add ? gemm<ADD, false, false>(m, p, a.T, a.d, a.f, lc, stream)
                 : gemm<PLAIN, false, false>(m, p, a.T, a.d, a.f, lc, stream);
}

cudaError_t launch_ffn_bwd(const FfnGradArgs &a, const GemmLaunch &lc, int *launches, cudaStream_t stream) {
    using namespace ff;
    const int64_t f = a.f;
    Params p = {};
    p.act = a.act, p.status = a.status, p.timeout_ns = a.timeout_ns;
    *launches = 0;
    const bool small = a.T <= 4096;  // (as in Ways)
    // da and h, from dh = dy W2 (W2 read as stored)
    if (small && prefer_few(a.T, a.f, a.d, false, FewShape(a.T, a.f, a.d, false, lc, DACT_TOKEN_NS).ns - DACT_NS, lc.ffn_pairs)) {
        FewParams fp = {};
        fp.act = a.act, fp.status = a.status, fp.timeout_ns = a.timeout_ns;
        fp.out = bf16(a.h), fp.pair = bf16(a.da), fp.in = bf16(a.preact);
        const cudaError_t e = few<DACT>(a.W2, a.dy, a.T, a.f, a.d, fp, lc, stream);
        if (e != cudaSuccess) return e;
    } else {
        Maps m = {};
        if (!operand(&m.a, a.dy, a.T, a.d, false) || !operand(&m.b, a.W2, a.d, f, true) ||
            !boxes(&m.in, a.preact, a.T, f, 2 * f) || !boxes(&m.in2, a.preact + f, a.T, f, 2 * f) ||
            !boxes(&m.more[0], a.da, a.T, f, 2 * f) || !boxes(&m.more[1], a.da + f, a.T, f, 2 * f) ||
            !boxes(&m.out, a.h, a.T, f, f))
            return cudaErrorInvalidValue;
        const cudaError_t e = gemm<DACT, false, true>(m, p, a.T, a.f, a.d, lc, stream);
        if (e != cudaSuccess) return e;
    }
    ++*launches;
    // The three products of these: one list of tiles, the longest ones first, handed
    // out as pairs fall free, so that one tail is left instead of three.
    GradMaps m = {};
    struct {
        int kind, M, N, K;
        const uint16_t *left, *right;
        void *out;
    } list[PRODUCTS];
    int n = 0;
    auto weights = [&] {
        if (a.dW1) list[n++] = {KIND_WEIGHTS, 2 * a.f, a.d, a.T, a.da, a.x, a.dW1};
        if (a.dW2) list[n++] = {KIND_WEIGHTS, a.d, a.f, a.T, a.dy, a.h, a.dW2};
    };
    // Slices of a product's tile, and of all tiles of the list.
    const auto slices = [](const Product &q) { return static_cast<int64_t>((q.K + BK - 1) / BK); };
    int64_t work = 0;
    double work_ns = 0;
    const auto count = [&](int M, int N, int K) {
        const Product q = product(M, N, K, false, 0);
        work += q.tiles * slices(q);
        work_ns += q.tiles * std::max(346.0 * slices(q), 1000.0);
    };
    if (a.dW1) count(2 * a.f, a.d, a.T);
    if (a.dW2) count(a.d, a.f, a.T);
    // dx has the longest tiles, and few of them where tokens and d are few: then it is better
    // made by the kernel that shares K, behind the others. By a model of both: 346 ns per slice
    // of a tile and 1000 at least, 274 per slice for the one that ends last, and 500 for
    // the launch. us in the list and apart: 200 tokens of d = 256, f = 8192 91 and 34,
    // d = 1024, f = 4096 58 and 41; d = 4096, f = 1536 51 and 59.
    bool few_dx = false;
    if (a.dx) {
        const double others = work_ns / lc.ffn_pairs;
        count(a.T, a.d, 2 * a.f);
        const double KB = (2 * a.f + BK - 1) / BK, listed = std::max(work_ns / lc.ffn_pairs, 274 * KB);
        few_dx = small && others + FewShape(a.T, a.d, 2 * a.f, false, lc).ns + 500 < listed;
        if (few_dx) work -= product(a.T, a.d, 2 * a.f, false, 0).tiles * static_cast<int64_t>(KB);
    }
    if (a.T > 2 * a.f) weights();
    if (a.dx && !few_dx) list[n++] = {KIND_DX, a.T, a.d, 2 * a.f, a.da, a.W1, a.dx};
    if (a.T <= 2 * a.f) weights();
    p.add = a.add != nullptr, p.products = n;
    for (int i = 0; i < n; ++i) {
        const auto &l = list[i];
        const bool dx = l.kind == KIND_DX;
        Product q = product(l.M, l.N, l.K, false, p.tiles);
        // tiles that take longer than a pair's share of all work are halved
        if (slices(q) * lc.ffn_pairs > work) cut(&q, 0);
        p.product[i] = q, p.kind[i] = l.kind, p.tiles += q.tiles;
        // the weights' gradients sum over the tokens, the rows of both operands; dx over W1's rows
        const int64_t K = l.K;
        if (!(dx ? operand(&m.a[i], l.left, l.M, K, false) : operand(&m.a[i], l.left, K, l.M, true)) ||
            !operand(&m.b[i], l.right, K, l.N, true))
            return cudaErrorInvalidValue;
        if (!dx && a.weights_f32 ? !make_tmap_2d(&m.out[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, l.out, l.M, l.N, CHUNK,
                                                 CHUNK, CU_TENSOR_MAP_SWIZZLE_128B)
                                 : !boxes(&m.out[i], l.out, l.M, l.N, l.N))
            return cudaErrorInvalidValue;
    }
    if (a.add && !boxes(&m.in, a.add, a.T, a.d, a.d)) return cudaErrorInvalidValue;
    if (n > 0) {
        p.tickets = p.tiles > lc.ffn_pairs ? gemm_tickets(lc, stream) : nullptr;
        const cudaError_t e = a.weights_f32 ? gradients<float>(m, p, lc, stream) : gradients<uint16_t>(m, p, lc, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (!few_dx) return cudaSuccess;
    ++*launches;
    FewParams fp = {};
    fp.status = a.status, fp.timeout_ns = a.timeout_ns;
    fp.out = bf16(a.dx), fp.in = bf16(a.add);
    return few<ADD>(a.W1, a.da, a.T, a.d, 2 * a.f, fp, lc, stream);
}

}  // namespace moe

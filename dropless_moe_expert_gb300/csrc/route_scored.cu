// Routing by scores of all experts, and the gradient of the logits.
//
// For each token, with l its fp32 logits and b a selection bias (fp32 [E] or
// none, e.g. one that balances the load; it enters the choice only):
//   s = sigmoid(l), or softmax(l) over the E experts;      c = s + b
//   the experts form n_group runs of E / n_group; a run's score is the sum of
//   its group_top largest c, and only the topk_group best runs stay open;
//   the K largest c of the open runs are chosen, descending;
//   w_k = scale * s_k / (sum_j s_j + 1e-20), or scale * s_k without renorm.
// Every tie, between experts or runs, goes to the lower index.  What is
// ranked is defined in 32 bits to the last bit, so that the choice does not
// depend on how the work is split: sigmoid is 1 / (1 + exp(-l)), and the
// softmax's sum adds element i + h to element i for h = 128, 64, .., 1 (E
// padded to 256 with zeros), which is what the registers of a warp and then
// its lanes do below.
//
// The gradient of sum(dw * w) to l, nothing through the choice or b:
//   ds_k = (scale dw_k - sum_j dw_j w_j) / (sum_j s_j + 1e-20), or scale dw_k;
//   sigmoid: dl_k = ds_k s_k (1 - s_k) for the chosen, 0 for the others;
//   softmax: dl_e = s_e (ds_e - sum_j s_j ds_j) for every expert.
//
// Latency and the instructions of a token bound it, not memory.  Measured on
// the device, all launches of a call: 1 token of 256 experts in 8 runs 5.1 us,
// 4096 of them 11.8, 32768 of 64 experts 14.2 (its bytes: 1.7); the gradient of
// 16381 x 128 softmax scores 5.9 us (its bytes: 2.6).
#include "kernels.h"
#include "ptx.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace rs {

constexpr int MAX_E = 256;
constexpr int CH = 16;             // tokens of a chunk, which a CTA of the top-K kernel takes
constexpr int OPEN = MAX_E / 16;   // words of a token's open runs
constexpr int SPANS = 152;         // CTAs of the dispatch kernel, each a run of chunks
// Of counts that every dispatch CTA adds up itself, not another launch before
// it (32768 x 64, 128 KB: 14.1 us, 18.7 with the launch; 131072 x 64, 512 KB:
// 46.2 and 42.6).
constexpr size_t SELF_SUM_BYTES = 256 * 1024;
constexpr unsigned FULL = 0xffffffffu;

// Of a dispatch CTA: 512 while it adds the counts up itself (4096 x 256: 11.8 us,
// 12.3 with 1024), 1024 where its span is long (131072 x 64: 42.6 us, 44.3 with 512).
__host__ __device__ constexpr int dispatch_threads(bool spanned) { return spanned ? 1024 : 512; }

// Bytes of a chunk's row of counts (one byte per expert, whole 16-byte words).
__host__ __device__ constexpr int count_pitch(int E) { return (E + 15) / 16 * 16; }
int num_chunks(int T) { return (T + CH - 1) / CH; }
int span_chunks(int chunks) { return (chunks + SPANS - 1) / SPANS; }

// Keys that order as the values do, -0.0 as +0.0; 0 is kept for "not there".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0.0 becomes +0.0
    return max(u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u), 1u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Over the LANES lanes (32, or a half of the warp) that hold a token.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES == 32) {
        return __reduce_max_sync(FULL, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(FULL, v, o));
        return v;
    }
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
    if constexpr (LANES == 32) {
        return __reduce_min_sync(FULL, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(FULL, v, o));
        return v;
    }
}

// Scores of one token: lane holds experts lane + LANES j in v (logits in, scores out).
template <int LANES, int EPL>
__device__ __forceinline__ void scores(float *v, int E, int lane, bool softmax) {
    if (!softmax) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = sigmoid(v[j]);
        return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (lane + LANES * j < E) top = max(top, order_key(v[j]));
    const float m = key_value(lanes_max<LANES>(top));
    float t[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) t[j] = v[j] = lane + LANES * j < E ? expf(v[j] - m) : 0.0f;
#pragma unroll
    for (int h = EPL / 2; h; h >>= 1) {
#pragma unroll
        for (int j = 0; j < h; ++j) t[j] += t[j + h];
    }
    const float sum = lanes_sum<LANES>(t[0]);
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = v[j] / sum;
}

// The runs that stay open, as a bit mask per LANES runs: `open`, filled by the
// token's lanes, and the first mask returned to all of them.  `keys`: the experts' keys in shared memory; `score`: room for a key
// per run.  Lanes share a run's experts; each keeps its two largest.
template <int LANES>
__device__ __forceinline__ uint32_t open_runs(const uint32_t *keys, uint32_t *score, uint32_t *open, int per,
                                          const RouteRule &rule, int lane) {
    const int G = rule.n_group;
    int share = 1;  // lanes per run: the largest power of two that leaves every run its own
    while (2 * share * G <= LANES && share < per) share *= 2;
    const int at_once = LANES / share;
    for (int g0 = 0; g0 < G; g0 += at_once) {
        const int g = g0 + lane / share;
        uint32_t a = 0, b = 0;
        if (g < G) {
#pragma unroll 4
            for (int i = lane % share; i < per; i += share) {
                const uint32_t k = keys[g * per + i];
                b = max(b, min(a, k));
                a = max(a, k);
            }
        }
        for (int o = share / 2; o; o >>= 1) {
            const uint32_t c = __shfl_xor_sync(FULL, a, o), d = __shfl_xor_sync(FULL, b, o);
            b = max(max(b, d), min(a, c));
            a = max(a, c);
        }
        if (g < G && lane % share == 0)
            score[g] = rule.group_top == 2 && b ? order_key(key_value(a) + key_value(b)) : a;
    }
    __syncwarp();
    uint32_t first = 0;
    for (int g0 = 0; g0 < G; g0 += LANES) {
        const int g = g0 + lane;
        const uint32_t mine = g < G ? score[g] : 0u;
        int above = 0;  // runs that come before this one
#pragma unroll 4
        for (int o = 0; o < G; ++o) above += score[o] > mine || (score[o] == mine && o < g);
        uint32_t bits = __ballot_sync(FULL, g < G && above < rule.topk_group);
        if (LANES < 32) bits = bits >> (threadIdx.x & 16) & 0xffffu;
        if (g0 == 0) first = bits;
        if (lane == 0) open[g0 / LANES] = bits;
    }
    __syncwarp();
    return first;
}

// LANES lanes per token, a chunk per CTA.  FINAL: the chunk holds every token
// and the CTA writes the dispatch order too; else it writes its chunk's counts
// and each pair's rank inside the chunk (in row_of) for the dispatch kernel.
// The instructions of a token bound it: half a warp per token up to 64 experts
// (32768 tokens, 64 experts, all routed by this kernel: 19.5 us for the whole
// routing, 20.9 with a warp; 128 experts the other way round, 17.7 and 18.8 for 16384).
template <int LANES, int EPL, bool FINAL>
__global__ void __launch_bounds__(CH *LANES, !FINAL && LANES == 32 ? 3 : 1)
route_scored_topk_kernel(const float *__restrict__ L, const float *__restrict__ bias, int T, int E, int K,
                         RouteRule rule, int32_t *__restrict__ topk_idx, float *__restrict__ topk_w,
                         int32_t *__restrict__ row_of, uint8_t *__restrict__ chunk_counts,
                         int32_t *__restrict__ counts, int32_t *__restrict__ offsets, int32_t *__restrict__ src_tok) {
    constexpr int THREADS = CH * LANES;
    __shared__ uint32_t chose[MAX_E];  // bit i: token i of the CTA chose the expert
    __shared__ int32_t s_off[MAX_E];
    extern __shared__ uint32_t s_groups[];  // with groups: keys [CH][E], scores [CH][n_group], open [CH][OPEN]
    const int tok = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int t = blockIdx.x * CH + tok;
    for (int e = threadIdx.x; e < E; e += THREADS) chose[e] = 0u;
    int my_e = 0;
    float w = 0.0f;  // lane k: the k-th choice and its weight
    if (t - (LANES < 32 ? tok & 1 : 0) < T) {  // the whole warp; a second token beyond the last is routed as the last
        const float *row = L + static_cast<size_t>(min(t, T - 1)) * E;
        float s[EPL];
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = lane + LANES * j < E ? row[lane + LANES * j] : 0.0f;
        scores<LANES, EPL>(s, E, lane, rule.softmax);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + LANES * j;
            key[j] = e < E ? order_key(bias ? s[j] + bias[e] : s[j]) : 0u;
        }
        if (rule.topk_group < rule.n_group) {
            uint32_t *keys = s_groups + tok * E;
            uint32_t *score = s_groups + CH * E + tok * rule.n_group;
            uint32_t *open = s_groups + CH * (E + rule.n_group) + tok * OPEN;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + LANES * j < E) keys[lane + LANES * j] = key[j];
            __syncwarp();
            const uint32_t first = open_runs<LANES>(keys, score, open, E / rule.n_group, rule, lane);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int g = ((lane + LANES * j) * rule.run_of) >> 20;
                const uint32_t bits = rule.n_group <= LANES ? first : lane + LANES * j < E ? open[g / LANES] : 0u;
                if (!((bits >> (g % LANES)) & 1u)) key[j] = 0u;
            }
        }
        // this lane's largest key, the lowest expert on ties, kept as the largest of two halves
        constexpr int HALF = (EPL + 1) / 2;
        uint32_t lo, hi = 0u;
        int lo_j, hi_j = HALF;
        auto find_lo = [&]() {
            lo = key[0], lo_j = 0;
#pragma unroll
            for (int j = 1; j < HALF; ++j)
                if (key[j] > lo) lo = key[j], lo_j = j;
        };
        auto find_hi = [&]() {
            if constexpr (EPL > 1) {
                hi = key[HALF], hi_j = HALF;
#pragma unroll
                for (int j = HALF + 1; j < EPL; ++j)
                    if (key[j] > hi) hi = key[j], hi_j = j;
            }
        };
        find_lo();
        find_hi();
        for (int k = 0; k < K; ++k) {
            const uint32_t best = max(lo, hi);
            const int mine = lane + LANES * (lo >= hi ? lo_j : hi_j);
            const uint32_t top = lanes_max<LANES>(best);
            const int e = static_cast<int>(lanes_min<LANES>(best == top ? static_cast<uint32_t>(mine) : FULL));
            if (lane == k) my_e = e;
            if (e == mine) {  // taken: the half that held it is searched again
                const int taken = e / LANES;
                if (taken < HALF) {
#pragma unroll
                    for (int j = 0; j < HALF; ++j) key[j] = j == taken ? 0u : key[j];
                    find_lo();
                } else {
#pragma unroll
                    for (int j = HALF; j < EPL; ++j) key[j] = j == taken ? 0u : key[j];
                    find_hi();
                }
            }
            if (LANES < 32) __syncwarp();  // the halves of a warp take different experts
        }
        float my_s = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float v = __shfl_sync(FULL, s[j], my_e % LANES, LANES);
            my_s = my_e / LANES == j ? v : my_s;
        }
        // the share first: that of a single choice is 1 to the last bit
        w = rule.scale * (rule.renorm ? my_s / (lanes_sum<LANES>(lane < K ? my_s : 0.0f) + kRouteEps) : my_s);
    }
    const bool write = t < T && lane < K;
    __syncthreads();  // `chose` is zero
    if (write) {
        const size_t p = static_cast<size_t>(t) * K + lane;
        topk_idx[p] = my_e;
        topk_w[p] = w;
        atomicOr(&chose[my_e], 1u << tok);  // the final mask does not depend on the order
    }
    __syncthreads();
    if constexpr (FINAL) {
        if (threadIdx.x < 32) {
            int carry = 0;
            for (int base = 0; base < E; base += 32) {
                const int e = base + static_cast<int>(threadIdx.x);
                const int c = e < E ? __popc(chose[e]) : 0;
                int incl = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(FULL, incl, o);
                    if (static_cast<int>(threadIdx.x) >= o) incl += v;
                }
                if (e < E) {
                    s_off[e] = offsets[e] = carry + incl - c;
                    counts[e] = c;
                }
                carry += __shfl_sync(FULL, incl, 31);
            }
            if (threadIdx.x == 0) offsets[E] = carry;
        }
        __syncthreads();
    } else {
        uint8_t *mine = chunk_counts + static_cast<size_t>(blockIdx.x) * count_pitch(E);
        for (int e = threadIdx.x; e < count_pitch(E); e += THREADS)
            mine[e] = static_cast<uint8_t>(e < E ? __popc(chose[e]) : 0);
    }
    if (write) {
        int r = __popc(chose[my_e] & ((1u << tok) - 1u));
        if constexpr (FINAL) {
            r += s_off[my_e];
            src_tok[r] = t;
        }
        row_of[static_cast<size_t>(t) * K + lane] = r;
    }
}

// The same for many tokens: 4 or 8 lanes per token, so that what is done
// per token and choice is shared by the 4 or 8 tokens of a warp (instructions of a
// token: 64 experts, softmax 164, half a warp 336; 256 in 8 runs 570 and 1250).
// Lane l holds the octets (8 neighbouring experts) l, l + LANES, ..; their keys
// also lie in shared memory, where the octet of a choice is read again for its next
// largest.  The same sums in the same order, so the same bits as above.  Us, all
// launches: 32768 tokens, 64 experts softmax 14.2, half a warp per token 19.2; 256
// in 8 runs 41.6 and 56.0; with 8192 tokens 15.0 and 19.0; but, fewer warps taking
// longer each, with 4096 tokens (no runs) 10.7 and 9.8, and for 8192 x 32 8.2 and 6.7;
// 6144 x 256 13.0 and 15.3, without runs 12.0 and 12.2, 6144 x 128 10.0 and 9.7.
// E and a run's experts are multiples of four, with at most RUNS runs.
constexpr int many(int E) { return E > 128 ? 5120 : 8192; }
constexpr int RUNS = 16;
constexpr int OCTET_THREADS = 128;
template <int LANES, int OCTETS>
__global__ void __launch_bounds__(OCTET_THREADS, 5)
route_scored_topk_octets_kernel(const float *__restrict__ L, const float *__restrict__ bias, int T, int E, int K,
                                RouteRule rule, int32_t *__restrict__ topk_idx, float *__restrict__ topk_w,
                                int32_t *__restrict__ row_of, uint8_t *__restrict__ chunk_counts) {
    constexpr int TOKENS = OCTET_THREADS / LANES, CHUNKS = TOKENS / CH, MOST = 8 * LANES * OCTETS;
    constexpr int PITCH = MOST + 8;
    static_assert(TOKENS % CH == 0, "whole chunks");
    __shared__ __align__(16) uint32_t s_keys[TOKENS * PITCH];
    __shared__ __align__(16) float s_chosen[TOKENS][16];  // the choices' scores
    __shared__ uint32_t s_runs[TOKENS][RUNS];             // the runs' scores
    __shared__ uint8_t s_e[TOKENS][16];                   // the choices
    __shared__ uint32_t chose[CHUNKS][MOST];              // bit i: token i of the chunk chose the expert
    const int tok = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int t = blockIdx.x * TOKENS + tok;
    const float *row = L + static_cast<size_t>(min(t, T - 1)) * E;  // a token beyond the last is routed as the last
    uint32_t *const keys = s_keys + tok * PITCH;
    for (int i = threadIdx.x; i < CHUNKS * MOST; i += OCTET_THREADS) (&chose[0][0])[i] = 0u;

    float v[OCTETS][8];
    auto load = [&](const float *from, float absent) {
#pragma unroll
        for (int j = 0; j < OCTETS; ++j)
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
                const int e = 8 * (l + LANES * j) + h;
                const float4 x = e < E ? *reinterpret_cast<const float4 *>(from + e)
                                       : make_float4(absent, absent, absent, absent);
                v[j][h] = x.x, v[j][h + 1] = x.y, v[j][h + 2] = x.z, v[j][h + 3] = x.w;
            }
    };
    load(row, -INFINITY);
    float m = -INFINITY, sum = 1.0f;
    if (rule.softmax) {
#pragma unroll
        for (int j = 0; j < OCTETS; ++j)
#pragma unroll
            for (int q = 0; q < 8; ++q) m = fmaxf(m, v[j][q]);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        float f[OCTETS][8];
#pragma unroll
        for (int j = 0; j < OCTETS; ++j)
#pragma unroll
            for (int q = 0; q < 8; ++q) f[j][q] = v[j][q] = expf(v[j][q] - m);
        // element i + h to element i: over a lane's octets, the lanes, an octet's experts
#pragma unroll
        for (int h = OCTETS / 2; h; h >>= 1)
#pragma unroll
            for (int j = 0; j < h; ++j)
#pragma unroll
                for (int q = 0; q < 8; ++q) f[j][q] += f[j + h][q];
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1)
#pragma unroll
            for (int q = 0; q < 8; ++q) f[0][q] += __shfl_xor_sync(FULL, f[0][q], o);
#pragma unroll
        for (int h = 4; h; h >>= 1)
#pragma unroll
            for (int q = 0; q < h; ++q) f[0][q] += f[0][q + h];
        sum = f[0][0];
    }
    auto score = [&](float x) { return rule.softmax ? x / sum : sigmoid(x); };  // of a logit, or its exponential
    uint32_t key[OCTETS][8];
#pragma unroll
    for (int j = 0; j < OCTETS; ++j)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[j][q] = score(v[j][q]);
#pragma unroll
    for (int j = 0; j < OCTETS; ++j)
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            const int e = 8 * (l + LANES * j) + h;
            float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (bias && e < E) b = *reinterpret_cast<const float4 *>(bias + e);
            const float add[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                key[j][h + q] = e < E ? order_key(bias ? v[j][h + q] + add[q] : v[j][h + q]) : 0u;
            *reinterpret_cast<uint4 *>(keys + e) =
                make_uint4(key[j][h], key[j][h + 1], key[j][h + 2], key[j][h + 3]);
        }
    __syncwarp();
    if (rule.topk_group < rule.n_group) {
        const int G = rule.n_group, per = E / G;
        for (int g = l; g < G; g += LANES) {
            uint32_t a = 0, b = 0;  // its two largest
            for (int i = 0, at = 4 * l % per; i < per; i += 4, at = at + 4 == per ? 0 : at + 4) {  // lanes off each other's banks
                const uint4 k = *reinterpret_cast<const uint4 *>(keys + g * per + at);
                b = max(b, min(a, k.x)), a = max(a, k.x);
                b = max(b, min(a, k.y)), a = max(a, k.y);
                b = max(b, min(a, k.z)), a = max(a, k.z);
                b = max(b, min(a, k.w)), a = max(a, k.w);
            }
            s_runs[tok][g] = rule.group_top == 2 && b ? order_key(key_value(a) + key_value(b)) : a;
        }
        __syncwarp();
        uint32_t open = 0;
        for (int g = l; g < G; g += LANES) {
            const uint32_t mine = s_runs[tok][g];
            int above = 0;  // runs that come before this one
            for (int o = 0; o < G; ++o) above += s_runs[tok][o] > mine || (s_runs[tok][o] == mine && o < g);
            open |= static_cast<uint32_t>(above < rule.topk_group) << g;
        }
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) open |= __shfl_xor_sync(FULL, open, o);
#pragma unroll
        for (int j = 0; j < OCTETS; ++j)
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
                const int e = 8 * (l + LANES * j) + h;
                if (open >> (e * rule.run_of >> 20) & 1u) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) key[j][h + q] = 0u;
                *reinterpret_cast<uint4 *>(keys + e) = make_uint4(0u, 0u, 0u, 0u);
            }
    }
    uint32_t best[OCTETS];
#pragma unroll
    for (int j = 0; j < OCTETS; ++j) {
        best[j] = key[j][0];
#pragma unroll
        for (int q = 1; q < 8; ++q) best[j] = max(best[j], key[j][q]);
    }
    for (int k = 0; k < K; ++k) {
        uint32_t top = best[0];
#pragma unroll
        for (int j = 1; j < OCTETS; ++j) top = max(top, best[j]);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
        int octet = MOST;  // the lowest that holds it
#pragma unroll
        for (int j = OCTETS - 1; j >= 0; --j) octet = best[j] == top ? l + LANES * j : octet;
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) octet = min(octet, __shfl_xor_sync(FULL, octet, o));
        if (octet % LANES == l) {  // taken: the octet is searched again
            const uint4 a = *reinterpret_cast<const uint4 *>(keys + 8 * octet);
            const uint4 b = *reinterpret_cast<const uint4 *>(keys + 8 * octet + 4);
            const uint32_t held[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            int q = 7;
#pragma unroll
            for (int i = 6; i >= 0; --i) q = held[i] == top ? i : q;
            uint32_t next = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) next = max(next, i == q ? 0u : held[i]);
            keys[8 * octet + q] = 0u;
            s_e[tok][k] = static_cast<uint8_t>(8 * octet + q);
#pragma unroll
            for (int j = 0; j < OCTETS; ++j) best[j] = octet / LANES == j ? next : best[j];
        }
        __syncwarp();
    }
    constexpr int MINE = 16 / LANES;  // choices l, l + LANES, .. are this lane's
    int my_e[MINE];
    float my_s[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        my_e[i] = l + LANES * i < K ? s_e[tok][l + LANES * i] : -1;
        my_s[i] = my_e[i] >= 0 ? row[my_e[i]] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        if (my_e[i] >= 0) my_s[i] = score(rule.softmax ? expf(my_s[i] - m) : my_s[i]);
        s_chosen[tok][l + LANES * i] = my_s[i];
    }
    __syncthreads();  // and `chose` is zero
    float total = 1.0f;
    if (rule.renorm) {
        float f[16];  // added as a warp does: element i + h to element i
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(&s_chosen[tok][i]);
            f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
        }
#pragma unroll
        for (int h = 8; h; h >>= 1)
#pragma unroll
            for (int i = 0; i < h; ++i) f[i] += f[i + h];
        total = f[0] + kRouteEps;
    }
    if (t >= T) {
#pragma unroll
        for (int i = 0; i < MINE; ++i) my_e[i] = -1;
    }
    const size_t p = static_cast<size_t>(t) * K + l;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        if (my_e[i] < 0) continue;
        topk_idx[p + LANES * i] = my_e[i];
        topk_w[p + LANES * i] = rule.scale * (rule.renorm ? my_s[i] / total : my_s[i]);
        atomicOr(&chose[tok / CH][my_e[i]], 1u << tok % CH);  // the final mask does not depend on the order
    }
    __syncthreads();
    const int pitch = count_pitch(E), first = blockIdx.x * CHUNKS, chunks = (T + CH - 1) / CH;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        if (first + c < chunks)
            for (int e = threadIdx.x; e < pitch; e += OCTET_THREADS)
                chunk_counts[static_cast<size_t>(first + c) * pitch + e] =
                    static_cast<uint8_t>(e < E ? __popc(chose[c][e]) : 0);
#pragma unroll
    for (int i = 0; i < MINE; ++i)
        if (my_e[i] >= 0) row_of[p + LANES * i] = __popc(chose[tok / CH][my_e[i]] & ((1u << tok % CH) - 1u));
}

// Sums of the rows [from, to) of byte counts: thread (word, slice) of the
// block adds 16 experts' bytes of every slice-th row, as sixteen 16-bit sums.
struct Sums16 {
    uint32_t even[4], odd[4];
    __device__ __forceinline__ void add(const uint4 &v) {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            even[i] += x[i] & 0x00ff00ffu;
            odd[i] += (x[i] >> 8) & 0x00ff00ffu;
        }
    }
};

// span_counts[s][e]: the pairs of expert e in span s.
__global__ void __launch_bounds__(256)
route_scored_span_kernel(const uint8_t *__restrict__ chunk_counts, int chunks, int per_span, int E,
                         int32_t *__restrict__ span_counts) {
    grid_dependency_wait();  // launched early: the counts
    const int c0 = blockIdx.x * per_span, c1 = min(chunks, c0 + per_span);
    for (int e = threadIdx.x; e < E; e += 256) {
        int sum = 0;
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += chunk_counts[static_cast<size_t>(c) * count_pitch(E) + e];
        span_counts[static_cast<size_t>(blockIdx.x) * E + e] = sum;
    }
}

// Counts, offsets and the dispatch order from the chunks' counts and the
// pairs' ranks.  CTA s takes the chunks of span s.  It needs the experts'
// totals and what the spans before it hold: summed from the chunks' bytes by
// every CTA itself, or from the spans' sums (SPANNED) where the bytes are many.
template <bool SPANNED>
__global__ void __launch_bounds__(dispatch_threads(SPANNED))
route_scored_dispatch_kernel(const int32_t *__restrict__ topk_idx, const uint8_t *__restrict__ chunk_counts,
                             const int32_t *__restrict__ span_counts, int T, int E, int K, int chunks, int per_span,
                             int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
                             int32_t *__restrict__ row_of, int32_t *__restrict__ src_tok) {
    constexpr int THREADS = dispatch_threads(SPANNED), WARPS = THREADS / 32;
    constexpr int BLOCK = 16;  // chunks whose first rows are held at a time
    __shared__ union {
        uint16_t part[2][WARPS][MAX_E];  // the warps' sums: all chunks, those before the span
        int32_t base[BLOCK][MAX_E];      // then the chunks' first rows
    } sh;
    __shared__ int32_t s_total[MAX_E], s_next[MAX_E], s_warp[MAX_E / 32];  // totals; the experts' next rows
    grid_dependency_wait();  // launched early: the choices, ranks and counts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = count_pitch(E);
    const int c0 = blockIdx.x * per_span, c1 = min(chunks, c0 + per_span);
    // of the first block of chunks: the counts and this thread's first pair, ahead of the sums
    uint8_t n[BLOCK] = {};
    auto load_counts = [&](int b0) {
        if (warp * 32 >= E) return;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i)
            n[i] = static_cast<int>(threadIdx.x) < E && b0 + i < c1
                       ? chunk_counts[static_cast<size_t>(b0 + i) * pitch + threadIdx.x] : 0;
    };
    load_counts(c0);
    const int64_t pairs = min(static_cast<int64_t>(T), static_cast<int64_t>(c1) * CH) * K;  // up to the span's end
    int64_t p = static_cast<int64_t>(c0) * CH * K + threadIdx.x;
    int next_e = 0, next_rank = 0;
    if (p < pairs) next_e = topk_idx[p], next_rank = row_of[p];
    if constexpr (SPANNED) {
        const int e = threadIdx.x;
        if (e < E) {
            int total = 0, before = 0;
#pragma unroll 8
            for (int s = 0; s < static_cast<int>(gridDim.x); ++s) {
                const int v = span_counts[static_cast<size_t>(s) * E + e];
                total += v;
                before += s < static_cast<int>(blockIdx.x) ? v : 0;
            }
            s_total[e] = total;
            s_next[e] = before;
        }
    } else {
        const int words = pitch / 16;  // at most 16; the words of a row lie in neighbouring lanes
        int lanes = 1;
        while (lanes < words) lanes *= 2;
        const int word = lane % lanes, slices = THREADS / lanes;
        Sums16 all = {}, before = {};
        if (word < words) {
#pragma unroll 4
            for (int c = threadIdx.x / lanes; c < chunks; c += slices) {
                const uint4 v = *reinterpret_cast<const uint4 *>(chunk_counts + static_cast<size_t>(c) * pitch + word * 16);
                all.add(v);
                if (c < c0) before.add(v);
            }
        }
        for (int o = lanes; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all.even[i] += __shfl_xor_sync(FULL, all.even[i], o);
                all.odd[i] += __shfl_xor_sync(FULL, all.odd[i], o);
                before.even[i] += __shfl_xor_sync(FULL, before.even[i], o);
                before.odd[i] += __shfl_xor_sync(FULL, before.odd[i], o);
            }
        }
        if (lane < words) {
            uint16_t *a = &sh.part[0][warp][word * 16], *b = &sh.part[1][warp][word * 16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // byte order: even 0, odd 0, even 1, odd 1 of each 32-bit word
                a[4 * i] = all.even[i] & 0xffffu, a[4 * i + 1] = all.odd[i] & 0xffffu;
                a[4 * i + 2] = all.even[i] >> 16, a[4 * i + 3] = all.odd[i] >> 16;
                b[4 * i] = before.even[i] & 0xffffu, b[4 * i + 1] = before.odd[i] & 0xffffu;
                b[4 * i + 2] = before.even[i] >> 16, b[4 * i + 3] = before.odd[i] >> 16;
            }
        }
        __syncthreads();
        if (threadIdx.x < 2 * MAX_E) {
            const int set = threadIdx.x / MAX_E, e = threadIdx.x % MAX_E;
            if (e < E) {
                int sum = 0;
#pragma unroll 8
                for (int w = 0; w < WARPS; ++w) sum += sh.part[set][w][e];
                (set ? s_next : s_total)[e] = sum;
            }
        }
    }
    __syncthreads();
    // offsets, and the span's first rows: the warps scan 32 experts each
    {
        const int e = threadIdx.x;
        int c = 0, incl = 0;
        if (warp < MAX_E / 32) {
            incl = c = e < E ? s_total[e] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) s_warp[warp] = incl;
        }
        __syncthreads();
        if (e < E) {
            int off = incl - c;
            for (int w = 0; w < warp; ++w) off += s_warp[w];
            s_next[e] += off;
            if (blockIdx.x == 0) {
                counts[e] = c;
                offsets[e] = off;
                if (e == E - 1) offsets[E] = off + c;
            }
        }
    }
    for (int b0 = c0; b0 < c1; b0 += BLOCK) {
        if (threadIdx.x < E) {
            const int e = threadIdx.x;
            int run = s_next[e];
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                sh.base[i][e] = run;
                run += n[i];
            }
            s_next[e] = run;
        }
        __syncthreads();
        const int64_t first = static_cast<int64_t>(b0) * CH * K;
        const int64_t last = min(pairs, static_cast<int64_t>(min(b0 + BLOCK, c1)) * CH * K);
        while (p < last) {
            const int i = static_cast<int>(p - first) / (CH * K);
            const int r = sh.base[i][next_e] + next_rank;
            row_of[p] = r;
            src_tok[r] = static_cast<int32_t>(p / K);
            p += THREADS;
            if (p < pairs) next_e = topk_idx[p], next_rank = row_of[p];
        }
        if (b0 + BLOCK < c1) {
            load_counts(b0 + BLOCK);
            __syncthreads();
        }
    }
}

// dlogits [T, E]: one warp per token; lane k < K holds the k-th choice.
template <int EPL>
__global__ void __launch_bounds__(256)
route_scored_bwd_kernel(const float *__restrict__ L, const int32_t *__restrict__ topk_idx,
                        const float *__restrict__ dw, int T, int E, int K, RouteRule rule, float *__restrict__ dL) {
    const int lane = threadIdx.x & 31;
    const int nw = (gridDim.x * blockDim.x) >> 5;
    for (int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < T; t += nw) {
        const float *row = L + static_cast<size_t>(t) * E;
        int e = -1;
        float g = 0.0f;
        if (lane < K) {
            e = topk_idx[static_cast<size_t>(t) * K + lane];
            g = dw[static_cast<size_t>(t) * K + lane];
            if (e < 0 || e >= E) e = -1;  // outside the contract: no access, no gradient
        }
        float s[EPL];
        float se = 0.0f;  // the score of this lane's choice
        if (rule.softmax) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) s[j] = lane + 32 * j < E ? row[lane + 32 * j] : 0.0f;
            scores<32, EPL>(s, E, lane, true);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const float v = __shfl_sync(FULL, s[j], e & 31);
                if ((e >> 5) == j) se = v;  // -1 >> 5 is no j
            }
        } else if (e >= 0) {
            se = sigmoid(row[e]);
        }
        float ds = e >= 0 ? rule.scale * g : 0.0f;
        if (rule.renorm) {
            // a division, not a product with 1 / total: the share of a single choice
            // is 1 to the last bit, and its gradient zero
            const float total = lanes_sum<32>(se) + kRouteEps;
            const float mean = lanes_sum<32>(e >= 0 ? g * (se / total) : 0.0f);
            ds = e >= 0 ? rule.scale * (g - mean) / total : 0.0f;
        }
        // every expert's entry as if it were not chosen, then the chosen ones over them
        float mean = 0.0f, mine;
        if (rule.softmax) {
            mean = lanes_sum<32>(se * ds);
            mine = se * (ds - mean);
        } else {
            mine = e >= 0 ? ds * se / (1.0f + expf(row[e])) : 0.0f;
        }
        float *out = dL + static_cast<size_t>(t) * E;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j < E) out[lane + 32 * j] = rule.softmax ? s[j] * -mean : 0.0f;
        __syncwarp();  // orders the warp's stores
        if (e >= 0) out[e] = mine;
    }
}

// The chosen experts' entries alone, for a layer's backward: with w saved by
// the forward, dl_k = w_k (dw_k - sum_j dw_j (w_j / scale) [renorm]), times
// 1 - s_k for sigmoid scores.  Softmax scores only with renorm: there the
// entries of the experts that were not chosen are zero (up to the 1e-20).
__global__ void __launch_bounds__(256)
route_scored_bwd_rows_kernel(const float *__restrict__ L, const int32_t *__restrict__ topk_idx,
                             const float *__restrict__ topk_w, const float *__restrict__ dw,
                             const int32_t *__restrict__ row_of, int T, int E, int K, RouteRule rule,
                             float *__restrict__ dl, float *__restrict__ dl_row, int TK) {
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= T) return;
    float mean = 0.0f;
    if (rule.renorm && rule.scale != 0.0f)
        for (int k = 0; k < K; ++k) {
            const size_t i = static_cast<size_t>(t) * K + k;
            mean = __fmaf_rn(topk_w[i] / rule.scale, dw[i], mean);  // the share of a single choice is 1 to the last bit
        }
    for (int k = 0; k < K; ++k) {
        const size_t i = static_cast<size_t>(t) * K + k;
        const int e = topk_idx[i];
        float v = topk_w[i] * (dw[i] - mean);
        if (!rule.softmax) v = e >= 0 && e < E ? v / (1.0f + expf(L[static_cast<size_t>(t) * E + e])) : 0.0f;
        dl[i] = v;
        const int r = row_of[i];
        if (r >= 0 && r < TK) dl_row[r] = v;
    }
}

}  // namespace rs

size_t route_scored_workspace_bytes(int T, int E) {
    return static_cast<size_t>(rs::num_chunks(T)) * rs::count_pitch(E) + sizeof(int32_t) * rs::SPANS * E;
}

cudaError_t launch_route_scored(const float *logits, const float *sel_bias, int T, int E, int K, const RouteRule &rule,
                                int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *row_of,
                                int32_t *src_tok, uint8_t *workspace, int *launches, cudaStream_t stream) {
    const int chunks = rs::num_chunks(T);
    const bool few = T <= rs::CH;
    const size_t smem =
        rule.topk_group < rule.n_group ? static_cast<size_t>(rs::CH) * (E + rule.n_group + rs::OPEN) * 4 : 0;
    auto topk = [&](auto kernel, int lanes) {
        static_assert(rs::CH * (2 * rs::MAX_E + rs::OPEN) * 4 < 40 * 1024, "the groups' keys fit without an attribute");
        kernel<<<few ? 1 : chunks, rs::CH * lanes, smem, stream>>>(logits, sel_bias, T, E, K, rule, topk_idx, topk_w, row_of,
                                                             workspace, counts, offsets, src_tok);
        return cudaGetLastError();
    };
    auto by_experts = [&](auto lanes, auto each) {
        constexpr int LANES = decltype(lanes)::value, EPL = decltype(each)::value;
        return few ? topk(rs::route_scored_topk_kernel<LANES, EPL, true>, LANES)
                   : topk(rs::route_scored_topk_kernel<LANES, EPL, false>, LANES);
    };
    auto octets = [&](auto kernel, int lanes) {
        const int tokens = rs::OCTET_THREADS / lanes;
        kernel<<<(T + tokens - 1) / tokens, rs::OCTET_THREADS, 0, stream>>>(logits, sel_bias, T, E, K, rule, topk_idx,
                                                                            topk_w, row_of, workspace);
        return cudaGetLastError();
    };
    const bool grouped = rule.topk_group < rule.n_group;
    const bool fours = E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(sel_bias) % 16 == 0 &&
                       (!grouped || (rule.n_group <= rs::RUNS && E / rule.n_group % 4 == 0));
    using std::integral_constant;
    const integral_constant<int, 16> half;
    const integral_constant<int, 32> whole;
    cudaError_t err = fours && E > 32 && T >= rs::many(E)
                          ? E <= 64    ? octets(rs::route_scored_topk_octets_kernel<4, 2>, 4)
                            : E <= 128 ? octets(rs::route_scored_topk_octets_kernel<4, 4>, 4)
                                       : octets(rs::route_scored_topk_octets_kernel<8, 4>, 8)
                      : E <= 16  ? by_experts(half, integral_constant<int, 1>{})
                      : E <= 32  ? by_experts(half, integral_constant<int, 2>{})
                      : E <= 64  ? by_experts(half, integral_constant<int, 4>{})
                      : E <= 128 ? by_experts(whole, integral_constant<int, 4>{})
                                 : by_experts(whole, integral_constant<int, 8>{});
    *launches = 1;
    if (err != cudaSuccess || few) return err;
    const int per_span = rs::span_chunks(chunks), spans = (chunks + per_span - 1) / per_span;
    const size_t count_bytes = static_cast<size_t>(chunks) * rs::count_pitch(E);
    int32_t *span_counts = reinterpret_cast<int32_t *>(workspace + count_bytes);
    const bool spanned = count_bytes > rs::SELF_SUM_BYTES;
    if (spanned) {
        err = launch_dependent(rs::route_scored_span_kernel, spans, 256, stream,
                               static_cast<const uint8_t *>(workspace), chunks, per_span, E, span_counts);
        if (err != cudaSuccess) return err;
        ++*launches;
    }
    ++*launches;
    return launch_dependent(spanned ? rs::route_scored_dispatch_kernel<true> : rs::route_scored_dispatch_kernel<false>,
                            spans, rs::dispatch_threads(spanned), stream, static_cast<const int32_t *>(topk_idx),
                            static_cast<const uint8_t *>(workspace), static_cast<const int32_t *>(span_counts), T, E,
                            K, chunks, per_span, counts, offsets, row_of, src_tok);
}

cudaError_t launch_route_scored_bwd(const float *logits, const int32_t *topk_idx, const float *dw, int T, int E, int K,
                                    const RouteRule &rule, float *dlogits, cudaStream_t stream) {
    const int blocks = std::min((T + 7) / 8, 152 * 8);
#define ROUTE_SCORED_BWD(EPL) \
    rs::route_scored_bwd_kernel<EPL><<<blocks, 256, 0, stream>>>(logits, topk_idx, dw, T, E, K, rule, dlogits)
    if (E <= 32) ROUTE_SCORED_BWD(1);
    else if (E <= 64) ROUTE_SCORED_BWD(2);
    else if (E <= 128) ROUTE_SCORED_BWD(4);
    else ROUTE_SCORED_BWD(8);
#undef ROUTE_SCORED_BWD
    return cudaGetLastError();
}

cudaError_t launch_route_scored_bwd_rows(const float *logits, const int32_t *topk_idx, const float *topk_w,
                                         const float *dw, const int32_t *row_of, int T, int E, int K,
                                         const RouteRule &rule, float *dl, float *dl_row, cudaStream_t stream) {
    rs::route_scored_bwd_rows_kernel<<<(T + 255) / 256, 256, 0, stream>>>(logits, topk_idx, topk_w, dw, row_of, T, E,
                                                                         K, rule, dl, dl_row, T * K);
    return cudaGetLastError();
}

}  // namespace moe

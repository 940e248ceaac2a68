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
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace rs {

constexpr int CH = kRouteChunk;  // tokens per CTA
constexpr int MAX_E = 256;
constexpr int MAX_K = 16;
constexpr int WARPS = 16;
constexpr int THREADS = WARPS * 32;
constexpr unsigned FULL = 0xffffffffu;

// Keys that order as the values do, -0.0 as +0.0; 0 is kept for "not there".
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v == 0.0f) v = 0.0f;
    const uint32_t u = __float_as_uint(v);
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return k ? k : 1u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// Scores of one token: lane holds experts lane + 32 j in v (logits in, scores out).
template <int EPL>
__device__ __forceinline__ void scores(float *v, int E, int lane, bool softmax) {
    if (!softmax) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = sigmoid(v[j]);
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (lane + 32 * j < E) m = fmaxf(m, v[j]);
    m = warp_max(m);
    float t[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) t[j] = v[j] = lane + 32 * j < E ? expf(v[j] - m) : 0.0f;
#pragma unroll
    for (int h = EPL / 2; h; h >>= 1) {
#pragma unroll
        for (int j = 0; j < h; ++j) t[j] += t[j + h];
    }
    const float sum = warp_sum(t[0]);
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = v[j] / sum;
}

// One CTA per chunk of CH tokens, one warp per token at a time.
template <int EPL>
__global__ void __launch_bounds__(THREADS)
route_scored_topk_kernel(const float *__restrict__ L, const float *__restrict__ bias, int T, int E, int K,
                         RouteRule rule, int32_t *__restrict__ topk_idx, float *__restrict__ topk_w,
                         int32_t *__restrict__ row_rank, int32_t *__restrict__ chunk_counts) {
    __shared__ uint32_t bits[MAX_E][CH / 32];
    __shared__ int32_t s_idx[CH * MAX_K];
    __shared__ uint32_t s_key[WARPS][MAX_E], s_group[WARPS][MAX_E];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * CH;
    const int nt = min(CH, T - t0);
    const int per = E / rule.n_group;
    for (int i = threadIdx.x; i < E * (CH / 32); i += THREADS) (&bits[0][0])[i] = 0u;
    __syncthreads();
    float b[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) b[j] = bias && lane + 32 * j < E ? bias[lane + 32 * j] : 0.0f;

    for (int tl = warp; tl < nt; tl += WARPS) {
        const int t = t0 + tl;
        const float *row = L + static_cast<size_t>(t) * E;
        float s[EPL];
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = lane + 32 * j < E ? row[lane + 32 * j] : 0.0f;
        scores<EPL>(s, E, lane, rule.softmax);
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = lane + 32 * j < E ? order_key(bias ? s[j] + b[j] : s[j]) : 0u;
        if (rule.topk_group < rule.n_group) {
            uint32_t *sk = s_key[warp], *sg = s_group[warp];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < E) sk[lane + 32 * j] = key[j];
            __syncwarp();
            for (int g = lane; g < rule.n_group; g += 32) {
                uint32_t a = 0, c = 0;  // the two largest
                for (int i = 0; i < per; ++i) {
                    const uint32_t k = sk[g * per + i];
                    c = max(c, min(a, k));
                    a = max(a, k);
                }
                sg[g] = rule.group_top == 2 && c ? order_key(key_value(a) + key_value(c)) : a;
            }
            __syncwarp();
            uint32_t open = 0;  // bit i: run lane + 32 i stays open
            for (int g = lane, i = 0; g < rule.n_group; g += 32, ++i) {
                const uint32_t mine = sg[g];
                int above = 0;
                for (int o = 0; o < rule.n_group; ++o) above += sg[o] > mine || (sg[o] == mine && o < g);
                if (above < rule.topk_group) open |= 1u << i;
            }
            __syncwarp();
            for (int g = lane, i = 0; g < rule.n_group; g += 32, ++i) sg[g] = (open >> i) & 1u;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < E && !sg[(lane + 32 * j) / per]) key[j] = 0u;
        }
        uint32_t best = 0;
        int bj = 0;
        float bs = 0.0f;
        auto find = [&]() {  // this lane's largest key, the lowest expert on ties
            best = key[0], bj = 0, bs = s[0];
#pragma unroll
            for (int j = 1; j < EPL; ++j)
                if (key[j] > best) best = key[j], bj = j, bs = s[j];
        };
        find();
        int my_e = 0;
        float my_s = 0.0f, sum = 0.0f;
        for (int k = 0; k < K; ++k) {
            const uint32_t top = __reduce_max_sync(FULL, best);
            const int e = static_cast<int>(
                __reduce_min_sync(FULL, best == top ? static_cast<uint32_t>(lane + 32 * bj) : FULL));
            const float se = __shfl_sync(FULL, bs, e & 31);
            if ((e & 31) == lane) {
#pragma unroll
                for (int j = 0; j < EPL; ++j) key[j] = j == bj ? 0u : key[j];
                find();
            }
            sum += se;
            if (lane == k) my_e = e, my_s = se;
        }
        if (lane < K) {
            const size_t p = static_cast<size_t>(t) * K + lane;
            topk_idx[p] = my_e;
            topk_w[p] = rule.renorm ? rule.scale * my_s / (sum + kRouteEps) : rule.scale * my_s;
            s_idx[tl * K + lane] = my_e;
            atomicOr(&bits[my_e][tl >> 5], 1u << (tl & 31));
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < CH / 32; ++w) c += __popc(bits[e][w]);
        chunk_counts[static_cast<size_t>(blockIdx.x) * E + e] = c;
    }
    for (int p = threadIdx.x; p < nt * K; p += THREADS) {
        const int tl = p / K, e = s_idx[p];
        int r = __popc(bits[e][tl >> 5] & ((1u << (tl & 31)) - 1u));
        for (int w = 0; w < (tl >> 5); ++w) r += __popc(bits[e][w]);
        row_rank[static_cast<size_t>(t0) * K + p] = r;
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
            scores<EPL>(s, E, lane, true);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const float v = __shfl_sync(FULL, s[j], e & 31);
                if (e >= 0 && (e >> 5) == j) se = v;
            }
        } else if (e >= 0) {
            se = sigmoid(row[e]);
        }
        float ds = e >= 0 ? rule.scale * g : 0.0f;
        if (rule.renorm) {
            const float inv = 1.0f / (warp_sum(se) + kRouteEps);
            const float mean = warp_sum(e >= 0 ? g * (se * inv) : 0.0f);
            ds = e >= 0 ? rule.scale * (g - mean) * inv : 0.0f;
        }
        // what this lane's choice adds to its expert's entry
        const float mine = rule.softmax ? ds : e >= 0 ? ds * se / (1.0f + expf(row[e])) : 0.0f;
        float o[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) o[j] = 0.0f;
        for (int k = 0; k < K; ++k) {
            const int ek = __shfl_sync(FULL, e, k);
            const float v = __shfl_sync(FULL, mine, k);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (ek == lane + 32 * j) o[j] = v;
        }
        if (rule.softmax) {
            const float mean = warp_sum(se * ds);
#pragma unroll
            for (int j = 0; j < EPL; ++j) o[j] = s[j] * (o[j] - mean);
        }
        float *out = dL + static_cast<size_t>(t) * E;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j < E) out[lane + 32 * j] = o[j];
    }
}

// The chosen experts' entries alone, for a layer's backward: with w saved by
// the forward, dl_k = w_k (dw_k - sum_j dw_j w_j / scale [renorm]), times
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
    if (rule.renorm && rule.scale != 0.0f) {
        for (int k = 0; k < K; ++k)
            mean = __fmaf_rn(topk_w[static_cast<size_t>(t) * K + k], dw[static_cast<size_t>(t) * K + k], mean);
        mean /= rule.scale;
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

cudaError_t launch_route_scored(const float *logits, const float *sel_bias, int T, int E, int K, const RouteRule &rule,
                                int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *row_of,
                                int32_t *src_tok, int32_t *workspace, cudaStream_t stream) {
    const int C = route_num_chunks(T);
#define ROUTE_SCORED(EPL)                                                                                       \
    rs::route_scored_topk_kernel<EPL><<<C, rs::THREADS, 0, stream>>>(logits, sel_bias, T, E, K, rule, topk_idx, \
                                                                     topk_w, row_of, workspace)
    if (E <= 32) ROUTE_SCORED(1);
    else if (E <= 64) ROUTE_SCORED(2);
    else if (E <= 128) ROUTE_SCORED(4);
    else ROUTE_SCORED(8);
#undef ROUTE_SCORED
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_route_dispatch(topk_idx, T, E, K, counts, offsets, row_of, src_tok, workspace, stream);
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

// router.cu -- the router's gate: the top_k largest of a token's E logits and
// their softmax weights, and the gradient.  With p = softmax(logits) over the
// token's E experts and S the chosen ones:
//
//   w_j = p_j                      or, renormalised,  w_j = p_j / sum_S p
//   dl_e = [e in S] w_e dw_e - p_e * sum_S w dw
//   renormalised: dl_e = w_e * (dw_e - sum_S w dw) for e in S, else 0
//
// Ties go to the lower index.  A logit of -inf closes its expert to the token:
// it is never chosen, and a token with fewer than top_k open experts gets id -1
// (which the routing plan drops) and weight 0 in the places left over.  A NaN
// or +inf among a token's logits makes its weights NaN; a NaN logit itself is
// never chosen.  One warp a token; everything is FP32.
#include <math_constants.h>

#include "hg_internal.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTopK = 32;       // one choice a lane

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Largest logit (NaN aside) and the sum of exp(logit - largest), NaN included;
// a row of -inf gives (-inf, 0).
__device__ __forceinline__ void softmax_stats(const float* row, int E, int lane, float& top,
                                              float& sum) {
    top = -CUDART_INF_F;
    for (int e = lane; e < E; e += 32) top = fmaxf(top, __ldg(row + e));
    top = warp_max(top);
    sum = 0.0f;
    for (int e = lane; e < E; e += 32) {
        const float l = __ldg(row + e);
        if (l != -CUDART_INF_F) sum += expf(l - top);
    }
    sum = warp_sum(sum);
}

__global__ void __launch_bounds__(kThreads)
router_topk_kernel(const float* __restrict__ logits, int M, int E, int top_k, int renormalize,
                   int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x & 31;
    const long long nw = (static_cast<long long>(gridDim.x) * kThreads) >> 5;
    for (long long t = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5; t < M;
         t += nw) {
        const float* row = logits + t * E;
        float top, sum;
        softmax_stats(row, E, lane, top, sum);
        // the largest logit below the one chosen before, in the order (value
        // descending, index ascending)
        float last = CUDART_INF_F, mine = 0.0f;
        int last_e = -1, mine_e = -1;
        for (int c = 0; c < top_k; ++c) {
            float best = -CUDART_INF_F;
            int best_e = 0x7FFFFFFF;
            for (int e = lane; e < E; e += 32) {
                const float l = __ldg(row + e);
                if ((l < last || (l == last && e > last_e)) &&
                    (l > best || (l == best && e < best_e))) {
                    best = l;
                    best_e = e;
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const float l = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                const int e = __shfl_xor_sync(0xFFFFFFFFu, best_e, o);
                if (l > best || (l == best && e < best_e)) {
                    best = l;
                    best_e = e;
                }
            }
            if (best == -CUDART_INF_F) break;      // no open expert is left
            last = best;
            last_e = best_e;
            if (lane == c) {
                mine = best;
                mine_e = best_e;
            }
        }
        float w = mine_e >= 0 ? expf(mine - top) : 0.0f;
        const float den = renormalize && !isnan(sum) ? warp_sum(w) : sum;
        if (mine_e >= 0) w /= den;
        if (lane < top_k) {
            ids[t * top_k + lane] = mine_e;
            weights[t * top_k + lane] = w;
        }
    }
}

__global__ void __launch_bounds__(kThreads)
router_topk_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                       const float* __restrict__ weights, const float* __restrict__ dweights,
                       int M, int E, int top_k, int renormalize, float* __restrict__ dlogits) {
    const int lane = threadIdx.x & 31;
    const long long nw = (static_cast<long long>(gridDim.x) * kThreads) >> 5;
    for (long long t = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5; t < M;
         t += nw) {
        int id = -1;
        float w = 0.0f, dw = 0.0f;
        if (lane < top_k) {
            id = __ldg(ids + t * top_k + lane);
            if (id >= 0 && id < E) {
                w = __ldg(weights + t * top_k + lane);
                dw = __ldg(dweights + t * top_k + lane);
            } else {
                id = -1;
            }
        }
        const float inner = warp_sum(w * dw);
        float top = 0.0f, sum = 1.0f;
        if (!renormalize) softmax_stats(logits + t * E, E, lane, top, sum);
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            float d = 0.0f;
            if (!renormalize && e < E) {
                const float l = __ldg(logits + t * E + e);
                if (l != -CUDART_INF_F) d = -(expf(l - top) / sum) * inner;
            }
            for (int c = 0; c < top_k; ++c) {
                const int ic = __shfl_sync(0xFFFFFFFFu, id, c);
                const float wc = __shfl_sync(0xFFFFFFFFu, w, c);
                const float dc = __shfl_sync(0xFFFFFFFFu, dw, c);
                if (ic == e) d += renormalize ? wc * (dc - inner) : wc * dc;
            }
            if (e < E) dlogits[t * E + e] = d;
        }
    }
}

int grid_blocks(int M, int num_sms) {
    const int blocks = (M + kThreads / 32 - 1) / (kThreads / 32);
    return blocks < num_sms * 8 ? blocks : num_sms * 8;
}

}  // namespace

int router_max_top_k() { return kMaxTopK; }

cudaError_t launch_router_topk(const float* logits, int M, int E, int top_k, int renormalize,
                               int32_t* ids, float* weights, int num_sms, cudaStream_t stream) {
    router_topk_kernel<<<grid_blocks(M, num_sms), kThreads, 0, stream>>>(logits, M, E, top_k,
                                                                         renormalize, ids, weights);
    return cudaGetLastError();
}

cudaError_t launch_router_topk_bwd(const float* logits, const int32_t* ids, const float* weights,
                                   const float* dweights, int M, int E, int top_k,
                                   int renormalize, float* dlogits, int num_sms,
                                   cudaStream_t stream) {
    router_topk_bwd_kernel<<<grid_blocks(M, num_sms), kThreads, 0, stream>>>(
        logits, ids, weights, dweights, M, E, top_k, renormalize, dlogits);
    return cudaGetLastError();
}

}  // namespace hg

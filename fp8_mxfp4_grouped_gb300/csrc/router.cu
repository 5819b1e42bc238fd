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
// never chosen.
//
// One warp a token, everything in FP32.  Both passes move one row of logits (the
// gradient also writes one), 640 bytes for 160 experts: little enough that
// instructions count.  The row stays in registers (up to 512 experts); a choice
// is a warp-wide maximum and a warp-wide minimum of the index, one reduction
// instruction each, and only the lane that owned it looks at its values again.
// The gradient needs no softmax of its own, as long as the first choice is there:
// it is the row's largest logit and its weight 1 / sum, so that p_e = exp(l_e -
// l_first) * w_first.  Gate and gradient of 16384 x 160, top-6, take 15.8 us (22 MB: 3.3 at
// the copy rate), bound by the rounds of choice; of 5 x 32, top-8, the gate 2.0.
#include <math_constants.h>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxTopK = 32;       // one choice a lane
constexpr int kMaxHeld = 16;       // logits a lane holds in registers

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The row of a token, lane l holding experts l, l + 32, ...: in registers
// (kHeld of them), or read again each time (kHeld = 0).  NaN reads as -inf.
template <int kHeld>
struct Row {
    const float* at;
    int E, lane;
    float v[kHeld ? kHeld : 1];
    bool nan = false;

    __device__ Row(const float* row, int E_, int lane_) : at(row), E(E_), lane(lane_) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = read(i);
        if (kHeld == 0) {
            for (int i = 0; lane + 32 * i < E; ++i) read(i);
        }
    }
    __device__ float read(int i) {
        if (lane + 32 * i >= E) return -CUDART_INF_F;
        const float l = ptx::load(at + lane + 32 * i);
        nan |= isnan(l);
        return isnan(l) ? -CUDART_INF_F : l;
    }
    template <class F>
    __device__ void each(F f) {
        if (kHeld) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) f(lane + 32 * i, v[i]);
        } else {
            for (int i = 0; lane + 32 * i < E; ++i) f(lane + 32 * i, read(i));
        }
    }
};

template <int kHeld>
__global__ void __launch_bounds__(kThreads)
router_topk_kernel(const float* logits, int M, int E, int top_k, int renormalize,
                   int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    start_dependent();
    if (t >= M) return;
    Row<kHeld> row(logits + t * E, E, lane);

    // This lane's largest logit below what it has given away (last, last_e), in
    // the order (value descending, index ascending).
    float best, last = CUDART_INF_F;
    int best_e, last_e = -1;
    auto look = [&]() {
        best = -CUDART_INF_F;
        best_e = 0x7FFFFFFF;
        row.each([&](int e, float l) {
            if (l > best && (l < last || (l == last && e > last_e))) {
                best = l;
                best_e = e;
            }
        });
    };
    look();
    const float top = warp_max(best);
    float sum = 0.0f;
    row.each([&](int e, float l) {
        if (l != -CUDART_INF_F) sum += expf(l - top);
    });
    sum = warp_sum(sum);
    if (__any_sync(0xFFFFFFFFu, row.nan)) sum = CUDART_NAN_F;

    float mine = 0.0f;
    int mine_e = -1;
    for (int c = 0; c < top_k; ++c) {
        const float l = warp_max(best);
        if (l == -CUDART_INF_F) break;       // no open expert is left
        const int e = __reduce_min_sync(0xFFFFFFFFu, best == l ? best_e : 0x7FFFFFFF);
        if (lane == c) {
            mine = l;
            mine_e = e;
        }
        if (best_e == e) {
            last = l;
            last_e = e;
            look();
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

// dw - c, with c = sum_j w_j dw_j, cancels for the largest weight where that is
// nearly 1.  There it is taken as dw (1 - w) - sum over the others of w_j dw_j, and
// 1 - w as the sum of all other probabilities.
//
// A choice whose id has been taken out since the gate (for an expert's capacity,
// say) has no dw, but its probability still counts: its weight does, and where it
// was the row's largest, or one before the last, the row's own softmax is taken.
template <int kHeld>
__global__ void __launch_bounds__(kThreads)
router_topk_bwd_kernel(const float* logits, const int32_t* ids, const float* weights,
                       const float* dweights, int M, int E, int top_k, int renormalize,
                       float* __restrict__ dlogits) {
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    start_dependent();
    if (t >= M) return;
    int id = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < top_k) {
        id = ptx::load(ids + t * top_k + lane);
        w = ptx::load(weights + t * top_k + lane);
        dw = ptx::load(dweights + t * top_k + lane);
    }
    const float* row = logits + t * E;
    float l[kHeld ? kHeld : 1];
    if (!renormalize) {                      // asked for ahead of what the choices decide
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            l[i] = lane + 32 * i < E ? ptx::load(row + lane + 32 * i) : -CUDART_INF_F;
    }
    float out_of = 0.0f;                     // the weight of a choice taken out
    if (id < 0 || id >= E) {
        id = -1;
        out_of = w;
        w = dw = 0.0f;
    }
    const uint32_t chosen = __ballot_sync(0xFFFFFFFFu, id >= 0);
    const int lead = chosen ? __ffs(chosen) - 1 : 0;         // the largest weight's
    const float others = warp_sum(lane != lead ? w * dw : 0.0f);
    const float c = __shfl_sync(0xFFFFFFFFu, w * dw, lead) + others;
    float rest = lane != lead ? w + out_of : 0.0f;           // probabilities but the largest
    float* out = dlogits + t * E;
    if (renormalize || !chosen) {
        for (int e = lane; e < E; e += 32) out[e] = 0.0f;
    } else {
        auto logit = [&](int e) {
            if (kHeld == 0) return ptx::load(row + e);
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) v = e >> 5 == i ? l[i] : v;
            return __shfl_sync(0xFFFFFFFFu, v, e & 31);
        };
        auto each = [&](auto f) {
            if (kHeld) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) f(lane + 32 * i, l[i]);
            } else {
                for (int e = lane; e < E; e += 32) f(e, ptx::load(row + e));
            }
        };
        const int last = 31 - __clz(chosen);
        float top = logit(__shfl_sync(0xFFFFFFFFu, id, lead));
        float p_top = __shfl_sync(0xFFFFFFFFu, w, lead);
        if (lead > 0) {                      // the row's largest was taken out
            float most = -CUDART_INF_F, sum = 0.0f;
            each([&](int, float le) { most = fmaxf(most, le); });
            top = warp_max(most);
            each([&](int, float le) { sum += expf(le - top); });
            p_top = 1.0f / warp_sum(sum);
        }
        // what comes after the last choice, in the choices' order, is not chosen;
        // weights taken out behind it are among that
        const int last_e = __shfl_sync(0xFFFFFFFFu, id, last);
        const float least = logit(last_e);
        if (lane > last) rest -= out_of;
        each([&](int e, float le) {
            const float p = expf(le - top) * p_top;
            if (le < least || (le == least && e > last_e)) rest += p;
            if (e < E) out[e] = -p * c;
        });
    }
    rest = warp_sum(rest);
    __syncwarp();                            // the chosen ones' values come last
    if (id >= 0) out[id] = w * (lane == lead ? fmaf(dw, rest, -others) : dw - c);
}

template <int kHeld>
cudaError_t launch_topk(const float* logits, int M, int E, int top_k, int renormalize,
                        int32_t* ids, float* weights, cudaStream_t stream) {
    const int grid = (M - 1) / (kThreads / 32) + 1;
    return launch_dependent(router_topk_kernel<kHeld>, grid, kThreads, 0, stream, logits, M, E,
                            top_k, renormalize, ids, weights);
}

}  // namespace

int router_max_top_k() { return kMaxTopK; }

cudaError_t launch_router_topk(const float* logits, int M, int E, int top_k, int renormalize,
                               int32_t* ids, float* weights, cudaStream_t stream) {
    const int held = (E + 31) / 32;
    // a lane looks through all that it holds at each of its choices: eight held
    // where five are needed take 13 us in place of 10 at 16384 x 160, top-6
    const auto launch = held <= 1          ? launch_topk<1>
                        : held <= 2        ? launch_topk<2>
                        : held <= 3        ? launch_topk<3>
                        : held <= 4        ? launch_topk<4>
                        : held <= 5        ? launch_topk<5>
                        : held <= 6        ? launch_topk<6>
                        : held <= 8        ? launch_topk<8>
                        : held <= 12       ? launch_topk<12>
                        : held <= kMaxHeld ? launch_topk<kMaxHeld>
                                           : launch_topk<0>;
    return launch(logits, M, E, top_k, renormalize, ids, weights, stream);
}

cudaError_t launch_router_topk_bwd(const float* logits, const int32_t* ids, const float* weights,
                                   const float* dweights, int M, int E, int top_k,
                                   int renormalize, float* dlogits, cudaStream_t stream) {
    const int grid = (M - 1) / (kThreads / 32) + 1, held = (E + 31) / 32;
    const auto kernel = renormalize        ? router_topk_bwd_kernel<0>
                        : held <= 1        ? router_topk_bwd_kernel<1>
                        : held <= 2        ? router_topk_bwd_kernel<2>
                        : held <= 5        ? router_topk_bwd_kernel<5>
                        : held <= 8        ? router_topk_bwd_kernel<8>
                        : held <= kMaxHeld ? router_topk_bwd_kernel<kMaxHeld>
                                           : router_topk_bwd_kernel<0>;
    return launch_dependent(kernel, grid, kThreads, 0, stream, logits, ids, weights, dweights, M, E,
                            top_k, renormalize, dlogits);
}

}  // namespace hg

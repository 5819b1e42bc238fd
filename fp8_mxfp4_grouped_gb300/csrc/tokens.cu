// tokens.cu -- token rows sorted by expert and back, with the router's
// weights, and the gradients of both directions.  With r(t, j) =
// src_to_sorted[t * top_k + j], the place that the routing plan gave choice j
// of token t:
//
//   dispatch        rows[r(t,j)] = w[t,j] * x[t]                (w = 1 when absent)
//   its gradient    dx[t]        = sum_j w[t,j] * drows[r(t,j)]
//                   dw[t,j]      = <drows[r(t,j)], x[t]>
//   combine         out[t]       = sum_j w[t,j] * y[r(t,j)]     (moe_io.cu)
//   its gradient    dy[r(t,j)]   = w[t,j] * dout[t]
//                   dw[t,j]      = <y[r(t,j)], dout[t]>
//
// Every row is read or written by one token only, so each kernel is organised
// per token: no atomics, and sums whose order is fixed.  Sums and dot products
// are FP32; each result is rounded once to BF16.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;

// Sum over the block, in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();   // s_part may still be read for the previous sum
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kThreads / 32; ++i) t += s_part[i];
    }
    return t;
}

__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ src_to_sorted,
                const float* __restrict__ weights, int M, int top_k, int K,
                uint16_t* __restrict__ rows) {
    const int R = M * top_k;
    for (int t = blockIdx.x; t < M; t += gridDim.x) {
        const uint16_t* xt = x + static_cast<long long>(t) * K;
        for (int n = 8 * threadIdx.x; n < K; n += 8 * kThreads) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(xt + n));
            for (int j = 0; j < top_k; ++j) {
                const int r = __ldg(src_to_sorted + t * top_k + j);
                if (r < 0 || r >= R) continue;
                uint4 o = v;
                if (weights) {
                    const float w = __ldg(weights + t * top_k + j);
                    float f[8];
                    bf16_unpack8(v, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= w;
                    o = bf16_pack8(f);
                }
                *reinterpret_cast<uint4*>(rows + static_cast<long long>(r) * K + n) = o;
            }
        }
    }
}

// kSum: the gradient of the dispatch (out[t] = sum of the weighted rows);
// otherwise the gradient of the combine (out rows = w * token row).
template <bool kSum>
__global__ void __launch_bounds__(kThreads)
token_grad_kernel(const uint16_t* __restrict__ rows, const uint16_t* __restrict__ token,
                  const int32_t* __restrict__ src_to_sorted, const float* __restrict__ weights,
                  int M, int top_k, int N, uint16_t* __restrict__ out, float* __restrict__ dw) {
    __shared__ float s_part[kThreads / 32];
    const int R = M * top_k;
    for (int t = blockIdx.x; t < M; t += gridDim.x) {
        const long long base = static_cast<long long>(t) * N;
        const int32_t* place = src_to_sorted + static_cast<long long>(t) * top_k;
        const float* wt = weights ? weights + static_cast<long long>(t) * top_k : nullptr;
        if (dw) {
            for (int j = 0; j < top_k; ++j) {
                const int r = __ldg(place + j);
                float dot = 0.0f;
                if (r >= 0 && r < R) {
                    const uint16_t* row = rows + static_cast<long long>(r) * N;
                    for (int n = 8 * threadIdx.x; n < N; n += 8 * kThreads) {
                        float a[8], b[8];
                        bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(row + n)), a);
                        bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(token + base + n)), b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot = fmaf(a[i], b[i], dot);
                    }
                }
                dot = block_sum(dot, s_part);
                if (threadIdx.x == 0) dw[static_cast<long long>(t) * top_k + j] = dot;
            }
        }
        for (int n = 8 * threadIdx.x; n < N; n += 8 * kThreads) {
            float acc[8] = {};
            for (int j = 0; j < top_k; ++j) {
                const int r = __ldg(place + j);
                if (r < 0 || r >= R) continue;
                const float w = wt ? __ldg(wt + j) : 1.0f;
                float f[8];
                if (kSum) {
                    bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(
                                     rows + static_cast<long long>(r) * N + n)), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
                } else {
                    bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(token + base + n)), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= w;
                    *reinterpret_cast<uint4*>(out + static_cast<long long>(r) * N + n) =
                        bf16_pack8(f);
                }
            }
            if (kSum) *reinterpret_cast<uint4*>(out + base + n) = bf16_pack8(acc);
        }
    }
}

int grid_blocks(long long work, int num_sms) {
    const long long cap = static_cast<long long>(num_sms) * 8;
    return static_cast<int>(work < cap ? work : cap);
}

}  // namespace

cudaError_t launch_dispatch(const uint16_t* x, const int32_t* d2s, const float* weights, int M,
                            int top_k, int K, uint16_t* rows, int num_sms, cudaStream_t stream) {
    dispatch_kernel<<<grid_blocks(M, num_sms), kThreads, 0, stream>>>(x, d2s, weights, M, top_k, K,
                                                                      rows);
    return cudaGetLastError();
}

cudaError_t launch_dispatch_bwd(const uint16_t* drows, const uint16_t* x, const int32_t* d2s,
                                const float* weights, int M, int top_k, int K, uint16_t* dx,
                                float* dw, int num_sms, cudaStream_t stream) {
    token_grad_kernel<true><<<grid_blocks(M, num_sms), kThreads, 0, stream>>>(
        drows, x, d2s, weights, M, top_k, K, dx, dw);
    return cudaGetLastError();
}

cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* d2s,
                               const float* weights, int M, int top_k, int N, uint16_t* dy,
                               float* dw, int num_sms, cudaStream_t stream) {
    token_grad_kernel<false><<<grid_blocks(M, num_sms), kThreads, 0, stream>>>(
        y, dout, d2s, weights, M, top_k, N, dy, dw);
    return cudaGetLastError();
}

}  // namespace hg

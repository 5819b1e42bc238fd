// matvec.cu -- few tokens times the routed experts' MXFP4 weights, on BF16
// activations: the single-token form of the grouped GEMM.  Slot s = t * top_k
// + j multiplies its input row with the weights of expert topk_ids[s]:
//
//   y[s, n] = sum_k x[row(s), k] * e2m1(w_fp4[e, n, k]) * 2^(w_scale[e, n, k/32] - 127)
//
// with row(s) = s / top_k (one row a token) or s (one row a slot).  The
// SwiGLU form writes h[s, f] = silu(y[s, f]) * y[s, F + f], F = N / 2.
// Products and sums are FP32; the result is rounded once to BF16.  A slot
// whose id is outside [0, E) gets a row of zeros.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;

// Four E2M1 codes of the low 16 bits (element i in bits 4i..4i+3) as floats.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7u;
    const float mag = m < 2u ? 0.5f * m
                             : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (code & 8u) ? -mag : mag;
}

__device__ __forceinline__ float dot_row(const uint16_t* x, const uint8_t* w, const uint8_t* ws,
                                         int K, int lane) {
    float acc = 0.0f;
    for (int g = lane; g < K / 32; g += 32) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(w + 16 * g));
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
            bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(x + 32 * g + 8 * i)), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) part = fmaf(f[e], e2m1_value(words[i] >> (4 * e)), part);
        }
        acc = fmaf(part, e8m0_value(__ldg(ws + g)), acc);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    return acc;
}

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads)
expert_matvec_kernel(const uint16_t* __restrict__ x, int slots_per_row,
                     const int32_t* __restrict__ ids, const uint8_t* __restrict__ w_fp4,
                     const uint8_t* __restrict__ w_scale, int slots, int E, int N, int K,
                     uint16_t* __restrict__ out) {
    const int lane = threadIdx.x & 31;
    const int cols = kSwiglu ? N / 2 : N;
    const long long items = static_cast<long long>(slots) * cols;
    const long long nw = (static_cast<long long>(gridDim.x) * kThreads) >> 5;
    for (long long it = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
         it < items; it += nw) {
        const int s = static_cast<int>(it / cols);
        const int n = static_cast<int>(it % cols);
        const int e = __ldg(ids + s);
        float y = 0.0f;
        if (e >= 0 && e < E) {
            const uint16_t* xr = x + static_cast<long long>(s / slots_per_row) * K;
            const long long row = static_cast<long long>(e) * N + n;
            y = dot_row(xr, w_fp4 + row * (K / 2), w_scale + row * (K / 32), K, lane);
            if (kSwiglu) {
                const long long up = row + cols;
                const float u = dot_row(xr, w_fp4 + up * (K / 2), w_scale + up * (K / 32), K, lane);
                y = y / (1.0f + expf(-y)) * u;
            }
        }
        if (lane == 0) out[it] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
}

}  // namespace

cudaError_t launch_expert_matvec(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    const long long items = static_cast<long long>(a.slots) * (a.swiglu ? a.N / 2 : a.N);
    long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > static_cast<long long>(num_sms) * 8) blocks = static_cast<long long>(num_sms) * 8;
    const int grid = static_cast<int>(blocks);
    if (a.swiglu) {
        expert_matvec_kernel<true><<<grid, kThreads, 0, stream>>>(
            a.x, a.slots_per_row, a.ids, a.w_fp4, a.w_scale, a.slots, a.E, a.N, a.K, a.out);
    } else {
        expert_matvec_kernel<false><<<grid, kThreads, 0, stream>>>(
            a.x, a.slots_per_row, a.ids, a.w_fp4, a.w_scale, a.slots, a.E, a.N, a.K, a.out);
    }
    return cudaGetLastError();
}

}  // namespace hg

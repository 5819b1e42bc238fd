// swiglu.cu -- the activation between an expert's two projections, and its
// gradient from an 8-bit checkpoint.  The gate/up GEMM leaves z = (g, u) per
// row, g in columns [0, F) and u in [F, 2F).  With s = 1 / (1 + exp(-g)):
//
//   forward    h  = g * s * u          quantised to E4M3 with one E8M0 scale per
//                                      128 elements: the down GEMM's input
//              z  quantised the same way: the checkpoint (half of BF16's bytes)
//   backward   dg = dh * u * s * (1 + g * (1 - s))
//              du = dh * g * s         with g and u decoded from the checkpoint
//
// A group of 128 is held by a half-warp, eight elements a lane, so that its
// largest magnitude is one shuffle reduction away and nothing is read twice.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128;

__global__ void __launch_bounds__(kThreads)
swiglu_quantize_kernel(const uint16_t* __restrict__ z, long long groups, int F,
                       uint8_t* __restrict__ a_fp8, uint8_t* __restrict__ a_scale,
                       uint8_t* __restrict__ z_fp8, uint8_t* __restrict__ z_scale) {
    const int G = F / kGroup;
    const int j = threadIdx.x & 15;
    const long long first = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 4;
    const long long step = (static_cast<long long>(gridDim.x) * kThreads) >> 4;
    // both half-warps of a warp stay in the loop together: the reductions
    // shuffle across the whole warp
    for (long long it = first - ((threadIdx.x >> 4) & 1); it < groups; it += step) {
        const long long i = it + ((threadIdx.x >> 4) & 1);
        const bool real = i < groups;
        const long long r = real ? i / G : 0;
        const int g = real ? static_cast<int>(i - r * G) : 0;
        const uint16_t* zr = z + 2 * r * F;
        const uint4 vg = __ldg(reinterpret_cast<const uint4*>(zr + g * kGroup) + j);
        const uint4 vu = __ldg(reinterpret_cast<const uint4*>(zr + F + g * kGroup) + j);
        float fg[8], fu[8], h[8];
        bf16_unpack8(vg, fg);
        bf16_unpack8(vu, fu);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = fg[e] / (1.0f + expf(-fg[e])) * fu[e];
        const GroupCodes ch = quantize_codes(h);
        if (real) {
            *reinterpret_cast<uint2*>(a_fp8 + r * F + g * kGroup + 8 * j) =
                make_uint2(ch.lo, ch.hi);
            if (j == 0) a_scale[r * G + g] = ch.scale;
        }
        if (z_fp8) {
            const GroupCodes cg = quantize_codes(fg);
            const GroupCodes cu = quantize_codes(fu);
            if (real) {
                uint8_t* q = z_fp8 + 2 * r * F + g * kGroup + 8 * j;
                *reinterpret_cast<uint2*>(q) = make_uint2(cg.lo, cg.hi);
                *reinterpret_cast<uint2*>(q + F) = make_uint2(cu.lo, cu.hi);
                if (j == 0) {
                    z_scale[2 * r * G + g] = cg.scale;
                    z_scale[2 * r * G + G + g] = cu.scale;
                }
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads)
swiglu_bwd_kernel(const uint16_t* __restrict__ dh, const uint8_t* __restrict__ z_fp8,
                  const uint8_t* __restrict__ z_scale, long long groups, int F,
                  uint16_t* __restrict__ dz) {
    const int G = F / kGroup;
    const int j = threadIdx.x & 15;
    const long long step = (static_cast<long long>(gridDim.x) * kThreads) >> 4;
    for (long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 4;
         i < groups; i += step) {
        const long long r = i / G;
        const int g = static_cast<int>(i - r * G);
        const long long at = r * F + g * kGroup + 8 * j;
        const long long zat = 2 * r * F + g * kGroup + 8 * j;
        float d[8], fg[8], fu[8], og[8], ou[8];
        bf16_unpack8(__ldg(reinterpret_cast<const uint4*>(dh + at)), d);
        e4m3_unpack8(__ldg(reinterpret_cast<const uint2*>(z_fp8 + zat)), fg);
        e4m3_unpack8(__ldg(reinterpret_cast<const uint2*>(z_fp8 + zat + F)), fu);
        const float sg = e8m0_value(__ldg(z_scale + 2 * r * G + g));
        const float su = e8m0_value(__ldg(z_scale + 2 * r * G + G + g));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float gv = fg[e] * sg;
            const float uv = fu[e] * su;
            const float s = 1.0f / (1.0f + expf(-gv));
            og[e] = d[e] * uv * s * (1.0f + gv * (1.0f - s));
            ou[e] = d[e] * gv * s;
        }
        *reinterpret_cast<uint4*>(dz + zat) = bf16_pack8(og);
        *reinterpret_cast<uint4*>(dz + zat + F) = bf16_pack8(ou);
    }
}

int grid_blocks(long long groups, int num_sms) {
    const long long blocks = (groups + kThreads / 16 - 1) / (kThreads / 16);
    const long long cap = static_cast<long long>(num_sms) * 8;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_swiglu_quantize(const uint16_t* z, int rows, int F, uint8_t* a_fp8,
                                   uint8_t* a_scale, uint8_t* z_fp8, uint8_t* z_scale, int num_sms,
                                   cudaStream_t stream) {
    const long long groups = static_cast<long long>(rows) * (F / kGroup);
    swiglu_quantize_kernel<<<grid_blocks(groups, num_sms), kThreads, 0, stream>>>(
        z, groups, F, a_fp8, a_scale, z_fp8, z_scale);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* z_fp8, const uint8_t* z_scale,
                              int rows, int F, uint16_t* dz, int num_sms, cudaStream_t stream) {
    const long long groups = static_cast<long long>(rows) * (F / kGroup);
    swiglu_bwd_kernel<<<grid_blocks(groups, num_sms), kThreads, 0, stream>>>(
        dh, z_fp8, z_scale, groups, F, dz);
    return cudaGetLastError();
}

}  // namespace hg

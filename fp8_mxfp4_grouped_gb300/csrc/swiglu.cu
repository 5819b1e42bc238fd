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
// What bounds both is memory, once the arithmetic is short enough: per element
// of h the forward moves 7 bytes (5 without the checkpoint), the backward 8.  A
// group of 128 belongs to one warp, four elements a lane, so that its largest
// magnitude is one warp-wide reduction instruction away and nothing is read
// twice; each warp has two groups under way.  exp is 2^x of the hardware and
// the reciprocal its approximation: off by some 2^-22 of the value, and by
// |g| * 2^-24 of it for the rounding of the exponent, against the formats'
// 2^-4 and 2^-8.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128;
constexpr int kUnder = 2;                    // groups under way per warp

// 1 / (1 + exp(-g)).  exp overflows to infinity below g = -88 and the result
// is 0 there; between -87.3 and -88 it is subnormal, which rcp keeps.
__device__ __forceinline__ float sigmoid(float g) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

// Where the warps' walk over groups (row r, group g) has come to: every
// `step`-th group of the rows in order.
struct Walk {
    int r, g;
    __device__ Walk(int first, int G) : r(first / G), g(first - first / G * G) {}
    __device__ void next(int step_r, int step_g, int G) {
        r += step_r;
        g += step_g;
        if (g >= G) {
            g -= G;
            ++r;
        }
    }
};

// Four elements a lane of a group -> four E4M3 codes and the group's scale.
__device__ __forceinline__ uint32_t quantize4(const float (&f)[4], uint32_t& scale) {
    const float top = warp_abs_max(max_nan(max_nan(fabsf(f[0]), fabsf(f[1])),
                                           max_nan(fabsf(f[2]), fabsf(f[3]))));
    scale = e8m0_scale_code(top);
    const float inv = scale == 255u ? __uint_as_float(0x7FC00000u)      // every code becomes NaN
                                    : __uint_as_float((254u - scale) << 23);
    return e4m3_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
}

template <bool kCheckpoint>
__global__ void __launch_bounds__(kThreads)
swiglu_quantize_kernel(const uint16_t* __restrict__ z, int rows, int F,
                       uint8_t* __restrict__ a_fp8, uint8_t* __restrict__ a_scale,
                       uint8_t* __restrict__ z_fp8, uint8_t* __restrict__ z_scale) {
    const int G = F / kGroup;
    const int lane = threadIdx.x & 31;
    const int step = gridDim.x * (kThreads / 32);
    const int step_r = step / G, step_g = step - step_r * G;
    Walk at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), G);
    while (at.r < rows) {
        int r[kUnder], g[kUnder];
        uint2 vg[kUnder], vu[kUnder];
#pragma unroll
        for (int k = 0; k < kUnder; ++k) {
            r[k] = at.r;
            g[k] = at.g;
            at.next(step_r, step_g, G);
            vg[k] = vu[k] = make_uint2(0, 0);
            if (r[k] < rows) {
                const uint16_t* p = z + 2ll * r[k] * F + g[k] * kGroup + 4 * lane;
                vg[k] = __ldcs(reinterpret_cast<const uint2*>(p));
                vu[k] = __ldcs(reinterpret_cast<const uint2*>(p + F));
            }
        }
#pragma unroll
        for (int k = 0; k < kUnder; ++k) {
            const float fg[4] = {bf16_lo(vg[k].x), bf16_hi(vg[k].x), bf16_lo(vg[k].y),
                                 bf16_hi(vg[k].y)};
            const float fu[4] = {bf16_lo(vu[k].x), bf16_hi(vu[k].x), bf16_lo(vu[k].y),
                                 bf16_hi(vu[k].y)};
            float h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = fg[e] * sigmoid(fg[e]) * fu[e];
            if (r[k] >= rows) break;         // the whole warp
            const long long row = r[k];
            uint32_t scale;
            const uint32_t codes = quantize4(h, scale);
            *reinterpret_cast<uint32_t*>(a_fp8 + row * F + g[k] * kGroup + 4 * lane) = codes;
            if (lane == 0) a_scale[row * G + g[k]] = static_cast<uint8_t>(scale);
            if (kCheckpoint) {
                uint32_t sg, su;
                const uint32_t cg = quantize4(fg, sg);
                const uint32_t cu = quantize4(fu, su);
                uint8_t* q = z_fp8 + 2 * row * F + g[k] * kGroup + 4 * lane;
                *reinterpret_cast<uint32_t*>(q) = cg;
                *reinterpret_cast<uint32_t*>(q + F) = cu;
                if (lane < 2)
                    z_scale[(2 * row + lane) * G + g[k]] = static_cast<uint8_t>(lane ? su : sg);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads)
swiglu_bwd_kernel(const uint16_t* __restrict__ dh, const uint8_t* __restrict__ z_fp8,
                  const uint8_t* __restrict__ z_scale, int rows, int F,
                  uint16_t* __restrict__ dz) {
    const int G = F / kGroup;
    const int lane = threadIdx.x & 31;
    const int step = gridDim.x * (kThreads / 32);
    const int step_r = step / G, step_g = step - step_r * G;
    Walk at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), G);
    while (at.r < rows) {
        int r[kUnder], g[kUnder];
        uint2 vd[kUnder];
        uint32_t vg[kUnder], vu[kUnder], sg[kUnder], su[kUnder];
#pragma unroll
        for (int k = 0; k < kUnder; ++k) {
            r[k] = at.r;
            g[k] = at.g;
            at.next(step_r, step_g, G);
            vd[k] = make_uint2(0, 0);
            vg[k] = vu[k] = sg[k] = su[k] = 0;
            if (r[k] < rows) {
                const long long row = r[k];
                const int col = g[k] * kGroup + 4 * lane;
                vd[k] = __ldcs(reinterpret_cast<const uint2*>(dh + row * F + col));
                vg[k] = __ldcs(reinterpret_cast<const uint32_t*>(z_fp8 + 2 * row * F + col));
                vu[k] = __ldcs(reinterpret_cast<const uint32_t*>(z_fp8 + (2 * row + 1) * F + col));
                sg[k] = __ldg(z_scale + 2 * row * G + g[k]);
                su[k] = __ldg(z_scale + (2 * row + 1) * G + g[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnder; ++k) {
            if (r[k] >= rows) break;
            const float d[4] = {bf16_lo(vd[k].x), bf16_hi(vd[k].x), bf16_lo(vd[k].y),
                                bf16_hi(vd[k].y)};
            float fg[4], fu[4], og[4], ou[4];
            e4m3_unpack4(vg[k], fg);
            e4m3_unpack4(vu[k], fu);
            const float scale_g = e8m0_value(sg[k]), scale_u = e8m0_value(su[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float gv = fg[e] * scale_g;
                const float uv = fu[e] * scale_u;
                const float s = sigmoid(gv);
                og[e] = d[e] * uv * s * (1.0f + gv * (1.0f - s));
                ou[e] = d[e] * gv * s;
            }
            uint16_t* o = dz + 2ll * r[k] * F + g[k] * kGroup + 4 * lane;
            *reinterpret_cast<uint2*>(o) = make_uint2(bf16_pack(og[0], og[1]),
                                                      bf16_pack(og[2], og[3]));
            *reinterpret_cast<uint2*>(o + F) = make_uint2(bf16_pack(ou[0], ou[1]),
                                                          bf16_pack(ou[2], ou[3]));
        }
    }
}

// Blocks: a warp for each pair of groups, at most what is resident at once.
int grid_blocks(int rows, int F, const void* kernel, int num_sms) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0) !=
            cudaSuccess ||
        per_sm < 1)
        per_sm = 1;
    const long long groups = static_cast<long long>(rows) * (F / kGroup);
    const long long per_block = kThreads / 32 * kUnder;
    const long long blocks = (groups + per_block - 1) / per_block;
    const long long cap = static_cast<long long>(num_sms) * per_sm;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_swiglu_quantize(const uint16_t* z, int rows, int F, uint8_t* a_fp8,
                                   uint8_t* a_scale, uint8_t* z_fp8, uint8_t* z_scale, int num_sms,
                                   cudaStream_t stream) {
    const auto kernel = z_fp8 ? swiglu_quantize_kernel<true> : swiglu_quantize_kernel<false>;
    const int grid = grid_blocks(rows, F, reinterpret_cast<const void*>(kernel), num_sms);
    kernel<<<grid, kThreads, 0, stream>>>(z, rows, F, a_fp8, a_scale, z_fp8, z_scale);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* z_fp8, const uint8_t* z_scale,
                              int rows, int F, uint16_t* dz, int num_sms, cudaStream_t stream) {
    const int grid = grid_blocks(rows, F, reinterpret_cast<const void*>(swiglu_bwd_kernel),
                                 num_sms);
    swiglu_bwd_kernel<<<grid, kThreads, 0, stream>>>(dh, z_fp8, z_scale, rows, F, dz);
    return cudaGetLastError();
}

}  // namespace hg

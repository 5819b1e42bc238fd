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
// group of 128 belongs to half a warp, eight elements a lane, so that its
// largest magnitude is a reduction instruction away and nothing is read twice
// (four elements a lane of a whole warp pay twice for addresses and scales:
// 390 us for 131072 x 2048 with the checkpoint; this form takes 287, 98 % of
// the measured HBM copy rate).  exp is 2^x of the hardware and
// the reciprocal its approximation: off by some 2^-22 of the value, and by
// |g| * 2^-24 of it for the rounding of the exponent, against the formats'
// 2^-4 and 2^-8.  Where s itself would leave FP32's normal numbers (g < -87), or
// dh * u or dh * g might pass its largest, the few elements concerned are computed
// again in wider steps: with a large u or dh beside a tiny s the result can be any
// number.
#include <atomic>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128;
constexpr int kBlockGroups = kThreads / 16;

// 1 / (1 + exp(-g)) of two values, for g >= kFar; 0 from about g = -87.3 down,
// where the result leaves FP32's normal numbers.
constexpr float kFar = -87.0f;
constexpr uint32_t kFarScale = 125u;         // E8M0 code from which E4M3 reaches kFar: 448 / 4
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
    const float2 t = ptx::f32x2_parts(
        ptx::mul_f32x2(g, ptx::f32x2(-1.4426950408889634f, -1.4426950408889634f)));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    const float2 d = ptx::f32x2_parts(ptx::add_f32x2(ptx::f32x2(e.x, e.y), ptx::f32x2(1.0f, 1.0f)));
    float2 s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
    return ptx::f32x2(s.x, s.y);
}

// g * s * u for g < kFar, where s is exp(g): a quarter of the exponent at a time,
// two of them with either factor, so that nothing underflows that the result does
// not.
__device__ __forceinline__ float far_silu_times(float g, float u) {
    const float q = expf(0.25f * g);
    return ((g * q) * q) * ((u * q) * q);
}

// Whether any of eight BF16 is below kFar (or a negative NaN): as numbers without
// sign the negative ones come after all others, in order of magnitude.
__device__ __forceinline__ bool any_far(const uint4 v) {
    const uint32_t two = __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w));
    constexpr uint32_t kCode = 0xC2AEu;      // of kFar
    return max(two & 0xFFFFu, two >> 16) > kCode;
}

__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) {
    return ptx::f32x2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ uint32_t bf16_pack_pair(uint64_t v) {
    const float2 f = ptx::f32x2_parts(v);
    return hg::bf16_pack(f.x, f.y);
}

// The two E4M3 codes of the low 16 bits.
__device__ __forceinline__ uint64_t e4m3_pair(uint32_t codes) {
    const float2 f = e4m3x2_to_f32(codes);
    return ptx::f32x2(f.x, f.y);
}

// A half-warp's walk over the groups of all rows, in order: group i of all, of row
// r, g-th in it.  (32 bits are enough for groups, and spare the registers that the
// flags below need: with 64, 131072 x 2048 with the checkpoint takes 296 us.)
struct Walk {
    int G, step, step_r, step_g;
    int i, r, g;
    __device__ explicit Walk(int F)
        : G(F / kGroup), step(gridDim.x * kBlockGroups), step_r(step / G),
          step_g(step - step_r * G), i(blockIdx.x * kBlockGroups + (threadIdx.x >> 4)), r(i / G),
          g(i - r * G) {}
    // where this lane's eight elements of h, of the gate and of its scale lie
    __device__ long long h_at() const {
        return static_cast<long long>(i) * kGroup + 8 * (threadIdx.x & 15);
    }
    __device__ long long z_at() const { return h_at() + static_cast<long long>(r) * G * kGroup; }
    __device__ long long scale_at() const { return i + static_cast<long long>(r) * G; }
    __device__ void next() {
        i += step;
        r += step_r;
        g += step_g;
        if (g >= G) {
            g -= G;
            ++r;
        }
    }
};

// h of all of this warp's groups that hold a gate below kFar, again.  Out of line:
// in the loop, or as a loop after it, it costs the kernel up to 9 %.
__device__ __noinline__ void far_groups(const uint16_t* z, int groups, int F, uint8_t* a_fp8,
                                        uint8_t* a_scale) {
    const int half = (threadIdx.x >> 4) & 1, j = threadIdx.x & 15;
    for (Walk at(F); at.i - half < groups; at.next()) {
        const bool real = at.i < groups;
        uint4 vg = make_uint4(0, 0, 0, 0), vu = vg;
        if (real) {
            vg = ptx::load(reinterpret_cast<const uint4*>(z + at.z_at()));
            vu = ptx::load(reinterpret_cast<const uint4*>(z + at.z_at() + F));
        }
        if (!__any_sync(0xFFFFFFFFu, any_far(vg))) continue;
        float g[8], u[8];
        bf16_unpack8(vg, g);
        bf16_unpack8(vu, u);
        uint64_t h[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint64_t g2 = ptx::f32x2(g[2 * p], g[2 * p + 1]);
            const uint64_t u2 = ptx::f32x2(u[2 * p], u[2 * p + 1]);
            const float2 v =
                ptx::f32x2_parts(ptx::mul_f32x2(ptx::mul_f32x2(g2, sigmoid2(g2)), u2));
            h[p] = ptx::f32x2(
                g[2 * p] < kFar ? far_silu_times(g[2 * p], u[2 * p]) : v.x,
                g[2 * p + 1] < kFar ? far_silu_times(g[2 * p + 1], u[2 * p + 1]) : v.y);
        }
        uint32_t scale;
        const uint2 codes = quantize8(h, half, scale);
        if (real) {
            *reinterpret_cast<uint2*>(a_fp8 + at.h_at()) = codes;
            if (j == 0) a_scale[at.i] = static_cast<uint8_t>(scale);
        }
    }
}

template <bool kCheckpoint>
__global__ void __launch_bounds__(kThreads)
swiglu_quantize_kernel(const uint16_t* z, int groups, int F, uint8_t* __restrict__ a_fp8,
                       uint8_t* __restrict__ a_scale, uint8_t* __restrict__ z_fp8,
                       uint8_t* __restrict__ z_scale) {
    __shared__ int s_far;                    // whether any gate may be below kFar
    const int half = (threadIdx.x >> 4) & 1, j = threadIdx.x & 15;
    Walk at(F);
    if (threadIdx.x == 0) s_far = 0;
    __syncthreads();
    start_dependent();
    // the group after this one is asked for before this one is worked on
    uint4 next_g = make_uint4(0, 0, 0, 0), next_u = next_g;
    auto load = [&]() {
        if (at.i >= groups) return;
        next_g = ptx::load(reinterpret_cast<const uint4*>(z + at.z_at()));
        next_u = ptx::load(reinterpret_cast<const uint4*>(z + at.z_at() + F));
    };
    load();
    while (at.i - half < groups) {
        const bool real = at.i < groups;     // the last group may have no partner
        const Walk now = at;
        const uint4 vg = next_g, vu = next_u;
        at.next();
        load();
        if (!kCheckpoint && any_far(vg)) s_far = 1;
        const uint64_t g[4] = {bf16_pair(vg.x), bf16_pair(vg.y), bf16_pair(vg.z), bf16_pair(vg.w)};
        const uint64_t u[4] = {bf16_pair(vu.x), bf16_pair(vu.y), bf16_pair(vu.z), bf16_pair(vu.w)};
        uint64_t h[4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
            h[p] = ptx::mul_f32x2(ptx::mul_f32x2(g[p], sigmoid2(g[p])), u[p]);
        uint32_t scale, sg, su;
        const uint2 codes = quantize8(h, half, scale);
        if (real) {
            *reinterpret_cast<uint2*>(a_fp8 + now.h_at()) = codes;
            if (j == 0) a_scale[now.i] = static_cast<uint8_t>(scale);
        }
        if (kCheckpoint) {
            const uint2 cg = quantize8(g, half, sg);
            if (sg >= kFarScale) s_far = 1;
            const uint2 cu = quantize8(u, half, su);
            if (real) {
                *reinterpret_cast<uint2*>(z_fp8 + now.z_at()) = cg;
                *reinterpret_cast<uint2*>(z_fp8 + now.z_at() + F) = cu;
                if (j < 2)
                    z_scale[now.scale_at() + (j ? now.G : 0)] = static_cast<uint8_t>(j ? su : sg);
            }
        }
    }
    __syncthreads();
    if (s_far) far_groups(z, groups, F, a_fp8, a_scale);
}

// The gradient's two elements in steps that nothing leaves the range of.
__device__ __forceinline__ void wide_gradient(float d, float g, float u, uint16_t* dg,
                                              uint16_t* du) {
    const float q = expf(-0.25f * fabsf(g)), e = q * q * q * q;      // e may be 0
    const float r = 1.0f / (1.0f + e);
    const double e_wide = static_cast<double>(q) * q * q * q;
    const double s = g < 0.0f ? e_wide * r : static_cast<double>(r);
    const float slope = fmaf(g, g < 0.0f ? r : e * r, 1.0f);         // 1 + g (1 - s)
    const double ds = s * d;
    *dg = __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<float>(ds * u * slope)));
    *du = __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<float>(ds * g)));
}

__global__ void __launch_bounds__(kThreads)
swiglu_bwd_kernel(const uint16_t* dh, const uint8_t* z_fp8, const uint8_t* z_scale, int groups,
                  int F, uint16_t* __restrict__ dz) {
    const uint64_t one = ptx::f32x2(1.0f, 1.0f), minus = ptx::f32x2(-1.0f, -1.0f);
    start_dependent();
    bool wide = false;                       // whether any element may need wide_gradient
    // eight elements of three inputs are enough loads under way: asking ahead as
    // above costs registers and with them warps (24.7 -> 25.9 us at 9223 x 2048)
    for (Walk at(F); at.i < groups; at.next()) {
        const long long z_at = at.z_at();
        const uint8_t* s_at = z_scale + at.scale_at();
        const uint4 vd = ptx::load(reinterpret_cast<const uint4*>(dh + at.h_at()));
        const uint2 vg = ptx::load(reinterpret_cast<const uint2*>(z_fp8 + z_at));
        const uint2 vu = ptx::load(reinterpret_cast<const uint2*>(z_fp8 + z_at + F));
        const float scale_g = e8m0_value(ptx::load(s_at));
        const float scale_u = e8m0_value(ptx::load(s_at + at.G));
        const uint64_t sg = ptx::f32x2(scale_g, scale_g), su = ptx::f32x2(scale_u, scale_u);
        uint32_t og[4], ou[4];
        float d_max = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint64_t d = bf16_pair(p == 0 ? vd.x : p == 1 ? vd.y : p == 2 ? vd.z : vd.w);
            const float2 d_parts = ptx::f32x2_parts(d);
            d_max = fmaxf(fmaxf(d_max, fabsf(d_parts.x)), fabsf(d_parts.y));
            const uint64_t g = ptx::mul_f32x2(e4m3_pair((p < 2 ? vg.x : vg.y) >> 16 * (p & 1)), sg);
            const uint64_t u = ptx::mul_f32x2(e4m3_pair((p < 2 ? vu.x : vu.y) >> 16 * (p & 1)), su);
            const uint64_t s = sigmoid2(g);
            const uint64_t slope = ptx::fma_f32x2(g, ptx::fma_f32x2(s, minus, one), one);
            og[p] = bf16_pack_pair(ptx::mul_f32x2(ptx::mul_f32x2(ptx::mul_f32x2(d, u), s), slope));
            ou[p] = bf16_pack_pair(ptx::mul_f32x2(ptx::mul_f32x2(d, g), s));
        }
        *reinterpret_cast<uint4*>(dz + z_at) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(dz + z_at + F) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        // only from these scales on can g be below kFar, or a product with dh pass
        // 2^120 (448 < 2^9)
        wide |= scale_g >= 0.25f || d_max * fmaxf(scale_g, scale_u) >= 0x1p111f;
    }
    if (!wide) return;                       // rare: those elements again, one by one
    for (Walk at(F); at.i < groups; at.next()) {
        const long long z_at = at.z_at();
        const uint8_t* s_at = z_scale + at.scale_at();
        const float scale_g = e8m0_value(ptx::load(s_at));
        const float scale_u = e8m0_value(ptx::load(s_at + at.G));
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const float d = bf16_lo(ptx::load(dh + at.h_at() + i));
            const float g = e4m3x2_to_f32(ptx::load(z_fp8 + z_at + i)).x * scale_g;
            const float u = e4m3x2_to_f32(ptx::load(z_fp8 + z_at + F + i)).x * scale_u;
            if (g < kFar || !(fabsf(d) * fmaxf(fabsf(g), fabsf(u)) < 0x1p120f))
                wide_gradient(d, g, u, dz + z_at + i, dz + z_at + F + i);
        }
    }
}

// Blocks: a half-warp for each group, at most what is resident at once (asked
// for once per kernel: it is a property of the code and of sm_103a).
int grid_blocks(int groups, const void* kernel, std::atomic<int>& known, int num_sms) {
    int per_sm = known.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0) !=
                cudaSuccess ||
            per_sm < 1)
            per_sm = 1;
        known.store(per_sm, std::memory_order_relaxed);
    }
    const int blocks = (groups + kBlockGroups - 1) / kBlockGroups, cap = num_sms * per_sm;
    return blocks < cap ? blocks : cap;
}

}  // namespace

// Groups at most: walks step past the last by less than the grid's half-warps.
int swiglu_max_groups() { return 0x7FFFFFFF - (1 << 20); }

cudaError_t launch_swiglu_quantize(const uint16_t* z, int rows, int F, uint8_t* a_fp8,
                                   uint8_t* a_scale, uint8_t* z_fp8, uint8_t* z_scale, int num_sms,
                                   cudaStream_t stream) {
    const auto kernel = z_fp8 ? swiglu_quantize_kernel<true> : swiglu_quantize_kernel<false>;
    static std::atomic<int> known[2];
    const int groups = rows * (F / kGroup);
    const int grid = grid_blocks(groups, reinterpret_cast<const void*>(kernel),
                                 known[z_fp8 != nullptr], num_sms);
    return launch_dependent(kernel, grid, kThreads, 0, stream, z, groups, F, a_fp8, a_scale, z_fp8,
                            z_scale);
}

cudaError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* z_fp8, const uint8_t* z_scale,
                              int rows, int F, uint16_t* dz, int num_sms, cudaStream_t stream) {
    static std::atomic<int> known;
    const int groups = rows * (F / kGroup);
    const int grid =
        grid_blocks(groups, reinterpret_cast<const void*>(swiglu_bwd_kernel), known, num_sms);
    return launch_dependent(swiglu_bwd_kernel, grid, kThreads, 0, stream, dh, z_fp8, z_scale,
                            groups, F, dz);
}

}  // namespace hg

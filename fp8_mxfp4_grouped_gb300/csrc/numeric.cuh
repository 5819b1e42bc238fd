// numeric.cuh -- element conversions shared by the kernels around the GEMM:
// the E8M0 scale rule of the activations, and BF16 pairs in 32-bit words.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx.cuh"

namespace hg {

// Value of an E8M0 code: 2^(code - 127); code 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
    const uint32_t bits = code == 0u ? 0x00400000u : code << 23;   // 2^-127 is subnormal
    return __uint_as_float(code == 255u ? 0x7FC00000u : bits);
}

// Values of the two E4M3 codes of the low 16 bits (the low byte first).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four floats as E4M3 codes, round to nearest even; finite values beyond the
// range saturate, NaN becomes NaN.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Larger of two floats; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Largest value over the warp, NaN aside.
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// Largest magnitude over the warp; NaN if any is.
__device__ __forceinline__ float warp_abs_max(float v) {
    float m;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// E8M0 code of the scale of a group whose largest magnitude is amax, from its bits
// (exact, no floating-point division or logarithm): 127 + e with e the smallest
// integer such that amax <= 448 * 2^e = 1.75 * 2^(e + 8), clamped to codes from 0
// (the carry of the addition is the step from 1.75 to the next power of two); 127
// for amax = 0, 255 (NaN) for an Inf or NaN.
__device__ __forceinline__ uint32_t e8m0_scale_code(float amax) {
    const uint32_t bits = __float_as_uint(amax) & 0x7FFFFFFFu;
    const int code = static_cast<int>((bits + 0x1FFFFFu) >> 23) - 8;
    if (bits >= 0x7F800000u) return 255u;
    return bits == 0u ? 127u : static_cast<uint32_t>(max(code, 0));
}

// The two BF16 values of a 32-bit word (element 2i in the low half).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats rounded to nearest even into one word of BF16.
__device__ __forceinline__ uint32_t bf16_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void bf16_unpack8(const uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 bf16_pack8(const float (&f)[8]) {
    return make_uint4(bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]),
                      bf16_pack(f[6], f[7]));
}

struct GroupCodes {
    uint32_t lo, hi;        // this lane's 8 E4M3 codes
    uint8_t scale;          // the group's E8M0 code
};

// Lane j of a half-warp holds elements 8j .. 8j+7 of one 128-element group;
// every lane of the warp must call this (the amax reduction shuffles).
__device__ __forceinline__ GroupCodes quantize_codes(const uint4 v) {
    float f[8];
    bf16_unpack8(v, f);
    float amax = 0.0f;                             // NaN if any element is
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    GroupCodes c;
    c.scale = static_cast<uint8_t>(e8m0_scale_code(amax));
    if (c.scale == 255u) {                         // an Inf or NaN: all of the group NaN
        c.lo = c.hi = 0x7F7F7F7Fu;
    } else {
        // 2^-e from its bits: finite inputs give codes up to 247, so that the
        // biased exponent 254 - code stays in [7, 254] (a normal float).
        const float inv = __uint_as_float((254u - c.scale) << 23);
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            b[i] = __nv_cvt_float_to_fp8(f[i] * inv, __NV_SATFINITE, __NV_E4M3);
        }
        c.lo = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
        c.hi = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
    }
    return c;
}

// Eight elements a lane of each half-warp's group -> eight E4M3 codes and the
// group's scale.  Every lane of the warp takes part.
__device__ __forceinline__ uint2 quantize8(const uint64_t (&f)[4], int half, uint32_t& scale) {
    float top = 0.0f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float2 v = ptx::f32x2_parts(f[p]);
        top = max_nan(top, max_nan(fabsf(v.x), fabsf(v.y)));
    }
    const float top0 = warp_abs_max(half ? 0.0f : top), top1 = warp_abs_max(half ? top : 0.0f);
    scale = e8m0_scale_code(half ? top1 : top0);
    const float inv = scale == 255u ? __uint_as_float(0x7FC00000u)      // every code becomes NaN
                                    : __uint_as_float((254u - scale) << 23);
    const uint64_t inv2 = ptx::f32x2(inv, inv);
    float2 q[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) q[p] = ptx::f32x2_parts(ptx::mul_f32x2(f[p], inv2));
    return make_uint2(e4m3_pack4(q[0].x, q[0].y, q[1].x, q[1].y),
                      e4m3_pack4(q[2].x, q[2].y, q[3].x, q[3].y));
}

// E8M0 code of the scale of 32 weights whose largest magnitude is amax: as above with
// 6 = 1.5 * 2^2 for E2M1 in the place of 448.
__device__ __forceinline__ uint32_t e8m0_weight_scale_code(float amax) {
    const uint32_t bits = __float_as_uint(amax) & 0x7FFFFFFFu;
    const int code = static_cast<int>((bits + 0x3FFFFFu) >> 23) - 2;
    if (bits >= 0x7F800000u) return 255u;
    return bits == 0u ? 127u : static_cast<uint32_t>(max(code, 0));
}

// Eight floats as E2M1 codes, round to nearest, ties to the even code, the first in
// the lowest four bits.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&f)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

}  // namespace hg

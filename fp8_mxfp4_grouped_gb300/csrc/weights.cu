// weights.cu -- BF16 or FP32 weights [E, N, K] as MXFP4: E2M1 codes, two to a byte, with
// one E8M0 scale per 32 of them along K (what the GEMM reads), and in the same pass along
// N (the transposed copy that the gradient of the activations goes through); and 4-bit
// weights back as numbers.  Per group of 32:
//
//   e = smallest integer with amax <= 6 * 2^e (0 for amax = 0), in [-127, 127]
//   code = nearest E2M1 value of w / 2^e, ties to the even code; scale = 127 + e
//
// Along K alone and back it is bound by memory: 32 x 4096 x 6144 from BF16 278 us (7.3 TB/s),
// from FP32 494; back to BF16 292 us, to FP32 525 (7.0 TB/s).  In both orientations 428 us from
// BF16 (5.8 TB/s; the ALU pipe is busy for 59 % of the time) and 691 from FP32 (5.9): the tiles
// of a persistent grid copied ahead into shared memory took 630 and 736.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kGroup = 32;
constexpr int kThreads = 256;

// 1 / scale; finite groups have codes up to 253.
__device__ __forceinline__ float inverse(uint32_t code) {
    return __uint_as_float((254u - code) << 23);
}
// (of code 255: any BF16, and nothing beyond its bits)
__device__ __forceinline__ uint32_t inverse_bf16(uint32_t code) {
    return ((254u - code) << 7) & 0xFFFFu;
}

// Eight consecutive weights, FP32 or BF16.  BF16 are taken two at a time where they can be,
// and away from the pipe of the integer instructions, comparisons and conversions, which
// bounds the kernel that quantises in both orientations: 32 x 4096 x 6144 in 615 us with
// every weight widened, 428 so.
//
// A lane holds kPieces of eight consecutive weights, 4 / kPieces lanes a group.
template <class T, int kPieces>
struct Run;

template <int kPieces>
struct Run<float, kPieces> {
    float f[kPieces][8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kPieces * 8; ++i) f[i / 8][i % 8] = 0.0f;
    }
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int h = 0; h < 2 * kPieces; ++h) {
            const uint4 v = ptx::load(reinterpret_cast<const uint4*>(p) + h);
            f[h / 2][h % 2 * 4] = __uint_as_float(v.x);
            f[h / 2][h % 2 * 4 + 1] = __uint_as_float(v.y);
            f[h / 2][h % 2 * 4 + 2] = __uint_as_float(v.z);
            f[h / 2][h % 2 * 4 + 3] = __uint_as_float(v.w);
        }
    }
    static constexpr int kWords = 8;         // of a piece
    __device__ __forceinline__ void store(int p, uint32_t* to) const {
        reinterpret_cast<float4*>(to)[0] = make_float4(f[p][0], f[p][1], f[p][2], f[p][3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[p][4], f[p][5], f[p][6], f[p][7]);
    }
    // E8M0 code of the group's scale
    __device__ __forceinline__ uint32_t scale() const {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kPieces * 8; ++i) m = max_nan(m, fabsf(f[i / 8][i % 8]));
#pragma unroll
        for (int o = 1; o < 4 / kPieces; o *= 2)
            m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        return e8m0_weight_scale_code(m);
    }
    __device__ __forceinline__ void codes(uint32_t scale, uint32_t (&c)[kPieces]) const {
        const float inv = inverse(scale);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = f[p][i] * inv;
            c[p] = scale == 255u ? 0u : e2m1_pack8(q);
        }
    }
};

// Larger magnitudes of pairs, whatever their signs; NaN if either is.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
// The two of a word times the two of another, in FP32, -0 staying -0.
__device__ __forceinline__ float2 scaled2(uint32_t w, uint32_t by) {
    float2 f;
    asm("{\n\t.reg .b16 lo, hi, i, j;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b32 {i, j}, %3;\n\t"
        "fma.rn.f32.bf16 %0, lo, i, 0f80000000;\n\tfma.rn.f32.bf16 %1, hi, j, 0f80000000;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(w), "r"(by));
    return f;
}

template <int kPieces>
struct Run<uint16_t, kPieces> {
    uint4 v[kPieces];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) v[p] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const uint16_t* from) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
            v[p] = ptx::load(reinterpret_cast<const uint4*>(from) + p);
    }
    static constexpr int kWords = 4;         // of a piece
    __device__ __forceinline__ void store(int p, uint32_t* to) const {
        *reinterpret_cast<uint4*>(to) = v[p];
    }
    __device__ __forceinline__ uint32_t scale() const {
        uint32_t m = abs_max2(abs_max2(v[0].x, v[0].y), abs_max2(v[0].z, v[0].w));
#pragma unroll
        for (int p = 1; p < kPieces; ++p)
            m = abs_max2(m, abs_max2(abs_max2(v[p].x, v[p].y), abs_max2(v[p].z, v[p].w)));
        // the other half too, then the other lanes
        m = abs_max2(m, __byte_perm(m, 0u, 0x1032));
#pragma unroll
        for (int o = 1; o < 4 / kPieces; o *= 2)
            m = abs_max2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        return e8m0_weight_scale_code(bf16_lo(m));       // which does not ask for the sign
    }
    __device__ __forceinline__ void codes(uint32_t scale, uint32_t (&c)[kPieces]) const {
        const uint32_t inv = inverse_bf16(scale) * 0x10001u;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
            float q[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = scaled2(w[i], inv);
                q[2 * i] = f.x;
                q[2 * i + 1] = f.y;
            }
            c[p] = scale == 255u ? 0u : e2m1_pack8(q);
        }
    }
};

// Along K alone the rows of all experts are one run of groups: eight weights a lane,
// kBatch of them in flight.
constexpr int kBatch = 4;

template <class T>
__global__ void __launch_bounds__(kThreads)
quantize_weights_kernel(const T* w, long long pieces, uint8_t* q, uint8_t* scale) {
    start_dependent();
    const int lane = threadIdx.x & 31;
    const long long warp = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    Run<T, 1> f[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p = (warp * kBatch + b) * 32 + lane;
        f[b].clear();
        if (p < pieces) f[b].load(w + 8 * p);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p = (warp * kBatch + b) * 32 + lane;
        const uint32_t code = f[b].scale();
        if (p >= pieces) continue;
        uint32_t c[1];
        f[b].codes(code, c);
        reinterpret_cast<uint32_t*>(q)[p] = c[0];
        if ((lane & 3) == 0) scale[p / 4] = static_cast<uint8_t>(code);
    }
}

// Both orientations: a tile of 128 rows (four groups along N) and 256 bytes a row goes
// through registers, where its rows are quantised, into shared memory, where a thread
// takes 32 rows of one 32-bit word's column(s).
constexpr int kTileRows = 128;

template <class T>
struct Tile {
    static constexpr int kCols = 256 / sizeof(T);
    static constexpr int kPerWord = 4 / sizeof(T);
    // 32-bit word w of row r; the groups of rows differ in their banks
    static __device__ __forceinline__ int word(int r, int w) {
        return r * 64 + (w ^ (8 * (r / kGroup)));
    }
};

// The 32 words of a column of FP32, or of two columns of BF16: codes and scales.
__device__ __forceinline__ void column_codes(const uint32_t (&w)[kGroup], uint4 (&codes)[1],
                                             uint32_t (&scale)[1]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) amax = max_nan(amax, fabsf(__uint_as_float(w[i])));
    scale[0] = e8m0_weight_scale_code(amax);
    const float inv = inverse(scale[0]);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = __uint_as_float(w[8 * i + j]) * inv;
        c[i] = scale[0] == 255u ? 0u : e2m1_pack8(q);
    }
    codes[0] = make_uint4(c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ void column_codes(const uint32_t (&w)[kGroup], uint4 (&codes)[2],
                                             uint32_t (&scale)[2]) {
    uint32_t amax = w[0];
#pragma unroll
    for (int i = 1; i < kGroup; ++i) amax = abs_max2(amax, w[i]);
    scale[0] = e8m0_weight_scale_code(bf16_lo(amax));    // which does not ask for the sign
    scale[1] = e8m0_weight_scale_code(bf16_hi(amax));
    const uint32_t inv = inverse_bf16(scale[0]) | (inverse_bf16(scale[1]) << 16);
    uint32_t c[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 q = scaled2(w[8 * i + j], inv);
            lo[j] = q.x;
            hi[j] = q.y;
        }
        c[0][i] = scale[0] == 255u ? 0u : e2m1_pack8(lo);
        c[1][i] = scale[1] == 255u ? 0u : e2m1_pack8(hi);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) codes[h] = make_uint4(c[h][0], c[h][1], c[h][2], c[h][3]);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4)
quantize_weights_both_kernel(const T* w, int N, int K, int tiles_n, int tiles_k, uint8_t* q,
                             uint8_t* scale, uint8_t* qt, uint8_t* scale_t) {
    using Tl = Tile<T>;
    __shared__ __align__(16) uint32_t s[kTileRows * 64];
    start_dependent();
    const int tn = blockIdx.x % tiles_n, tk = blockIdx.x / tiles_n % tiles_k;
    const long long e = blockIdx.x / tiles_n / tiles_k;
    const int n0 = tn * kTileRows, k0 = tk * Tl::kCols;
    // BF16: sixteen weights a lane, so that two share the work of a scale (428 us, with eight
    // 511); FP32: eight, since with sixteen a load instruction's lanes lie 64 bytes apart (917
    // against 690 us)
    constexpr int kPer = sizeof(T) == 2 ? 2 : 1, kAhead = 4;
    constexpr int kLanes = Tl::kCols / (8 * kPer), kRowsAtOnce = kThreads / kLanes;
    constexpr int kSteps = kTileRows / kRowsAtOnce;
    const int piece = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
    const int k = k0 + 8 * kPer * piece;
    const long long first = (e * N + n0 + r0) * K + k;
#pragma unroll
    for (int b0 = 0; b0 < kSteps; b0 += kAhead) {
        Run<T, kPer> f[kAhead];
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
            const int r = (b0 + b) * kRowsAtOnce;
            f[b].clear();
            if (n0 + r0 + r < N && k < K) f[b].load(w + first + static_cast<long long>(r) * K);
        }
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
            const int r = (b0 + b) * kRowsAtOnce;
            const uint32_t code = f[b].scale();
            if (n0 + r0 + r < N && k < K) {
                const long long at = first + static_cast<long long>(r) * K;
                uint32_t c[kPer];
                f[b].codes(code, c);
                if constexpr (kPer == 2) {
                    *reinterpret_cast<uint2*>(q + at / 2) = make_uint2(c[0], c[1]);
                } else {
                    *reinterpret_cast<uint32_t*>(q + at / 2) = c[0];
                }
                if (piece % (4 / kPer) == 0) scale[at / kGroup] = static_cast<uint8_t>(code);
            }
            // (the swizzle keeps runs of eight words)
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                f[b].store(p, &s[Tl::word(r0 + r, (kPer * piece + p) * Run<T, kPer>::kWords)]);
        }
    }
    __syncthreads();
    // lane = (group of rows, word): four lanes write 64 bytes of a column's codes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane & 3, word = 8 * warp + (lane >> 2);
    const int n = n0 + g * kGroup, col = k0 + word * Tl::kPerWord;
    if (n >= N || col >= K) return;
    uint32_t v[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) v[i] = s[Tl::word(g * kGroup + i, word)];
    uint4 codes[Tl::kPerWord];
    uint32_t code[Tl::kPerWord];
    column_codes(v, codes, code);
#pragma unroll
    for (int h = 0; h < Tl::kPerWord; ++h) {
        const long long at = (e * K + col + h) * N + n;
        *reinterpret_cast<uint4*>(qt + at / 2) = codes[h];
        scale_t[at / kGroup] = static_cast<uint8_t>(code[h]);
    }
}

// Eight E2M1 values in FP16 times a scale's.
__device__ __forceinline__ void decode(uint32_t (&h)[4], float value, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = v.x * value;
        f[2 * i + 1] = v.y * value;
    }
}

// A warp's 256 consecutive weights from the lanes' eight codes each and their scales, of the
// lanes with `mine`.  Every lane takes part.
__device__ __forceinline__ void store256(uint16_t* w, uint32_t codes, float value, bool mine) {
    uint32_t h[4];
    ptx::e2m1x8_to_f16(codes, h);
    float f[8];
    decode(h, value, f);
    if (mine) reinterpret_cast<uint4*>(w)[threadIdx.x & 31] = bf16_pack8(f);
}
// FP32: a lane's eight would be 32 bytes, of which an instruction stores 16: the lanes
// exchange halves, so that 32 lanes store 512 consecutive bytes twice.
__device__ __forceinline__ void store256(float* w, uint32_t codes, float value, bool mine) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int from = 16 * j + lane / 2;
        const uint32_t c = __shfl_sync(0xFFFFFFFFu, codes, from);
        const float v = __shfl_sync(0xFFFFFFFFu, value, from);
        const bool there = __shfl_sync(0xFFFFFFFFu, mine, from);
        uint32_t h[4];
        ptx::e2m1x8_to_f16(lane & 1 ? c >> 16 : c & 0xFFFFu, h);
        float f[8];
        decode(h, v, f);
        if (there) reinterpret_cast<float4*>(w)[32 * j + lane] = make_float4(f[0], f[1], f[2], f[3]);
    }
}

// Eight codes a lane, kBatch times.
template <class T>
__global__ void __launch_bounds__(kThreads)
dequantize_weights_kernel(const uint8_t* q, const uint8_t* scale, long long pieces, T* w) {
    start_dependent();
    const int lane = threadIdx.x & 31;
    const long long warp = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    uint32_t c[kBatch], code[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p = (warp * kBatch + b) * 32 + lane;
        c[b] = code[b] = 0u;
        if (p >= pieces) continue;
        c[b] = ptx::load(reinterpret_cast<const uint32_t*>(q) + p);
        code[b] = ptx::load(scale + p / 4);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p0 = (warp * kBatch + b) * 32;
        store256(w + 8 * p0, c[b], e8m0_value(code[b]), p0 + lane < pieces);
    }
}

int flat_blocks(long long pieces) {
    const long long per_block = static_cast<long long>(kThreads) * kBatch;
    return static_cast<int>((pieces + per_block - 1) / per_block);
}

template <class T>
cudaError_t quantize(const T* w, int E, int N, int K, uint8_t* q, uint8_t* scale, uint8_t* qt,
                     uint8_t* scale_t, cudaStream_t stream) {
    if (!qt) {
        const long long pieces = static_cast<long long>(E) * N * (K / 8);
        return launch_dependent(quantize_weights_kernel<T>, flat_blocks(pieces), kThreads, 0,
                                stream, w, pieces, q, scale);
    }
    const int tiles_n = (N + kTileRows - 1) / kTileRows;
    const int tiles_k = (K + Tile<T>::kCols - 1) / Tile<T>::kCols;
    return launch_dependent(quantize_weights_both_kernel<T>, E * tiles_n * tiles_k, kThreads, 0,
                            stream, w, N, K, tiles_n, tiles_k, q, scale, qt, scale_t);
}

}  // namespace

cudaError_t launch_quantize_weights(const void* w, bool f32, int E, int N, int K, uint8_t* q,
                                    uint8_t* scale, uint8_t* qt, uint8_t* scale_t,
                                    cudaStream_t stream) {
    return f32 ? quantize(static_cast<const float*>(w), E, N, K, q, scale, qt, scale_t, stream)
               : quantize(static_cast<const uint16_t*>(w), E, N, K, q, scale, qt, scale_t, stream);
}

cudaError_t launch_dequantize_weights(const uint8_t* q, const uint8_t* scale, int E, int N, int K,
                                      void* w, bool f32, cudaStream_t stream) {
    const long long pieces = static_cast<long long>(E) * N * (K / 8);
    return f32 ? launch_dependent(dequantize_weights_kernel<float>, flat_blocks(pieces), kThreads,
                                  0, stream, q, scale, pieces, static_cast<float*>(w))
               : launch_dependent(dequantize_weights_kernel<uint16_t>, flat_blocks(pieces),
                                  kThreads, 0, stream, q, scale, pieces,
                                  static_cast<uint16_t*>(w));
}

}  // namespace hg

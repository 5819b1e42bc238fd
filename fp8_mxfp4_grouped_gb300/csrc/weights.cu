// weights.cu -- BF16 or FP32 weights [E, N, K] as MXFP4: E2M1 codes, two to a byte, with
// one E8M0 scale per 32 of them along K (what the GEMM reads), and in the same pass along
// N (the transposed copy that the gradient of the activations goes through); and 4-bit
// weights back as numbers.  Per group of 32:
//
//   e = smallest integer with amax <= 6 * 2^e (0 for amax = 0), in [-127, 127]
//   code = nearest E2M1 value of w / 2^e, ties to the even code; scale = 127 + e
//
// Both directions are bound by memory.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kGroup = 32;
constexpr int kThreads = 256;

// Eight consecutive weights in FP32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
    bf16_unpack8(ptx::load(reinterpret_cast<const uint4*>(p)), f);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 v = ptx::load(reinterpret_cast<const uint4*>(p) + h);
        f[4 * h] = __uint_as_float(v.x);
        f[4 * h + 1] = __uint_as_float(v.y);
        f[4 * h + 2] = __uint_as_float(v.z);
        f[4 * h + 3] = __uint_as_float(v.w);
    }
}

// 1 / scale; finite groups have codes up to 253.
__device__ __forceinline__ float inverse(uint32_t code) {
    return __uint_as_float((254u - code) << 23);
}

// Codes of eight of a group's weights and the group's scale; the group's largest
// magnitude is amax (NaN if any weight is).
__device__ __forceinline__ uint32_t codes8(const float (&f)[8], float amax, uint32_t& scale) {
    scale = e8m0_weight_scale_code(amax);
    if (scale == 255u) return 0u;
    const float inv = inverse(scale);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = f[i] * inv;
    return e2m1_pack8(q);
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
    return m;
}

// Four lanes hold a group.
__device__ __forceinline__ float quad_max(float m) {
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// Along K alone the rows of all experts are one run of groups: eight weights a lane,
// kBatch of them in flight.
constexpr int kBatch = 4;

template <class T>
__global__ void __launch_bounds__(kThreads)
quantize_weights_kernel(const T* w, long long pieces, uint8_t* q, uint8_t* scale) {
    start_dependent();
    const int lane = threadIdx.x & 31;
    const long long warp = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    float f[kBatch][8];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p = (warp * kBatch + b) * 32 + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[b][i] = 0.0f;
        if (p < pieces) load8(w + 8 * p, f[b]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const long long p = (warp * kBatch + b) * 32 + lane;
        uint32_t code;
        const uint32_t c = codes8(f[b], quad_max(amax8(f[b])), code);
        if (p >= pieces) continue;
        reinterpret_cast<uint32_t*>(q)[p] = c;
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
    static constexpr int kPieces = kCols / 8;            // of a row
    static constexpr int kPerWord = 4 / sizeof(T);
    // 32-bit word w of row r; the groups of rows differ in their banks
    static __device__ __forceinline__ int word(int r, int w) {
        return r * 64 + (w ^ (8 * (r / kGroup)));
    }
};

__device__ __forceinline__ void word_values(uint32_t w, float (&v)[2], const uint16_t*) {
    v[0] = bf16_lo(w);
    v[1] = bf16_hi(w);
}
__device__ __forceinline__ void word_values(uint32_t w, float (&v)[2], const float*) {
    v[0] = __uint_as_float(w);
}

template <class T>
__global__ void __launch_bounds__(kThreads)
quantize_weights_both_kernel(const T* w, int N, int K, int tiles_n, int tiles_k, uint8_t* q,
                             uint8_t* scale, uint8_t* qt, uint8_t* scale_t) {
    using Tl = Tile<T>;
    __shared__ __align__(16) uint32_t s[kTileRows * 64];
    start_dependent();
    const long long tile = blockIdx.x;
    const int tn = static_cast<int>(tile % tiles_n);
    const int tk = static_cast<int>(tile / tiles_n % tiles_k);
    const long long e = tile / tiles_n / tiles_k;
    const int n0 = tn * kTileRows, k0 = tk * Tl::kCols;
    const T* we = w + e * N * K;
    constexpr int kRowsAtOnce = kThreads / Tl::kPieces, kSteps = kTileRows / kRowsAtOnce;
    const int piece = threadIdx.x % Tl::kPieces, r0 = threadIdx.x / Tl::kPieces;
    const int k = k0 + 8 * piece;
#pragma unroll
    for (int b0 = 0; b0 < kSteps; b0 += kBatch) {
        float f[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int n = n0 + r0 + (b0 + b) * kRowsAtOnce;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[b][i] = 0.0f;
            if (n < N && k < K) load8(we + static_cast<long long>(n) * K + k, f[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + (b0 + b) * kRowsAtOnce, n = n0 + r;
            uint32_t code;
            const uint32_t c = codes8(f[b], quad_max(amax8(f[b])), code);
            if (n < N && k < K) {
                const long long at = (e * N + n) * K + k;
                *reinterpret_cast<uint32_t*>(q + at / 2) = c;
                if (piece % 4 == 0) scale[at / kGroup] = static_cast<uint8_t>(code);
            }
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(&s[Tl::word(r, 4 * piece)]) = bf16_pack8(f[b]);
            } else {
                *reinterpret_cast<float4*>(&s[Tl::word(r, 8 * piece)]) =
                    make_float4(f[b][0], f[b][1], f[b][2], f[b][3]);
                *reinterpret_cast<float4*>(&s[Tl::word(r, 8 * piece + 4)]) =
                    make_float4(f[b][4], f[b][5], f[b][6], f[b][7]);
            }
        }
    }
    __syncthreads();
    // lane = (group of rows, word): four lanes write 64 bytes of a column's codes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane & 3, word = 8 * warp + (lane >> 2);
    const int n = n0 + g * kGroup;
    if (n >= N) return;
#pragma unroll
    for (int h = 0; h < Tl::kPerWord; ++h) {
        const int col = k0 + word * Tl::kPerWord + h;
        if (col >= K) return;
        float f[4][8], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            float v[2];
            word_values(s[Tl::word(g * kGroup + i, word)], v, w);
            f[i / 8][i % 8] = v[h];
            amax = max_nan(amax, fabsf(v[h]));
        }
        uint32_t code = 0, c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = codes8(f[i], amax, code);
        const long long at = (e * K + col) * N + n;
        *reinterpret_cast<uint4*>(qt + at / 2) = make_uint4(c[0], c[1], c[2], c[3]);
        scale_t[at / kGroup] = static_cast<uint8_t>(code);
    }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = bf16_pack8(f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
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
        const long long p = (warp * kBatch + b) * 32 + lane;
        if (p >= pieces) continue;
        const float value = e8m0_value(code[b]);
        uint32_t h[4];
        ptx::e2m1x8_to_f16(c[b], h);
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            f[2 * i] = v.x * value;
            f[2 * i + 1] = v.y * value;
        }
        store8(w + 8 * p, f);
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

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
//
// All three are bound by memory: each row is read or written once, in 16-byte
// pieces.  A token is the work of a team of 1, 2, 4 or 8 warps, as many as give
// each lane one to four pieces of a row (rows of more than 8192 elements take
// several passes); a block holds eight warps of whole teams.  The token's own
// pieces stay in registers while the rows of its choices go by.  Measured: the
// combine's gradient of 16384 x 6144, top-8, 489 us for 3424 MB (7.0 TB/s); the
// dispatch's with dw at that size 320 us for 2015 MB (6.3 TB/s); the dispatch of
// 768 x 6144, top-8, 14.7 us for 85 MB.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPieces = 4;                // of a row per lane and pass
constexpr int kBatch = 8;                    // choices whose dot products are reduced together

// The token of this thread's team, and the lane's place in the team.
struct Team {
    int warps, rank;                         // rank: of the thread, 0 .. 32 * warps - 1
    long long token;
    __device__ explicit Team(int team_warps)
        : warps(team_warps),
          rank(threadIdx.x & (32 * team_warps - 1)),
          token(static_cast<long long>(blockIdx.x) * (kWarps / team_warps) +
                threadIdx.x / (32 * team_warps)) {}
    // first element of piece c of pass p
    __device__ __forceinline__ int at(int pass, int pieces, int c) const {
        return 8 * (rank + 32 * warps * (pass * pieces + c));
    }
    __device__ __forceinline__ int pass_elements(int pieces) const { return 256 * warps * pieces; }
};

// Rows (-1: none) and weights of up to 32 of a token's choices, one a lane.
struct Choices {
    int row = -1;
    float weight = 0.0f;
    __device__ Choices(const int32_t* place, const float* weights, long long first, int n,
                       long long rows) {
        const int lane = threadIdx.x & 31;
        if (lane < n) {
            row = ptx::load(place + first + lane);
            weight = weights ? ptx::load(weights + first + lane) : 1.0f;
            if (row < 0 || row >= rows) row = -1;
        }
    }
};

template <int kPieces>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const uint16_t* x, const int32_t* place,
                const float* weights, int M, int top_k, int K, int team_warps,
                uint16_t* __restrict__ rows) {
    const Team team(team_warps);
    start_dependent();
    if (team.token >= M) return;
    const uint16_t* xt = x + team.token * K;
    for (int pass = 0; pass * team.pass_elements(kPieces) < K; ++pass) {
        uint4 v[kPieces];
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            const int n = team.at(pass, kPieces, c);
            v[c] = make_uint4(0, 0, 0, 0);
            if (n < K) v[c] = ptx::load(reinterpret_cast<const uint4*>(xt + n));
        }
        for (int j0 = 0; j0 < top_k; j0 += 32) {
            const Choices mine(place, weights, team.token * top_k + j0, min(32, top_k - j0),
                               static_cast<long long>(M) * top_k);
            for (int j = j0; j < min(top_k, j0 + 32); ++j) {
                const int r = __shfl_sync(0xFFFFFFFFu, mine.row, j - j0);
                const float w = __shfl_sync(0xFFFFFFFFu, mine.weight, j - j0);
                if (r < 0) continue;
                uint16_t* out = rows + static_cast<long long>(r) * K;
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    const int n = team.at(pass, kPieces, c);
                    if (n >= K) continue;
                    uint4 o = v[c];
                    if (weights) {
                        float f[8];
                        bf16_unpack8(v[c], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] *= w;
                        o = bf16_pack8(f);
                    }
                    *reinterpret_cast<uint4*>(out + n) = o;
                }
            }
        }
    }
}

// Sums over the warp of eight values a lane: the lane gets the sum of value
// lane >> 2, in halving steps (nine shuffles for the eight sums).
__device__ __forceinline__ float warp_sum8(const float (&d)[8]) {
    const int lane = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        a[i] = (up ? d[i + 4] : d[i]) +
               __shfl_xor_sync(0xFFFFFFFFu, up ? d[i] : d[i + 4], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + 2], 8);
    }
    const bool up = lane & 4;
    float v = (up ? b[1] : b[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? b[0] : b[1], 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
    return v;
}

// kSum: the gradient of the dispatch (out[t] = sum of the weighted rows);
// otherwise the gradient of the combine (out rows = w * token row).
// kDots: dw as well (always with the combine).  kFlight: rows in flight; kBlocks:
// blocks per SM.
template <bool kSum, bool kDots, int kPieces, int kFlight, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks)
token_grad_kernel(const uint16_t* rows, const uint16_t* token,
                  const int32_t* place, const float* weights, int M,
                  int top_k, int N, int team_warps, uint16_t* __restrict__ out,
                  float* __restrict__ dw) {
    __shared__ float s_part[kWarps * kBatch];
    static_assert(kBatch % kFlight == 0, "a batch is whole groups of rows in flight");
    const Team team(team_warps);
    start_dependent();
    const bool real = team.token < M;        // a block's last teams may have no token
    const long long first = team.token * top_k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int pass = 0; pass * team.pass_elements(kPieces) < N; ++pass) {
        float acc[kSum ? kPieces : 1][8];
        uint4 own[kPieces];
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            const int n = team.at(pass, kPieces, c);
            own[c] = make_uint4(0, 0, 0, 0);
            if ((!kSum || kDots) && real && n < N)
                own[c] = ptx::load(reinterpret_cast<const uint4*>(token + team.token * N + n));
            if (kSum) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
            }
        }
        int my_row = -1;
        float my_weight = 0.0f;
        for (int j0 = 0; j0 < top_k; j0 += kBatch) {
            if (j0 % 32 == 0) {
                const Choices mine(place, weights, first + j0, real ? min(32, top_k - j0) : 0,
                                   static_cast<long long>(M) * top_k);
                my_row = mine.row;
                my_weight = mine.weight;
            }
            float dots[kBatch] = {};
#pragma unroll
            for (int f0 = 0; f0 < kBatch; f0 += kFlight) {
                if (j0 + f0 >= top_k) break;
                int r[kFlight];
                float w[kFlight];
                uint4 v[kFlight][kPieces];
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    // lanes past top_k hold row -1
                    r[f] = __shfl_sync(0xFFFFFFFFu, my_row, (j0 + f0 + f) & 31);
                    w[f] = __shfl_sync(0xFFFFFFFFu, my_weight, (j0 + f0 + f) & 31);
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        const int n = team.at(pass, kPieces, c);
                        v[f][c] = make_uint4(0, 0, 0, 0);
                        if (r[f] >= 0 && n < N)
                            v[f][c] = ptx::load(reinterpret_cast<const uint4*>(
                                rows + static_cast<long long>(r[f]) * N + n));
                    }
                }
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    if (r[f] < 0) continue;
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        const int n = team.at(pass, kPieces, c);
                        float a[8], t[8];
                        bf16_unpack8(v[f][c], a);
                        bf16_unpack8(own[c], t);
                        if (kDots) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dots[f0 + f] = fmaf(a[i], t[i], dots[f0 + f]);
                        }
                        if (kSum) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[c][i] = fmaf(w[f], a[i], acc[c][i]);
                        } else if (n < N) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) t[i] *= w[f];
                            *reinterpret_cast<uint4*>(out + static_cast<long long>(r[f]) * N + n) =
                                bf16_pack8(t);
                        }
                    }
                }
            }
            if (kDots) {
                float sum = warp_sum8(dots);
                int j = lane >> 2;
                bool writes = (lane & 3) == 0;
                if (team.warps > 1) {
                    __syncthreads();         // the sums before have been read
                    if (writes) s_part[warp * kBatch + j] = sum;
                    __syncthreads();
                    j = lane;
                    writes = team.rank < kBatch;
                    if (writes) {
                        sum = 0.0f;
                        for (int i = 0; i < team.warps; ++i) sum += s_part[(warp + i) * kBatch + j];
                    }
                }
                if (writes && real && j0 + j < top_k) {
                    float* to = dw + first + j0 + j;
                    *to = pass ? *to + sum : sum;            // by the same lane each pass
                }
            }
        }
        if (kSum && real) {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int n = team.at(pass, kPieces, c);
                if (n < N)
                    *reinterpret_cast<uint4*>(out + team.token * N + n) = bf16_pack8(acc[c]);
            }
        }
    }
}

// Warps per token and pieces per lane for rows of n elements.
struct Shape {
    int team_warps, pieces;
    explicit Shape(int n, int most_warps = kWarps, int most_pieces = kMaxPieces) {
        const int chunks = (n + 7) / 8;
        team_warps = 1;
        while (team_warps < most_warps && 32 * team_warps * most_pieces < chunks) team_warps *= 2;
        pieces = (chunks + 32 * team_warps - 1) / (32 * team_warps);
        if (pieces > most_pieces) pieces = most_pieces;
    }
    int blocks(int M) const {
        const int teams = kWarps / team_warps;
        return static_cast<int>((static_cast<long long>(M) + teams - 1) / teams);
    }
};

// With tokens enough for every SM's warps (16 a SM), a warp for itself takes a
// token in several passes where a team would mostly wait: for one choice's row
// (16384 x 2056: 42 us, a team 46 to 55), and for the dispatch's gradient with
// dw, whose dot products join across a team's warps (16384 x 6144, top-8: 320
// us, a team 352; 8004 x 3336, top-3: 54 and 65).
constexpr int kManyTokens = 16 * 152;
template <bool kSum, bool kDots>
Shape grad_shape(int M, int top_k, int N) {
    if (M >= kManyTokens && top_k == 1) return Shape(N, 1);
    if (M >= kManyTokens && kSum && kDots) return Shape(N, 1, 2);
    return Shape(N);
}

// Two rows in flight and three or four blocks per SM against four rows and two
// blocks: 489 against 504 us for the combine's gradient (M = 16384, N = 6144,
// top-8), 63 against 77 for the dispatch's without dw (M = 4096), where the sums
// alone leave registers for a fourth block.  With
// one choice a second row would be no row.  The block counts were found at 6144 columns and
// a few other widths; they make some forms spill, most of all the dispatch's gradient
// with dw at three pieces a lane (120 bytes; 2880 or 6144 columns, for fewer tokens than
// kManyTokens) and the combine's at four (76 bytes; 2048, 4096 or 8192 columns).
template <bool kSum, bool kDots, int kPieces>
cudaError_t launch_pieces(const Shape& s, const uint16_t* rows, const uint16_t* token,
                          const int32_t* d2s, const float* weights, int M, int top_k, int N,
                          uint16_t* out, float* dw, cudaStream_t stream) {
    constexpr int kBlocks = kPieces == 4 ? (kSum ? 2 : 3) : kDots && kPieces == 3 ? 3 : 4;
    constexpr int kSingleBlocks = kPieces < 3 ? 4 : kSum && kPieces == 4 ? 2 : 3;
    const auto kernel = top_k == 1 ? token_grad_kernel<kSum, kDots, kPieces, 1, kSingleBlocks>
                                   : token_grad_kernel<kSum, kDots, kPieces, 2, kBlocks>;
    return launch_dependent(kernel, s.blocks(M), kThreads, 0, stream, rows, token, d2s, weights, M,
                            top_k, N, s.team_warps, out, dw);
}

template <bool kSum, bool kDots>
cudaError_t launch_grad(const uint16_t* rows, const uint16_t* token, const int32_t* d2s,
                        const float* weights, int M, int top_k, int N, uint16_t* out, float* dw,
                        cudaStream_t stream) {
    const Shape s = grad_shape<kSum, kDots>(M, top_k, N);
    const auto launch = s.pieces == 1   ? launch_pieces<kSum, kDots, 1>
                        : s.pieces == 2 ? launch_pieces<kSum, kDots, 2>
                        : s.pieces == 3 ? launch_pieces<kSum, kDots, 3>
                                        : launch_pieces<kSum, kDots, 4>;
    return launch(s, rows, token, d2s, weights, M, top_k, N, out, dw, stream);
}

}  // namespace

cudaError_t launch_dispatch(const uint16_t* x, const int32_t* d2s, const float* weights, int M,
                            int top_k, int K, uint16_t* rows, cudaStream_t stream) {
    const Shape s(K);
    const auto kernel = s.pieces == 1   ? dispatch_kernel<1>
                        : s.pieces == 2 ? dispatch_kernel<2>
                        : s.pieces == 3 ? dispatch_kernel<3>
                                        : dispatch_kernel<4>;
    return launch_dependent(kernel, s.blocks(M), kThreads, 0, stream, x, d2s, weights, M, top_k, K,
                            s.team_warps, rows);
}

cudaError_t launch_dispatch_bwd(const uint16_t* drows, const uint16_t* x, const int32_t* d2s,
                                const float* weights, int M, int top_k, int K, uint16_t* dx,
                                float* dw, cudaStream_t stream) {
    return dw ? launch_grad<true, true>(drows, x, d2s, weights, M, top_k, K, dx, dw, stream)
              : launch_grad<true, false>(drows, x, d2s, weights, M, top_k, K, dx, dw, stream);
}

cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* d2s,
                               const float* weights, int M, int top_k, int N, uint16_t* dy,
                               float* dw, cudaStream_t stream) {
    return launch_grad<false, true>(y, dout, d2s, weights, M, top_k, N, dy, dw, stream);
}

}  // namespace hg

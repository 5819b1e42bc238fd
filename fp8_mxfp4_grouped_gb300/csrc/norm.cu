// norm.cu -- the root-mean-square norm in front of a layer, with the addition to the
// residual stream before it, and its gradient.  Per row of D elements:
//
//   s = bf16(x + residual)                      (s = x without a residual)
//   r = 1 / sqrt(mean(s^2) + eps)
//   v = s r gain;  y = bf16(v);  (a_fp8, a_scale) = v in E4M3 with E8M0 per 128
//
// and backward, with n = s r and u = r dy gain:
//
//   dx    = dsum + u - n mean(u n)              (for x and for the residual alike)
//   dgain = sum over the rows of dy n
//
// All of it is bound by memory.  A row is the work of a team of 1, 2, 4, 8 or 16 warps
// that holds it in registers, up to four pieces of eight elements a lane, so that
// everything is read once; a half-warp's sixteen pieces are one 128-element group of
// the scales.
#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kWarps = 8;                    // of a block, or one team where that has more
constexpr int kMaxTeamWarps = 16;
constexpr int kMaxPieces = 4;

// The row of this thread's team, and the lane's place in the team.
struct Team {
    int warps, rank, in_block, per_block;
    __device__ explicit Team(int team_warps)
        : warps(team_warps),
          rank(threadIdx.x & (32 * team_warps - 1)),
          in_block(threadIdx.x / (32 * team_warps)),
          per_block(blockDim.x / (32 * team_warps)) {}
    __device__ __forceinline__ int at(int c) const { return 8 * (rank + 32 * warps * c); }
    // A barrier of the team's own: other teams of the block may be at other rows.
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + in_block), "r"(32 * warps) : "memory");
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the team, the same in every lane: a butterfly in each warp, the warps' sums
// in their order.  part: a slot per warp of the block, read by all until the team's next
// barrier.
__device__ __forceinline__ float team_sum(const Team& team, float v, float* part) {
    v = warp_sum(v);
    if (team.warps == 1) return v;
    const int first = team.in_block * team.warps;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    team.sync();
    v = 0.0f;
    for (int i = 0; i < team.warps; ++i) v += part[first + i];
    return v;
}

// 1 / sqrt(mean + eps) where the squares pass FP32's range: in 64 bits, from the row of s
// as it stands in memory (this thread's own pieces).
__device__ __noinline__ float wide_rstd(const Team team, const uint16_t* row, int D, float eps,
                                        double* part) {
    double sum = 0.0;
    for (int c = 0; team.at(c) < D; ++c) {
        float f[8];
        bf16_unpack8(ptx::load(reinterpret_cast<const uint4*>(row + team.at(c))), f);
        for (int i = 0; i < 8; ++i) sum += static_cast<double>(f[i]) * f[i];
    }
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (team.warps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        team.sync();
        sum = 0.0;
        for (int i = 0; i < team.warps; ++i) sum += part[team.in_block * team.warps + i];
    }
    return static_cast<float>(1.0 / sqrt(sum / D + eps));
}

constexpr float kWide = 1e37f;               // sums of squares from here on are done again

template <int kPieces>
__global__ void __launch_bounds__(kMaxTeamWarps * 32)
rmsnorm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* gain, int M, int D,
               float eps, int team_warps, uint16_t* sum, uint16_t* y, uint8_t* a_fp8,
               uint8_t* a_scale, float* rstd) {
    __shared__ float part[kMaxTeamWarps];
    __shared__ double wide_part[kMaxTeamWarps];
    const Team team(team_warps);
    const long long row = static_cast<long long>(blockIdx.x) * team.per_block + team.in_block;
    start_dependent();
    if (row >= M) return;
    uint4 s[kPieces], add[kPieces];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        const int n = team.at(c);
        s[c] = add[c] = make_uint4(0, 0, 0, 0);
        if (n >= D) continue;
        s[c] = ptx::load(reinterpret_cast<const uint4*>(x + row * D + n));
        if (residual) add[c] = ptx::load(reinterpret_cast<const uint4*>(residual + row * D + n));
    }
    float squares = 0.0f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        float f[8];
        bf16_unpack8(s[c], f);
        if (residual) {
            float g[8];
            bf16_unpack8(add[c], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += g[i];
            s[c] = bf16_pack8(f);
            bf16_unpack8(s[c], f);
            const int n = team.at(c);
            if (n < D) *reinterpret_cast<uint4*>(sum + row * D + n) = s[c];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = fmaf(f[i], f[i], squares);
    }
    squares = team_sum(team, squares, part);
    const float r = squares < kWide ? 1.0f / sqrtf(squares / static_cast<float>(D) + eps)
                                    : wide_rstd(team, (residual ? sum : x) + row * D, D, eps, wide_part);
    if (rstd && team.rank == 0) rstd[row] = r;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        const int n = team.at(c);
        float f[8], g[8];
        bf16_unpack8(s[c], f);
        uint4 vg = make_uint4(0, 0, 0, 0);
        if (n < D) vg = ptx::load(reinterpret_cast<const uint4*>(gain + n));
        bf16_unpack8(vg, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * r * g[i];
        if (y && n < D) *reinterpret_cast<uint4*>(y + row * D + n) = bf16_pack8(f);
        if (!a_fp8) continue;
        // whole groups: D is a multiple of 128 here
        const uint64_t v[4] = {ptx::f32x2(f[0], f[1]), ptx::f32x2(f[2], f[3]),
                               ptx::f32x2(f[4], f[5]), ptx::f32x2(f[6], f[7])};
        uint32_t scale;
        const uint2 codes = quantize8(v, (threadIdx.x >> 4) & 1, scale);
        if (n < D) {
            *reinterpret_cast<uint2*>(a_fp8 + row * D + n) = codes;
            if ((threadIdx.x & 15) == 0)
                a_scale[row * (D / 128) + n / 128] = static_cast<uint8_t>(scale);
        }
    }
}

// Blocks of the gradient's grid: two a SM.  Each team takes every so-manieth row and
// keeps its columns' part of dgain in registers; the parts go to the workspace, a row a
// team, and are added in the order of the teams.
constexpr int kBwdBlocks = 2 * 152;

template <int kPieces>
__global__ void __launch_bounds__(kMaxTeamWarps * 32)
rmsnorm_bwd_kernel(const uint16_t* dy, const uint16_t* dsum, const uint16_t* sum,
                   const uint16_t* gain, const float* rstd, int M, int D, int team_warps,
                   uint16_t* dx, float* parts) {
    __shared__ float part[2][kMaxTeamWarps];
    const Team team(team_warps);
    const int teams = gridDim.x * team.per_block;
    const int first = blockIdx.x * team.per_block + team.in_block;
    start_dependent();
    if (first >= M) return;
    float dg[kPieces][8] = {};
    int turn = 0;
    for (long long row = first; row < M; row += teams, turn ^= 1) {
        uint4 vd[kPieces], vs[kPieces];
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            const int n = team.at(c);
            vd[c] = vs[c] = make_uint4(0, 0, 0, 0);
            if (n >= D) continue;
            vd[c] = ptx::load(reinterpret_cast<const uint4*>(dy + row * D + n));
            vs[c] = ptx::load(reinterpret_cast<const uint4*>(sum + row * D + n));
        }
        const float r = ptx::load(rstd + row);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            const int n = team.at(c);
            float d[8], s[8], g[8];
            bf16_unpack8(vd[c], d);
            bf16_unpack8(vs[c], s);
            uint4 vg = make_uint4(0, 0, 0, 0);
            if (n < D) vg = ptx::load(reinterpret_cast<const uint4*>(gain + n));
            bf16_unpack8(vg, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float norm = s[i] * r;
                dg[c][i] = fmaf(d[i], norm, dg[c][i]);
                dot = fmaf(d[i] * r * g[i], norm, dot);
            }
        }
        const float mean = team_sum(team, dot, part[turn]) / static_cast<float>(D);
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            const int n = team.at(c);
            if (n >= D) continue;
            float d[8], s[8], g[8], o[8] = {};
            bf16_unpack8(vd[c], d);
            bf16_unpack8(vs[c], s);
            bf16_unpack8(ptx::load(reinterpret_cast<const uint4*>(gain + n)), g);
            if (dsum) bf16_unpack8(ptx::load(reinterpret_cast<const uint4*>(dsum + row * D + n)), o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += fmaf(-s[i] * r, mean, d[i] * r * g[i]);
            *reinterpret_cast<uint4*>(dx + row * D + n) = bf16_pack8(o);
        }
    }
    if (!parts) return;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        const int n = team.at(c);
        if (n >= D) continue;
        float4* to = reinterpret_cast<float4*>(parts + static_cast<long long>(first) * D + n);
        to[0] = make_float4(dg[c][0], dg[c][1], dg[c][2], dg[c][3]);
        to[1] = make_float4(dg[c][4], dg[c][5], dg[c][6], dg[c][7]);
    }
}

// dgain[n] = sum over the teams' parts, in an order that depends on the sizes alone.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32)
rmsnorm_join_kernel(const float* parts, int teams, int D, float* dgain) {
    __shared__ float s[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    start_dependent();
    float v = 0.0f;
    if (n < D) {
#pragma unroll 4
        for (int t = warp; t < teams; t += kJoinWarps)
            v += ptx::load(parts + static_cast<long long>(t) * D + n);
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || n >= D) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) v += s[w][lane];
    dgain[n] = v;
}

// Warps per row, pieces per lane and threads per block for rows of D elements.
struct Shape {
    int team_warps = 1, pieces, threads;
    explicit Shape(int D) {
        const int chunks = (D + 7) / 8;
        while (32 * team_warps * kMaxPieces < chunks) team_warps *= 2;
        pieces = (chunks + 32 * team_warps - 1) / (32 * team_warps);
        threads = 32 * (team_warps > kWarps ? team_warps : kWarps);
    }
    int teams_per_block() const { return threads / (32 * team_warps); }
};

int bwd_teams(int M, int D) {
    const int most = kBwdBlocks * Shape(D).teams_per_block();
    return M < most ? M : most;
}

template <int kPieces>
cudaError_t launch_fwd(const Shape& s, const RmsnormArgs& a, cudaStream_t stream) {
    const int teams = s.teams_per_block();
    const int grid = static_cast<int>((static_cast<long long>(a.M) + teams - 1) / teams);
    return launch_dependent(rmsnorm_kernel<kPieces>, grid, s.threads, 0, stream, a.x, a.residual,
                            a.gain, a.M, a.D, a.eps, s.team_warps, a.sum, a.y, a.a_fp8, a.a_scale,
                            a.rstd);
}

template <int kPieces>
cudaError_t launch_bwd(const Shape& s, const RmsnormBwdArgs& a, cudaStream_t stream) {
    const int teams = bwd_teams(a.M, a.D), per_block = s.teams_per_block();
    const cudaError_t err = launch_dependent(
        rmsnorm_bwd_kernel<kPieces>, (teams + per_block - 1) / per_block, s.threads, 0, stream,
        a.dy, a.dsum, a.sum, a.gain, a.rstd, a.M, a.D, s.team_warps, a.dx,
        a.dgain ? a.parts : nullptr);
    if (err != cudaSuccess || !a.dgain) return err;
    return launch_dependent(rmsnorm_join_kernel, (a.D + 31) / 32, kJoinWarps * 32, 0, stream,
                            a.parts, teams, a.D, a.dgain);
}

}  // namespace

int rmsnorm_max_elements() { return kMaxTeamWarps * 32 * kMaxPieces * 8; }

size_t rmsnorm_bwd_workspace(int M, int D) {
    return static_cast<size_t>(bwd_teams(M, D)) * static_cast<size_t>(D) * sizeof(float);
}

cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream) {
    const Shape s(a.D);
    const auto launch = s.pieces == 1   ? launch_fwd<1>
                        : s.pieces == 2 ? launch_fwd<2>
                        : s.pieces == 3 ? launch_fwd<3>
                                        : launch_fwd<4>;
    return launch(s, a, stream);
}

cudaError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, cudaStream_t stream) {
    const Shape s(a.D);
    const auto launch = s.pieces == 1   ? launch_bwd<1>
                        : s.pieces == 2 ? launch_bwd<2>
                        : s.pieces == 3 ? launch_bwd<3>
                                        : launch_bwd<4>;
    return launch(s, a, stream);
}

}  // namespace hg

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
// A row is the work of a team of 1, 2, 4, 8 or 16 warps that takes it into registers, up to
// four pieces of eight elements a lane, so that everything is read once; a half-warp's
// sixteen pieces are one 128-element group of the scales.
//
// Long rows with a residual, and their gradient, are bound by memory: 16384 x 6144 with all
// outputs 131 us for 907 MB (6.9 TB/s; a persistent grid that asks for the next row ahead 149),
// the gradient with the residual's 125 us for 805 MB (6.4 TB/s), of 8199 x 6144 69 us (5.9),
// of which some 6 us join the parts of dgain.  Those 6 us show in short rows: the gradient of
// 16384 x 1024 takes 30 us for a floor of 20.  With the rows in registers, and loads that waited
// for the row before, the gradient took 106 us at 8199 x 6144 and 78 at 16384 x 1024.
//
// One output without a residual is not: BF16 67 us for 403 MB (6.0 TB/s), FP8, a quarter less,
// 72 us (4.2 TB/s).  A block has one row and loads, sums, quantises and stores it one after the
// other, with six rows on an SM; three blocks of up to 512 threads leave 40 registers a thread, of
// which rows of two to four pieces spill 24, 40 and 72 bytes (with a residual: 64 registers, 12
// bytes at four pieces).
#include <atomic>

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
    // A barrier of the team's own: other teams of the block may be at other rows.  (Barriers by
    // number: one in a register would take all sixteen of the SM's per block.)
    __device__ __forceinline__ void sync() const {
        switch (in_block) {
            case 0: named_sync<1>(); break;
            case 1: named_sync<2>(); break;
            case 2: named_sync<3>(); break;
            default: named_sync<4>(); break;             // teams of two warps: four a block
        }
    }
    template <int kName>
    __device__ __forceinline__ void named_sync() const {
        asm volatile("bar.sync %0, %1;" ::"n"(kName), "r"(32 * warps) : "memory");
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

template <int kPieces, bool kResidual>
__global__ void __launch_bounds__(kMaxTeamWarps * 32, kResidual ? 2 : 3)
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
        if (kResidual) add[c] = ptx::load(reinterpret_cast<const uint4*>(residual + row * D + n));
    }
    float squares = 0.0f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        float f[8];
        bf16_unpack8(s[c], f);
        if (kResidual) {
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
    const float r = squares < kWide
                        ? 1.0f / sqrtf(squares / static_cast<float>(D) + eps)
                        : wide_rstd(team, (kResidual ? sum : x) + row * D, D, eps, wide_part);
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

// The gradient: a block takes groups of consecutive rows in turn, some 6144 elements of each
// array a group, which bulk copies bring into one half of its shared memory while the other
// half is worked on.  Rows stay there for their second pass; a thread keeps its columns'
// gains and its part of dgain in registers.  The parts of a block's teams are added up, then
// written to the workspace, a row a block, and joined in the order of the blocks.
constexpr int kGroupElements = 6144;

// Blocks of an SM that there are registers for.
constexpr int bwd_blocks(int threads, int pieces) {
    return threads > kWarps * 32 ? 1 : pieces < kMaxPieces ? 3 : 2;
}

template <int kPieces, int kThreads>
__global__ void __launch_bounds__(kThreads, bwd_blocks(kThreads, kPieces))
rmsnorm_bwd_kernel(const uint16_t* dy, const uint16_t* dsum, const uint16_t* sum,
                   const uint16_t* gain, const float* rstd, int M, int D, int team_warps,
                   int group_rows, uint16_t* dx, float* parts, uint32_t* status,
                   uint64_t timeout_ns) {
    extern __shared__ __align__(16) uint8_t smem[];      // two halves of dy, sum and dsum
    __shared__ float part[2][kMaxTeamWarps];
    __shared__ __align__(8) uint64_t s_bar[2];
    __shared__ uint32_t s_abort;
    const Team team(team_warps);
    const uint32_t bars = ptx::smem_u32(s_bar);
    if (threadIdx.x == 0) {
        for (int h = 0; h < 2; ++h) ptx::mbar_init(bars + 8 * h, 1);
        s_abort = 0u;
        ptx::fence_barrier_init();
    }
    __syncthreads();
    start_dependent();
    const int arrays = dsum ? 3 : 2;
    const int array_bytes = group_rows * D * 2;
    const int groups = (M - 1) / group_rows + 1;
    const WaitCtx ctx{status, &s_abort, timeout_ns};
    auto load = [&](int group, int half) {
        const long long row = static_cast<long long>(group) * group_rows;
        const int rows = static_cast<int>(min(static_cast<long long>(group_rows), M - row));
        const uint32_t bytes = static_cast<uint32_t>(rows) * D * 2;
        const uint16_t* from[3] = {dy, sum, dsum};
        ptx::mbar_arrive_expect_tx(bars + 8 * half, bytes * arrays);
        for (int i = 0; i < arrays; ++i)
            ptx::bulk_load(ptx::smem_u32(smem) + (half * 3 + i) * array_bytes, from[i] + row * D,
                           bytes, bars + 8 * half);
    };
    if (threadIdx.x == 0) {
        for (int h = 0; h < 2; ++h) {
            const long long group = blockIdx.x + static_cast<long long>(h) * gridDim.x;
            if (group < groups) load(static_cast<int>(group), h);
        }
    }
    uint4 g16[kPieces];
    float dg[kPieces][8] = {};
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        const int n = team.at(c);
        g16[c] = make_uint4(0, 0, 0, 0);
        if (n < D) g16[c] = ptx::load(reinterpret_cast<const uint4*>(gain + n));
    }
    int turn = 0, step = 0;
    long long group = blockIdx.x;
    for (; group < groups; group += gridDim.x, ++step) {
        const int half = step & 1;
        const long long row0 = group * group_rows;
        const int rows = static_cast<int>(min(static_cast<long long>(group_rows), M - row0));
        const bool came = wait_bounded(bars + 8 * half, (step >> 1) & 1u, ctx, kRoleNorm, half);
        if (__syncthreads_or(!came)) break;
        const uint8_t* base = smem + half * 3 * array_bytes;
        for (int j = team.in_block; j < rows; j += team.per_block, turn ^= 1) {
            const float r = ptx::load(rstd + row0 + j);
            const uint16_t* at = reinterpret_cast<const uint16_t*>(base) + j * D;
            float dot = 0.0f;
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int n = team.at(c);
                if (n >= D) continue;
                float d[8], s[8], g[8];
                bf16_unpack8(*reinterpret_cast<const uint4*>(at + n), d);
                bf16_unpack8(*reinterpret_cast<const uint4*>(at + array_bytes / 2 + n), s);
                bf16_unpack8(g16[c], g);
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
                bf16_unpack8(*reinterpret_cast<const uint4*>(at + n), d);
                bf16_unpack8(*reinterpret_cast<const uint4*>(at + array_bytes / 2 + n), s);
                bf16_unpack8(g16[c], g);
                if (dsum) bf16_unpack8(*reinterpret_cast<const uint4*>(at + array_bytes + n), o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += fmaf(-s[i] * r, mean, d[i] * r * g[i]);
                *reinterpret_cast<uint4*>(dx + (row0 + j) * D + n) = bf16_pack8(o);
            }
        }
        __syncthreads();                                 // this half has been read
        if (threadIdx.x == 0 && group + 2ll * gridDim.x < groups)
            load(static_cast<int>(group + 2ll * gridDim.x), half);
    }
    if (s_abort) {                                       // copies in flight land first
        for (int i = 0; i < 2; ++i, ++step)
            if (threadIdx.x == 0 && blockIdx.x + static_cast<long long>(step) * gridDim.x < groups)
                wait_drain(bars + 8 * (step & 1), (step >> 1) & 1u);
        return;
    }
    if (!parts) return;
    float* sums = reinterpret_cast<float*>(smem);        // [teams, D]; nothing is in flight
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
        const int n = team.at(c);
        if (n >= D) continue;
        float4* to = reinterpret_cast<float4*>(
            team.per_block > 1 ? sums + team.in_block * D + n
                               : parts + static_cast<long long>(blockIdx.x) * D + n);
        to[0] = make_float4(dg[c][0], dg[c][1], dg[c][2], dg[c][3]);
        to[1] = make_float4(dg[c][4], dg[c][5], dg[c][6], dg[c][7]);
    }
    if (team.per_block == 1) return;
    __syncthreads();
    for (int n = threadIdx.x; n < D; n += blockDim.x) {
        float v = sums[n];
        for (int t = 1; t < team.per_block; ++t) v += sums[t * D + n];
        parts[static_cast<long long>(blockIdx.x) * D + n] = v;
    }
}

// dgain[n] = sum over the blocks' parts, in an order that depends on the sizes alone.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32)
rmsnorm_join_kernel(const float* parts, int blocks, int D, float* dgain) {
    __shared__ float s[kJoinWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    start_dependent();
    float v = 0.0f;
    if (n < D) {
#pragma unroll 10
        for (int b = warp; b < blocks; b += kJoinWarps)
            v += ptx::load(parts + static_cast<long long>(b) * D + n);
    }
    s[warp][lane] = v;
    __syncthreads();
    v = warp_sum(s[lane][warp]);                         // of column `warp`
    if (lane == 0 && blockIdx.x * 32 + warp < D) dgain[blockIdx.x * 32 + warp] = v;
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

// The gradient's grid: groups of whole teams' rows, shorter where there would be fewer
// groups than blocks, and as many blocks as 152 SMs hold at once.
constexpr size_t kSmSmem = 228 * 1024, kBlockSmem = 2048;      // of an SM; beside the groups
struct BwdShape : Shape {
    int group_rows, blocks;
    int parts;                               // room for parts: the most blocks of up to M rows
    size_t smem;
    BwdShape(int M, int D) : Shape(D) {
        const int teams = teams_per_block();
        group_rows = kGroupElements / D / teams * teams;
        if (group_rows < teams) group_rows = teams;
        const auto bytes = [&] { return 6ull * group_rows * D * sizeof(uint16_t); };
        int per_sm = bwd_blocks(threads, pieces);
        if (per_sm > static_cast<int>(kSmSmem / (bytes() + kBlockSmem)))
            per_sm = static_cast<int>(kSmSmem / (bytes() + kBlockSmem));
        const int most = 152 * per_sm, fair = ((M - 1) / most / teams + 1) * teams;
        if (group_rows > fair) group_rows = fair;
        const int groups = (M - 1) / group_rows + 1;
        blocks = groups < most ? groups : most;
        const int shortest = (M - 1) / teams + 1;        // groups of M rows, a row a team
        parts = shortest < most ? shortest : most;
        smem = bytes();                      // and room for the teams' sums
    }
};

template <int kPieces>
cudaError_t launch_fwd(const Shape& s, const RmsnormArgs& a, cudaStream_t stream) {
    const int teams = s.teams_per_block();
    const int grid = static_cast<int>((static_cast<long long>(a.M) + teams - 1) / teams);
    const auto kernel = a.residual ? rmsnorm_kernel<kPieces, true> : rmsnorm_kernel<kPieces, false>;
    return launch_dependent(kernel, grid, s.threads, 0, stream, a.x, a.residual, a.gain, a.M, a.D,
                            a.eps, s.team_warps, a.sum, a.y, a.a_fp8, a.a_scale, a.rstd);
}

// Devices (a bit each) on which a gradient's kernel may use its shared memory, by pieces and
// whether a team has sixteen warps.
std::atomic<uint64_t> g_ready[kMaxPieces + 1][2];

template <int kPieces, int kThreads>
cudaError_t launch_bwd(const BwdShape& s, const RmsnormBwdArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const auto kernel = rmsnorm_bwd_kernel<kPieces, kThreads>;
    std::atomic<uint64_t>& ready = g_ready[kPieces][kThreads > kWarps * 32];
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   6 * kMaxTeamWarps * 32 * kMaxPieces * 8 * 2);
        if (err != cudaSuccess) return err;
        ready.fetch_or(bit);
    }
    err = launch_dependent(kernel, s.blocks, s.threads, s.smem, stream, a.dy, a.dsum, a.sum, a.gain,
                           a.rstd, a.M, a.D, s.team_warps, s.group_rows, a.dx,
                           a.dgain ? a.parts : nullptr, a.status, a.timeout_ns);
    if (err != cudaSuccess || !a.dgain) return err;
    return launch_dependent(rmsnorm_join_kernel, (a.D + 31) / 32, kJoinWarps * 32, 0, stream,
                            a.parts, s.blocks, a.D, a.dgain);
}

}  // namespace

int rmsnorm_max_elements() { return kMaxTeamWarps * 32 * kMaxPieces * 8; }

// The blocks themselves fall where a group's rows rise: the workspace of a batch has to do for
// smaller ones too.
size_t rmsnorm_bwd_workspace(int M, int D) {
    return static_cast<size_t>(BwdShape(M, D).parts) * static_cast<size_t>(D) * sizeof(float);
}

void rmsnorm_reset_caches() {
    for (auto& pieces : g_ready)
        for (auto& ready : pieces) ready.store(0);
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
    constexpr int kSmall = kWarps * 32, kLarge = kMaxTeamWarps * 32;
    const BwdShape s(a.M, a.D);
    if (s.threads == kSmall) {
        const auto launch = s.pieces == 1   ? launch_bwd<1, kSmall>
                            : s.pieces == 2 ? launch_bwd<2, kSmall>
                            : s.pieces == 3 ? launch_bwd<3, kSmall>
                                            : launch_bwd<4, kSmall>;
        return launch(s, a, stream);
    }
    // more than 8192 elements: at least three pieces a lane
    return s.pieces == 3 ? launch_bwd<3, kLarge>(s, a, stream)
                         : launch_bwd<4, kLarge>(s, a, stream);
}

}  // namespace hg

// matvec.cu -- few tokens times the routed experts' MXFP4 weights, on BF16
// activations: the single-token form of the grouped GEMM.  Slot s = t * top_k
// + j multiplies its input row with the weights of expert topk_ids[s]:
//
//   y[s, n] = sum_k x[row(s), k] * e2m1(w_fp4[e, n, k]) * 2^(w_scale[e, n, k/32] - 127)
//
// with row(s) = s / top_k (one row a token) or s (one row a slot).  The
// SwiGLU form writes h[s, f] = silu(y[s, f]) * y[s, F + f], F = N / 2.  A slot
// whose id is outside [0, E) gets a row of zeros.
//
// What bounds it: the weights, N * K * 17/32 bytes per expert in use, read
// once from HBM.  Every block first lists the slots by expert in shared
// memory, in chunks of up to eight slots (the columns of one MMA), so that an
// expert's weights are read once for all of a chunk's slots; a work unit is
// (chunk, 16 weight rows), and each block takes one contiguous range of units.
//
// Warps stream: each warp owns a ring of 16-row x 256-K boxes that its lane 0
// fills by TMA, runs ahead of its own use of them by the ring's depth, and
// waits for nobody else to do so.  A team of T warps splits a unit's K range
// box by box and joins its partial sums in shared memory, in warp order, so
// that results do not depend on timing.
//
// Arithmetic: a box's E2M1 codes become FP16 (exact) in registers and meet x
// in mma.sync m16n8k16: with eight columns at most the tensor work is small,
// and tcgen05 would want the 16-bit weights written back to shared memory
// first.  x is BF16, wider than FP16's range: each row's 256 elements of a box
// are scaled by the power of two that takes their largest magnitude into
// [2^14, 2^15).  An element keeps its 8 bits down to 2^-32 of that largest,
// and what lies below is off by 2^-40 of it at most, far below the FP32 sum's
// own rounding.  The sums of a 32-K group come out of the MMA in FP32 and are
// added up in FP32 times the product of the two scales.
#include <cuda_fp16.h>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
static_assert(kThreads >= kMatvecMaxSlots, "a thread lists one slot");
constexpr int kRows = 16;                    // weight rows of a unit: the MMA's M
constexpr int kMaxCols = 8;                  // slots of a chunk: the MMA's N
constexpr int kBoxK = 256;                   // elements of a box's rows: 128 bytes
constexpr int kBoxBytes = kRows * kBoxK / 2;
constexpr int kBoxScaleBytes = kRows * kBoxK / 32;
constexpr int kMaxSlots = kMatvecMaxSlots;
constexpr int kMaxRing = 6;                  // boxes in flight per warp
constexpr int kSmemLimit = 232448 - 256;     // beside a few static bytes

// One entry per slot or chunk (there are at most as many chunks as slots).
struct Tables {
    int id[kMaxSlots];
    int expert[kMaxSlots];                   // of a chunk
    int ncols[kMaxSlots];                    // of a chunk
    uint16_t chunk_of[kMaxSlots];            // of a chunk's first slot
    uint16_t slot[kMaxSlots * kMaxCols];     // of a chunk's columns
    uint8_t same_rows[kMaxSlots];            // the chunk's input rows are those of the one before
    int warp_count[kWarps];
};

struct Layout {
    int ring;          // boxes per warp
    int cols;          // most slots of a chunk
    int x_stride;      // bytes between the columns of x
    int scales, partial, x, x_scale, bars, tables, total;   // byte offsets
};

// As many columns as fit beside a ring of at least two boxes a warp, then as
// deep a ring as fits.  Columns stay 64 bytes off a multiple of 128 apart, so
// that the eight lanes of a 16-byte load phase (two columns) meet no bank
// twice.
bool make_layout(int K, int slots, int tokens, Layout* out) {
    const int nb = (K + kBoxK - 1) / kBoxK;
    Layout l;
    l.x_stride = nb * kBoxK * 2 + 64;
    const int fixed = 1024 + kWarps * 2 * 512 + nb * kMaxCols * 4 + kWarps * kMaxRing * 8 +
                      static_cast<int>(sizeof(Tables));
    const int box = kWarps * (kBoxBytes + kBoxScaleBytes);
    int cols = tokens < kMaxCols ? tokens : kMaxCols;   // a token's choices are distinct experts
    if (cols > slots) cols = slots;
    while (cols > 1 && fixed + cols * l.x_stride + 2 * box > kSmemLimit) --cols;
    l.cols = cols;
    l.ring = (kSmemLimit - fixed - cols * l.x_stride) / box;
    if (l.ring > kMaxRing) l.ring = kMaxRing;
    if (l.ring < 2) return false;
    l.scales = kWarps * l.ring * kBoxBytes;
    l.partial = l.scales + kWarps * l.ring * kBoxScaleBytes;
    l.x = l.partial + kWarps * 2 * 512;
    l.x_scale = l.x + cols * l.x_stride;
    l.bars = l.x_scale + nb * kMaxCols * 4;
    l.tables = l.bars + kWarps * l.ring * 8;
    l.total = l.tables + static_cast<int>(sizeof(Tables)) + 1024;
    *out = l;
    return true;
}

struct KernelArgs {
    const uint16_t* x;
    const int32_t* ids;
    const uint8_t* w_scale;
    uint16_t* out;
    uint32_t* status;
    uint64_t timeout_ns;
    int slots_per_row, slots, E, N, K;
    Layout l;
};

// List the slots by expert in chunks of up to `cols`: thread s handles slot s.
// Returns the number of chunks.
__device__ int list_slots(const KernelArgs& a, Tables& tb) {
    const int s = threadIdx.x;
    const bool mine = s < a.slots;
    if (mine) {
        tb.id[s] = __ldg(a.ids + s);
        tb.ncols[s] = 0;
    }
    __syncthreads();
    // rank among the slots of the same expert; the first slot of this one's chunk
    int rank = 0, lead = s;
    const int e = mine ? tb.id[s] : -1;
    const bool valid = mine && e >= 0 && e < a.E;
    if (valid) {
        for (int j = 0; j < s; ++j) {
            if (tb.id[j] == e) {
                if (rank % a.l.cols == 0) lead = j;
                ++rank;
            }
        }
        if (rank % a.l.cols == 0) lead = s;
    }
    const bool leads = valid && lead == s;
    const uint32_t vote = __ballot_sync(0xFFFFFFFFu, leads);
    const int lane = s & 31, warp = s >> 5;
    if (lane == 0) tb.warp_count[warp] = __popc(vote);
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < kWarps; ++i) {
        const int c = tb.warp_count[i];
        if (i < warp) before += c;
        total += c;
    }
    if (leads) {
        const int c = before + __popc(vote & ((1u << lane) - 1u));
        tb.chunk_of[s] = static_cast<uint16_t>(c);
        tb.expert[c] = e;
    }
    __syncthreads();
    if (valid) {
        const int c = tb.chunk_of[lead];
        tb.slot[c * kMaxCols + rank % a.l.cols] = static_cast<uint16_t>(s);
        atomicAdd(&tb.ncols[c], 1);
    }
    __syncthreads();
    if (s < total) {
        bool same = s > 0 && tb.ncols[s] == tb.ncols[s - 1];
        for (int i = 0; same && i < tb.ncols[s]; ++i) {
            same = tb.slot[s * kMaxCols + i] / a.slots_per_row ==
                   tb.slot[(s - 1) * kMaxCols + i] / a.slots_per_row;
        }
        tb.same_rows[s] = same;
    }
    __syncthreads();
    return total;
}

// The chunk's input rows into shared memory as scaled FP16, with one scale per
// row and box: a warp handles 256 elements at a time, eight a lane.
__device__ void load_x(const KernelArgs& a, const Tables& tb, uint8_t* smem, int chunk, int nb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ncols = tb.ncols[chunk];
    float* scale = reinterpret_cast<float*>(smem + a.l.x_scale);
    for (int i = warp; i < nb * kMaxCols; i += kWarps) {
        const int b = i / kMaxCols, c = i % kMaxCols;
        if (c >= ncols) {
            if (lane == 0) scale[i] = 0.0f;
            continue;
        }
        const int row = tb.slot[chunk * kMaxCols + c] / a.slots_per_row;
        const int k = b * kBoxK + 8 * lane;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < a.K)
            v = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<long long>(row) * a.K + k));
        float f[8];
        bf16_unpack8(v, f);
        uint32_t top = 0;                    // largest magnitude's bits; NaN counts as the largest
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        int be = static_cast<int>(top >> 23);
        float mult, back;
        if (be == 255) {
            // an Inf or NaN decides the sum: the finite elements may be dropped
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = isfinite(f[e]) ? 0.0f : f[e];
            mult = back = 1.0f;
        } else {
            be = max(be, 15);                // both factors stay normal numbers
            mult = __uint_as_float(static_cast<uint32_t>(268 - be) << 23);   // 2^(14 - (be - 127))
            back = __uint_as_float(static_cast<uint32_t>(be - 14) << 23);
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 p = __floats2half2_rn(f[2 * e] * mult, f[2 * e + 1] * mult);
            h[e] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *reinterpret_cast<uint4*>(smem + a.l.x + c * a.l.x_stride + 2 * k) =
            make_uint4(h[0], h[1], h[2], h[3]);
        if (lane == 0) scale[i] = back;
    }
}

// 2^(code - 127) for the byte `i` of the group's eight codes; 255 becomes Inf
// (not a supported code).
__device__ __forceinline__ float scale_of(const uint2 codes, int i) {
    const uint32_t c = ((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xFFu;
    return __uint_as_float(max(c << 23, 0x00400000u));
}

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1)
expert_matvec_kernel(const __grid_constant__ CUtensorMap map_w, const KernelArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_abort;
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    Tables& tb = *reinterpret_cast<Tables*>(smem + a.l.tables);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = (a.K + kBoxK - 1) / kBoxK;
    const int out_cols = kSwiglu ? a.N / 2 : a.N;
    const int tile_cols = kSwiglu ? kRows / 2 : kRows;       // outputs of a unit
    const int tiles = (out_cols + tile_cols - 1) / tile_cols;

    if (lane == 0) {
        for (int i = 0; i < a.l.ring; ++i)
            ptx::mbar_init(base + a.l.bars + 8 * (warp * a.l.ring + i), 33);
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) s_abort = 0;
    const int chunks = list_slots(a, tb);    // has block barriers

    // slots without an expert: zeros, spread over the grid
    for (int s = 0; s < a.slots; ++s) {
        if (tb.id[s] >= 0 && tb.id[s] < a.E) continue;
        for (int n = blockIdx.x * kThreads + threadIdx.x; n < out_cols; n += gridDim.x * kThreads)
            a.out[static_cast<long long>(s) * out_cols + n] = 0;
    }

    const long long units = static_cast<long long>(chunks) * tiles;
    const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    if (u0 >= u1) return;

    // Warps per team: the fewest box steps of a warp, with more warps on ties.
    const int most = static_cast<int>((units + gridDim.x - 1) / gridDim.x);
    int team_warps = 1, best = 0x7FFFFFFF;
    for (int t = 1; t <= kWarps; t *= 2) {
        const int teams = kWarps / t;
        const int cost = ((most + teams - 1) / teams) * ((nb + t - 1) / t);
        if (cost <= best) {
            best = cost;
            team_warps = t;
        }
    }
    const int teams = kWarps / team_warps;
    const int team = warp / team_warps, member = warp % team_warps;

    // End of the run of units from `u` that share their input rows.
    auto run_end = [&](int u) {
        int c = u / tiles + 1;
        while (c < chunks && tb.same_rows[c]) ++c;
        return min(c * tiles, u1);
    };

    // This warp's boxes in order: units u (every teams-th of a run), boxes b
    // (every team_warps-th of a unit).
    int p_u = u0 + team, p_end = run_end(u0), p_b = member, issued = 0;
    const uint32_t ring_w = base + warp * a.l.ring * kBoxBytes;
    const uint32_t ring_s = base + a.l.scales + warp * a.l.ring * kBoxScaleBytes;
    const uint32_t bars = base + a.l.bars + 8 * warp * a.l.ring;
    const long long last_row = static_cast<long long>(a.E) * a.N - 1;
    const int groups = a.K / 32;
    auto issue = [&]() {
        if (member >= nb) return;
        while (p_u >= p_end) {
            if (p_end >= u1) return;
            p_u = p_end + team;
            p_end = run_end(p_end);
        }
        const int chunk = p_u / tiles, tile = p_u - chunk * tiles;
        const int n0 = tile * tile_cols;
        const int second = kSwiglu ? a.N / 2 : 8;            // rows 8..15 of the unit
        const int row0 = tb.expert[chunk] * a.N + n0;
        const int at = issued % a.l.ring;
        const uint32_t bar = bars + 8 * at;
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, kBoxBytes);
            ptx::tma_load_2d_nohint(ring_w + at * kBoxBytes, &map_w, p_b * (kBoxK / 2), row0, bar);
            ptx::tma_load_2d_nohint(ring_w + at * kBoxBytes + kBoxBytes / 2, &map_w,
                                    p_b * (kBoxK / 2), row0 + second, bar);
        }
        const int r = lane >> 1, g = 8 * p_b + 4 * (lane & 1);
        const bool there = g < groups;
        const long long row = min(static_cast<long long>(row0) + (r < 8 ? r : second + r - 8),
                                  last_row);
        ptx::cp_async_4(ring_s + at * kBoxScaleBytes + 4 * lane,
                        a.w_scale + row * groups + (there ? g : 0), there);
        ptx::cp_async_mbar_arrive(bar);
        ++issued;
        p_b += team_warps;
        if (p_b >= nb) {
            p_b = member;
            p_u += teams;
        }
    };
    for (int i = 0; i < a.l.ring; ++i) issue();

    const WaitCtx ctx{a.status, &s_abort, a.timeout_ns};
    const float2* x_scale = reinterpret_cast<const float2*>(smem + a.l.x_scale);
    float4* partial = reinterpret_cast<float4*>(smem + a.l.partial);
    const int q = lane & 3, g8 = lane >> 2;
    // ldmatrix: lane l addresses row l % 8 of matrix l / 8: rows 0-7 and 8-15
    // of one group, then of the next; 16-byte chunks are XOR-swizzled by row
    const uint32_t lm_row = ((lane >> 3) & 1) * (kBoxBytes / 2) + (lane & 7) * 128;
    int used = 0, turn = 0;
    for (int run = u0; run < u1;) {
        const int end = run_end(run);
        const int ncols = tb.ncols[run / tiles];
        if (run > u0) __syncthreads();       // everybody is done with the rows before
        load_x(a, tb, smem, run / tiles, nb);
        __syncthreads();
        const bool col = g8 < ncols;
        const uint32_t x_at = base + a.l.x + g8 * a.l.x_stride + 16 * q;
        for (int u = run + team; u < end; u += teams, ++turn) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int b = member; b < nb; b += team_warps, ++used) {
                const int at = used % a.l.ring;
                const bool ok = __all_sync(0xFFFFFFFFu, wait_bounded(bars + 8 * at,
                                                                     (used / a.l.ring) & 1, ctx,
                                                                     kRoleMatvec, used));
                if (ok) {
                    const uint32_t w_at = ring_w + at * kBoxBytes + lm_row;
                    const uint32_t s_at = a.l.scales + (warp * a.l.ring + at) * kBoxScaleBytes;
                    const uint2 code_lo = *reinterpret_cast<const uint2*>(smem + s_at + 8 * g8);
                    const uint2 code_hi = *reinterpret_cast<const uint2*>(smem + s_at + 64 + 8 * g8);
                    const float2 sx = x_scale[b * (kMaxCols / 2) + q];
#pragma unroll
                    for (int g = 0; g < 8; g += 2) {
                        uint32_t w[4];
                        ptx::ldmatrix_x4(w_at + (((g + (lane >> 4)) ^ (lane & 7)) << 4), w);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint4 xv = make_uint4(0, 0, 0, 0);
                            if (col) xv = ptx::lds_v4(x_at + 2 * (b * kBoxK + 32 * (g + i)));
                            uint32_t lo[4], hi[4];
                            ptx::e2m1x8_to_f16(w[2 * i], lo);
                            ptx::e2m1x8_to_f16(w[2 * i + 1], hi);
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            ptx::mma_f16_16816(d, lo[0], hi[0], lo[1], hi[1], xv.x, xv.y);
                            ptx::mma_f16_16816(d, lo[2], hi[2], lo[3], hi[3], xv.z, xv.w);
                            const float s_lo = scale_of(code_lo, g + i);
                            const float s_hi = scale_of(code_hi, g + i);
                            acc[0] = fmaf(d[0], s_lo * sx.x, acc[0]);
                            acc[1] = fmaf(d[1], s_lo * sx.y, acc[1]);
                            acc[2] = fmaf(d[2], s_hi * sx.x, acc[2]);
                            acc[3] = fmaf(d[3], s_hi * sx.y, acc[3]);
                        }
                    }
                }
                __syncwarp();                // the box is read: its place may be refilled
                if (ok) issue();
            }
            // join: two buffers, so that one barrier a unit is enough
            float4* part = partial + (turn & 1) * kWarps * 32 + team * team_warps * 32;
            if (team_warps > 1) {
                part[member * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                ptx::named_barrier(1 + team, 32 * team_warps);
                if (member != turn % team_warps) continue;
                acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
                for (int m = 0; m < min(team_warps, nb); ++m) {
                    const float4 v = part[m * 32 + lane];
                    acc[0] += v.x;
                    acc[1] += v.y;
                    acc[2] += v.z;
                    acc[3] += v.w;
                }
            }
            const int chunk = u / tiles;
            const int n0 = (u - chunk * tiles) * tile_cols + g8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (2 * q + i >= ncols) continue;
                const long long o =
                    static_cast<long long>(tb.slot[chunk * kMaxCols + 2 * q + i]) * out_cols;
                if (kSwiglu) {
                    const float y = acc[i], up = acc[2 + i];
                    if (n0 < out_cols)
                        a.out[o + n0] = __bfloat16_as_ushort(
                            __float2bfloat16_rn(y / (1.0f + expf(-y)) * up));
                } else {
                    if (n0 < out_cols)
                        a.out[o + n0] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i]));
                    if (n0 + 8 < out_cols)
                        a.out[o + n0 + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[2 + i]));
                }
            }
        }
        run = end;
    }
    // After a wait that gave up, copies may still be in flight: wait for them,
    // again with a limit, before the shared memory is given back.
    if (*ctx.abort) {
        const uint64_t t0 = ptx::globaltimer_ns();
        for (int i = max(0, issued - a.l.ring); i < issued; ++i) {
            while (!ptx::mbar_try_wait(bars + 8 * (i % a.l.ring), (i / a.l.ring) & 1) &&
                   ptx::globaltimer_ns() - t0 < a.timeout_ns) {
            }
        }
    }
}

template <bool kSwiglu>
cudaError_t launch(const CUtensorMap& map, const KernelArgs& k, int grid, cudaStream_t stream) {
    const cudaError_t err = cudaFuncSetAttribute(expert_matvec_kernel<kSwiglu>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kSmemLimit);
    if (err != cudaSuccess) return err;
    expert_matvec_kernel<kSwiglu><<<grid, kThreads, k.l.total, stream>>>(map, k);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_matvec(const MatvecArgs& a, const CUtensorMap& map_w, int num_sms,
                                 cudaStream_t stream) {
    KernelArgs k;
    k.x = a.x;
    k.ids = a.ids;
    k.w_scale = a.w_scale;
    k.out = a.out;
    k.status = a.status;
    k.timeout_ns = a.timeout_ns;
    k.slots_per_row = a.slots_per_row;
    k.slots = a.slots;
    k.E = a.E;
    k.N = a.N;
    k.K = a.K;
    if (!make_layout(a.K, a.slots, a.tokens, &k.l)) return cudaErrorInvalidValue;
    const int tile_cols = a.swiglu ? kRows / 2 : kRows;
    const long long tiles = ((a.swiglu ? a.N / 2 : a.N) + tile_cols - 1) / tile_cols;
    const long long units = tiles * a.slots;
    const int grid = static_cast<int>(units < num_sms ? units : num_sms);
    return a.swiglu ? launch<true>(map_w, k, grid, stream) : launch<false>(map_w, k, grid, stream);
}

}  // namespace hg

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
// fills by TMA, and runs ahead of its own use of them by the ring's depth.  The
// boxes of a block's units, in order, go to its 16 warps in turn, so that all
// have the same work whatever K is; a unit's partial sums meet in shared memory,
// in a fixed order (the result does not depend on timing), and the warp of the
// unit's last box writes the outputs.  Nobody else waits for that: the sums of
// several units may be under way at once.
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
constexpr int kTileCols = 8;                 // slots of an MMA: its N
constexpr int kMaxCols = 16;                 // slots of a chunk: at most two MMAs
constexpr int kHalfK = 256;                  // elements of 128 bytes of a weight row
constexpr int kHalfBytes = kRows * kHalfK / 2;
constexpr int kHalfScaleBytes = kRows * kHalfK / 32;
constexpr int kMaxRing = 4;                  // boxes in flight per warp
constexpr int kMaxUnderWay = 4;              // units whose partial sums are kept at once
constexpr int kSmemLimit = 232448 - 256;     // beside a few static bytes

// The slots by expert: an entry per slot or chunk (there are at most as many
// chunks as slots).
struct Tables {
    int* id;
    int* expert;             // of a chunk
    int* ncols;              // of a chunk
    uint16_t* chunk_of;      // of a chunk's first slot
    uint16_t* slot;          // of a chunk's columns: chunk * cols + column
    uint8_t* same_rows;      // the chunk's input rows are those of the one before
    int* warp_count;
};

// For n slots; in multiples of 4 bytes.
__host__ __device__ inline int table_bytes(int slots, int cols) {
    const int n = (slots + 3) & ~3;
    return n * (3 * 4 + 2 + 2 * cols + 1) + kWarps * 4;
}

__device__ inline Tables tables_at(uint8_t* p, int slots, int cols) {
    const int n = (slots + 3) & ~3;
    Tables t;
    t.warp_count = reinterpret_cast<int*>(p);
    t.id = t.warp_count + kWarps;
    t.expert = t.id + n;
    t.ncols = t.expert + n;
    t.chunk_of = reinterpret_cast<uint16_t*>(t.ncols + n);
    t.slot = t.chunk_of + n;
    t.same_rows = reinterpret_cast<uint8_t*>(t.slot + n * cols);
    return t;
}

struct Layout {
    int ring;          // boxes per warp
    int cols;          // most slots of a chunk
    int x_stride;      // bytes between the columns of x
    int scales, partial, x, x_scale, zeros, bars, tables, total;   // byte offsets
};

// 256-K halves of a box: a single column's work is light, and two at a time
// halve what a box costs besides.
__host__ __device__ constexpr int box_halves(int cols) { return cols == 1 ? 2 : 1; }

// Partial sums of the units under way: a float per weight row of a single
// column, 16 x 8 floats per MMA otherwise, from every warp.
int partial_bytes(int cols) {
    return kWarps * (cols == 1 ? kMaxUnderWay * kRows * 4 : kMaxUnderWay * kRows * kTileCols * 4);
}

// As many columns as fit beside a ring of at least two boxes a warp, then as
// deep a ring as fits.  Columns stay 64 bytes off a multiple of 128 apart, so
// that the eight lanes of a 16-byte load phase (two columns) meet no bank
// twice.
bool make_layout(int K, int slots, int tokens, Layout* out) {
    const int halves = (K + kHalfK - 1) / kHalfK + 1;   // a box may reach one past the end
    Layout l;
    l.x_stride = halves * kHalfK * 2 + 64;
    auto box = [](int cols) { return kWarps * box_halves(cols) * (kHalfBytes + kHalfScaleBytes); };
    auto needs = [&](int cols) {
        return 1024 + partial_bytes(cols) + cols * l.x_stride + halves * kMaxCols * 4 +
               2 * kHalfK + (kWarps * kMaxRing + 2 * kMaxUnderWay) * 8 + table_bytes(slots, cols);
    };
    int cols = tokens < kMaxCols ? tokens : kMaxCols;   // a token's choices are distinct experts
    if (cols > slots) cols = slots;
    while (cols > 1 && needs(cols) + 2 * box(cols) > kSmemLimit) --cols;
    l.cols = cols;
    l.ring = (kSmemLimit - needs(cols)) / box(cols);
    if (l.ring > kMaxRing) l.ring = kMaxRing;
    if (l.ring < 1) return false;
    const int ring = kWarps * l.ring * box_halves(cols);
    l.scales = ring * kHalfBytes;
    l.partial = l.scales + ring * kHalfScaleBytes;
    l.x = l.partial + partial_bytes(cols);
    l.x_scale = l.x + cols * l.x_stride;
    l.zeros = l.x_scale + halves * kMaxCols * 4;
    l.bars = l.zeros + 2 * kHalfK;
    l.tables = l.bars + (kWarps * l.ring + 2 * kMaxUnderWay) * 8;
    l.total = l.tables + table_bytes(slots, cols) + 1024;
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
__device__ int list_slots(const KernelArgs& a, const Tables& tb) {
    const int s = threadIdx.x;
    const bool mine = s < a.slots;
    if (a.slots <= 32) {                     // one warp sees all slots at once
        if (s < 32) {
            const int e = mine ? __ldg(a.ids + s) : -1;
            const bool valid = e >= 0 && e < a.E;
            const uint32_t below = (1u << s) - 1u;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, valid ? e : -1);
            const int rank = __popc(same & below);
            const int col = rank % a.l.cols;
            const uint32_t leads = __ballot_sync(0xFFFFFFFFu, valid && col == 0);
            // the chunk's first slot: the last leader of this expert up to here
            const int lead = 31 - __clz(same & leads & (below | (1u << s)));
            const int c = __popc(leads & ((1u << (lead & 31)) - 1u));
            if (mine) tb.id[s] = e;
            if (valid) tb.slot[c * a.l.cols + col] = static_cast<uint16_t>(s);
            const int cols_here = min(a.l.cols, __popc(same) - (rank - col));
            if (valid && col == 0) {
                tb.expert[c] = e;
                tb.ncols[c] = cols_here;
            }
            __syncwarp();
            const int total = __popc(leads);
            if (s < total) {
                bool rows = s > 0 && tb.ncols[s] == tb.ncols[s - 1];
                for (int i = 0; rows && i < tb.ncols[s]; ++i) {
                    rows = tb.slot[s * a.l.cols + i] / a.slots_per_row ==
                           tb.slot[(s - 1) * a.l.cols + i] / a.slots_per_row;
                }
                tb.same_rows[s] = rows;
            }
            if (s == 0) tb.warp_count[0] = total;
        }
        __syncthreads();
        return tb.warp_count[0];
    }
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
        tb.slot[c * a.l.cols + rank % a.l.cols] = static_cast<uint16_t>(s);
        atomicAdd(&tb.ncols[c], 1);
    }
    __syncthreads();
    if (s < total) {
        bool same = s > 0 && tb.ncols[s] == tb.ncols[s - 1];
        for (int i = 0; same && i < tb.ncols[s]; ++i) {
            same = tb.slot[s * a.l.cols + i] / a.slots_per_row ==
                   tb.slot[(s - 1) * a.l.cols + i] / a.slots_per_row;
        }
        tb.same_rows[s] = same;
    }
    __syncthreads();
    return total;
}

// The chunk's input rows into shared memory as scaled FP16, with one scale per
// row and 256 elements: a warp handles these at a time, eight a lane.
__device__ void load_x(const KernelArgs& a, const Tables& tb, uint8_t* smem, int chunk, int halves) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ncols = tb.ncols[chunk];
    float* scale = reinterpret_cast<float*>(smem + a.l.x_scale);
    for (int i = threadIdx.x; i < halves * kMaxCols; i += kThreads) {
        if (i % kMaxCols >= ncols) scale[i] = 0.0f;
    }
    for (int i = warp; i < halves * ncols; i += kWarps) {
        const int c = i / halves, b = i - c * halves;
        const int row = tb.slot[chunk * a.l.cols + c] / a.slots_per_row;
        const int k = b * kHalfK + 8 * lane;
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
        if (lane == 0) scale[b * kMaxCols + c] = back;
    }
}

// 256 K of 16 weight rows times one column.  Were the column alone in the
// MMA's eight, each 32-K group would need its own scaling of 16 x 8 sums.
// Instead column c of x holds the elements of group c, so that one load serves
// all eight groups, and of group g's product only column g is kept: a lane
// keeps groups 2q and 2q + 1 of its two rows, and scales four sums in place of
// thirty-two.
__device__ __forceinline__ void single_half(uint32_t w_at, uint32_t x_at, uint32_t code_lo,
                                            uint32_t code_hi, float sx, int lane,
                                            float (&acc)[2]) {
    const int q = lane & 3;
    const uint4 xv = ptx::lds_v4(x_at + 16 * lane);
    float v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {                            // groups 2p and 2p + 1
        uint32_t w[4];
        ptx::ldmatrix_x4(w_at + (((2 * p + (lane >> 4)) ^ (lane & 7)) << 4), w);
        float d[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t lo[4], hi[4];
            ptx::e2m1x8_to_f16(w[2 * i], lo);
            ptx::e2m1x8_to_f16(w[2 * i + 1], hi);
            d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
            ptx::mma_f16_16816(d[i], lo[0], hi[0], lo[1], hi[1], xv.x, xv.y);
            ptx::mma_f16_16816(d[i], lo[2], hi[2], lo[3], hi[3], xv.z, xv.w);
        }
        if (p == 0 || q == p) {
            v[0] = d[0][0];
            v[1] = d[1][1];
            v[2] = d[0][2];
            v[3] = d[1][3];
        }
    }
    const float2 s_lo = ptx::e8m0x2_to_f32(code_lo), s_hi = ptx::e8m0x2_to_f32(code_hi);
    acc[0] = fmaf(v[0], s_lo.x * sx, acc[0]);
    acc[0] = fmaf(v[1], s_lo.y * sx, acc[0]);
    acc[1] = fmaf(v[2], s_hi.x * sx, acc[1]);
    acc[1] = fmaf(v[3], s_hi.y * sx, acc[1]);
}

// kTiles: MMAs side by side, eight slots each; 0: a single slot.
template <bool kSwiglu, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
expert_matvec_kernel(const __grid_constant__ CUtensorMap map_w, const KernelArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_abort;
    constexpr bool kSingle = kTiles == 0;
    constexpr int kT = kSingle ? 1 : kTiles;
    constexpr int kUnderWay = kMaxUnderWay / kT;
    constexpr int kHalves = box_halves(kSingle ? 1 : kTileCols);
    constexpr int kBoxK = kHalves * kHalfK;
    constexpr int kBoxBytes = kHalves * kHalfBytes;
    constexpr int kBoxScaleBytes = kHalves * kHalfScaleBytes;
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const Tables tb = tables_at(smem + a.l.tables, a.slots, a.l.cols);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = (a.K + kBoxK - 1) / kBoxK;
    const int sharers = min(nb, kWarps);                     // warps that work on one unit
    const int out_cols = kSwiglu ? a.N / 2 : a.N;
    const int tile_cols = kSwiglu ? kRows / 2 : kRows;       // outputs of a unit
    const int tiles = (out_cols + tile_cols - 1) / tile_cols;
    const uint32_t bars = base + a.l.bars + 8 * warp * a.l.ring;
    const uint32_t full = base + a.l.bars + 8 * kWarps * a.l.ring;
    const uint32_t empty = full + 8 * kMaxUnderWay;

    if (lane == 0) {
        for (int i = 0; i < a.l.ring; ++i) ptx::mbar_init(bars + 8 * i, 33);
        if (warp == 0) {
            ptx::prefetch_tensormap(&map_w);
            s_abort = 0;
            for (int i = 0; i < kUnderWay; ++i) {
                ptx::mbar_init(full + 8 * i, sharers);
                ptx::mbar_init(empty + 8 * i, 1);
            }
        }
        ptx::fence_barrier_init();
    }
    if (!kSingle && threadIdx.x < kHalfK / 2)
        reinterpret_cast<uint32_t*>(smem + a.l.zeros)[threadIdx.x] = 0;
    const int chunks = list_slots(a, tb);    // has block barriers

    const long long units = static_cast<long long>(chunks) * tiles;
    const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);

    // End of the run of units from `u` that share their input rows.
    auto run_end = [&](int u) {
        int c = u / tiles + 1;
        while (c < chunks && tb.same_rows[c]) ++c;
        return min(c * tiles, u1);
    };

    // Boxes of a run in order, box b of unit u at (u - run) * nb + b: this warp
    // takes every 16th.
    const int step_u = kWarps / nb, step_b = kWarps % nb;
    const int first_u = warp / nb, first_b = warp % nb;

    // What this warp has asked for so far.
    const int groups = a.K / 32;
    const uint32_t ring_w = base + warp * a.l.ring * kBoxBytes;
    const uint32_t ring_s = base + a.l.scales + warp * a.l.ring * kBoxScaleBytes;
    int p_u = u0 + first_u, p_b = first_b, p_end = u0 < u1 ? run_end(u0) : u0;
    int p_chunk = u0 / tiles, p_known = -1, p_n0 = 0, p_expert = 0, p_at = 0, issued = 0;
    const uint8_t* p_scale = nullptr;
    auto issue = [&]() {
        while (p_u >= p_end) {
            if (p_end >= u1) return;
            p_u = p_end + first_u;
            p_b = first_b;
            p_end = run_end(p_end);
        }
        if (p_u != p_known) {
            p_known = p_u;
            while (p_u >= (p_chunk + 1) * tiles) ++p_chunk;
            p_n0 = (p_u - p_chunk * tiles) * tile_cols;
            p_expert = tb.expert[p_chunk];
            // lane l copies half of row l / 2's scales; rows past the end of the
            // expert's are not used
            const int r = lane >> 1;
            const int n = kSwiglu ? min(p_n0 + (r & 7), out_cols - 1) + (r >> 3) * out_cols
                                  : min(p_n0 + r, out_cols - 1);
            p_scale = a.w_scale + (static_cast<long long>(p_expert) * a.N + n) * groups;
        }
        const uint32_t bar = bars + 8 * p_at;
        if (lane == 0) {
            const uint32_t dst = ring_w + p_at * kBoxBytes;
            const int z = kSwiglu ? 2 * p_expert : p_expert;
            ptx::mbar_arrive_expect_tx(bar, kBoxBytes);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
                ptx::tma_load_3d(dst + h * kHalfBytes, &map_w, (kHalves * p_b + h) * (kHalfK / 2),
                                 p_n0, z, bar);
        }
        const int g = kHalves * (8 * p_b + 4 * (lane & 1));
        const uint32_t to = ring_s + p_at * kBoxScaleBytes + 4 * kHalves * lane;
        if (kHalves == 1) {
            ptx::cp_async_4(to, p_scale + (g < groups ? g : 0), g < groups);
        } else if (groups & 7) {             // rows of scales start at multiples of 4 bytes
            ptx::cp_async_4(to, p_scale + (g < groups ? g : 0), g < groups);
            ptx::cp_async_4(to + 4, p_scale + (g + 4 < groups ? g + 4 : 0), g + 4 < groups);
        } else {
            ptx::cp_async_8(to, p_scale + (g < groups ? g : 0), g < groups);
        }
        ptx::cp_async_mbar_arrive(bar);
        ++issued;
        if (++p_at == a.l.ring) p_at = 0;
        p_u += step_u;
        p_b += step_b;
        if (p_b >= nb) {
            p_b -= nb;
            ++p_u;
        }
    };
    for (int i = 0; i < a.l.ring; ++i) issue();

    // slots without an expert: zeros, spread over the grid
    for (int s = 0; s < a.slots; ++s) {
        if (tb.id[s] >= 0 && tb.id[s] < a.E) continue;
        for (int n = blockIdx.x * kThreads + threadIdx.x; n < out_cols; n += gridDim.x * kThreads)
            a.out[static_cast<long long>(s) * out_cols + n] = 0;
    }

    const WaitCtx ctx{a.status, &s_abort, a.timeout_ns};
    const float* x_scale = reinterpret_cast<const float*>(smem + a.l.x_scale);
    float* partial = reinterpret_cast<float*>(smem + a.l.partial);
    const int q = lane & 3, g8 = lane >> 2;
    // ldmatrix: lane l addresses row l % 8 of matrix l / 8: rows 0-7 and 8-15
    // of one group, then of the next; 16-byte chunks are XOR-swizzled by row
    const uint32_t lm_row = ring_w + ((lane >> 3) & 1) * (kHalfBytes / 2) + (lane & 7) * 128;
    const uint8_t* my_scales = smem + a.l.scales + warp * a.l.ring * kBoxScaleBytes;
    int at = 0;
    uint32_t phase = 0;
    for (int run = u0, before = 0; run < u1;) {              // before: units of earlier runs
        const int end = run_end(run);
        const int ncols = tb.ncols[run / tiles];
        if (run > u0) __syncthreads();       // everybody is done with the rows before
        load_x(a, tb, smem, run / tiles, kHalves * nb);
        __syncthreads();
        int chunk = run / tiles;
        // lanes of columns that the chunk does not have read zeros
        uint32_t x_at[kT], x_step[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const bool there = 8 * t + g8 < ncols;
            x_at[t] = base + (there ? a.l.x + (8 * t + g8) * a.l.x_stride : a.l.zeros) + 16 * q;
            x_step[t] = there ? 2 * kHalfK : 0;
        }
        float acc[kT][4];
#pragma unroll
        for (int i = 0; i < 4 * kT; ++i) acc[i >> 2][i & 3] = 0.0f;
        float one[2] = {0.0f, 0.0f};
        for (int u = run + first_u, b = first_b; u < end;) {
            const bool ok = __all_sync(0xFFFFFFFFu,
                                       wait_bounded(bars + 8 * at, phase, ctx, kRoleMatvec, at));
            if (ok) {
                const uint8_t* codes = my_scales + at * kBoxScaleBytes + 8 * kHalves * g8;
                if (kSingle) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        single_half(lm_row + at * kBoxBytes + h * kHalfBytes,
                                    base + a.l.x + (2 * b + h) * (2 * kHalfK),
                                    *reinterpret_cast<const uint16_t*>(codes + 8 * h + 2 * q),
                                    *reinterpret_cast<const uint16_t*>(codes + 128 + 8 * h + 2 * q),
                                    x_scale[(2 * b + h) * kMaxCols], lane, one);
                    }
                } else {
                    const uint2 code_lo = *reinterpret_cast<const uint2*>(codes);
                    const uint2 code_hi = *reinterpret_cast<const uint2*>(codes + 64);
                    const uint32_t w_at = lm_row + at * kBoxBytes;
                    float2 sx[kT];
#pragma unroll
                    for (int t = 0; t < kT; ++t)
                        sx[t] = *reinterpret_cast<const float2*>(x_scale + b * kMaxCols + 8 * t +
                                                                 2 * q);
                    float s_lo[4], s_hi[4];
#pragma unroll
                    for (int g = 0; g < 8; g += 2) {
                        if (g % 4 == 0) {
                            ptx::e8m0x4_to_f32(g ? code_lo.y : code_lo.x, s_lo);
                            ptx::e8m0x4_to_f32(g ? code_hi.y : code_hi.x, s_hi);
                        }
                        uint32_t w[4];
                        ptx::ldmatrix_x4(w_at + (((g + (lane >> 4)) ^ (lane & 7)) << 4), w);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t lo[4], hi[4];
                            ptx::e2m1x8_to_f16(w[2 * i], lo);
                            ptx::e2m1x8_to_f16(w[2 * i + 1], hi);
#pragma unroll
                            for (int t = 0; t < kT; ++t) {
                                const uint4 xv =
                                    ptx::lds_v4(x_at[t] + b * x_step[t] + 64 * (g + i));
                                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                ptx::mma_f16_16816(d, lo[0], hi[0], lo[1], hi[1], xv.x, xv.y);
                                ptx::mma_f16_16816(d, lo[2], hi[2], lo[3], hi[3], xv.z, xv.w);
                                const float a_lo = s_lo[g % 4 + i], a_hi = s_hi[g % 4 + i];
                                acc[t][0] = fmaf(d[0], a_lo * sx[t].x, acc[t][0]);
                                acc[t][1] = fmaf(d[1], a_lo * sx[t].y, acc[t][1]);
                                acc[t][2] = fmaf(d[2], a_hi * sx[t].x, acc[t][2]);
                                acc[t][3] = fmaf(d[3], a_hi * sx[t].y, acc[t][3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();                    // the box is read: its place may be refilled
            if (ok) issue();
            if (++at == a.l.ring) {
                at = 0;
                phase ^= 1;
            }
            const int done = u;
            const bool last_box = b == nb - 1;
            u += step_u;
            b += step_b;
            if (b >= nb) {
                b -= nb;
                ++u;
            }
            if (u == done) continue;

            // This warp's part of unit `done` is complete: leave it, and if the
            // unit's last box was here, join the parts and write the outputs.
            const int n_unit = before + done - run;
            const int place = n_unit % kUnderWay;
            const uint32_t round = (n_unit / kUnderWay) & 1;
            const int w0 = warp - (sharers - 1);             // the unit's first sharer, cyclically
            wait_bounded(empty + 8 * place, round ^ 1, ctx, kRoleMatvec, 0x100 + place);
            if (kSingle) {
                float* part = partial + place * kWarps * kRows;
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
                    one[0] += __shfl_xor_sync(0xFFFFFFFFu, one[0], o);
                    one[1] += __shfl_xor_sync(0xFFFFFFFFu, one[1], o);
                }
                if (q < 2) part[warp * kRows + 8 * q + g8] = q ? one[1] : one[0];
                one[0] = one[1] = 0.0f;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full + 8 * place);
                if (!last_box) continue;
                wait_bounded(full + 8 * place, round, ctx, kRoleMatvec, 0x200 + place);
                float y = 0.0f;
#pragma unroll 4
                for (int j = 0; j < sharers; ++j)
                    y += part[((w0 + j) & (kWarps - 1)) * kRows + (lane & 15)];
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty + 8 * place);
                while (done >= (chunk + 1) * tiles) ++chunk;
                const int n = (done - chunk * tiles) * tile_cols + lane;
                if (kSwiglu) {
                    const float up = __shfl_down_sync(0xFFFFFFFFu, y, 8);
                    y = y / (1.0f + expf(-y)) * up;
                }
                if (lane < tile_cols && n < out_cols)
                    a.out[static_cast<long long>(tb.slot[chunk]) * out_cols + n] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(y));
            } else {
                float4* part = reinterpret_cast<float4*>(partial) + place * kWarps * kT * 32 + lane;
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    part[(warp * kT + t) * 32] =
                        make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full + 8 * place);
                if (!last_box) continue;
                wait_bounded(full + 8 * place, round, ctx, kRoleMatvec, 0x200 + place);
                while (done >= (chunk + 1) * tiles) ++chunk;
                const int n0 = (done - chunk * tiles) * tile_cols + g8;
                float4 sum[kT];
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    sum[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int j = 0; j < sharers; ++j) {
                        const float4 v = part[(((w0 + j) & (kWarps - 1)) * kT + t) * 32];
                        sum[t].x += v.x;
                        sum[t].y += v.y;
                        sum[t].z += v.z;
                        sum[t].w += v.w;
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty + 8 * place);
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    const float y[4] = {sum[t].x, sum[t].y, sum[t].z, sum[t].w};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = 8 * t + 2 * q + i;
                        if (c >= ncols) continue;
                        uint16_t* o = a.out + static_cast<long long>(
                                                  tb.slot[chunk * a.l.cols + c]) * out_cols + n0;
                        if (kSwiglu) {
                            if (n0 < out_cols)
                                o[0] = __bfloat16_as_ushort(
                                    __float2bfloat16_rn(y[i] / (1.0f + expf(-y[i])) * y[2 + i]));
                        } else {
                            if (n0 < out_cols)
                                o[0] = __bfloat16_as_ushort(__float2bfloat16_rn(y[i]));
                            if (n0 + 8 < out_cols)
                                o[8] = __bfloat16_as_ushort(__float2bfloat16_rn(y[2 + i]));
                        }
                    }
                }
            }
        }
        before += end - run;
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

template <bool kSwiglu, int kTiles>
cudaError_t launch(const CUtensorMap& map, const KernelArgs& k, int grid, cudaStream_t stream) {
    const cudaError_t err = cudaFuncSetAttribute(expert_matvec_kernel<kSwiglu, kTiles>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kSmemLimit);
    if (err != cudaSuccess) return err;
    expert_matvec_kernel<kSwiglu, kTiles><<<grid, kThreads, k.l.total, stream>>>(map, k);
    return cudaGetLastError();
}

template <bool kSwiglu>
cudaError_t launch_cols(const CUtensorMap& map, const KernelArgs& k, int grid,
                        cudaStream_t stream) {
    if (k.l.cols == 1) return launch<kSwiglu, 0>(map, k, grid, stream);
    if (k.l.cols <= kTileCols) return launch<kSwiglu, 1>(map, k, grid, stream);
    return launch<kSwiglu, 2>(map, k, grid, stream);
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
    return a.swiglu ? launch_cols<true>(map_w, k, grid, stream)
                    : launch_cols<false>(map_w, k, grid, stream);
}

}  // namespace hg

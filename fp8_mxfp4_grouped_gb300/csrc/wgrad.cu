// wgrad.cu -- the gradient of every expert's weights, a matrix product over the rows
// that the plan gave to the expert:
//
//   dw[e, n, k] (+)= sum over r in [off[e], off[e+1]) of dy[r, n] * x[r, k]
//
// with dy and x in BF16, or x as the forward pass had it, E4M3 codes with one E8M0 scale
// per 128 of a row.  Sums in FP32.
//
// A CTA pair computes 256 x 256 of one expert's dw with tcgen05 cta_group::2 MMAs (M = 256,
// N = 256, K = 16 rows).  The rows of dy and x are the K of the product, so that both
// operands lie in memory with K as the slow axis: TMA boxes of 128 rows x 64 columns are
// MN-major panels as they are.  Roles in a CTA: warp 0 TMA producer, warp 1 TMEM
// allocation and (in the even CTA) MMA issue, warp 2 the last stage of an expert, warps
// 4-11 epilogue.  An expert's last stage can hold rows of the next expert: warp 2 clears
// them in both operands (a NaN there must not meet a zero) before the MMAs see them.
//
// FP8 codes are turned into BF16 by a kernel of its own before, which is exact (three
// mantissa bits times a power of two): 46 us for 16384 x 6144.  Turning them on their way
// through shared memory, by eight warps beside the others, was slower by more than that
// (1002 us against 795 for the product itself at 32 x 4096 x 6144): the codes' write and read
// and the BF16's write come on top of 128 bytes a cycle that the MMAs and the copies use
// of shared memory.
//
// The tensor core adds to its accumulator by cutting, not by rounding: the sum loses some
// 2^-24 of itself with each MMA, 9e-7 of a sum of positive terms over 512 rows and 1.8e-4
// over 32768.  After kChunk stages the epilogue therefore takes an accumulator over into
// its registers, where sums round.
//
// What bounds it: for long sums the tensor cores (4 x 4096 x 4096 over 32768 rows, BF16, 597 us,
// 1840 TFLOP/s).  For experts of some 512 rows nothing that was measured is full: 8 x 4096 x 6144
// in FP32 of 512 rows each keep the SMs' ports to the L2 busy for 74 % of the time (49 % with the
// stores of dw), HBM for 57 %, the L2 for 52 % and the tensor cores for 48 %.  32 x 4096 x 6144
// over 16384 rows, BF16 x, take 794 us with skewed routing (512 rows each 715 to 731), 836 from FP8
// (764 to 769).  Copies alone take 396 us there, the stores 494, both 709, which is neither the
// larger nor the sum; the MMAs at the rate of long sums would take 454.  How the rows fall on the
// pairs counts too: 10 % with these many tiles, and with few the fullest expert's tiles decide
// (8 x 1024 x 512 over 32768 rows 57 us against 30 with equal experts, a floor of 18), since a
// tile is one pair's and wgrad_splits knows the average expert only.
//
// Tried and not kept, at the 794 us: stores by the threads instead of TMA (955 us, from
// registers 890), 16 KB store boxes (809), two store buffers a warp for a stage less (867), dy
// kept in shared memory for several tiles with x in the two remaining slots (1040: too few
// bytes of x in flight), the tiles walked along k (795), pairs started apart in time (no
// change), 256 x 512 a pair for experts of up to 1024 rows and two passes for longer ones (869;
// 512 rows each 700 against 714; 32 x 4096 x 2048 to BF16 of 200 rows each 123 against 130).
#include <atomic>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kTile = 256;                   // dw rows and columns of a pair's unit
constexpr int kHalf = 128;                   // dy columns and x columns that a CTA loads
constexpr int kEpiWarps = 8;                 // four lane quarters x two halves of the columns
constexpr int kEpiCols = kTile * 4 / kEpiWarps;
constexpr int kPanel = kWgradRows * 128;     // bytes of a stage of 64 16-bit columns
constexpr int kOperand = 2 * kPanel;         // a CTA's part of an operand's stage
constexpr int kOutBuf = 32 * 128;            // a warp's 32 rows x 128 bytes of output
constexpr int kTmemCols = 512;               // two accumulators of 256 columns
constexpr int kMmaRows = 16;                 // K of an MMA

// Stages of an accumulator: 512 rows.
constexpr int kChunk = 512 / kWgradRows;

constexpr int kThreads = 384;
constexpr int kStages = 3;
constexpr int kOffA = 0;
constexpr int kOffB = kOffA + kStages * kOperand;
constexpr int kOffOut = kOffB + kStages * kOperand;
constexpr int kOffBar = kOffOut + kEpiWarps * kOutBuf;
constexpr int kOffMisc = kOffBar + 8 * (4 * kStages + 5);
constexpr int kSmem = kOffMisc + 16 + 1024;  // with room to align to 1024
static_assert(kSmem <= 227 * 1024, "shared memory of an SM");

struct Shape {
    int E, N, K, rows, splits, tiles_n, tiles_k;
    int dy_panels, x_panels;                 // of 64 columns in a box: 1 or 2
};

// A unit of work: the tile's place, and the rows that are summed.
struct Unit {
    int e, n0, k0, split, row0, rows;
    bool bad;
    // u may be past the last unit: any expert's offsets are read then
    __device__ __forceinline__ Unit(const Shape& s, const int32_t* offsets, int u) {
        const int tn = u % s.tiles_n;
        u /= s.tiles_n;
        const int tk = u % s.tiles_k;
        u /= s.tiles_k;
        split = u % s.splits;
        e = min(u / s.splits, s.E - 1);
        n0 = tn * kTile;
        k0 = tk * kTile;
        const int lo = ptx::load(offsets + e), hi = ptx::load(offsets + e + 1);
        bad = lo < 0 || hi < lo || hi > s.rows;
        const int all = bad ? 0 : hi - lo;
        const int stages = (all + kWgradRows - 1) / kWgradRows;
        const int part = (stages + s.splits - 1) / s.splits * kWgradRows;
        row0 = lo + split * part;
        rows = max(0, min(part, all - split * part));
    }
    __device__ __forceinline__ int stages() const { return (rows + kWgradRows - 1) / kWgradRows; }
    // whether the MMAs of a stage meet rows that are not the unit's
    __device__ __forceinline__ bool mixed(int stage) const {
        return rows - stage * kWgradRows < kWgradRows && rows % kMmaRows != 0;
    }
    // rows of a stage that belong to the unit
    __device__ __forceinline__ int valid(int stage) const {
        return min(kWgradRows, rows - stage * kWgradRows);
    }
};

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Clear rows [first, last) of an operand's stage (whole warp).
__device__ __forceinline__ void clear_rows(uint32_t operand, int first, int last) {
    operand += first * 128;
    for (int i = threadIdx.x & 31; i < (last - first) * 16; i += 32)
        sts_v4(operand + ((i >> 3) & 1) * kPanel + (i >> 4) * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
}

// A CTA's 128 columns of a stage, counted on a barrier of either CTA: two panels of 64
// columns, one behind the other.
__device__ __forceinline__ void load_stage(uint32_t to, const CUtensorMap* map, int panels, int col,
                                           int row, uint32_t bar, uint64_t policy) {
    if (panels == 2) {
        ptx::tma_load_3d_pair_elect(to, map, 0, row, col / 64, bar, policy);
    } else {
        ptx::tma_load_3d_pair_elect(to, map, col, row, 0, bar, policy);
        ptx::tma_load_3d_pair_elect(to + kPanel, map, col + 64, row, 0, bar, policy);
    }
}

template <bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ WgradMaps maps, const Shape shape, const int32_t* offsets,
             int accumulate, int parts, uint32_t* status, uint64_t timeout_ns) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = ptx::smem_u32(smem_raw);
    const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (sbase - raw_u32);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;

    // full (even CTA): both CTAs' bytes of a stage have landed.  empty: its MMAs are done.
    // last: this CTA's bytes of an expert's last stage have landed; clear (even CTA): the odd
    // CTA's are cleared.
    const uint32_t bar_full = sbase + kOffBar;
    const uint32_t bar_empty = bar_full + 8 * kStages;
    const uint32_t bar_tfull = bar_empty + 8 * kStages;
    const uint32_t bar_tempty = bar_tfull + 16;          // even CTA: both have read TMEM
    const uint32_t bar_last = bar_tempty + 16;
    const uint32_t bar_clear = bar_last + 8 * kStages;
    const uint32_t bar_done = bar_clear + 8 * kStages;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(base + kOffMisc);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
            ptx::mbar_init(bar_last + 8 * s, 1);
            ptx::mbar_init(bar_clear + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_tfull + 8 * b, 1);
            ptx::mbar_init(bar_tempty + 8 * b, 2 * kEpiWarps);
        }
        ptx::mbar_init(bar_done, 1);
        misc[1] = 0u;                                    // abort flag
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(sbase + kOffMisc, kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&maps.dy);
        ptx::prefetch_tensormap(&maps.x);
        ptx::prefetch_tensormap(&maps.out);
    }
    // Nothing above reads global memory.
    start_dependent();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();                                 // both CTAs' barriers and TMEM exist
    ptx::tc_fence_after();

    const uint32_t tmem = misc[0];
    const WaitCtx wctx{status, misc + 1, timeout_ns};
    const int units = shape.E * shape.splits * shape.tiles_n * shape.tiles_k;
    const int pairs = static_cast<int>(gridDim.x >> 1);
    const int first = static_cast<int>(blockIdx.x >> 1);
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t role, uint32_t where) {
        return __all_sync(0xFFFFFFFFu, wait_bounded<true>(bar, parity, wctx, role, where));
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        const uint64_t policy = ptx::policy_evict_last();    // read again by other tiles
        const uint32_t full = ptx::mapa_shared(bar_full, 0), last = ptx::mapa_shared(bar_last, rank);
        uint32_t g = 0;
        bool ok = true;
        Unit next(shape, offsets, first);
        for (int u = first; ok && u < units; u += pairs) {
            const Unit t = next;
            next = Unit(shape, offsets, u + pairs);
            if (t.bad && lane == 0) record_error(status, HG_ERR_BAD_OFFSETS, t.e);
            const int n = t.n0 + static_cast<int>(rank) * kHalf;
            const int k = t.k0 + static_cast<int>(rank) * kHalf;
            const int stages = t.stages();
            for (int s = 0; s < stages; ++s, ++g) {
                const uint32_t slot = g % kStages;
                if (!(ok = wait(bar_empty + 8 * slot, ((g / kStages) & 1u) ^ 1u, kRoleProducer,
                                slot)))
                    break;
                const int row = t.row0 + s * kWgradRows;
                uint32_t bar = full + 8 * slot;
                if (t.mixed(s)) {
                    bar = last + 8 * slot;
                    ptx::mbar_arrive_expect_tx_elect(bar_last + 8 * slot, 2 * kOperand);
                } else if (leader) {
                    ptx::mbar_arrive_expect_tx_elect(bar_full + 8 * slot, 4 * kOperand);
                }
                load_stage(sbase + kOffA + slot * kOperand, &maps.dy, shape.dy_panels, n, row, bar,
                           policy);
                load_stage(sbase + kOffB + slot * kOperand, &maps.x, shape.x_panels, k, row, bar,
                           policy);
            }
        }
        // No copy may land, and no release of a stage arrive, after the CTA has gone.  What the
        // MMAs have released has landed.  What they will not release, since a wait gave up, has
        // landed once a drain has waited for its whole limit: those behind it need no other.
        for (uint32_t gg = g > kStages ? g - kStages : 0; gg < g; ++gg)
            if (!wait_drain(bar_empty + 8 * (gg % kStages), (gg / kStages) & 1u)) break;
    } else if (warp == 1) {
        // ------------------------------------------------- MMA issuer ---
        if (leader) {
            const uint32_t idesc = ptx::idesc_bf16_mnmajor(kTile, kTile);
            uint32_t g = 0, tc = 0;
            bool ok = true;
            Unit next(shape, offsets, first);
            for (int u = first; ok && u < units; u += pairs) {
                const Unit t = next;
                next = Unit(shape, offsets, u + pairs);
                const int stages = t.stages();
                for (int s = 0; s < stages; ++s, ++g) {
                    const uint32_t b = tc & 1u, slot = g % kStages;
                    if (s % kChunk == 0 && !(ok = wait(bar_tempty + 8 * b, ((tc >> 1) & 1u) ^ 1u,
                                                       kRoleMma, 0x100u | b)))
                        break;
                    if (!(ok = wait(bar_full + 8 * slot, (g / kStages) & 1u, kRoleMma, slot)))
                        break;
                    ptx::tc_fence_after();
                    const uint64_t a =
                        ptx::desc_mnmajor_sw128(sbase + kOffA + slot * kOperand, kPanel);
                    const uint64_t x =
                        ptx::desc_mnmajor_sw128(sbase + kOffB + slot * kOperand, kPanel);
                    const int steps = (t.valid(s) + kMmaRows - 1) / kMmaRows;
                    for (int i = 0; i < steps; ++i) {
                        // 16 rows of 128 bytes on, in the descriptor's 16-byte units
                        ptx::mma_f16_pair_elect(tmem + b * kTile, a + i * kMmaRows * 8,
                                                x + i * kMmaRows * 8, idesc,
                                                s % kChunk != 0 || i != 0);
                    }
                    ptx::tc_commit_pair_multicast_elect(bar_empty + 8 * slot, 0x3);
                    if (s % kChunk == kChunk - 1 || s == stages - 1) {
                        ptx::tc_commit_pair_multicast_elect(bar_tfull + 8 * b, 0x3);
                        ++tc;
                    }
                }
            }
            // Everything issued must finish before either CTA gives TMEM back.
            ptx::tc_commit_pair_multicast_elect(bar_done, 0x1);
            wait_drain(bar_done, 0u);
        }
    } else if (warp >= 4 && warp < 4 + kEpiWarps) {
        // ---------------------------------------------------- epilogue --
        constexpr int kCols = kF32 ? 32 : 64;            // 128 bytes of output
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty = ptx::mapa_shared(bar_tempty, 0);
        const uint32_t buf = sbase + kOffOut + (warp - 4) * kOutBuf;
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * kEpiCols;
        const bool add = accumulate && !parts;
        uint32_t tc = 0;
        bool ok = true;
        for (int u = first; ok && u < units; u += pairs) {
            const Unit t(shape, offsets, u);
            const int stages = t.stages();
            if (stages == 0 && add) continue;
            float sum[kEpiCols];
            if (stages == 0) {
#pragma unroll
                for (int i = 0; i < kEpiCols; ++i) sum[i] = 0.0f;
            }
            for (int s = 0; s < stages; s += kChunk, ++tc) {
                const uint32_t b = tc & 1u;
                if (!(ok = wait(bar_tfull + 8 * b, (tc >> 1) & 1u, kRoleEpilogue, b))) break;
                ptx::tc_fence_after();
                if (s == 0) {
#pragma unroll
                    for (int c = 0; c < kEpiCols; c += 16)
                        ptx::tmem_ld_32x32b_x16(from + b * kTile + c,
                                                reinterpret_cast<uint32_t(&)[16]>(sum[c]));
                    ptx::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < kEpiCols; c += 16) {
                        uint32_t v[16];
                        ptx::tmem_ld_32x32b_x16(from + b * kTile + c, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_remote(tempty + 8 * b);
            }
            if (!ok) break;
            const int n = t.n0 + static_cast<int>(rank) * kHalf + 32 * q;
            const int k = t.k0 + half * kEpiCols;
            const int z = parts ? t.split * shape.E + t.e : t.e;
#pragma unroll
            for (int c = 0; c < kEpiCols; c += kCols) {
                if (n >= shape.N || k + c >= shape.K) continue;
                if (lane == 0) ptx::bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t to = buf + lane * 128 + ((i ^ (lane & 7)) << 4);
                    const float* v = sum + c + i * (kCols / 8);
                    if constexpr (kF32) {
                        sts_v4(to, __float_as_uint(v[0]), __float_as_uint(v[1]),
                               __float_as_uint(v[2]), __float_as_uint(v[3]));
                    } else {
                        sts_v4(to, bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3]),
                               bf16_pack(v[4], v[5]), bf16_pack(v[6], v[7]));
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (kF32 && add) {
                        ptx::tma_add_3d(&maps.out, buf, k + c, n, z);
                    } else {
                        ptx::tma_store_3d(&maps.out, buf, k + c, n, z);
                    }
                    ptx::bulk_commit_group();
                }
            }
        }
        // After giving up, the MMAs may still hand over this accumulator and the next one: those
        // arrivals come before the CTA goes, or not at all.
        for (uint32_t i = 0; !ok && i < 2; ++i)
            if (!wait_drain(bar_tfull + 8 * ((tc + i) & 1u), ((tc + i) >> 1) & 1u)) break;
        // every store has completed before the CTA can exit
        if (lane == 0) ptx::bulk_wait_group_all();
        __syncwarp();
    } else if (warp == 2) {
        // --------------------------------------- experts' last stages ---
        const uint32_t clear = ptx::mapa_shared(bar_clear, 0);
        uint32_t g = 0, parities = 0;                    // a bit per slot
        bool ok = true;
        Unit next(shape, offsets, first);
        for (int u = first; ok && u < units; u += pairs) {
            const Unit t = next;
            next = Unit(shape, offsets, u + pairs);
            const int s = t.stages() - 1;
            if (s >= 0 && t.mixed(s)) {
                const uint32_t slot = (g + s) % kStages, parity = (parities >> slot) & 1u;
                const int valid = t.valid(s);
                const int used = (valid + kMmaRows - 1) / kMmaRows * kMmaRows;
                if (!(ok = wait(bar_last + 8 * slot, parity, kRoleWorker, slot))) break;
                clear_rows(sbase + kOffA + slot * kOperand, valid, used);
                clear_rows(sbase + kOffB + slot * kOperand, valid, used);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (leader && !(ok = wait(bar_clear + 8 * slot, parity, kRoleWorker, 0x100u | slot)))
                    break;
                if (lane == 0) {
                    if (leader) {
                        ptx::mbar_arrive(bar_full + 8 * slot);
                    } else {
                        ptx::mbar_arrive_remote(clear + 8 * slot);
                    }
                }
                parities ^= 1u << slot;
            }
            g += s + 1;
        }
    }

    // Neither CTA may give up TMEM or shared memory while the pair's MMAs or the other
    // CTA's arrivals can still touch them.
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// dw = (dw +) the splits' parts, in their order.
constexpr int kJoinThreads = 256;
template <bool kF32>
__global__ void __launch_bounds__(kJoinThreads)
wgrad_join_kernel(const float* parts, int splits, long long pieces, int accumulate, void* dw) {
    start_dependent();
    const long long p = static_cast<long long>(blockIdx.x) * kJoinThreads + threadIdx.x;
    if (p >= pieces) return;                             // of four elements
    float v[4] = {};
    if (kF32 && accumulate) {
        const uint4 o = ptx::load(static_cast<const uint4*>(dw) + p);
        v[0] = __uint_as_float(o.x);
        v[1] = __uint_as_float(o.y);
        v[2] = __uint_as_float(o.z);
        v[3] = __uint_as_float(o.w);
    }
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const uint4 o = ptx::load(reinterpret_cast<const uint4*>(parts) + s * pieces + p);
        v[0] += __uint_as_float(o.x);
        v[1] += __uint_as_float(o.y);
        v[2] += __uint_as_float(o.z);
        v[3] += __uint_as_float(o.w);
    }
    if (kF32) {
        static_cast<float4*>(dw)[p] = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        static_cast<uint2*>(dw)[p] = make_uint2(bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3]));
    }
}

int tiles(int n) { return (n - 1) / kTile + 1; }

// x in BF16 from its codes, sixteen a thread.
constexpr int kDecodeThreads = 256;
__global__ void __launch_bounds__(kDecodeThreads)
wgrad_decode_kernel(const uint8_t* a, const uint8_t* scale, const int32_t* offsets, int E, int rows,
                    int K, uint16_t* x) {
    __shared__ int s_rows;
    if (threadIdx.x == 0) s_rows = 0;
    __syncthreads();
    start_dependent();
    // rows behind the last expert's are in no sum (the last offset need not be the largest)
    for (int e = threadIdx.x; e <= E; e += kDecodeThreads)
        atomicMax(&s_rows, min(ptx::load(offsets + e), rows));
    __syncthreads();
    const long long pieces = static_cast<long long>(s_rows) * (K / 16);
    const long long step = static_cast<long long>(gridDim.x) * kDecodeThreads;
    for (long long p = static_cast<long long>(blockIdx.x) * kDecodeThreads + threadIdx.x; p < pieces;
         p += step) {
        const uint4 v = ptx::load(reinterpret_cast<const uint4*>(a) + p);
        const float value = e8m0_value(ptx::load(scale + p / 8));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 lo = e4m3x2_to_f32(w[i]), hi = e4m3x2_to_f32(w[i] >> 16);
            o[2 * i] = bf16_pack(lo.x * value, lo.y * value);
            o[2 * i + 1] = bf16_pack(hi.x * value, hi.y * value);
        }
        uint4* to = reinterpret_cast<uint4*>(x) + 2 * p;
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Pairs that can be resident at once: the kernel's clusters are placed whole, and the
// occupancy calculator misjudges kernels that use TMEM, so that it is asked about a
// stand-in of the same size.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) stand_in() {}

constexpr int kMaxDevices = 64;
std::atomic<int> g_pairs[kMaxDevices];                   // 0: not set up

cudaError_t pairs_of(int num_sms, int* pairs) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::atomic<int>& known = g_pairs[dev % kMaxDevices];
    if ((*pairs = known.load()) > 0) return cudaSuccess;
    for (const void* kernel : {reinterpret_cast<const void*>(wgrad_kernel<false>),
                               reinterpret_cast<const void*>(wgrad_kernel<true>),
                               reinterpret_cast<const void*>(stand_in)}) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, stand_in, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    *pairs = n > 0 && n < num_sms / 2 ? n : num_sms / 2;
    known.store(*pairs);
    return cudaSuccess;
}

}  // namespace

void wgrad_reset_caches() {
    for (auto& pairs : g_pairs) pairs.store(0);
}

// Whole panels of 64 columns go two in a box (else a box's columns would run into the next
// row): a copy costs the engine some 80 cycles beside its bytes.  32 x 4096 x 6144, 16384
// rows: 793 us, with a box a panel 803.
int wgrad_panels(int cols) { return cols % 64 == 0 ? 2 : 1; }

// With fewer tiles than pairs (76, those of a whole GPU) the rows are split, as long as a part has
// some 2048 rows: dense
// 1024 x 1024 over 32768 rows 55 us in four parts, 157 in one; over 4096 rows 20 in two,
// 25 in one; over 2048 rows 18 to 22 in two or four, 17 in one, since joining is a launch more.
int wgrad_splits(int E, int N, int K, int rows) {
    constexpr long long kPairs = 76, kLeast = 2048;
    const long long t = static_cast<long long>(E) * tiles(N) * tiles(K);
    const long long by_rows = rows / (kLeast * E);
    const long long s = kPairs / t < by_rows ? kPairs / t : by_rows;
    return s < 1 ? 1 : static_cast<int>(s);
}

size_t wgrad_parts_bytes(int E, int N, int K, int rows) {
    const int s = wgrad_splits(E, N, K, rows);
    return s == 1 ? 0 : sizeof(float) * s * static_cast<size_t>(E) * N * K;
}

bool wgrad_fits(int E, int N, int K, int rows) {
    const long long units = static_cast<long long>(wgrad_splits(E, N, K, rows)) * E * tiles(N);
    const long long longest = 4ll * (N > K ? N : K);     // bytes of a row of any operand, at most
    constexpr long long kMost = 0x7FFF0000ll;            // with room to go on past the last
    return rows <= kMost && units <= kMost / tiles(K) &&
           longest * (rows > N ? rows : N) < 1ll << 40;  // a tensor map's stride
}

cudaError_t launch_wgrad(const WgradArgs& a, const WgradMaps& maps, int num_sms,
                         cudaStream_t stream) {
    int pairs = 0;
    cudaError_t err = pairs_of(num_sms, &pairs);
    if (err != cudaSuccess) return err;
    if (a.codes && a.rows > 0) {
        const long long blocks =
            (static_cast<long long>(a.rows) * (a.K / 16) + kDecodeThreads - 1) / kDecodeThreads;
        err = launch_dependent(wgrad_decode_kernel,
                               static_cast<int>(blocks < 16ll * num_sms ? blocks : 16ll * num_sms),
                               kDecodeThreads, 0, stream, a.codes, a.code_scale, a.offsets, a.E,
                               a.rows, a.K, a.x);
        if (err != cudaSuccess) return err;
    }
    const Shape s{a.E,        a.N,        a.K,
                  a.rows,     wgrad_splits(a.E, a.N, a.K, a.rows),
                  tiles(a.N), tiles(a.K), wgrad_panels(a.N), wgrad_panels(a.K)};
    const long long units = static_cast<long long>(s.E) * s.splits * s.tiles_n * s.tiles_k;
    const int grid = 2 * static_cast<int>(units < pairs ? units : pairs);
    err = launch_dependent(a.f32 || a.parts ? wgrad_kernel<true> : wgrad_kernel<false>, grid,
                           kThreads, kSmem, stream, maps, s, a.offsets, a.accumulate ? 1 : 0,
                           a.parts ? 1 : 0, a.status, a.timeout_ns);
    if (err != cudaSuccess || !a.parts) return err;
    const long long pieces = static_cast<long long>(a.E) * a.N * a.K / 4;
    const int blocks = static_cast<int>((pieces + kJoinThreads - 1) / kJoinThreads);
    return launch_dependent(a.f32 ? wgrad_join_kernel<true> : wgrad_join_kernel<false>, blocks,
                            kJoinThreads, 0, stream, a.parts, s.splits, pieces,
                            a.accumulate ? 1 : 0, a.dw);
}

}  // namespace hg

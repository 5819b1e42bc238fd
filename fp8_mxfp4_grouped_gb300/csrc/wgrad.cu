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
// operands lie in memory with K as the slow axis: TMA boxes of 64 rows x 64 columns are
// MN-major panels as they are.  Roles in a CTA, by warpgroup of four warps: the first holds
// the TMA producer, the MMA issuer (its warp in the odd CTA only allocates TMEM) and, where
// x is BF16, a worker; the second and third are the epilogue; where x is FP8 the fourth are
// workers.  A worker sees a stage after its bytes have landed and before the MMAs do: it
// clears the rows of an expert's last stage that belong to the next expert (in both
// operands: a NaN there must not meet a zero), and where x is FP8 turns the codes into
// BF16, which is exact (three mantissa bits times a power of two).
//
// The tensor core adds to its accumulator by cutting, not by rounding: the sum loses some
// 2^-24 of itself with each MMA, 9e-7 of a sum of positive terms over 512 rows and 1.8e-4
// over 32768.  After kChunk stages the epilogue therefore takes an accumulator over into
// its registers, where sums round.
#include <atomic>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kTile = 256;                   // dw rows and columns of a pair's unit
constexpr int kHalf = 128;                   // dy columns and x columns that a CTA loads
constexpr int kEpiWarps = 8;                 // four lane quarters x two halves of the columns
constexpr int kEpiCols = kTile * 4 / kEpiWarps;
constexpr int kPanel = kWgradRows * 128;     // bytes of 64 rows x 64 16-bit columns
constexpr int kOperand = 2 * kPanel;         // a CTA's part of an operand's stage
constexpr int kOutBuf = 32 * 128;            // a warp's 32 rows x 128 bytes of output
constexpr int kTmemCols = 512;               // two accumulators of 256 columns
constexpr int kMmaRows = 16;                 // K of an MMA

// Stages of an accumulator: 512 rows.
constexpr int kChunk = 8;

template <bool kFp8>
struct Cfg {
    static constexpr int kWorkers = kFp8 ? 4 : 1;        // warps that work on one stage
    static constexpr int kGroups = kFp8 ? 2 : 1;         // of them, taking stages in turn
    static constexpr int kFirstWorker = kFp8 ? 12 : 2;
    static constexpr int kThreads = 32 * (kFp8 ? 20 : 12);
    static constexpr int kStages = kFp8 ? 4 : 6;
    static constexpr int kRaw = kFp8 ? kWgradRows * kHalf : 0;
    static constexpr int kFactors = kFp8 ? (2 * kWgradRows + 4) * 4 : 0;
    static constexpr int kTx = kOperand + (kFp8 ? kRaw : kOperand);
    static constexpr int kOffA = 0;
    static constexpr int kOffB = kOffA + kStages * kOperand;
    static constexpr int kOffRaw = kOffB + kStages * kOperand;
    static constexpr int kOffOut = kOffRaw + kStages * kRaw;
    static constexpr int kOffFactors = kOffOut + kEpiWarps * kOutBuf;
    static constexpr int kOffBar = kOffFactors + kStages * kFactors;
    static constexpr int kOffMisc = kOffBar + 8 * (3 * kStages + 5);
    static constexpr int kSmem = kOffMisc + 16 + 1024;   // with room to align to 1024
    static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
    // registers of a thread by role: their sum over the warpgroups is the launch's
    static constexpr int kLaunchRegs = kFp8 ? 96 : 168;
    static constexpr int kControlRegs = kFp8 ? 48 : 88;
    static constexpr int kEpiRegs = kFp8 ? 168 : 208;
    static constexpr int kWorkerRegs = kFp8 ? 48 : 0;
    static_assert(kControlRegs + 2 * kEpiRegs + kGroups * kWorkerRegs <=
                      kLaunchRegs * kThreads / 128,
                  "setmaxnreg takes only what the launch has");
};

struct Shape {
    int E, N, K, rows, splits, tiles_n, tiles_k;
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
    // rows of a stage that belong to the unit
    __device__ __forceinline__ int valid(int stage) const {
        return min(kWgradRows, rows - stage * kWgradRows);
    }
};

// Eight E4M3 codes as BF16 times f, a pair of BF16 2^120 times the scale: shifted into place
// a code is its value times 2^-120 (the exponents' biases differ by as much; subnormal codes
// become subnormal numbers).  The four words' steps stand in turn, so that none waits for
// the one before.
__device__ __forceinline__ uint4 e4m3x8_to_bf16(uint2 v, uint32_t f) {
    uint4 o;
    asm("{\n\t.reg .b32 a, b, c, d, p, q, r, s;\n\t"
        "prmt.b32 a, %4, 0, 0x1404;\n\tprmt.b32 b, %4, 0, 0x3424;\n\t"
        "prmt.b32 c, %5, 0, 0x1404;\n\tprmt.b32 d, %5, 0, 0x3424;\n\t"
        "shr.b32 p, a, 4;\n\tshr.b32 q, b, 4;\n\tshr.b32 r, c, 4;\n\tshr.b32 s, d, 4;\n\t"
        "and.b32 p, p, 0x07F007F0;\n\tand.b32 q, q, 0x07F007F0;\n\t"
        "and.b32 r, r, 0x07F007F0;\n\tand.b32 s, s, 0x07F007F0;\n\t"
        "lop3.b32 p, a, 0x80008000, p, 0xEA;\n\tlop3.b32 q, b, 0x80008000, q, 0xEA;\n\t"
        "lop3.b32 r, c, 0x80008000, r, 0xEA;\n\tlop3.b32 s, d, 0x80008000, s, 0xEA;\n\t"
        "mul.rn.bf16x2 %0, p, %6;\n\tmul.rn.bf16x2 %1, q, %6;\n\t"
        "mul.rn.bf16x2 %2, r, %6;\n\tmul.rn.bf16x2 %3, s, %6;\n\t}"
        : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
        : "r"(v.x), "r"(v.y), "r"(f));
    return o;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// Clear rows [first, last) of an operand's stage (whole warp).
__device__ __forceinline__ void clear_rows(uint32_t operand, int first, int last) {
    for (int i = threadIdx.x & 31; i < (last - first) * 16; i += 32) {
        const int r = first + (i >> 4), panel = (i >> 3) & 1;
        sts_v4(operand + panel * kPanel + r * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
    }
}

template <bool kFp8, bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<kFp8>::kThreads, 1)
wgrad_kernel(const __grid_constant__ WgradMaps maps, const Shape shape, const uint8_t* x_scale,
             const int32_t* offsets, int accumulate, int parts, uint32_t* status,
             uint64_t timeout_ns) {
    using C = Cfg<kFp8>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = ptx::smem_u32(smem_raw);
    const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (sbase - raw_u32);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;

    // full: this CTA's bytes of a stage have landed.  ready (even CTA): the workers of
    // both CTAs are done with it.  empty: its MMAs are.
    const uint32_t bar_full = sbase + C::kOffBar;
    const uint32_t bar_ready = bar_full + 8 * kStages;
    const uint32_t bar_empty = bar_ready + 8 * kStages;
    const uint32_t bar_tfull = bar_empty + 8 * kStages;
    const uint32_t bar_tempty = bar_tfull + 16;          // even CTA: both have read TMEM
    const uint32_t bar_done = bar_tempty + 16;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, kFp8 ? 2 : 1);
            ptx::mbar_init(bar_ready + 8 * s, 2 * C::kWorkers);
            ptx::mbar_init(bar_empty + 8 * s, 1);
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
        ptx::tmem_alloc_pair(sbase + C::kOffMisc, kTmemCols);
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
    if (warp < 4) ptx::setmaxnreg_dec<C::kControlRegs>();
    if (C::kWorkerRegs && warp >= 4 + kEpiWarps) ptx::setmaxnreg_dec<C::kWorkerRegs>();
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t role, uint32_t where) {
        return __all_sync(0xFFFFFFFFu, wait_bounded<true>(bar, parity, wctx, role, where));
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        const uint64_t policy = ptx::policy_evict_last();    // read again by other tiles
        uint32_t g = 0;
        bool ok = true;
        Unit next(shape, offsets, first);
        for (int u = first; ok && u < units; u += pairs) {
            const Unit t = next;
            next = Unit(shape, offsets, u + pairs);
            if (t.bad && lane == 0) record_error(status, HG_ERR_BAD_OFFSETS, t.e);
            const int n = t.n0 + static_cast<int>(rank) * kHalf;
            const int k = t.k0 + static_cast<int>(rank) * kHalf;
            for (int s = 0; s < t.stages(); ++s, ++g) {
                const uint32_t slot = g % kStages;
                if (!(ok = wait(bar_empty + 8 * slot, ((g / kStages) & 1u) ^ 1u, kRoleProducer,
                                slot)))
                    break;
                const uint32_t bar = bar_full + 8 * slot;
                const int row = t.row0 + s * kWgradRows;
                ptx::mbar_arrive_expect_tx_elect(bar, C::kTx);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    ptx::tma_load_3d_elect(sbase + C::kOffA + slot * kOperand + p * kPanel,
                                           &maps.dy, n + 64 * p, row, 0, bar, policy);
                if (kFp8) {
                    ptx::tma_load_3d_elect(sbase + C::kOffRaw + slot * C::kRaw, &maps.x, k, row, 0,
                                           bar, policy);
                } else {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        ptx::tma_load_3d_elect(sbase + C::kOffB + slot * kOperand + p * kPanel,
                                               &maps.x, k + 64 * p, row, 0, bar, policy);
                }
            }
        }
        // No copy may land, and no release of a stage arrive, after the CTA has gone.
        for (uint32_t gg = g > kStages ? g - kStages : 0; gg < g; ++gg) {
            wait_drain(bar_full + 8 * (gg % kStages), (gg / kStages) & 1u);
            if (!*wctx.abort) wait_drain(bar_empty + 8 * (gg % kStages), (gg / kStages) & 1u);
        }
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
                    if (!(ok = wait(bar_ready + 8 * slot, (g / kStages) & 1u, kRoleMma, slot)))
                        break;
                    ptx::tc_fence_after();
                    const uint64_t a =
                        ptx::desc_mnmajor_sw128(sbase + C::kOffA + slot * kOperand, kPanel);
                    const uint64_t x =
                        ptx::desc_mnmajor_sw128(sbase + C::kOffB + slot * kOperand, kPanel);
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
        ptx::setmaxnreg_inc<C::kEpiRegs>();
        constexpr int kCols = kF32 ? 32 : 64;            // 128 bytes of output
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty = ptx::mapa_shared(bar_tempty, 0);
        const uint32_t buf = sbase + C::kOffOut + (warp - 4) * kOutBuf;
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
        // every store has completed before the CTA can exit
        if (lane == 0) ptx::bulk_wait_group_all();
        __syncwarp();
    } else if (kFp8 && warp == 2) {
        // ------------------------------------------------------ scales --
        // One factor a row for the workers: 2^120 times the row's scale as a pair of BF16, in
        // two factors where BF16 ends, and 0 for rows that are not the unit's.  The scales of
        // four stages are asked for while those of the four before are handed over.
        const int groups = shape.K / kHalf;
        uint32_t* factors = reinterpret_cast<uint32_t*>(base + C::kOffFactors);
        int u = first, s = 0;                            // the next stage to ask for
        Unit t(shape, offsets, u);
        constexpr uint32_t kNone = 256u;
        uint32_t now[8], later[8];
        auto ask = [&](uint32_t (&code)[8]) {            // how many stages were left
            int n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                code[2 * i] = code[2 * i + 1] = kNone;
                while (u < units && s >= t.stages()) {
                    u += pairs;
                    s = 0;
                    t = Unit(shape, offsets, u);
                }
                if (u >= units) continue;
                const int group = (t.k0 >> 7) + static_cast<int>(rank);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = s * kWgradRows + 32 * h + lane;
                    if (r < t.rows && group < groups)
                        code[2 * i + h] =
                            ptx::load(x_scale + static_cast<long long>(t.row0 + r) * groups + group);
                }
                ++s;
                ++n;
            }
            return n;
        };
        int n = ask(now);
        uint32_t g = 0;
        bool ok = true;
        while (ok && n > 0) {
            const int more = ask(later);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= n) break;
                const uint32_t slot = g % kStages;
                if (!(ok = wait(bar_empty + 8 * slot, ((g / kStages) & 1u) ^ 1u, kRoleScale, slot)))
                    break;
                uint32_t* to = factors + slot * (C::kFactors / 4);
                bool wide = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t code = now[2 * i + h];
                    const uint32_t one = code == 255u ? 0x7FC0u : (min(code, 134u) + 120u) << 7;
                    const bool over = code > 134u && code < 255u;
                    const uint32_t two = (over ? code - 7u : 127u) << 7;
                    to[32 * h + lane] = code == kNone ? 0u : one * 0x10001u;
                    to[kWgradRows + 32 * h + lane] = two * 0x10001u;
                    wide |= over;
                }
                wide = __any_sync(0xFFFFFFFFu, wide);
                if (lane == 0) to[2 * kWgradRows] = wide;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_full + 8 * slot);
                ++g;
            }
            n = more;
#pragma unroll
            for (int i = 0; i < 8; ++i) now[i] = later[i];
        }
    } else if (warp >= C::kFirstWorker && warp < C::kFirstWorker + C::kWorkers * C::kGroups) {
        // ----------------------------------------------------- workers --
        const int w = (warp - C::kFirstWorker) % C::kWorkers;
        const uint32_t turn = (warp - C::kFirstWorker) / C::kWorkers;
        const uint32_t ready = ptx::mapa_shared(bar_ready, 0);
        // FP8: this warp's 16 rows of a stage two at a time, a lane eight codes of one
        const int row0 = kMmaRows * w + (lane >> 4);
        const uint32_t from = row0 * kHalf + (lane & 15) * 8;
        const uint32_t to = ((lane >> 3) & 1) * kPanel + row0 * 128;
        uint32_t g = 0;
        bool ok = true;
        Unit next(shape, offsets, first);
        for (int u = first; ok && u < units; u += pairs) {
            const Unit t = next;
            next = Unit(shape, offsets, u + pairs);
            const int stages = t.stages();
            for (int s = 0; s < stages; ++s, ++g) {
                if (C::kGroups > 1 && g % C::kGroups != turn) continue;
                const uint32_t slot = g % kStages;
                const uint32_t a = sbase + C::kOffA + slot * kOperand;
                const int valid = t.valid(s);
                const int used = (valid + kMmaRows - 1) / kMmaRows * kMmaRows;
                if (!(ok = wait(bar_full + 8 * slot, (g / kStages) & 1u, kRoleWorker, slot))) break;
                if constexpr (kFp8) {
                    if (kMmaRows * w < used) {
                        const uint8_t* raw = base + C::kOffRaw + slot * C::kRaw + from;
                        uint8_t* out = base + C::kOffB + slot * kOperand + to;
                        const uint32_t* factor = reinterpret_cast<const uint32_t*>(
                                                     base + C::kOffFactors + slot * C::kFactors) + row0;
                        const bool wide = factor[2 * kWgradRows - row0] != 0u;
#pragma unroll
                        for (int i0 = 0; i0 < 8; i0 += 4) {
                            uint2 v[4];
                            uint32_t f[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[i] = *reinterpret_cast<const uint2*>(raw + 2 * (i0 + i) * kHalf);
                                f[i] = factor[2 * (i0 + i)];
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint4 o = e4m3x8_to_bf16(v[i], f[i]);
                                if (wide) {
                                    const uint32_t f2 = factor[kWgradRows + 2 * (i0 + i)];
                                    o = make_uint4(mul_bf16x2(o.x, f2), mul_bf16x2(o.y, f2),
                                                   mul_bf16x2(o.z, f2), mul_bf16x2(o.w, f2));
                                }
                                // row 2i + lane / 16 of 16, its chunk swizzled by the row mod 8
                                const int chunk = (lane & 7) ^ ((2 * i + (lane >> 4)) & 7);
                                *reinterpret_cast<uint4*>(out + 256 * (i0 + i) + (chunk << 4)) = o;
                            }
                        }
                        if (valid < kMmaRows * (w + 1))
                            clear_rows(a, max(valid, kMmaRows * w), min(used, kMmaRows * (w + 1)));
                    }
                } else if (valid < used) {
                    clear_rows(a, valid, used);
                    clear_rows(sbase + C::kOffB + slot * kOperand, valid, used);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_remote(ready + 8 * slot);
            }
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

// Pairs that can be resident at once: the kernel's clusters are placed whole, and the
// occupancy calculator misjudges kernels that use TMEM, so that it is asked about a
// stand-in of the same size.
template <int kThreads>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) stand_in() {}

constexpr int kMaxDevices = 64;
std::atomic<int> g_pairs[2][2][kMaxDevices];             // by x's and dw's type; 0: not set up

template <bool kFp8, bool kF32>
cudaError_t pairs_of(int num_sms, int* pairs) {
    using C = Cfg<kFp8>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::atomic<int>& known = g_pairs[kFp8][kF32][dev % kMaxDevices];
    if ((*pairs = known.load()) > 0) return cudaSuccess;
    err = cudaFuncSetAttribute(wgrad_kernel<kFp8, kF32>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (err != cudaSuccess) return err;
    // setmaxnreg in the kernel counts on the launch's registers, and would wait for ever for others
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, wgrad_kernel<kFp8, kF32>);
    if (err != cudaSuccess) return err;
    if (attr.numRegs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
    err = cudaFuncSetAttribute(stand_in<C::kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, stand_in<C::kThreads>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    *pairs = n > 0 && n < num_sms / 2 ? n : num_sms / 2;
    known.store(*pairs);
    return cudaSuccess;
}

template <bool kFp8, bool kF32>
cudaError_t launch(const WgradArgs& a, const Shape& s, const WgradMaps& maps, int num_sms,
                   cudaStream_t stream) {
    int pairs = 0;
    const cudaError_t err = pairs_of<kFp8, kF32>(num_sms, &pairs);
    if (err != cudaSuccess) return err;
    const long long units = static_cast<long long>(s.E) * s.splits * s.tiles_n * s.tiles_k;
    const int grid = 2 * static_cast<int>(units < pairs ? units : pairs);
    return launch_dependent(wgrad_kernel<kFp8, kF32>, grid, Cfg<kFp8>::kThreads, Cfg<kFp8>::kSmem,
                            stream, maps, s, a.x_scale, a.offsets, a.accumulate ? 1 : 0,
                            a.parts ? 1 : 0, a.status, a.timeout_ns);
}

}  // namespace

void wgrad_reset_caches() {
    for (auto& x : g_pairs)
        for (auto& dw : x)
            for (auto& pairs : dw) pairs.store(0);
}

// With fewer tiles than pairs the rows are split, as long as a part has some 512 rows.
int wgrad_splits(int E, int N, int K, int rows) {
    constexpr long long kPairs = 76, kLeast = 512;
    const long long t = static_cast<long long>(E) * tiles(N) * tiles(K);
    const long long by_rows = rows / (kLeast * E);
    const long long s = kPairs / t < by_rows ? kPairs / t : by_rows;
    return s < 1 ? 1 : static_cast<int>(s);
}

size_t wgrad_workspace(int E, int N, int K, int rows) {
    const int s = wgrad_splits(E, N, K, rows);
    return s == 1 ? 0 : sizeof(float) * s * static_cast<size_t>(E) * N * K;
}

bool wgrad_fits(int E, int N, int K, int rows) {
    const long long units = static_cast<long long>(wgrad_splits(E, N, K, rows)) * E * tiles(N);
    const long long longest = 4ll * (N > K ? N : K);     // bytes of a row of any operand, at most
    return units <= 0x7FFFFFFFll / tiles(K) &&
           longest * (rows > N ? rows : N) < 1ll << 40;  // a tensor map's stride
}

cudaError_t launch_wgrad(const WgradArgs& a, const WgradMaps& maps, int num_sms,
                         cudaStream_t stream) {
    const Shape s{a.E, a.N, a.K, a.rows, wgrad_splits(a.E, a.N, a.K, a.rows), tiles(a.N),
                  tiles(a.K)};
    const bool f32 = a.f32 || a.parts;
    const auto run = a.x_scale ? (f32 ? launch<true, true> : launch<true, false>)
                               : (f32 ? launch<false, true> : launch<false, false>);
    const cudaError_t err = run(a, s, maps, num_sms, stream);
    if (err != cudaSuccess || !a.parts) return err;
    const long long pieces = static_cast<long long>(a.E) * a.N * a.K / 4;
    const int blocks = static_cast<int>((pieces + kJoinThreads - 1) / kJoinThreads);
    return launch_dependent(a.f32 ? wgrad_join_kernel<true> : wgrad_join_kernel<false>, blocks,
                            kJoinThreads, 0, stream, a.parts, s.splits, pieces,
                            a.accumulate ? 1 : 0, a.dw);
}

}  // namespace hg

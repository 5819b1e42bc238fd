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
// memory, in chunks of up to sixteen slots (the columns of two MMAs), so that
// an expert's weights are read once for all of a chunk's slots; a work unit is
// (chunk, 16 or 32 weight rows), and each block takes one contiguous range of
// units.
//
// Warps stream: each warp owns a ring of 4-KB boxes of weights that its lane 0
// fills by TMA, and runs ahead of its own use of them by the ring's depth.  The
// boxes of a block's units, in order, are cut into one contiguous range per
// warp, so that all have the same work whatever K is.  A warp leaves the sums
// of a unit that began before its range in shared memory; the warp of a unit's
// first box adds those to its own, in the order of the warps (the result does
// not depend on timing), and writes the outputs.  It does so at the end of its
// range, and the others did theirs at the start: nobody waits, mostly.  (Boxes
// dealt to the warps in turn, and sums added in the order of the boxes, had the
// warps wait a third of their time: 13 tokens on 12 experts 47.4 us.)
//
// Arithmetic: a box's E2M1 codes become FP16 (exact) in registers and meet x
// in mma.sync m16n8k16: with sixteen columns at most the tensor work is small,
// and tcgen05 would want the 16-bit weights written back to shared memory
// first.  x is BF16, wider than FP16's range: each row's 256 elements of a box
// are scaled by the power of two that takes their largest magnitude into
// [2^14, 2^15).  An element keeps its 8 bits down to 2^-31 of that largest.  The
// sums of a 32-K group come out of the MMA in FP32 and are added up in FP32
// times the two scales, one after the other (their product can leave FP32's range
// where the term does not).  Where 256 elements span more than that, or are
// outside 2^+-86 or so, Inf or NaN, outputs in which that can show are computed
// once more at the end, from memory, x split into levels of 32 powers of two: an
// element counts in full whatever lies beside it, as the largest may meet a weight
// of zero.
//
// Measured (E = 32, top-8; bytes of the experts that the timed ids name): gate/up of
// one token, 4096 x 6144 with SwiGLU, 20.8 to 21.2 us for 107 MB, of which 3.5 pass
// before the first weights arrive; from there on the weights stream at the measured
// copy rate.  Down, 6144 x 2048: 13.1 us for 54 MB.  4 tokens, gate/up, 18 experts in
// use: 42.6 us for 236 MB; 8 tokens, down, 21 experts: 29.4 us for 139 MB.  13 tokens
// on 12 experts, 6144 x 3584: 39.4 us for 142 MB, of which about 7 pass before the
// first product; then it is bound by the instructions issued: conversion, MMA and
// scaling.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "hg_internal.cuh"
#include "numeric.cuh"

namespace hg {
namespace {

constexpr int kTileCols = 8;                 // slots of an MMA: its N
constexpr int kMaxCols = 16;                 // slots of a chunk: at most two MMAs
constexpr int kSingleRows = 4;               // input rows held for single columns
constexpr int kPartK = 256;                  // elements of 128 bytes of a weight row
constexpr int kBlockBytes = 8 * kPartK / 2;  // 8 rows of a part: one swizzle pattern
constexpr int kSmemLimit = 232448 - 256;     // beside a few static bytes

// The forms of the kernel.  A single column's MMAs are light, and its boxes
// are long in K: 16 rows x 512 K.  With more columns the fragments of x weigh
// more than the weights, and 32 rows x 256 K share each of them between two
// MMAs.  There twelve warps where they leave room for x, else eight: what
// bounds them is the instructions they issue, and eight leave gaps between
// them; sixteen are short of registers (13 tokens on 12 experts 45.5 us, twelve
// 42.4).  Two boxes a warp cover the memory's latency; three or four change
// nothing.
struct Form {
    int warps, row_tiles, parts;             // parts: of 256 K in a box
    int ring;                                // boxes in flight per warp, at most
    __host__ __device__ constexpr int rows() const { return 16 * row_tiles; }
    __host__ __device__ constexpr int box_bytes() const {
        return 2 * row_tiles * parts * kBlockBytes;
    }
    // of two boxes
    __host__ __device__ constexpr int scale_bytes() const { return box_bytes() / 8; }
};
// tiles: MMAs side by side, 0 for a single column.
__host__ __device__ constexpr Form form_of(int tiles, int warps) {
    return tiles == 0 ? Form{warps, 1, 2, 2} : Form{warps, 2, 1, 2};
}
// The sums that each warp but the first may leave: a float per weight row and column.
__host__ __device__ constexpr int partial_bytes(int tiles, const Form& f) {
    return (f.warps - 1) * f.rows() * 4 * (tiles == 0 ? 1 : tiles * kTileCols);
}
__host__ __device__ constexpr int tiles_of(int cols) {
    return cols == 1 ? 0 : cols <= kTileCols ? 1 : 2;
}
constexpr int kSingleWarps = 16;
constexpr int kWarpChoices[2] = {12, 8};             // with more columns

struct __align__(8) Entry {
    int expert;                              // -1: free
    int first;                               // the expert's first slot
    uint8_t slots[kMatvecMaxSlots / 32];     // how many it has in each 32 slots
};

// The slots by expert: entries per slot and per chunk, and a hash table of the
// experts.
struct Tables {
    int* count;              // [0] chunks, [1] slots without an expert
    int* id;                 // of a slot; -1 without an expert
    int* expert;             // of a chunk
    int* ncols;              // of a chunk
    uint16_t* slot;          // of a chunk's columns: chunk * cols + column
    // more than 32 slots only
    uint32_t* leads;         // a bit per slot: the first of a chunk
    Entry* hash;             // by expert; where the warps' sums come later
};

// A power of two, twice the slots at least.
__host__ __device__ inline int hash_entries(int slots) {
    int n = 64;
    while (n < 2 * slots) n *= 2;
    return n;
}

// Chunks at most: each expert in use has one that is not full.
__host__ __device__ inline int max_chunks(int slots, int cols, int E) {
    const int n = slots / cols + (E < slots ? E : slots);
    return n < slots ? n : slots;
}

__host__ __device__ inline int table_bytes(int slots, int cols, int E) {
    const int n = (slots + 3) & ~3, c = (max_chunks(slots, cols, E) + 3) & ~3;
    return 16 + 4 * n + c * (2 * 4 + 2 * cols) + (slots > 32 ? kMatvecMaxSlots / 8 : 0);
}

__host__ __device__ inline int hash_bytes(int slots) {
    return slots > 32 ? static_cast<int>(sizeof(Entry)) * hash_entries(slots) : 0;
}

__device__ inline Tables tables_at(uint8_t* p, uint8_t* hash, int slots, int cols, int E) {
    const int n = (slots + 3) & ~3, c = (max_chunks(slots, cols, E) + 3) & ~3;
    Tables t;
    t.count = reinterpret_cast<int*>(p);
    t.id = t.count + 4;
    t.expert = t.id + n;
    t.ncols = t.expert + c;
    t.slot = reinterpret_cast<uint16_t*>(t.ncols + c);
    t.leads = reinterpret_cast<uint32_t*>(t.slot + c * cols);
    t.hash = reinterpret_cast<Entry*>(hash);
    return t;
}

struct Layout {
    int warps;
    int ring;          // boxes per warp
    int cols;          // most slots of a chunk
    int x_rows;        // input rows held at once
    int x_stride;      // bytes between them
    int scales, partial, x, x_scale, bars, tables, total;   // byte offsets
};

// Columns: up to eight (one MMA) where an expert has few slots on average, up
// to sixteen otherwise: a second MMA costs a quarter more, and reading the
// weights of an expert with more slots twice costs twice.  Warps: as many as
// leave a ring of two boxes each beside that.  Input rows: as many as still fit.
// They stay 64 bytes off a multiple of 128 apart, so that the eight lanes of a
// 16-byte load phase (two columns, whose rows mostly follow one another) meet
// no bank twice.
bool make_layout(int K, int slots, int tokens, int E, int x_rows, Layout* out) {
    int pieces = 0;
    Layout l{};
    Form f;
    auto box = [&]() { return f.warps * (f.box_bytes() + f.scale_bytes()); };
    auto sums = [&]() {
        const int left = partial_bytes(tiles_of(l.cols), f), hash = hash_bytes(slots);
        return left > hash ? left : hash;
    };
    auto bars = [&](int ring) { return (f.warps * ring + f.warps + 1) * 8 + (f.warps + 1) * 4; };
    auto needs = [&](int rows) {
        const int parts = f.parts * kPartK;              // the rows reach to the end of a box
        pieces = (K + parts - 1) / parts * f.parts;
        l.x_stride = pieces * kPartK * 2 + 64;
        return 1024 + sums() + rows * (l.x_stride + pieces * 4) + 32 + bars(f.ring) +
               table_bytes(slots, l.cols, E);
    };
    auto fits = [&]() { return needs(l.cols) + 2 * box() <= kSmemLimit; };
    auto choose = [&](int cols) {            // the most warps with which so many columns fit
        l.cols = cols;
        if (cols == 1) {
            f = form_of(0, kSingleWarps);
            return fits();
        }
        for (int warps : kWarpChoices) {
            f = form_of(tiles_of(cols), warps);
            if (fits()) return true;
        }
        return false;
    };
    int cols = tokens < slots ? tokens : slots;          // a token's choices are distinct experts
    const int most = slots > 6ll * E ? kMaxCols : kTileCols;
    if (cols > most) cols = most;
    // where not all of an expert's slots fit, two chunks of one MMA take less
    // than one of two and one of one
    if (!choose(cols) && cols > kTileCols) cols = kTileCols;
    while (!choose(cols) && cols > 1) --cols;
    l.warps = f.warps;
    const int useful = cols == 1 ? kSingleRows : 3 * kMaxCols;
    const int beside_rows = needs(0);
    l.x_rows = (kSmemLimit - 2 * box() - beside_rows) / (l.x_stride + pieces * 4);
    if (l.x_rows > useful) l.x_rows = useful;
    if (l.x_rows > x_rows) l.x_rows = x_rows;
    if (l.x_rows < cols) l.x_rows = cols;
    l.ring = (kSmemLimit - needs(l.x_rows)) / box();
    if (l.ring > f.ring) l.ring = f.ring;
    if (l.ring < 1) return false;
    const int ring = f.warps * l.ring;
    l.scales = ring * f.box_bytes();
    l.partial = l.scales + ring * f.scale_bytes();
    l.x = (l.partial + sums() + 15) & ~15;
    l.x_scale = l.x + l.x_rows * l.x_stride;
    l.bars = (l.x_scale + l.x_rows * pieces * 4 + 15) & ~15;
    l.tables = (l.bars + bars(l.ring) + 15) & ~15;
    l.total = l.tables + table_bytes(slots, cols, E) + 1024 - 16;
    *out = l;
    return true;
}

// Division by a number that the host knows, of n in [0, 2^31).
struct Divisor {
    uint32_t d, m;                           // m = 2^32 / d, at most 2^32 - 1
    explicit Divisor(int by = 1)
        : d(by), m(by == 1 ? 0xFFFFFFFFu : static_cast<uint32_t>((1ull << 32) / by)) {}
    __device__ __forceinline__ int of(int n) const {
        const uint32_t q = __umulhi(static_cast<uint32_t>(n), m);       // or one less
        return static_cast<int>(q + (static_cast<uint32_t>(n) - q * d >= d));
    }
};

struct KernelArgs {
    const uint16_t* x;
    const int32_t* ids;
    const uint8_t* w_fp4;
    const uint8_t* w_scale;
    uint16_t* out;
    uint32_t* status;
    uint64_t timeout_ns;
    int x_rows, slots_per_row, slots, E, N, K;
    Divisor boxes, tiles, blocks;            // boxes of a unit, units of a chunk, blocks
    bool wide_scales;                        // rows of scales start at multiples of 16 bytes
    Layout l;
};

// List the slots by expert in chunks of up to `cols`, in the order of the
// chunks' first slots: every block makes the same list.  Returns the number of
// chunks.
template <int kThreads>
__device__ int list_slots(const KernelArgs& a, const Tables& tb) {
    const int tid = threadIdx.x;
    const int cols = a.l.cols;
    auto expert_of = [&](int s) {
        const int e = s < a.slots ? ptx::load(a.ids + s) : -1;
        return e >= 0 && e < a.E ? e : -1;
    };
    if (a.slots <= 32) {                     // one warp sees all slots at once
        if (tid < 32) {
            const int e = expert_of(tid);
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
            const uint32_t below = (1u << tid) - 1u;
            const int rank = __popc(same & below);
            const int nth = rank / cols, col = rank - nth * cols;
            const uint32_t leads = __ballot_sync(0xFFFFFFFFu, e >= 0 && col == 0);
            const uint32_t valid = __ballot_sync(0xFFFFFFFFu, e >= 0);
            if (tid < a.slots) tb.id[tid] = e;
            if (e >= 0) {
                // the chunk's first slot: the last leader of this expert up to here
                const int lead = 31 - __clz(same & leads & (below | (1u << tid)));
                const int c = __popc(leads & ((1u << lead) - 1u));
                tb.slot[c * cols + col] = static_cast<uint16_t>(tid);
                if (col == 0) {
                    tb.expert[c] = e;
                    tb.ncols[c] = min(cols, __popc(same) - rank);
                }
            }
            if (tid == 0) {
                tb.count[0] = __popc(leads);
                tb.count[1] = a.slots - __popc(valid);
            }
        }
        __syncthreads();
        return tb.count[0];
    }
    constexpr int kTurns = (kMatvecMaxSlots + kThreads - 1) / kThreads;      // slots per thread
    const int mask = hash_entries(a.slots) - 1, words = (a.slots + 31) / 32;
    int e[kTurns], h[kTurns], rank[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) e[i] = expert_of(tid + i * kThreads);
    for (int i = tid; i <= mask; i += kThreads) {
        Entry& t = tb.hash[i];
        t.expert = -1;
        t.first = kMatvecMaxSlots;
#pragma unroll
        for (int w = 0; w < kMatvecMaxSlots / 32; w += 4)
            *reinterpret_cast<uint32_t*>(t.slots + w) = 0;
    }
    for (int i = tid; i < max_chunks(a.slots, cols, a.E); i += kThreads) tb.ncols[i] = 0;
    if (tid == 0) tb.count[1] = 0;
    __syncthreads();
    // each expert's slots of each 32, by the first lane that has it
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int s = tid + i * kThreads, lane = tid & 31;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e[i]);
        const int leader = __ffs(same) - 1;
        rank[i] = __popc(same & ((1u << lane) - 1u));
        h[i] = 0;
        if (e[i] >= 0 && lane == leader) {
            h[i] = static_cast<int>((static_cast<uint32_t>(e[i]) * 2654435761u) >> 16) & mask;
            for (;; h[i] = (h[i] + 1) & mask) {              // at most half of the entries are used
                const int there = atomicCAS(&tb.hash[h[i]].expert, -1, e[i]);
                if (there == -1 || there == e[i]) break;
            }
            atomicMin(&tb.hash[h[i]].first, s);
            tb.hash[h[i]].slots[s >> 5] = static_cast<uint8_t>(__popc(same));
        }
        h[i] = __shfl_sync(0xFFFFFFFFu, h[i], leader);
        if (s < a.slots) tb.id[s] = e[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int s = tid + i * kThreads;
        if (e[i] >= 0) {
            for (int w = 0; w < s >> 5; ++w) rank[i] += tb.hash[h[i]].slots[w];
        }
        const uint32_t leads = __ballot_sync(0xFFFFFFFFu, e[i] >= 0 && rank[i] % cols == 0);
        const uint32_t none = __ballot_sync(0xFFFFFFFFu, s < a.slots && e[i] < 0);
        if ((tid & 31) == 0 && s < a.slots) {
            tb.leads[s >> 5] = leads;
            if (none) atomicAdd(&tb.count[1], __popc(none));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        if (e[i] < 0) continue;
        int lead = tb.hash[h[i]].first, skip = rank[i] / cols * cols;
        const int col = rank[i] - skip;
        for (; skip > 0; ++lead) skip -= tb.id[lead] == e[i];    // a later chunk of the expert
        while (tb.id[lead] != e[i]) ++lead;
        int c = __popc(tb.leads[lead >> 5] & ((1u << (lead & 31)) - 1u));
        for (int w = 0; w < lead >> 5; ++w) c += __popc(tb.leads[w]);
        tb.slot[c * cols + col] = static_cast<uint16_t>(tid + i * kThreads);
        atomicAdd(&tb.ncols[c], 1);
        if (col == 0) tb.expert[c] = e[i];
    }
    if (tid == 0) {
        int total = 0;
        for (int w = 0; w < words; ++w) total += __popc(tb.leads[w]);
        tb.count[0] = total;
    }
    __syncthreads();
    return tb.count[0];
}

// Input rows come to shared memory as they are and are rewritten in place as
// scaled FP16, 256 elements of a row at a time, eight a lane: piece p is part
// p % parts of held row p / parts, and belongs to warp p % warps.  The one to four
// rows of single columns come by cp.async of the lanes that rewrite them (0.5 us
// less than with bulk copies for a dense 500 x 640), the many rows of the other
// forms by a bulk copy each (1.4 us less for 13 tokens on 12 experts).  Those are
// rewritten four pieces a warp at once, which hides the latency of the maximum
// over the lanes: one at a time takes 13 tokens' 182 pieces 2.5 us longer.
//
// What a row's 256 elements of a piece are scaled by follows from `be`, the
// biased exponent of the largest: an element goes to FP16 times 2^(141 - be), and
// sums come back times 2^(be - 141).  FP16 holds an element's 8 bits down to 31
// powers of two below the largest.  Pieces that span more are multiplied in
// levels: level l has the elements of exponents be - 32 l down to be - 32 l - 31,
// scaled as if be - 32 l were the largest's.
constexpr int kFp16Exponent = 141;           // of an element that stays as it is
constexpr int kLevel = 32;
constexpr int kLeastExponent = 15;           // both factors are normal numbers from here on
// A sum of the MMA, 2^-25 to 2^23 or zero, times a factor of up to 2^+-100 is
// exact and a normal number, and is then multiplied with the weights' scale as it
// is added.
constexpr int kQuickExponents = 100;
__device__ __forceinline__ float to_fp16_range(int be) {
    return __uint_as_float(static_cast<uint32_t>(kFp16Exponent + 127 - be) << 23);
}
// Biased exponent of a magnitude; a subnormal's lowest bit is that of exponent 1.
__device__ __forceinline__ int exponent_of(uint32_t magnitude) {
    return max(static_cast<int>(magnitude >> 7), 1);
}
__device__ __forceinline__ int level_exponent(int be, int level) {
    return be == 255 ? kFp16Exponent : max(be - kLevel * level, kLeastExponent);
}
// Level `level` of eight elements as FP16, zeros in the others' places.  be = 255:
// Inf and NaN alone, as they are, which decide a sum.
__device__ __forceinline__ uint4 level_part(const uint4 v, int be, int level) {
    const float mult = be == 255 ? 1.0f : to_fp16_range(level_exponent(be, level));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t bits = e ? w[i] >> 16 : w[i] & 0xFFFFu;
            const int below = be - exponent_of(bits & 0x7FFFu);
            const bool here = be == 255 ? below == 0 && level == 0 : below >> 5 == level;
            f[e] = here ? __uint_as_float(bits << 16) * mult : 0.0f;
        }
        const __half2 p = __floats2half2_rn(f[0], f[1]);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}
static_assert(kLevel == 32, "levels are told by a shift of five");

__device__ __forceinline__ uint4* piece_at(const KernelArgs& a, uint8_t* smem, int p, int parts,
                                           float per_row, int lane) {
    const int held = static_cast<int>((p + 0.5f) * per_row);
    return reinterpret_cast<uint4*>(smem + a.l.x + held * a.l.x_stride +
                                    (p - held * parts) * (2 * kPartK) + 16 * lane);
}
__device__ __forceinline__ float* factor_of(const KernelArgs& a, uint8_t* smem, int p) {
    return reinterpret_cast<float*>(smem + a.l.x_scale) + p;
}
// Largest and least magnitude of BF16 elements.  Magnitudes compare as integers,
// NaN the largest.  For the least, with the highest bit set and less one they are
// signed numbers in order, but zero, which comes out the largest.
struct Span {
    uint32_t top = 0, low = 0x7FFF7FFFu;
    __device__ __forceinline__ void add(uint32_t two) {
        top = __vmaxu2(top, two & 0x7FFF7FFFu);
        low = __vmins2(low, (two | 0x80008000u) - 0x00010001u);
    }
    __device__ __forceinline__ void add(const uint4 v) {
        add(v.x);
        add(v.y);
        add(v.z);
        add(v.w);
    }
    __device__ __forceinline__ uint32_t largest() const { return max(top & 0xFFFFu, top >> 16); }
    __device__ __forceinline__ int least_code() const {
        return min(static_cast<int>(low << 16) >> 16, static_cast<int>(low) >> 16);
    }
    // whether any element but zero is below 2^(exponent - 127), exponent above 0
    __device__ __forceinline__ bool any_below(int exponent) const {
        const int bound = static_cast<int>(static_cast<uint32_t>(exponent * 128 - 32769) << 16);
        return min(static_cast<int>(low << 16), static_cast<int>(low)) < bound;
    }
};
// Whether a lane's elements, with `top` the largest magnitude of the piece, allow
// it to be a plain one: of zeros, or neither Inf, NaN, extreme nor wide.
__device__ __forceinline__ bool is_plain(const Span& span, uint32_t top) {
    constexpr uint32_t kLow = (kFp16Exponent - kQuickExponents) << 7;
    constexpr uint32_t kHigh = (kFp16Exponent + kQuickExponents + 1) << 7;
    return top - 1u >= kLow - 1u && top < kHigh &&
           !span.any_below(static_cast<int>(top >> 7) - (kLevel - 1));
}

// Rows as they came become scaled FP16 where they lie.  Returns whether this lane
// has seen anything that makes its piece more than a plain one: Inf, NaN, extreme
// or wide elements.  (A vote and a branch here would stand in the way of the pieces'
// overlap: 41.1 us for 13 tokens on 12 experts where the flag alone took 39.0.)
template <int kPieces>
__device__ __forceinline__ bool scale_pieces(const KernelArgs& a, uint8_t* smem, int first,
                                             int step, int parts, float per_row, int lane) {
    uint4* at[kPieces];
    uint4 v[kPieces];
    uint32_t top[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        at[i] = piece_at(a, smem, first + i * step, parts, per_row, lane);
        v[i] = *at[i];
    }
    Span span[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        span[i].add(v[i]);
        top[i] = __reduce_max_sync(0xFFFFFFFFu, span[i].largest());
    }
    bool plain = true;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        float f[8];
        bf16_unpack8(v[i], f);
        plain &= is_plain(span[i], top[i]);
        const int be = max(static_cast<int>(top[i] >> 7), kLeastExponent);
        const float mult = to_fp16_range(be);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 p = __floats2half2_rn(f[2 * e] * mult, f[2 * e + 1] * mult);
            h[e] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *at[i] = make_uint4(h[0], h[1], h[2], h[3]);
        if (lane == 0)
            *factor_of(a, smem, first + i * step) =
                __uint_as_float(static_cast<uint32_t>(be + 127 - kFp16Exponent) << 23);
    }
    return !plain;
}

// acc + d * 2^(code - 127) * 2^(be - 141).  The product of the two powers can
// lie far outside FP32's range where the term does not: half of its exponent at
// a time.  Code 255 is NaN.
__device__ __forceinline__ float add_scaled(float d, uint32_t code, int be, float acc) {
    const int e = static_cast<int>(code) - 127 + be - kFp16Exponent, half = e >> 1;
    return fmaf(d * e8m0_value(127 + half), e8m0_value(code == 255u ? 255u : 127 + e - half), acc);
}

// 256 K of 16 weight rows times one column.  Were the column alone in the
// MMA's eight, each 32-K group would need its own scaling of 16 x 8 sums.
// Instead column c of x holds the elements of group c, so that one load serves
// all eight groups, and of group g's product only column g is kept: a lane
// keeps groups 2q and 2q + 1 of its two rows, and scales four sums in place of
// thirty-two.
__device__ __forceinline__ void single_part(uint32_t w_at, const uint8_t* x_at, uint32_t code_lo,
                                            uint32_t code_hi, float sx, int lane,
                                            float (&acc)[2]) {
    const int q = lane & 3;
    const uint4 xv = *reinterpret_cast<const uint4*>(x_at);
    float v[4];
    uint32_t w[2][4];
    ptx::ldmatrix_x4(w_at + (((lane >> 4) ^ (lane & 7)) << 4), w[0]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {                            // groups 2p and 2p + 1
        if (p < 3)
            ptx::ldmatrix_x4(w_at + (((2 * p + 2 + (lane >> 4)) ^ (lane & 7)) << 4), w[~p & 1]);
        float d[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t lo[4], hi[4];
            ptx::e2m1x8_to_f16(w[p & 1][2 * i], lo);
            ptx::e2m1x8_to_f16(w[p & 1][2 * i + 1], hi);
            ptx::mma_f16_16816_first(d[i], lo[0], hi[0], lo[1], hi[1], xv.x, xv.y);
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
    acc[0] = fmaf(v[0] * sx, s_lo.x, acc[0]);
    acc[0] = fmaf(v[1] * sx, s_lo.y, acc[0]);
    acc[1] = fmaf(v[2] * sx, s_hi.x, acc[1]);
    acc[1] = fmaf(v[3] * sx, s_hi.y, acc[1]);
}

// kTiles: MMAs side by side, eight slots each; 0: a single slot.
template <bool kSwiglu, int kTiles, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1)
expert_matvec_kernel(const __grid_constant__ CUtensorMap map_w, const KernelArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_abort, s_other;
    constexpr bool kSingle = kTiles == 0;
    constexpr int kT = kSingle ? 1 : kTiles;
    constexpr Form kForm = form_of(kTiles, kWarps);
    constexpr int kThreads = kWarps * 32;
    constexpr int kR = kForm.row_tiles;
    constexpr int kRows = 16 * kR;
    constexpr int kParts = kForm.parts;
    constexpr int kBoxBytes = kForm.box_bytes();
    constexpr int kScaleBytes = kForm.scale_bytes();         // of two boxes side by side
    static_assert(kScaleBytes == 32 * 16, "a warp copies two boxes' scales at once");
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const Tables tb = tables_at(smem + a.l.tables, smem + a.l.partial, a.slots, a.l.cols,
                                a.E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t bars = base + a.l.bars + 8 * warp * a.l.ring;
    const uint32_t left_bar = bars + 8 * (kWarps - warp) * a.l.ring;     // one per warp
    const uint32_t x_bar = left_bar + 8 * kWarps;
    // the first box of each warp's range in the run
    int* bound = reinterpret_cast<int*>(smem + a.l.bars + 8 * (kWarps * a.l.ring + kWarps + 1));
    const int nb = a.boxes.d;
    const int out_cols = kSwiglu ? a.N / 2 : a.N;
    const int tile_cols = kSwiglu ? kRows / 2 : kRows;       // outputs of a unit
    const int tiles = a.tiles.d;

    if (lane == 0) {
        for (int i = 0; i < a.l.ring; ++i) ptx::mbar_init(bars + 8 * i, 33);
        ptx::mbar_init(left_bar + 8 * warp, 1);
        if (warp == 0) {
            ptx::prefetch_tensormap(&map_w);
            s_abort = s_other = 0;
            ptx::mbar_init(x_bar, 1);
        }
        ptx::fence_barrier_init();
    }
    start_dependent();                       // nothing global is read or written before

    // x goes ahead of the weights, behind which it would wait for the whole
    // ring; where all rows are held, ahead of the ids, too.
    const int parts = kParts * nb;
    uint32_t x_phase = 0, x_asked = 1;       // of x_bar: the next to wait for, the last asked for
    bool rows_came = true;
    const bool hold_all = a.x_rows <= a.l.x_rows;
    auto each_piece = [&](int rows, auto f) {
        for (int p = warp, held = 0, part = warp; p < parts * rows; p += kWarps) {
            while (part >= parts) {
                part -= parts;
                ++held;
            }
            f(held, part);
            part += kWarps;
        }
    };
    auto load_rows = [&](int rows, auto row_of) {
        if (kSingle) {
            each_piece(rows, [&](int held, int part) {
                const int k = part * kPartK + 8 * lane;
                const uint16_t* src = a.x + static_cast<long long>(row_of(held)) * a.K;
                ptx::cp_async_16(base + a.l.x + held * a.l.x_stride + 2 * k,
                                 src + (k < a.K ? k : 0), k < a.K);
            });
            ptx::cp_async_commit();
            return;
        }
        // none are asked for in a phase that follows one that did not end
        if (warp != 0 || !rows_came) return;
        x_asked = x_phase;
        if (lane == 0) ptx::mbar_arrive_expect_tx(x_bar, rows * 2 * a.K);
        __syncwarp();
        ptx::fence_proxy_async_smem();       // the rows before were rewritten in place
        for (int held = lane; held < rows; held += 32)
            ptx::bulk_load(base + a.l.x + held * a.l.x_stride,
                           a.x + static_cast<long long>(row_of(held)) * a.K, 2 * a.K, x_bar);
    };
    if (hold_all) load_rows(a.x_rows, [](int held) { return held; });
    // zeros behind the rows, up to the end of their last box (cp.async writes them itself)
    if constexpr (!kSingle) {
        const int tail = (2 * kPartK * parts - 2 * a.K) / 16;
        for (int i = threadIdx.x; i < tail * a.l.x_rows; i += kThreads)
            *reinterpret_cast<uint4*>(smem + a.l.x + i / tail * a.l.x_stride + 2 * a.K +
                                      16 * (i % tail)) = make_uint4(0, 0, 0, 0);
    }
    const int chunks = list_slots<kThreads>(a, tb);          // has block barriers

    const int units = chunks * tiles;
    const int each = a.blocks.of(units);
    const int left = units - each * static_cast<int>(gridDim.x);
    int u0 = static_cast<int>(blockIdx.x) * each + min(static_cast<int>(blockIdx.x), left);
    int u1 = u0 + each + (static_cast<int>(blockIdx.x) < left);
    if (kTiles == 2 && chunks <= 32) {
        // A unit of a chunk with two MMAs a row tile takes about 5/4 of the
        // time of one with one: blocks get equal shares of that.
        const bool wide = lane < chunks && tb.ncols[lane] > kTileCols;
        const uint32_t wides = __ballot_sync(0xFFFFFFFFu, wide);
        const long long cost = 4 * lane + __popc(wides & ((1u << lane) - 1u));   // chunks before
        const long long all = static_cast<long long>(tiles) * (4 * chunks + __popc(wides));
        auto unit_at = [&](long long target) {
            const int c = __popc(__ballot_sync(0xFFFFFFFFu, lane < chunks &&
                                                                tiles * cost <= target)) - 1;
            const int weight = (wides >> c) & 1u ? 5 : 4;
            const int inside = static_cast<int>(
                target - tiles * __shfl_sync(0xFFFFFFFFu, cost, c));
            return c * tiles + min(tiles, (inside + weight - 1) / weight);
        };
        u0 = chunks ? unit_at(all * blockIdx.x / gridDim.x) : 0;
        u1 = chunks ? unit_at(all * (blockIdx.x + 1) / gridDim.x) : 0;
    }
    const int chunk0 = a.tiles.of(u0);

    // A run: the units of as many chunks, from chunk c on, as rows can be held.
    auto run_end = [&](int c) {
        if (hold_all) return u1;
        int rows = 0;
        while (c * tiles < u1 && rows + tb.ncols[c] <= a.l.x_rows) rows += tb.ncols[c++];
        return min(c * tiles, u1);
    };
    auto run_rows = [&](int c, int end) {
        int rows = 0;
        for (; c * tiles < end; ++c) rows += tb.ncols[c];
        return rows;
    };
    auto load_run = [&](int c, int end) {
        int before = 0;                      // rows of the run's chunks before c
        load_rows(run_rows(c, end), [&](int held) {
            while (held >= before + tb.ncols[c]) before += tb.ncols[c++];
            return tb.slot[c * a.l.cols + held - before] / a.slots_per_row;
        });
    };
    if (!hold_all && u0 < u1) load_run(chunk0, run_end(chunk0));

    // The run's boxes, in order, box b of unit u at (u - run) * nb + b, are cut
    // into equal ranges, with two MMAs a row tile by the times above.  The first
    // box of the range of warp `lane`:
    auto first_box = [&](int run, int end) {
        const int w = min(lane, kWarps);
        if (kTiles != 2 || chunks > 32)
            return static_cast<int>(static_cast<long long>(end - run) * nb * w / kWarps);
        auto weight_of = [&](int c) { return tb.ncols[c] > kTileCols ? 5 : 4; };
        auto units_of = [&](int c) { return min((c + 1) * tiles, end) - max(c * tiles, run); };
        const int c0 = a.tiles.of(run);
        long long all = 0;
        for (int c = c0; c * tiles < end; ++c) all += units_of(c) * weight_of(c);
        long long want = all * nb * w / kWarps;
        int box = 0;
        for (int c = c0; c * tiles < end; ++c) {
            const int weight = weight_of(c);
            const long long here = static_cast<long long>(units_of(c)) * nb * weight;
            const long long take = want < here ? want : here;
            box += static_cast<int>((take + weight - 1) / weight);
            want -= take;
        }
        return box;
    };

    // What this warp has asked for so far.
    const int groups = a.K / 32;
    const bool wide_scales = a.wide_scales;
    const uint32_t ring_w = base + warp * a.l.ring * kBoxBytes;
    const uint32_t ring_s = base + a.l.scales + warp * a.l.ring * kScaleBytes;
    int p_u = 0, p_b = 0, p_left = 0, p_end = u0;            // p_left: boxes of the range
    int p_slot = -1;                         // of the ring of scales
    int p_chunk = chunk0, p_known = -1, p_n0 = 0, p_expert = 0, p_at = 0, issued = 0;
    const uint8_t* p_scale = nullptr;
    auto issue = [&]() {
        bool first = false;
        while (p_left == 0) {
            if (p_end >= u1) return;
            const int run = p_end;
            while (run >= (p_chunk + 1) * tiles) ++p_chunk;
            p_end = run_end(p_chunk);
            const int mine = first_box(run, p_end);
            const int lo = __shfl_sync(0xFFFFFFFFu, mine, warp);
            p_left = __shfl_sync(0xFFFFFFFFu, mine, warp + 1) - lo;
            if (p_left == 0) continue;
            const int units_before = a.boxes.of(lo);
            p_u = run + units_before;
            p_b = lo - units_before * nb;
            first = true;
        }
        if (p_u != p_known) {
            p_known = p_u;
            while (p_u >= (p_chunk + 1) * tiles) ++p_chunk;
            p_n0 = (p_u - p_chunk * tiles) * tile_cols;
            p_expert = tb.expert[p_chunk];
            // the row whose scales this lane copies; rows past the end of the
            // expert's are not used
            const int r = lane / kParts;
            const int n = kSwiglu ? min(p_n0 + r % (kRows / 2), out_cols - 1) +
                                        r / (kRows / 2) * out_cols
                                  : min(p_n0 + r, out_cols - 1);
            p_scale = a.w_scale + (static_cast<long long>(p_expert) * a.N + n) * groups;
        }
        const uint32_t bar = bars + 8 * p_at;
        if (lane == 0) {
            const uint32_t dst = ring_w + p_at * kBoxBytes;
            const int z = kSwiglu ? 2 * p_expert : p_expert;
            ptx::mbar_arrive_expect_tx(bar, kBoxBytes);
#pragma unroll
            for (int h = 0; h < kParts; ++h)
                ptx::tma_load_3d(dst + h * (kBoxBytes / kParts), &map_w,
                                 (kParts * p_b + h) * (kPartK / 2), p_n0, z, bar);
        }
        // The scales come for two boxes at once, sixteen a lane: a row's 512 K,
        // or half of a row's 1024 K.  (Eight at a time, through an L1 that has
        // little room beside the ring, 4 tokens take 53 us in place of 43.)
        if (first || p_b % 2 == 0) {
            if (++p_slot == a.l.ring) p_slot = 0;
            const int g = 16 * (p_b / 2 * kParts + lane % kParts);
            const uint32_t to = ring_s + p_slot * kScaleBytes + 16 * lane;
            if (wide_scales) {
                ptx::cp_async_16(to, p_scale + (g < groups ? g : 0), g < groups);
            } else {                         // at multiples of 4
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    ptx::cp_async_4(to + i, p_scale + (g + i < groups ? g + i : 0), g + i < groups);
            }
        }
        ptx::cp_async_mbar_arrive(bar);
        ++issued;
        if (++p_at == a.l.ring) p_at = 0;
        --p_left;
        if (++p_b == nb) {
            p_b = 0;
            ++p_u;
        }
    };
    for (int i = 0; i < a.l.ring; ++i) issue();

    // slots without an expert: zeros, spread over the grid
    for (int s = 0; tb.count[1] > 0 && s < a.slots; ++s) {
        if (tb.id[s] >= 0) continue;
        for (int n = blockIdx.x * kThreads + threadIdx.x; n < out_cols; n += gridDim.x * kThreads)
            a.out[static_cast<long long>(s) * out_cols + n] = 0;
    }

    // Sixteen weight rows of unit u (row tile r), of chunk c, times eight columns in
    // levels, from memory: a lane loads the words that ldmatrix would give it.
    auto rows_in_levels = [&](int u, int r, int c, int t) {
        const int q = lane & 3, g8 = lane >> 2, ncols = tb.ncols[c];
        const int n0 = (u - c * tiles) * tile_cols + 8 * (kSwiglu ? r : 2 * r) + g8;
        auto slot_of = [&](int col) { return tb.slot[c * a.l.cols + min(col, ncols - 1)]; };
        const uint16_t* row =
            a.x + static_cast<long long>(slot_of(8 * t + g8) / a.slots_per_row) * a.K + 8 * q;
        // the lane's two weight rows' first groups
        const long long base_row = static_cast<long long>(tb.expert[c]) * a.N;
        const long long lo = (base_row + min(n0, out_cols - 1)) * (a.K / 32);
        const long long hi = (base_row + (kSwiglu ? out_cols + min(n0, out_cols - 1)
                                                  : min(n0 + 8, out_cols - 1))) * (a.K / 32);
        float sum[4] = {};
#pragma unroll 1
        for (int part = 0; part * kPartK < a.K; ++part) {
            const int groups = min(8, a.K / 32 - 8 * part);
            auto x_of = [&](int g) {
                return ptx::load(reinterpret_cast<const uint4*>(row + part * kPartK + 32 * g));
            };
            Span span;
#pragma unroll 4
            for (int g = 0; g < groups; ++g) span.add(x_of(g));
            uint32_t top = span.largest();
            int low = span.least_code();
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {               // over the column's four lanes
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                low = min(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
            }
            const int be = exponent_of(top);
            const int mine = be == 255 || top == 0 ? 1 : (be - exponent_of(low + 32769)) / kLevel + 1;
            const int count = __reduce_max_sync(0xFFFFFFFFu, mine);
#pragma unroll 1
            for (int l = 0; l < count; ++l) {
                // of the columns whose sums the lane holds
                const int be0 = __shfl_sync(0xFFFFFFFFu, level_exponent(be, l), 8 * q);
                const int be1 = __shfl_sync(0xFFFFFFFFu, level_exponent(be, l), 8 * q + 4);
#pragma unroll 4
                for (int g = 0; g < groups; ++g) {
                    const uint4 x = level_part(x_of(g), be, l);
                    uint32_t w_lo[4], w_hi[4];
                    auto weights = [&](long long first, uint32_t(&w)[4]) {
                        const long long at = first + 8 * part + g;
                        ptx::e2m1x8_to_f16(
                            ptx::load(reinterpret_cast<const uint32_t*>(a.w_fp4 + 16 * at + 4 * q)), w);
                        return ptx::load(a.w_scale + at);
                    };
                    const uint32_t code_lo = weights(lo, w_lo), code_hi = weights(hi, w_hi);
                    float d[4];
                    ptx::mma_f16_16816_first(d, w_lo[0], w_hi[0], w_lo[1], w_hi[1], x.x, x.y);
                    ptx::mma_f16_16816(d, w_lo[2], w_hi[2], w_lo[3], w_hi[3], x.z, x.w);
                    sum[0] = add_scaled(d[0], code_lo, be0, sum[0]);
                    sum[1] = add_scaled(d[1], code_lo, be1, sum[1]);
                    sum[2] = add_scaled(d[2], code_hi, be0, sum[2]);
                    sum[3] = add_scaled(d[3], code_hi, be1, sum[3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int col = 8 * t + 2 * q + i;
            if (col >= ncols) continue;
            uint16_t* to = a.out + static_cast<long long>(slot_of(col)) * out_cols + n0;
            const float y = sum[i], y2 = sum[2 + i];
            const float v = kSwiglu ? y / (1.0f + expf(-y)) * y2 : y;
            if (n0 < out_cols) to[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            if (!kSwiglu && n0 + 8 < out_cols) to[8] = __bfloat16_as_ushort(__float2bfloat16_rn(y2));
        }
    };
    // What FP16 cut of a slot's row: a bound on the sum of the errors of its elements;
    // infinity where the quick result says nothing (Inf, NaN, extreme pieces).
    auto cut_of = [&](int slot) {
        const uint16_t* row = a.x + static_cast<long long>(slot / a.slots_per_row) * a.K;
        float cut = 0.0f;
#pragma unroll 1
        for (int k = 0; k < a.K; k += kPartK) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k + 8 * lane < a.K) v = ptx::load(reinterpret_cast<const uint4*>(row + k + 8 * lane));
            Span span;
            span.add(v);
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, span.largest());
            if (is_plain(span, top)) continue;
            const int be = exponent_of(top);
            if (abs(be - kFp16Exponent) > kQuickExponents) {
                cut = __uint_as_float(0x7F800000u);
                continue;
            }
            // an element is off by half of 2^-24 times 2^(be - 141), or by itself
            const float most = __uint_as_float(static_cast<uint32_t>(be - 39) << 23);
            float f[8];
            bf16_unpack8(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (be - exponent_of(__float_as_uint(f[e]) >> 16 & 0x7FFFu) >= kLevel)
                    cut += fminf(fabsf(f[e]), most);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) cut += __shfl_xor_sync(0xFFFFFFFFu, cut, o);
        return cut;
    };
    // Whether the cuts can show in sixteen rows' outputs (row tile r of unit u, eight
    // columns): they are 2^-11 of none of them, a quarter of BF16's step, with every
    // weight taken as 6 times the row's largest scale.
    auto cuts_show = [&](int u, int r, int c, int t, const float* cut) {
        const int q = lane & 3, g8 = lane >> 2, ncols = tb.ncols[c];
        const int n0 = (u - c * tiles) * tile_cols + 16 * r;
        // two lanes a row look for its largest scale, 4 codes at a time
        const long long first = (static_cast<long long>(tb.expert[c]) * a.N +
                                 min(n0 + (lane >> 1), out_cols - 1)) * (a.K / 32);
        uint32_t even = 0, odd = 0;
#pragma unroll 1
        for (int g = 4 * (lane & 1); g < a.K / 32; g += 8) {
            const uint32_t w = ptx::load(reinterpret_cast<const uint32_t*>(a.w_scale + first + g));
            even = __vmaxu2(even, w & 0x00FF00FFu);
            odd = __vmaxu2(odd, w >> 8 & 0x00FF00FFu);
        }
        const uint32_t two = __vmaxu2(even, odd);
        uint32_t code = max(two & 0xFFFFu, two >> 16);
        code = max(code, __shfl_xor_sync(0xFFFFFFFFu, code, 1));
        bool show = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float w = 6.0f * e8m0_value(__shfl_sync(0xFFFFFFFFu, code, 2 * (g8 + 8 * h)));
            const int n = n0 + g8 + 8 * h;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 8 * t + 2 * q + i;
                if (col >= ncols || n >= out_cols) continue;
                const int slot = tb.slot[c * a.l.cols + col];
                const float y = bf16_lo(ptx::load(a.out + static_cast<long long>(slot) * out_cols + n));
                const bool hidden = fabsf(y) >= 0x1p11f * cut[slot] * w && isfinite(y);
                show |= cut[slot] > 0.0f && !hidden;
            }
        }
        return static_cast<bool>(__any_sync(0xFFFFFFFFu, show));
    };
    // This block's units again, in levels, where FP16 has cut something off a row
    // that can show.  Which rows these are is found anew, a row a warp: rows that
    // nobody multiplies are held, too, and may hold anything.  SwiGLU's outputs do not
    // tell what can show: there all units of such a row are done again.
    //
    // With SwiGLU's outputs of gates beyond +-20 as x, one token's down takes 18 in
    // place of 13 us, 8 tokens' 41 for 28; where the cuts show in many outputs, some
    // ten times as long (gate/up of one token with a row that spans too much: 180
    // us).  At the very end, since the registers that this asks for, the loop of the
    // boxes does not get.
    auto units_in_levels = [&]() {
        float* cut = reinterpret_cast<float*>(smem + a.l.partial);           // by slot
        const int last = a.tiles.of(u1 - 1);
        __syncthreads();                     // outputs and sums: all is done
        for (int c = chunk0, col = warp; c <= last; col += kWarps) {
            for (; c <= last && col >= tb.ncols[c]; ++c) col -= tb.ncols[c];
            if (c > last) break;
            const int slot = tb.slot[c * a.l.cols + col];
            const float of_slot = cut_of(slot);
            if (lane == 0) cut[slot] = of_slot;
        }
        __syncthreads();
#pragma unroll 1
        for (int i = u0 * kR + warp, c = chunk0; i < u1 * kR; i += kWarps) {
            const int u = i / kR;
            while (u >= (c + 1) * tiles) ++c;
#pragma unroll 1
            for (int t = 0; 8 * t < tb.ncols[c]; ++t) {
                const int col = 8 * t + (lane & 7);
                const bool any = __any_sync(
                    0xFFFFFFFFu, col < tb.ncols[c] && cut[tb.slot[c * a.l.cols + col]] > 0.0f);
                if (any && (kSwiglu || cuts_show(u, i % kR, c, t, cut)))
                    rows_in_levels(u, i % kR, c, t);
            }
        }
    };

    const WaitCtx ctx{a.status, &s_abort, a.timeout_ns};
    const int q = lane & 3, g8 = lane >> 2;
    // ldmatrix: lane l addresses row l % 8 of matrix l / 8: the MMA's rows 0-7
    // and 8-15 of one group, then of the next; 16-byte chunks are XOR-swizzled
    // by row.  The 8-row blocks of a box follow one another; MMA r takes blocks
    // 2r and 2r + 1, or with SwiGLU block r of the gate's and of the up rows.
    constexpr int kHiBlock = kSwiglu ? kR : 1, kTileBlock = kSwiglu ? 1 : 2;
    const uint32_t lm_row =
        ring_w + ((lane >> 3) & 1) * (kHiBlock * kBlockBytes) + (lane & 7) * 128;
    constexpr int kScaleRow = 16 * kParts;
    const uint8_t* my_scales = smem + a.l.scales + warp * a.l.ring * kScaleBytes +
                               g8 * kScaleRow;
    int at = 0, slot = -1;
    uint32_t phase = 0, left_phase = 0;
    if (!kSingle && hold_all && u0 >= u1) {  // no work here, but rows are on their way
        wait_bounded(x_bar, x_phase, ctx, kRoleMatvec, 0x300);
        x_phase ^= 1;
    }
    for (int run = u0, chunk = chunk0; run < u1;) {
        while (run >= (chunk + 1) * tiles) ++chunk;
        const int end = run_end(chunk);
        if (run > u0) {
            __syncthreads();                 // everybody is done with the rows before
            load_run(chunk, end);
        }
        if (kSingle) {
            ptx::cp_async_wait_all_groups();
            __syncwarp();
        } else {
            rows_came = __any_sync(0xFFFFFFFFu,
                                   wait_bounded(x_bar, x_phase, ctx, kRoleMatvec, 0x300));
            x_phase ^= 1;
        }
        const int pieces = (hold_all ? a.x_rows : run_rows(chunk, end)) * parts;
        int piece = warp;
        bool other = false;
        if constexpr (!kSingle) {
            for (; piece + 3 * kWarps < pieces; piece += 4 * kWarps)
                other |= scale_pieces<4>(a, smem, piece, kWarps, parts, 1.0f / parts, lane);
        }
        for (; piece < pieces; piece += kWarps)
            other |= scale_pieces<1>(a, smem, piece, kWarps, parts, 1.0f / parts, lane);
        if (other) s_other = 1;              // and it stays
        const int mine = first_box(run, end);
        if (warp == 0 && lane <= kWarps) bound[lane] = mine;
        __syncthreads();
        const int lo = bound[warp], hi = bound[warp + 1];
        // Where this lane's columns of the current chunk lie; lanes of columns
        // that the chunk does not have read its last one, for sums nobody writes.
        int ncols = 0, rows_before = 0, x_chunk = chunk - 1;
        int x_at[kT], s_at[kT][2];           // offsets in shared memory
        auto next_chunk = [&]() {
            rows_before += ncols;
            ncols = tb.ncols[++x_chunk];
            auto held_row = [&](int c) {
                c = kSingle ? 0 : min(c, ncols - 1);
                return hold_all ? tb.slot[x_chunk * a.l.cols + c] / a.slots_per_row
                                : rows_before + c;
            };
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                x_at[t] = a.l.x + held_row(8 * t + g8) * a.l.x_stride + 16 * (kSingle ? lane : q);
#pragma unroll
                for (int i = 0; i < (kSingle ? 1 : 2); ++i)
                    s_at[t][i] = a.l.x_scale + 4 * held_row(8 * t + 2 * q + i) * parts;
            }
        };
        auto x_scale = [&](int t, int i, int part) {
            return *reinterpret_cast<const float*>(smem + s_at[t][i] + 4 * part);
        };
        uint64_t acc[kR][kT][2];             // rows g8 and g8 + 8, each of columns 2q and 2q + 1
#pragma unroll
        for (int i = 0; i < kR * kT * 2; ++i) acc[i / (2 * kT)][i / 2 % kT][i % 2] = 0;
        float one[2] = {0.0f, 0.0f};
        // 256 K of kRows weight rows times the chunk's columns, in `tiles_here`
        // MMAs side by side.
        auto multiply = [&](auto tiles_here, int b, const uint8_t* codes) {
            constexpr int kHere = decltype(tiles_here)::value;
            uint64_t sx[kHere];
#pragma unroll
            for (int t = 0; t < kHere; ++t)
                sx[t] = ptx::f32x2(x_scale(t, 0, b), x_scale(t, 1, b));
            uint2 code[kR][2];
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int hi = 0; hi < 2; ++hi)
                    code[r][hi] = *reinterpret_cast<const uint2*>(
                        codes + (r * kTileBlock + hi * kHiBlock) * 8 * kScaleRow);
            }
#pragma unroll
            for (int g = 0; g < 8; g += 2) {
                uint4 xf[2][kHere];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int t = 0; t < kHere; ++t)
                        xf[i][t] = *reinterpret_cast<const uint4*>(smem + x_at[t] + b * (2 * kPartK) +
                                                                   64 * (g + i));
                }
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    uint32_t w[4];
                    ptx::ldmatrix_x4(lm_row + at * kBoxBytes + r * kTileBlock * kBlockBytes +
                                         (((g + (lane >> 4)) ^ (lane & 7)) << 4), w);
                    const uint2 c0 = code[r][0], c1 = code[r][1];
                    const float2 s0 = ptx::e8m0x2_to_f32((g < 4 ? c0.x : c0.y) >> (g & 2) * 8);
                    const float2 s1 = ptx::e8m0x2_to_f32((g < 4 ? c1.x : c1.y) >> (g & 2) * 8);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t lo[4], hi[4];
                        ptx::e2m1x8_to_f16(w[2 * i], lo);
                        ptx::e2m1x8_to_f16(w[2 * i + 1], hi);
                        const uint64_t s_lo = i ? ptx::f32x2(s0.y, s0.y) : ptx::f32x2(s0.x, s0.x);
                        const uint64_t s_hi = i ? ptx::f32x2(s1.y, s1.y) : ptx::f32x2(s1.x, s1.x);
#pragma unroll
                        for (int t = 0; t < kHere; ++t) {
                            const uint4 x = xf[i][t];
                            float d[4];
                            ptx::mma_f16_16816_first(d, lo[0], hi[0], lo[1], hi[1], x.x, x.y);
                            ptx::mma_f16_16816(d, lo[2], hi[2], lo[3], hi[3], x.z, x.w);
                            acc[r][t][0] = ptx::fma_f32x2(
                                ptx::mul_f32x2(ptx::f32x2(d[0], d[1]), sx[t]), s_lo, acc[r][t][0]);
                            acc[r][t][1] = ptx::fma_f32x2(
                                ptx::mul_f32x2(ptx::f32x2(d[2], d[3]), sx[t]), s_hi, acc[r][t][1]);
                        }
                    }
                }
            }
        };
        bool left = false;                   // whether this warp has left its sums
        const int u_lo = a.boxes.of(lo);
        int begun = lo - u_lo * nb;          // where its part of unit u begins
        for (int i = lo, u = run + u_lo, b = begun; i < hi; ++i) {
            while (u >= (x_chunk + 1) * tiles) next_chunk();
            const bool ok = __all_sync(0xFFFFFFFFu,
                                       wait_bounded(bars + 8 * at, phase, ctx, kRoleMatvec, at));
            if ((i == lo || b % 2 == 0) && ++slot == a.l.ring) slot = 0;
            if (ok) {
                const uint8_t* codes = my_scales + slot * kScaleBytes + b % 2 * (8 * kParts);
                if (kSingle) {
#pragma unroll 1                             // fewer instructions to fetch: 20.7 us, else 22.6
                    for (int h = 0; h < kParts; ++h) {
                        const uint8_t* c = codes + 8 * h + 2 * q;
                        single_part(lm_row + at * kBoxBytes + h * (kBoxBytes / kParts),
                                    smem + x_at[0] + (kParts * b + h) * (2 * kPartK),
                                    *reinterpret_cast<const uint16_t*>(c),
                                    *reinterpret_cast<const uint16_t*>(c + 8 * kScaleRow),
                                    x_scale(0, 0, kParts * b + h), lane, one);
                    }
                } else if (kT == 2 && ncols > kTileCols) {
                    multiply(std::integral_constant<int, kT>(), b, codes);
                } else {
                    multiply(std::integral_constant<int, 1>(), b, codes);
                }
            }
            __syncwarp();                    // the box is read: its place may be refilled
            if (ok) issue();
            if (++at == a.l.ring) {
                at = 0;
                phase ^= 1;
            }
            const int done = u;
            const bool whole = ++b == nb;
            if (!whole && i + 1 < hi) continue;
            const bool own = begun == 0;     // this warp has the unit's first box
            begun = 0;
            if (whole) {
                b = 0;
                ++u;
            }

            // This warp's part of unit `done` is complete.
            uint8_t* sums = smem + a.l.partial;
            // the parts of the warps behind
            auto each_other = [&](auto f) {
                if (whole) return;
                const int unit_end = (done - run + 1) * nb;
                for (int w = warp + 1; bound[w] < unit_end; ++w) {
                    if (bound[w + 1] == bound[w]) continue;
                    wait_bounded(left_bar + 8 * w, left_phase, ctx, kRoleMatvec, 0x200 + w);
                    f(w);
                }
            };
            auto leave = [&]() {
                left = true;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(left_bar + 8 * warp);
            };
            if (kSingle) {
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
                    one[0] += __shfl_xor_sync(0xFFFFFFFFu, one[0], o);
                    one[1] += __shfl_xor_sync(0xFFFFFFFFu, one[1], o);
                }
                const float lo8 = __shfl_sync(0xFFFFFFFFu, one[0], 4 * (lane & 7));
                const float hi8 = __shfl_sync(0xFFFFFFFFu, one[1], 4 * (lane & 7));
                float y = lane & 8 ? hi8 : lo8;              // of weight row lane % 16
                one[0] = one[1] = 0.0f;
                float* sum = reinterpret_cast<float*>(sums) + (lane & 15);
                if (!own) {
                    if (lane < 16) sum[(warp - 1) * kRows] = y;
                    leave();
                    continue;
                }
                each_other([&](int w) { y += sum[(w - 1) * kRows]; });
                const int n = (done - x_chunk * tiles) * tile_cols + lane;
                if (kSwiglu) {
                    const float up = __shfl_down_sync(0xFFFFFFFFu, y, 8);
                    y = y / (1.0f + expf(-y)) * up;
                }
                if (lane < tile_cols && n < out_cols)
                    a.out[static_cast<long long>(tb.slot[x_chunk]) * out_cols + n] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(y));
            } else {
                constexpr int kA = kR * kT;
                ulonglong2* sum = reinterpret_cast<ulonglong2*>(sums) + lane;
                if (!own) {
#pragma unroll
                    for (int j = 0; j < kA; ++j) {
                        uint64_t(&mine)[2] = acc[j / kT][j % kT];
                        sum[((warp - 1) * kA + j) * 32] = make_ulonglong2(mine[0], mine[1]);
                        mine[0] = mine[1] = 0;
                    }
                    leave();
                    continue;
                }
                each_other([&](int w) {
#pragma unroll
                    for (int j = 0; j < kA; ++j) {
                        uint64_t(&mine)[2] = acc[j / kT][j % kT];
                        const ulonglong2 v = sum[((w - 1) * kA + j) * 32];
                        mine[0] = ptx::add_f32x2(mine[0], v.x);
                        mine[1] = ptx::add_f32x2(mine[1], v.y);
                    }
                });
                uint16_t* to[2 * kT];        // the lane's columns' outputs
#pragma unroll
                for (int c = 0; c < 2 * kT; ++c) {
                    const int col = min(8 * (c / 2) + 2 * q + c % 2, ncols - 1);
                    to[c] = a.out + static_cast<long long>(tb.slot[x_chunk * a.l.cols + col]) *
                                        out_cols;
                }
#pragma unroll
                for (int j = 0; j < kA; ++j) {
                    uint64_t(&mine)[2] = acc[j / kT][j % kT];
                    const float2 lo8 = ptx::f32x2_parts(mine[0]), hi8 = ptx::f32x2_parts(mine[1]);
                    const float y[4] = {lo8.x, lo8.y, hi8.x, hi8.y};
                    mine[0] = mine[1] = 0;
                    const int n = (done - x_chunk * tiles) * tile_cols +
                                  j / kT * (kSwiglu ? 8 : 16) + g8;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (8 * (j % kT) + 2 * q + c >= ncols) continue;
                        uint16_t* o = to[2 * (j % kT) + c] + n;
                        const float v = kSwiglu ? y[c] / (1.0f + expf(-y[c])) * y[2 + c] : y[c];
                        if (n < out_cols) o[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        if (!kSwiglu && n + 8 < out_cols)
                            o[8] = __bfloat16_as_ushort(__float2bfloat16_rn(y[2 + c]));
                    }
                }
            }
        }
        // once a run, whether or not there was anything to leave
        if (!left && lane == 0) ptx::mbar_arrive(left_bar + 8 * warp);
        left_phase ^= 1;
        run = end;
    }
    if (u0 < u1 && s_other) units_in_levels();
    // After a wait that gave up, copies may still be in flight: they land before
    // the shared memory is given back.
    if (*ctx.abort) {
        for (int i = max(0, issued - a.l.ring); i < issued; ++i)
            wait_drain(bars + 8 * (i % a.l.ring), (i / a.l.ring) & 1);
        if (!kSingle && warp == 0) wait_drain(x_bar, x_asked);
    }
}

// Devices (a bit each) on which a kernel's shared-memory limit has been set:
// by epilogue, MMAs, warps / 4.
std::atomic<uint64_t> g_ready[2][3][5];

template <bool kSwiglu, int kTiles, int kWarps>
cudaError_t launch(const CUtensorMap& map, const KernelArgs& k, int grid, cudaStream_t stream) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::atomic<uint64_t>& ready = g_ready[kSwiglu][kTiles][kWarps / 4];
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        err = cudaFuncSetAttribute(expert_matvec_kernel<kSwiglu, kTiles, kWarps>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (err != cudaSuccess) return err;
        ready.fetch_or(bit);
    }
    return launch_dependent(expert_matvec_kernel<kSwiglu, kTiles, kWarps>, grid, kWarps * 32,
                            k.l.total, stream, map, k);
}

template <bool kSwiglu, int kTiles>
cudaError_t launch_warps(const CUtensorMap& map, const KernelArgs& k, int grid,
                         cudaStream_t stream) {
    return k.l.warps == kWarpChoices[0]
               ? launch<kSwiglu, kTiles, kWarpChoices[0]>(map, k, grid, stream)
               : launch<kSwiglu, kTiles, kWarpChoices[1]>(map, k, grid, stream);
}

template <bool kSwiglu>
cudaError_t launch_cols(const CUtensorMap& map, const KernelArgs& k, int grid,
                        cudaStream_t stream) {
    switch (tiles_of(k.l.cols)) {
        case 0: return launch<kSwiglu, 0, kSingleWarps>(map, k, grid, stream);
        case 1: return launch_warps<kSwiglu, 1>(map, k, grid, stream);
        default: return launch_warps<kSwiglu, 2>(map, k, grid, stream);
    }
}

}  // namespace

void matvec_reset_caches() {
    for (auto& epilogue : g_ready) {
        for (auto& tiles : epilogue) {
            for (auto& ready : tiles) ready.store(0);
        }
    }
}

int matvec_unit_rows(const MatvecArgs& a) {
    Layout l;
    return make_layout(a.K, a.slots, a.tokens, a.E, a.slots / a.slots_per_row, &l)
               ? form_of(tiles_of(l.cols), l.warps).rows()
               : 0;
}

cudaError_t launch_expert_matvec(const MatvecArgs& a, const CUtensorMap& map_w, int num_sms,
                                 cudaStream_t stream) {
    KernelArgs k;
    k.x = a.x;
    k.ids = a.ids;
    k.w_fp4 = a.w_fp4;
    k.w_scale = a.w_scale;
    k.out = a.out;
    k.status = a.status;
    k.timeout_ns = a.timeout_ns;
    k.x_rows = a.slots / a.slots_per_row;
    k.slots_per_row = a.slots_per_row;
    k.slots = a.slots;
    k.E = a.E;
    k.N = a.N;
    k.K = a.K;
    if (!make_layout(a.K, a.slots, a.tokens, a.E, k.x_rows, &k.l)) return cudaErrorInvalidValue;
    const Form form = form_of(tiles_of(k.l.cols), k.l.warps);
    const int tile_cols = form.rows() / (a.swiglu ? 2 : 1), box_k = form.parts * kPartK;
    const int tiles = ((a.swiglu ? a.N / 2 : a.N) + tile_cols - 1) / tile_cols;
    const long long units = static_cast<long long>(tiles) * a.slots;
    const int grid = static_cast<int>(units < num_sms ? units : num_sms);
    k.wide_scales = ((reinterpret_cast<uintptr_t>(a.w_scale) | (a.K / 32)) & 15) == 0;
    k.boxes = Divisor((a.K + box_k - 1) / box_k);
    k.tiles = Divisor(tiles);
    k.blocks = Divisor(grid);
    return a.swiglu ? launch_cols<true>(map_w, k, grid, stream)
                    : launch_cols<false>(map_w, k, grid, stream);
}

}  // namespace hg

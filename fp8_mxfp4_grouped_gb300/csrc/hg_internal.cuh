// hg_internal.cuh -- declarations shared by the library's translation units:
// the device status word protocol, the bounded barrier wait, and the host
// launchers each kernel file exports to the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hg.h"
#include "ptx.cuh"

namespace hg {

// Device status word (3 x uint32, library-owned, one per device):
//   [0] first error code recorded since the last read (0 = none)
//   [1] detail of that first error
//   [2] number of expert ids dropped by the plan (out of range)
enum { kStatusCode = 0, kStatusDetail = 1, kStatusBadIds = 2, kStatusWords = 4 };

__device__ __forceinline__ void record_error(uint32_t* status, uint32_t code, uint32_t detail) {
    if (atomicCAS(&status[kStatusCode], 0u, code) == 0u) {
        atomicExch(&status[kStatusDetail], detail);
    }
}

// Where a wait happened, packed into the status detail of a timeout:
// role in bits 24..31, ring slot / buffer in bits 0..23.
enum WaitRole : uint32_t {
    kRoleProducer = 1,
    kRoleScale = 2,
    kRoleMma = 3,
    kRoleEpilogue = 4,
    kRoleTeardown = 5,
    kRoleSelftest = 6,
    kRoleRelay = 7,
    kRoleMatvec = 8,
    kRoleWorker = 9,
    kRoleNorm = 10,
};

struct WaitCtx {
    uint32_t* status;             // device status word
    volatile uint32_t* abort;     // shared-memory abort flag of this CTA
    uint64_t timeout_ns;
};

// Wait for the phase of `bar` with parity `parity` to complete.  Gives up
// after ctx.timeout_ns (records HG_ERR_TIMEOUT and raises the CTA's abort
// flag) or as soon as another role of the CTA raised the abort flag.
// Returns true when the phase completed.  kCluster: acquire at cluster scope
// (for barriers that threads of another CTA of the cluster arrive on).
template <bool kCluster = false>
__device__ __forceinline__ bool try_wait_scoped(uint32_t bar, uint32_t parity) {
    return kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
}

template <bool kCluster = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const WaitCtx& ctx,
                                             uint32_t role, uint32_t where) {
    if (try_wait_scoped<kCluster>(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (try_wait_scoped<kCluster>(bar, parity)) return true;
        if (*ctx.abort) return false;
        if ((it & 7u) == 0u && ptx::globaltimer_ns() - t0 > ctx.timeout_ns) {
            *ctx.abort = 1u;
            record_error(ctx.status, HG_ERR_TIMEOUT, (role << 24) | (where & 0xFFFFFFu));
            return false;
        }
    }
}

// Wait for asynchronous work in flight before a CTA gives up what it writes to.
// It ignores the abort flag, and its limit is its own: the caller's (down to a
// microsecond) may have run out on copies that are merely not there yet.
constexpr uint64_t kDrainNs = 1000000000ull;

// Returns whether the phase completed; false: the whole limit has passed.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::globaltimer_ns() - t0 > kDrainNs) return false;
    }
    return true;
}

// ------------------------------------------------- host-side launchers --

// Launch with programmatic dependent launch: blocks may start while the kernel
// before on the stream drains.  The kernel calls start_dependent first of all,
// so that stream order holds for everything it reads and writes.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int block, size_t smem,
                             cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// Wait until the kernel before has completed, and let the one after be launched.
__device__ __forceinline__ void start_dependent() {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
}

struct GemmArgs {
    const uint8_t* a_fp8;
    const uint8_t* a_scale;
    const uint8_t* w_fp4;
    const uint8_t* w_scale;
    const int32_t* offsets;
    int32_t E, N, K, rows;
    int32_t as_rs, as_ks;   // a_scale element (row r, group g) is at r * as_rs + g * as_ks
    uint16_t* out;
    uint32_t* status;
    uint64_t timeout_ns;
    int num_sms;
    int variant;   // 1, 2, 4 (CTA pairs), 6 (split-K), 8: see hg_set_gemm_variant
};

// Lanes of the warp whose key equals this lane's, for keys in [0, 2^nbits)
// and negative keys (all negative keys of the warp share one class here,
// separate from the valid ones).  Every lane of the warp must call it with
// the same nbits.
__device__ __forceinline__ uint32_t lanes_with_equal_key(int key, int nbits) {
    uint32_t m = __ballot_sync(0xFFFFFFFFu, key < 0);
    if (key >= 0) m = ~m;
    for (int b = 0; b < nbits; ++b) {
        const bool bit = (key >> b) & 1;
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, bit);
        m &= bit ? bal : ~bal;
    }
    return m;
}

// Activation tensor maps over the same [rows, K] bytes, 128-byte swizzle,
// with boxes of 128 K x (16 << i) rows: any multiple of 16 rows up to 240
// loads in at most four boxes (one TMA instruction each).
struct AMaps {
    CUtensorMap box[4];
};

// map_out: the output [rows, N] BF16 with boxes of 16 rows x 32 columns, for
// kernels that write whole 16-row chunks with TMA stores; nullptr: plain
// stores only.
cudaError_t launch_grouped_gemm(const GemmArgs& a, const CUtensorMap& map_w, const AMaps& map_a,
                                const CUtensorMap* map_out, cudaStream_t stream);
size_t gemm_smem_bytes(int variant, int32_t E);
long long gemm_launch_ctas(const GemmArgs& a);   // CTAs the launch would use
int gemm_max_experts();
// Forget the per-device kernel settings and occupancy answers (hg_shutdown).
void gemm_reset_caches();
// Forget the plan scratch array's per-device addresses (hg_shutdown).
void plan_noalloc_reset();
// Forget on which devices the few-token product's kernels are set up (hg_shutdown).
void matvec_reset_caches();
int gemm_pick_variant(int32_t E, int32_t N, int32_t K, int32_t rows, int num_sms);
int gemm_variant_token_tile(int variant);
int gemm_variant_max_experts(int variant);

struct PlanArgs {
    const int32_t* ids;
    int32_t R, E;
    int32_t* offsets;
    int32_t* sorted_to_src;
    int32_t* src_to_sorted;
    int32_t* ws_counts;
    uint32_t* status;
    int threads;   // block size chosen by the shared-memory fit
    int nblk;      // number of blocks of the histogram / scatter grids
    int chunk;     // ids per block (multiple of 32)
    int cluster_ctas;   // > 0: whole plan in one cluster of this many CTAs (plan_cluster_ctas)
};

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream);
size_t plan_smem_bytes(int32_t E, int threads);
// CTAs of the one-cluster plan for R routed rows and E experts (1..8), or 0
// when R or the count tables exceed what one cluster holds.
int plan_cluster_ctas(int32_t R, int32_t E, int smem_limit);

cudaError_t launch_selftest_wait(uint32_t* status, uint64_t timeout_ns, cudaStream_t stream);

cudaError_t launch_quantize_gather(const uint16_t* x, int K, int top_k, const int32_t* s2d,
                                   int rows, uint8_t* a_fp8, uint8_t* a_scale, int num_sms,
                                   cudaStream_t stream);
cudaError_t launch_quantize_scatter(const uint16_t* x, int M, int K, int top_k, const int32_t* d2s,
                                    int rows, uint8_t* a_fp8, uint8_t* a_scale, int num_sms,
                                    cudaStream_t stream);
int quantize_scatter_max_top_k();
cudaError_t launch_combine_topk(const uint16_t* y, const int32_t* d2s, const float* weights,
                                int M, int top_k, int N, uint16_t* out, int num_sms,
                                cudaStream_t stream);

cudaError_t launch_dispatch(const uint16_t* x, const int32_t* d2s, const float* weights, int M,
                            int top_k, int K, uint16_t* rows, cudaStream_t stream);
cudaError_t launch_dispatch_acts(const uint8_t* a, const uint8_t* scale, const int32_t* d2s, int M,
                                 int top_k, int K, uint8_t* rows, uint8_t* rows_scale,
                                 cudaStream_t stream);
cudaError_t launch_dispatch_bwd(const uint16_t* drows, const uint16_t* x, const int32_t* d2s,
                                const float* weights, int M, int top_k, int K, uint16_t* dx,
                                float* dw, cudaStream_t stream);
cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* d2s,
                               const float* weights, int M, int top_k, int N, uint16_t* dy,
                               float* dw, cudaStream_t stream);

int swiglu_max_groups();     // of 128 elements of h
cudaError_t launch_swiglu_quantize(const uint16_t* z, int rows, int F, uint8_t* a_fp8,
                                   uint8_t* a_scale, uint8_t* z_fp8, uint8_t* z_scale, int num_sms,
                                   cudaStream_t stream);
cudaError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* z_fp8, const uint8_t* z_scale,
                              int rows, int F, uint16_t* dz, int num_sms, cudaStream_t stream);

struct MatvecArgs {
    const uint16_t* x;
    int slots_per_row;      // consecutive slots that share an input row: 1 or top_k
    const int32_t* ids;     // one expert id a slot
    const uint8_t* w_fp4;
    const uint8_t* w_scale;
    int tokens, slots, E, N, K;
    bool swiglu;
    uint16_t* out;
    uint32_t* status;
    uint64_t timeout_ns;
};
// Weight rows of a work unit for these sizes.
int matvec_unit_rows(const MatvecArgs& a);
// map_w: the weights' bytes, 128-byte swizzle, boxes of a unit's rows x 128
// bytes; with swiglu half of them the gate's and half the up projection's.
cudaError_t launch_expert_matvec(const MatvecArgs& a, const CUtensorMap& map_w, int num_sms,
                                 cudaStream_t stream);
// Limits of the few-token product: a block lists the slots by expert in shared
// memory, and holds at least one input row there.
constexpr int kMatvecMaxSlots = 512;
constexpr int kMatvecMaxK = 32768;

cudaError_t launch_router_topk(const float* logits, int M, int E, int top_k, int renormalize,
                               int32_t* ids, float* weights, cudaStream_t stream);
cudaError_t launch_router_topk_bwd(const float* logits, const int32_t* ids, const float* weights,
                                   const float* dweights, int M, int E, int top_k,
                                   int renormalize, float* dlogits, cudaStream_t stream);
int router_max_top_k();

struct RmsnormArgs {
    const uint16_t *x, *residual, *gain;
    int M, D;
    float eps;
    uint16_t *sum, *y;      // y, a_fp8 (with a_scale) and rstd may be null
    uint8_t *a_fp8, *a_scale;
    float* rstd;
};
struct RmsnormBwdArgs {
    const uint16_t *dy, *dsum, *sum, *gain;     // dsum may be null
    const float* rstd;
    int M, D;
    uint16_t* dx;
    float *dgain, *parts;   // dgain may be null; parts: rmsnorm_bwd_workspace
    uint32_t* status;
    uint64_t timeout_ns;
};
int rmsnorm_max_elements();
size_t rmsnorm_bwd_workspace(int M, int D);
// Forget on which devices the norm's gradient is set up (hg_shutdown).
void rmsnorm_reset_caches();
cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream);
cudaError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, cudaStream_t stream);

// qt, scale_t: null for no transposed copy.
cudaError_t launch_quantize_weights(const void* w, bool f32, int E, int N, int K, uint8_t* q,
                                    uint8_t* scale, uint8_t* qt, uint8_t* scale_t,
                                    cudaStream_t stream);
cudaError_t launch_dequantize_weights(const uint8_t* q, const uint8_t* scale, int E, int N, int K,
                                      void* w, bool f32, cudaStream_t stream);

struct WgradArgs {
    const uint8_t *codes, *code_scale;  // an FP8 x, to be decoded into x; else null
    uint16_t* x;
    const int32_t* offsets;
    int E, N, K, rows;
    bool accumulate, f32;       // f32: dw is FP32, else BF16
    void* dw;
    float* parts;               // wgrad_parts_bytes, where the rows are split
    uint32_t* status;
    uint64_t timeout_ns;
};
// Parts that an expert's rows are split into for these sizes.
int wgrad_splits(int E, int N, int K, int rows);
size_t wgrad_parts_bytes(int E, int N, int K, int rows);
bool wgrad_fits(int E, int N, int K, int rows);     // the grid's numbers and the maps' strides
// Tensor maps, all with the 128-byte swizzle: dy [rows, N] and x [rows, K] in boxes of
// kWgradRows rows x wgrad_panels panels of 64 columns, as [rows, N] or as [N/64, rows, 64];
// the output (the parts where the rows are split) [E or parts, N, K] in boxes of 32 rows x
// 128 bytes.
constexpr int kWgradRows = 128;
int wgrad_panels(int cols);
struct WgradMaps {
    CUtensorMap dy, x, out;
};
cudaError_t launch_wgrad(const WgradArgs& a, const WgradMaps& maps, int num_sms,
                         cudaStream_t stream);
// Forget on which devices the weight gradient's kernels are set up (hg_shutdown).
void wgrad_reset_caches();

}  // namespace hg

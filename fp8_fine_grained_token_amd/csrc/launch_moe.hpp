// Host-side launchers of the operators around the expert products
// (argument checking happens in abi_moe.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8blk {

// ---- tokens by expert (moe.hip) ----
constexpr int64_t kSortMaxExperts = 1024;
size_t moe_sort_workspace_bytes(int64_t slots, int64_t E);

struct MoeRouting {
    const void *ids;  // int32 or int64 [T][k]
    bool wide_ids;
    int64_t T, k, E;
    int32_t *offsets, *slot_row, *row_slot;
    void *workspace;
};
hipError_t launch_moe_sort(const MoeRouting &r, hipStream_t stream);

// One plane of a gather: rows of `bytes` bytes, `ld` bytes apart in the
// source and dense in the destination.
struct GatherPlane {
    const void *src;
    void *dst;
    int64_t bytes, ld;
};
hipError_t launch_moe_dispatch(const GatherPlane &rows, const GatherPlane *scales,
                               const int32_t *slot_row, int64_t T, int64_t k, int64_t R,
                               hipStream_t stream);
hipError_t launch_moe_dispatch_quant(const void *x, int64_t ldx, int64_t T, int64_t H,
                                     const int32_t *slot_row, int64_t k, void *q, float *scales,
                                     int64_t R, bool pow2, hipStream_t stream);

// Sort and gather: one launch for few slots.
hipError_t launch_moe_sort_dispatch(const MoeRouting &r, const GatherPlane &rows,
                                    hipStream_t stream);
hipError_t launch_moe_sort_dispatch_quant(const MoeRouting &r, const void *x, int64_t ldx,
                                          int64_t H, void *q, float *scales, bool pow2,
                                          hipStream_t stream);

hipError_t launch_moe_combine(const void *ys, bool ys_bf16, int64_t ld, int64_t R,
                              const int32_t *slot_row, const float *weights, int64_t T,
                              int64_t k, int64_t H, const void *residual, int64_t ld_residual,
                              void *out, bool out_bf16, hipStream_t stream);
hipError_t launch_moe_combine_grad(const void *dout, int64_t ld_dout, const void *ys,
                                   int64_t ld_ys, bool bf16, int64_t R, const int32_t *slot_row,
                                   const float *weights, int64_t T, int64_t k, int64_t H,
                                   void *dys, float *dweights, hipStream_t stream);

// ---- norms round a block (norm.hip) ----
constexpr int64_t kNormMaxWidth = 32768;

struct NormArgs {
    const void *y, *r;            // forward: y, r; gradient: y, r_out
    int64_t ldy, ldr;
    const void *w_post, *gate, *w_pre;
    bool y_bf16, r_bf16, param_bf16, post;
    int64_t T, H, gate_rows;      // gate_rows: 1 without a gate
    float residual_scale, branch_scale, eps;
    // forward
    void *r_out, *n, *q;
    float *scales, *rstd_post, *rstd_pre;
    bool pow2;
    // gradient
    const void *dn, *dr_out;
    int64_t ld_dn, ld_dr_out;
    const float *in_rstd_post, *in_rstd_pre;
    void *dy, *dr;
    float *dw_post, *dgate, *dw_pre;
    float *workspace;
};
hipError_t launch_norm_residual(const NormArgs &a, hipStream_t stream);
size_t norm_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows);
hipError_t launch_norm_residual_grad(const NormArgs &a, hipStream_t stream);

// ---- 4-bit weights (w4.hip) ----
hipError_t launch_w4_quant(const void *w, int64_t N, int64_t K, void *codes, void *scales,
                           bool e8m0, hipStream_t stream);
// offsets NULL: dense (E = 1).
hipError_t launch_w4_matvec(const void *x, int64_t ldx, const void *codes, const void *scales,
                            bool e8m0, const int32_t *offsets, int64_t E, int64_t R, int64_t N,
                            int64_t K, void *y, bool bf16_out, hipStream_t stream);

}  // namespace fp8blk

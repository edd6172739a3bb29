// C ABI of the operators around the expert products (include/fp8moe.h):
// argument validation, then dispatch to the launchers.  Every check runs
// before anything is enqueued; on error nothing is written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8moe.h"
#include "launch_moe.hpp"

namespace {

using namespace fp8blk;

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline fp8_status from_hip(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }
inline hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }
// an error that an earlier HIP call left on this thread is not this call's
inline void clear_last_error() { (void)hipGetLastError(); }

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxInner = (int64_t)1 << 24;  // inner dimension of a 4-bit product
constexpr int64_t kMaxWidth = (int64_t)1 << 28;  // a token's row: 32-bit byte offsets

inline bool dim_ok(int64_t n) { return n >= 0 && n < kMaxDim; }
inline bool matrix_ok(int64_t rows, int64_t cols) {
    return dim_ok(rows) && dim_ok(cols) && rows * cols < kMaxElems;
}
// rows `ld` elements apart: a row stride that keeps every address in range
inline bool stride_ok(int64_t rows, int64_t ld) {
    return ld >= 0 && ld < kMaxElems && (rows <= 1 || ld < kMaxElems / rows);
}
inline bool type_ok(int t) { return t == FP8_OUT_F32 || t == FP8_OUT_BF16; }
inline uintptr_t bytes_of(int t) { return t == FP8_OUT_BF16 ? 2 : 4; }

// ---- tokens by expert ----

fp8_status check_routing(const MoeRouting &r, int id_bytes, size_t workspace_bytes) {
    if (id_bytes != 4 && id_bytes != 8) return FP8_ERR_DTYPE;
    if (!dim_ok(r.T) || !dim_ok(r.k) || r.T * r.k >= kMaxDim) return FP8_ERR_SHAPE;
    if (r.E < 1 || r.E > kSortMaxExperts) return FP8_ERR_SHAPE;
    if (!r.offsets) return FP8_ERR_NULL;
    const bool any = r.T * r.k > 0;
    if (any && (!r.ids || !r.slot_row || !r.row_slot)) return FP8_ERR_NULL;
    if (!aligned(r.offsets, 4)) return FP8_ERR_ALIGN;
    if (any && (!aligned(r.ids, id_bytes) || !aligned(r.slot_row, 4) || !aligned(r.row_slot, 4)))
        return FP8_ERR_ALIGN;
    const size_t need = moe_sort_workspace_bytes(r.T * r.k, r.E);
    if (workspace_bytes < need || (need && !r.workspace)) return FP8_ERR_WORKSPACE;
    if (r.workspace && !aligned(r.workspace, 16)) return FP8_ERR_WORKSPACE;
    return FP8_OK;
}

// A plan and the rows it names: T x k slots into R rows.
fp8_status check_plan(const int32_t *slot_row, int64_t T, int64_t k, int64_t H, int64_t R) {
    if (!matrix_ok(T, H) || !matrix_ok(R, H) || H >= kMaxWidth) return FP8_ERR_SHAPE;
    if (!dim_ok(k) || T * k >= kMaxDim) return FP8_ERR_SHAPE;
    if (T * k > 0 && H > 0) {
        if (!slot_row) return FP8_ERR_NULL;
        if (!aligned(slot_row, 4)) return FP8_ERR_ALIGN;
    }
    return FP8_OK;
}

fp8_status check_rows(const void *x, int elem_bytes, int64_t ldx, int64_t T) {
    if (!stride_ok(T, ldx)) return FP8_ERR_SHAPE;
    if (!x) return FP8_ERR_NULL;
    return aligned(x, elem_bytes) ? FP8_OK : FP8_ERR_ALIGN;
}

fp8_status dispatch_quant(const void *x, int64_t ldx, int64_t T, int64_t H,
                          const int32_t *slot_row, int64_t k, void *q, float *scales, int64_t R,
                          bool pow2, void *stream) {
    fp8_status st = check_plan(slot_row, T, k, H, R);
    if (st != FP8_OK) return st;
    if (T * k == 0 || H == 0 || R == 0) return FP8_OK;
    st = check_rows(x, 2, ldx, T);
    if (st != FP8_OK) return st;
    if (!q || !scales) return FP8_ERR_NULL;
    if (!aligned(scales, 4)) return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(
        launch_moe_dispatch_quant(x, ldx, T, H, slot_row, k, q, scales, R, pow2, as_stream(stream)));
}

fp8_status sort_dispatch_quant(const void *x, int64_t ldx, int64_t T, int64_t H, const void *ids,
                               int id_bytes, int64_t k, int64_t E, int32_t *offsets,
                               int32_t *slot_row, int32_t *row_slot, void *q, float *scales,
                               void *ws, size_t ws_bytes, bool pow2, void *stream) {
    const MoeRouting r{ids, id_bytes == 8, T, k, E, offsets, slot_row, row_slot, ws};
    fp8_status st = check_routing(r, id_bytes, ws_bytes);
    if (st != FP8_OK) return st;
    st = check_plan(slot_row, T, k, H, T * k);
    if (st != FP8_OK) return st;
    const bool rows = T * k > 0 && H > 0;
    if (rows) {
        st = check_rows(x, 2, ldx, T);
        if (st != FP8_OK) return st;
        if (!q || !scales) return FP8_ERR_NULL;
        if (!aligned(scales, 4)) return FP8_ERR_ALIGN;
    }
    clear_last_error();
    if (!rows) return from_hip(launch_moe_sort(r, as_stream(stream)));
    return from_hip(
        launch_moe_sort_dispatch_quant(r, x, ldx, H, q, scales, pow2, as_stream(stream)));
}

// ---- norms ----

fp8_status check_norm(const NormArgs &a, int y_type, int r_type, int param_type, bool has_gate) {
    if (!type_ok(y_type) || !type_ok(r_type) || !type_ok(param_type)) return FP8_ERR_DTYPE;
    if (y_type == FP8_OUT_F32 && r_type == FP8_OUT_BF16) return FP8_ERR_DTYPE;
    if (!matrix_ok(a.T, a.H) || a.H > kNormMaxWidth) return FP8_ERR_SHAPE;
    if (!stride_ok(a.T, a.ldy) || !stride_ok(a.T, a.ldr)) return FP8_ERR_SHAPE;
    if (has_gate) {
        if (a.gate_rows < 1 || !matrix_ok(a.gate_rows, a.H)) return FP8_ERR_SHAPE;
        if (a.T % a.gate_rows != 0) return FP8_ERR_SHAPE;
    }
    const uintptr_t b = bytes_of(param_type);
    if (!aligned(a.w_post, b) || !aligned(a.gate, b) || !aligned(a.w_pre, b))
        return FP8_ERR_ALIGN;
    return FP8_OK;
}

fp8_status norm_residual(const void *y, int y_dtype, int64_t ldy, const void *r, int r_dtype,
                         int64_t ldr, const void *w_post, const void *gate, const void *w_pre,
                         int param_dtype, int64_t T, int64_t H, int64_t gate_rows, int post_norm,
                         float residual_scale, float branch_scale, float eps, void *r_out,
                         void *n, bool quant, void *q, float *scales, float *rstd_post,
                         float *rstd_pre, bool pow2, void *stream) {
    NormArgs a = {};
    a.y = y; a.r = r; a.ldy = ldy; a.ldr = ldr;
    a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
    a.y_bf16 = y_dtype == FP8_OUT_BF16;
    a.r_bf16 = r_dtype == FP8_OUT_BF16;
    a.param_bf16 = param_dtype == FP8_OUT_BF16;
    a.post = post_norm != 0;
    a.T = T; a.H = H; a.gate_rows = gate ? gate_rows : 1;
    a.residual_scale = residual_scale; a.branch_scale = branch_scale; a.eps = eps;
    a.r_out = r_out; a.n = n; a.q = q; a.scales = scales;
    a.rstd_post = rstd_post; a.rstd_pre = rstd_pre; a.pow2 = pow2;
    const fp8_status st = check_norm(a, y_dtype, r_dtype, param_dtype, gate != nullptr);
    if (st != FP8_OK || T == 0 || H == 0) return st;
    if (!y || !r || !r_out || (quant && (!q || !scales))) return FP8_ERR_NULL;
    const uintptr_t by = bytes_of(y_dtype), br = bytes_of(r_dtype);
    if (!aligned(y, by) || !aligned(n, by) || !aligned(r, br) || !aligned(r_out, br) ||
        !aligned(scales, 4) || !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
        return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_norm_residual(a, as_stream(stream)));
}

// ---- 4-bit weights ----

fp8_status w4_quant(const void *w, int64_t N, int64_t K, void *codes, void *scales, bool e8m0,
                    void *stream) {
    if (!matrix_ok(N, K)) return FP8_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8_OK;
    if (!w || !codes || !scales) return FP8_ERR_NULL;
    if (!aligned(w, 2) || !aligned(scales, e8m0 ? 1 : 4)) return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_w4_quant(w, N, K, codes, scales, e8m0, as_stream(stream)));
}

fp8_status w4_matvec(const void *x, int64_t ldx, const void *codes, const void *scales, int kind,
                     const int32_t *offsets, bool grouped, int64_t E, int64_t R, int64_t N,
                     int64_t K, void *y, int out_dtype, void *stream) {
    if (!type_ok(out_dtype)) return FP8_ERR_DTYPE;
    if (kind != FP8_W4_F32_1X128 && kind != FP8_W4_E8M0_1X32) return FP8_ERR_DTYPE;
    // a tile's 16 rows of codes are addressed with 32-bit offsets
    if (!matrix_ok(R, K) || !matrix_ok(R, N) || !matrix_ok(N, K) || K >= kMaxInner)
        return FP8_ERR_SHAPE;
    if (!stride_ok(R, ldx)) return FP8_ERR_SHAPE;
    if (E < 0 || E > 65535 || N * K >= kMaxElems / (E > 0 ? E : 1)) return FP8_ERR_SHAPE;
    if (R == 0 || N == 0) return FP8_OK;
    if (E == 0) return FP8_ERR_SHAPE;
    if (!y || (K > 0 && (!x || !codes || !scales)) || (grouped && !offsets)) return FP8_ERR_NULL;
    if (!aligned(x, 2) || !aligned(y, bytes_of(out_dtype)) || !aligned(offsets, 4) ||
        !aligned(scales, kind == FP8_W4_F32_1X128 ? 4 : 1))
        return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_w4_matvec(x, ldx, codes, scales, kind == FP8_W4_E8M0_1X32,
                                     grouped ? offsets : nullptr, E, R, N, K, y,
                                     out_dtype == FP8_OUT_BF16, as_stream(stream)));
}

}  // namespace

extern "C" {

size_t fp8_moe_sort_workspace_bytes(int64_t T, int64_t top_k, int64_t E) {
    if (!dim_ok(T) || !dim_ok(top_k) || T * top_k >= kMaxDim || E < 1 || E > kSortMaxExperts)
        return 0;
    return moe_sort_workspace_bytes(T * top_k, E);
}

fp8_status fp8_moe_sort(const void *expert_ids, int id_bytes, int64_t T, int64_t top_k,
                        int64_t E, int32_t *group_offsets, int32_t *slot_row,
                        int32_t *row_slot, void *workspace, size_t workspace_bytes,
                        void *hip_stream) {
    const MoeRouting r{expert_ids,    id_bytes == 8, T,        top_k,    E,
                       group_offsets, slot_row,      row_slot, workspace};
    const fp8_status st = check_routing(r, id_bytes, workspace_bytes);
    if (st != FP8_OK) return st;
    clear_last_error();
    return from_hip(launch_moe_sort(r, as_stream(hip_stream)));
}

fp8_status fp8_moe_dispatch(const void *x, int elem_bytes, int64_t ldx, const float *x_scales,
                            int64_t ldx_scales, int64_t T, int64_t H, int64_t G,
                            const int32_t *slot_row, int64_t top_k, void *xs, float *xs_scales,
                            int64_t R, void *hip_stream) {
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return FP8_ERR_DTYPE;
    fp8_status st = check_plan(slot_row, T, top_k, H, R);
    if (st != FP8_OK) return st;
    if (x_scales && (!matrix_ok(T, G) || !matrix_ok(R, G) || !stride_ok(T, ldx_scales)))
        return FP8_ERR_SHAPE;
    if (T * top_k == 0 || H == 0 || R == 0) return FP8_OK;
    st = check_rows(x, elem_bytes, ldx, T);
    if (st != FP8_OK) return st;
    if (!xs || (x_scales != nullptr) != (xs_scales != nullptr)) return FP8_ERR_NULL;
    if (!aligned(xs, elem_bytes) || !aligned(x_scales, 4) || !aligned(xs_scales, 4))
        return FP8_ERR_ALIGN;
    const GatherPlane rows{x, xs, H * elem_bytes, ldx * elem_bytes};
    const GatherPlane scales{x_scales, xs_scales, G * 4, ldx_scales * 4};
    clear_last_error();
    return from_hip(launch_moe_dispatch(rows, x_scales ? &scales : nullptr, slot_row, T, top_k, R,
                                        as_stream(hip_stream)));
}

fp8_status fp8_moe_dispatch_quant_1x128(const void *x_bf16, int64_t ldx, int64_t T, int64_t H,
                                        const int32_t *slot_row, int64_t top_k, void *q,
                                        float *scales, int64_t R, void *hip_stream) {
    return dispatch_quant(x_bf16, ldx, T, H, slot_row, top_k, q, scales, R, false, hip_stream);
}

fp8_status fp8_moe_dispatch_quant_1x128_pow2(const void *x_bf16, int64_t ldx, int64_t T,
                                             int64_t H, const int32_t *slot_row, int64_t top_k,
                                             void *q, float *scales, int64_t R,
                                             void *hip_stream) {
    return dispatch_quant(x_bf16, ldx, T, H, slot_row, top_k, q, scales, R, true, hip_stream);
}

fp8_status fp8_moe_sort_dispatch(const void *x, int elem_bytes, int64_t ldx, int64_t T,
                                 int64_t H, const void *expert_ids, int id_bytes,
                                 int64_t top_k, int64_t E, int32_t *group_offsets,
                                 int32_t *slot_row, int32_t *row_slot, void *xs,
                                 void *workspace, size_t workspace_bytes, void *hip_stream) {
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return FP8_ERR_DTYPE;
    const MoeRouting r{expert_ids,    id_bytes == 8, T,        top_k,    E,
                       group_offsets, slot_row,      row_slot, workspace};
    fp8_status st = check_routing(r, id_bytes, workspace_bytes);
    if (st != FP8_OK) return st;
    st = check_plan(slot_row, T, top_k, H, T * top_k);
    if (st != FP8_OK) return st;
    const bool rows = T * top_k > 0 && H > 0;
    if (rows) {
        st = check_rows(x, elem_bytes, ldx, T);
        if (st != FP8_OK) return st;
        if (!xs) return FP8_ERR_NULL;
        if (!aligned(xs, elem_bytes)) return FP8_ERR_ALIGN;
    }
    clear_last_error();
    if (!rows) return from_hip(launch_moe_sort(r, as_stream(hip_stream)));
    return from_hip(launch_moe_sort_dispatch(
        r, GatherPlane{x, xs, H * elem_bytes, ldx * elem_bytes},
        as_stream(hip_stream)));
}

fp8_status fp8_moe_sort_dispatch_quant_1x128(const void *x_bf16, int64_t ldx, int64_t T,
                                             int64_t H, const void *expert_ids, int id_bytes,
                                             int64_t top_k, int64_t E, int32_t *group_offsets,
                                             int32_t *slot_row, int32_t *row_slot, void *q,
                                             float *scales, void *workspace,
                                             size_t workspace_bytes, void *hip_stream) {
    return sort_dispatch_quant(x_bf16, ldx, T, H, expert_ids, id_bytes, top_k, E, group_offsets,
                               slot_row, row_slot, q, scales, workspace, workspace_bytes, false,
                               hip_stream);
}

fp8_status fp8_moe_sort_dispatch_quant_1x128_pow2(
    const void *x_bf16, int64_t ldx, int64_t T, int64_t H, const void *expert_ids, int id_bytes,
    int64_t top_k, int64_t E, int32_t *group_offsets, int32_t *slot_row, int32_t *row_slot,
    void *q, float *scales, void *workspace, size_t workspace_bytes, void *hip_stream) {
    return sort_dispatch_quant(x_bf16, ldx, T, H, expert_ids, id_bytes, top_k, E, group_offsets,
                               slot_row, row_slot, q, scales, workspace, workspace_bytes, true,
                               hip_stream);
}

fp8_status fp8_moe_combine(const void *ys, int in_dtype, int64_t ld_ys, int64_t R,
                           const int32_t *slot_row, const float *weights, int64_t T,
                           int64_t top_k, int64_t H, const void *residual, int64_t ld_residual,
                           void *out, int out_dtype, void *hip_stream) {
    if (!type_ok(in_dtype) || !type_ok(out_dtype)) return FP8_ERR_DTYPE;
    fp8_status st = check_plan(slot_row, T, top_k, H, R);
    if (st != FP8_OK) return st;
    if (!stride_ok(R, ld_ys) || (residual && !stride_ok(T, ld_residual))) return FP8_ERR_SHAPE;
    if (T == 0 || H == 0) return FP8_OK;
    if (!out || (!ys && R > 0 && top_k > 0)) return FP8_ERR_NULL;
    if (!aligned(ys, bytes_of(in_dtype)) || !aligned(out, bytes_of(out_dtype)) ||
        !aligned(residual, bytes_of(out_dtype)) || !aligned(weights, 4))
        return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_moe_combine(ys, in_dtype == FP8_OUT_BF16, ld_ys, R, slot_row, weights,
                                       T, top_k, H, residual, ld_residual, out,
                                       out_dtype == FP8_OUT_BF16, as_stream(hip_stream)));
}

fp8_status fp8_moe_dispatch_grad(const void *dxs, int in_dtype, int64_t ld_dxs, int64_t R,
                                 const int32_t *slot_row, int64_t T, int64_t top_k, int64_t H,
                                 void *dx, int out_dtype, void *hip_stream) {
    return fp8_moe_combine(dxs, in_dtype, ld_dxs, R, slot_row, nullptr, T, top_k, H, nullptr, 0,
                           dx, out_dtype, hip_stream);
}

fp8_status fp8_moe_combine_grad(const void *dout, int64_t ld_dout, const void *ys,
                                int64_t ld_ys, int dtype, int64_t R, const int32_t *slot_row,
                                const float *weights, int64_t T, int64_t top_k, int64_t H,
                                void *dys, float *dweights, void *hip_stream) {
    if (!type_ok(dtype)) return FP8_ERR_DTYPE;
    const fp8_status st = check_plan(slot_row, T, top_k, H, R);
    if (st != FP8_OK) return st;
    if (!stride_ok(T, ld_dout) || !stride_ok(R, ld_ys)) return FP8_ERR_SHAPE;
    if (T * top_k == 0 || (!dys && !dweights) || (H == 0 && !dweights)) return FP8_OK;
    // with no columns every dot product is an empty sum: slot_row is needed
    // only to be read where H > 0, but the gradient is still written
    if (H > 0 && (!dout || (dweights && !ys && R > 0))) return FP8_ERR_NULL;
    if (H == 0 && !slot_row) return FP8_ERR_NULL;
    const uintptr_t b = bytes_of(dtype);
    if (!aligned(dout, b) || !aligned(ys, b) || !aligned(dys, b) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_moe_combine_grad(dout, ld_dout, ys, ld_ys, dtype == FP8_OUT_BF16, R,
                                            slot_row, weights, T, top_k, H, dys, dweights,
                                            as_stream(hip_stream)));
}

fp8_status fp8_norm_residual(const void *y, int y_dtype, int64_t ldy, const void *r, int r_dtype,
                             int64_t ldr, const void *w_post, const void *gate,
                             const void *w_pre, int param_dtype, int64_t T, int64_t H,
                             int64_t gate_rows, int post_norm, float residual_scale,
                             float branch_scale, float eps, void *r_out, void *n,
                             float *rstd_post, float *rstd_pre, void *hip_stream) {
    return norm_residual(y, y_dtype, ldy, r, r_dtype, ldr, w_post, gate, w_pre, param_dtype, T, H,
                         gate_rows, post_norm, residual_scale, branch_scale, eps, r_out, n, false,
                         nullptr, nullptr, rstd_post, rstd_pre, false, hip_stream);
}

fp8_status fp8_norm_residual_quant_1x128(const void *y, int y_dtype, int64_t ldy, const void *r,
                                         int r_dtype, int64_t ldr, const void *w_post,
                                         const void *gate, const void *w_pre, int param_dtype,
                                         int64_t T, int64_t H, int64_t gate_rows, int post_norm,
                                         float residual_scale, float branch_scale, float eps,
                                         void *r_out, void *n, void *q, float *scales,
                                         float *rstd_post, float *rstd_pre, void *hip_stream) {
    return norm_residual(y, y_dtype, ldy, r, r_dtype, ldr, w_post, gate, w_pre, param_dtype, T, H,
                         gate_rows, post_norm, residual_scale, branch_scale, eps, r_out, n, true,
                         q, scales, rstd_post, rstd_pre, false, hip_stream);
}

fp8_status fp8_norm_residual_quant_1x128_pow2(
    const void *y, int y_dtype, int64_t ldy, const void *r, int r_dtype, int64_t ldr,
    const void *w_post, const void *gate, const void *w_pre, int param_dtype, int64_t T,
    int64_t H, int64_t gate_rows, int post_norm, float residual_scale, float branch_scale,
    float eps, void *r_out, void *n, void *q, float *scales, float *rstd_post, float *rstd_pre,
    void *hip_stream) {
    return norm_residual(y, y_dtype, ldy, r, r_dtype, ldr, w_post, gate, w_pre, param_dtype, T, H,
                         gate_rows, post_norm, residual_scale, branch_scale, eps, r_out, n, true,
                         q, scales, rstd_post, rstd_pre, true, hip_stream);
}

size_t fp8_norm_residual_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows) {
    if (!matrix_ok(T, H) || H > kNormMaxWidth || gate_rows < 0) return 0;
    if (gate_rows == 0) gate_rows = 1;
    if (T % gate_rows != 0) return 0;
    return norm_grad_workspace_bytes(T, H, gate_rows);
}

fp8_status fp8_norm_residual_grad(const void *dn, int64_t ld_dn, const void *dr_out,
                                  int64_t ld_dr_out, const void *y, int y_dtype, int64_t ldy,
                                  const void *r_out, int r_dtype, int64_t ld_r_out,
                                  const float *rstd_post, const float *rstd_pre,
                                  const void *w_post, const void *gate, const void *w_pre,
                                  int param_dtype, int64_t T, int64_t H, int64_t gate_rows,
                                  int post_norm, float residual_scale, float branch_scale,
                                  void *dy, void *dr, float *dw_post, float *dgate,
                                  float *dw_pre, void *workspace, size_t workspace_bytes,
                                  void *hip_stream) {
    NormArgs a = {};
    a.dn = dn; a.ld_dn = ld_dn; a.dr_out = dr_out; a.ld_dr_out = ld_dr_out;
    a.y = y; a.ldy = ldy; a.r = r_out; a.ldr = ld_r_out;
    a.in_rstd_post = rstd_post; a.in_rstd_pre = rstd_pre;
    a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
    a.y_bf16 = y_dtype == FP8_OUT_BF16;
    a.r_bf16 = r_dtype == FP8_OUT_BF16;
    a.param_bf16 = param_dtype == FP8_OUT_BF16;
    a.post = post_norm != 0;
    a.T = T; a.H = H; a.gate_rows = gate ? gate_rows : 1;
    a.residual_scale = residual_scale; a.branch_scale = branch_scale;
    a.dy = dy; a.dr = dr; a.dw_post = dw_post; a.dgate = dgate; a.dw_pre = dw_pre;
    a.workspace = static_cast<float *>(workspace);
    const fp8_status st = check_norm(a, y_dtype, r_dtype, param_dtype, gate != nullptr);
    if (st != FP8_OK) return st;
    if (!stride_ok(T, ld_dn) || !stride_ok(T, ld_dr_out)) return FP8_ERR_SHAPE;
    if ((dgate && !gate) || (dw_post && !post_norm)) return FP8_ERR_NULL;
    if (H == 0) return FP8_OK;
    if (T > 0) {
        if (!y || !dy || !dr || (a.post && !rstd_post) || (dn && (!r_out || !rstd_pre)))
            return FP8_ERR_NULL;
        const size_t need = norm_grad_workspace_bytes(T, H, a.gate_rows);
        if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
            return FP8_ERR_WORKSPACE;
    }
    const uintptr_t by = bytes_of(y_dtype), br = bytes_of(r_dtype);
    if (!aligned(dn, by) || !aligned(y, by) || !aligned(dy, by) || !aligned(dr_out, br) ||
        !aligned(r_out, br) || !aligned(dr, br) || !aligned(rstd_post, 4) ||
        !aligned(rstd_pre, 4) || !aligned(dw_post, 4) || !aligned(dgate, 4) ||
        !aligned(dw_pre, 4))
        return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_norm_residual_grad(a, as_stream(hip_stream)));
}

fp8_status fp8_w4_quant_1x128(const void *w_bf16, int64_t N, int64_t K, void *codes,
                              float *scales, void *hip_stream) {
    return w4_quant(w_bf16, N, K, codes, scales, false, hip_stream);
}

fp8_status fp8_w4_quant_1x32(const void *w_bf16, int64_t N, int64_t K, void *codes,
                             void *scales_e8m0, void *hip_stream) {
    return w4_quant(w_bf16, N, K, codes, scales_e8m0, true, hip_stream);
}

fp8_status fp8_w4_matvec(const void *x_bf16, int64_t ldx, const void *codes, const void *scales,
                         int scale_kind, int64_t M, int64_t N, int64_t K, void *y,
                         int out_dtype, void *hip_stream) {
    return w4_matvec(x_bf16, ldx, codes, scales, scale_kind, nullptr, false, 1, M, N, K, y,
                     out_dtype, hip_stream);
}

fp8_status fp8_w4_grouped_matvec(const void *x_bf16, int64_t ldx, const void *codes,
                                 const void *scales, int scale_kind,
                                 const int32_t *group_offsets, int64_t E, int64_t R, int64_t N,
                                 int64_t K, void *y, int out_dtype, void *hip_stream) {
    return w4_matvec(x_bf16, ldx, codes, scales, scale_kind, group_offsets, true, E, R, N, K, y,
                     out_dtype, hip_stream);
}

}  // extern "C"

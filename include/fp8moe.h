/*
 * fp8moe — the operators around the expert products of a mixture-of-experts
 * block, for MI355X (gfx950).  C ABI, in the same library as fp8blk.h
 * (libfp8blk.so) and under its conventions: device pointers owned by the
 * caller, nothing allocated, freed or synchronized, work enqueued on
 * `hip_stream`, arguments validated before anything is enqueued, no C++
 * exception across the boundary, calls reentrant and thread-safe.
 *
 * Conventions of this header:
 *   - Type codes are fp8_out_dtype's: FP8_OUT_F32 (0) and FP8_OUT_BF16 (1).
 *   - An input matrix [rows][cols] has unit stride along cols and a row stride
 *     `ld...` in elements (0 repeats one row); outputs, integer inputs, codes
 *     and scales are dense.  Pointers need the alignment of one element (or
 *     what the call states); wider accesses are the kernels' own matter.
 *   - Outputs and workspaces must not overlap inputs or each other, but where
 *     a call says so: inputs are still read when outputs are begun.
 *   - NaN and infinities propagate as the formulas have it (fp8blk.h leaves
 *     them out of its contract; here they are in it); in a dropped slot
 *     nothing is read at all, so whatever stands there has no effect.  A 1x128
 *     group that holds one is quantized so that it reads back as NaN: its
 *     scale is the largest magnitude (NaN, else infinity), with power-of-two
 *     scales too, and its codes are NaN.
 *   - Sums, norms and products are FP32 (the squares of a norm too: values
 *     from about 1e19 on are past their range); an output is rounded once, to
 *     nearest even.  Results do not depend on the run: no sum uses
 *     floating-point atomics.
 *   - Sizes of zero are valid; nothing is written but what a sum over nothing
 *     gives (zeros), where the call says so.
 *   - Limits (FP8_ERR_SHAPE): any one size below 2^31, a matrix below 2^40
 *     elements, and those a call states.
 */
#ifndef FP8MOE_H_
#define FP8MOE_H_

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- tokens sorted by expert and back ---------------------------------- */
/* H < 2^28 in all of them. */

/*
 * Stable counting sort of the slots (t, j) of a routing by expert: what the
 * grouped GEMM's rows are.  Slot s = t top_k + j.
 *   expert_ids    [T][top_k] int32 (id_bytes 4) or int64 (id_bytes 8); an id
 *                 outside [0, E) drops its slot (another rank's expert, a
 *                 padded token)
 *   group_offsets [E+1] int32: rows [off[e], off[e+1]) are expert e's, in
 *                 slot order; off[E] is the number of kept slots
 *   slot_row      [T][top_k] int32: the slot's row, -1 for a dropped slot
 *   row_slot      [T top_k] int32: the row's slot; -1 from row off[E] on
 *   workspace     fp8_moe_sort_workspace_bytes() bytes, 16-byte aligned
 *                 (NULL where that is 0); contents need no initialization
 * 1 <= E <= 1024, T top_k < 2^31.  T = 0 writes group_offsets (zeros) only.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_DTYPE (id_bytes),
 * FP8_ERR_ALIGN, FP8_ERR_WORKSPACE (too small), FP8_ERR_HIP.
 */
fp8_status fp8_moe_sort(const void *expert_ids, int id_bytes, int64_t T, int64_t top_k,
                        int64_t E, int32_t *group_offsets, int32_t *slot_row,
                        int32_t *row_slot, void *workspace, size_t workspace_bytes,
                        void *hip_stream);
size_t fp8_moe_sort_workspace_bytes(int64_t T, int64_t top_k, int64_t E);

/*
 * Rows gathered into expert order: xs[slot_row[t][j]] = x[t].
 *   x         [T][H] of elem_bytes 1, 2 or 4 (copied bit for bit)
 *   x_scales  [T][G] fp32 or NULL: scales that travel with quantized rows
 *   xs        [R][H], xs_scales [R][G] (NULL with x_scales)
 * Rows that no slot names are left untouched; a slot_row entry outside [0, R)
 * is a dropped slot.
 */
fp8_status fp8_moe_dispatch(const void *x, int elem_bytes, int64_t ldx, const float *x_scales,
                            int64_t ldx_scales, int64_t T, int64_t H, int64_t G,
                            const int32_t *slot_row, int64_t top_k, void *xs, float *xs_scales,
                            int64_t R, void *hip_stream);

/*
 * The same with the 1x128 quantizer in the gather: q[row], scales[row] are
 * the E4M3 bytes and scales fp8_quant_act_1x128 (or its _pow2 form) gives for
 * a finite x[t]; each token is read and quantized once.
 *   x_bf16 [T][H] bf16; q [R][H]; scales [R][ceil(H/128)]
 */
fp8_status fp8_moe_dispatch_quant_1x128(const void *x_bf16, int64_t ldx, int64_t T, int64_t H,
                                        const int32_t *slot_row, int64_t top_k, void *q,
                                        float *scales, int64_t R, void *hip_stream);
fp8_status fp8_moe_dispatch_quant_1x128_pow2(const void *x_bf16, int64_t ldx, int64_t T,
                                             int64_t H, const int32_t *slot_row, int64_t top_k,
                                             void *q, float *scales, int64_t R,
                                             void *hip_stream);

/*
 * fp8_moe_sort and the gather in one call (for few slots, in one launch).
 * Arguments as for the two calls; xs, q and scales have R = T top_k rows.
 */
fp8_status fp8_moe_sort_dispatch(const void *x, int elem_bytes, int64_t ldx, int64_t T,
                                 int64_t H, const void *expert_ids, int id_bytes,
                                 int64_t top_k, int64_t E, int32_t *group_offsets,
                                 int32_t *slot_row, int32_t *row_slot, void *xs,
                                 void *workspace, size_t workspace_bytes, void *hip_stream);
fp8_status fp8_moe_sort_dispatch_quant_1x128(const void *x_bf16, int64_t ldx, int64_t T,
                                             int64_t H, const void *expert_ids, int id_bytes,
                                             int64_t top_k, int64_t E, int32_t *group_offsets,
                                             int32_t *slot_row, int32_t *row_slot, void *q,
                                             float *scales, void *workspace,
                                             size_t workspace_bytes, void *hip_stream);
fp8_status fp8_moe_sort_dispatch_quant_1x128_pow2(
    const void *x_bf16, int64_t ldx, int64_t T, int64_t H, const void *expert_ids, int id_bytes,
    int64_t top_k, int64_t E, int32_t *group_offsets, int32_t *slot_row, int32_t *row_slot,
    void *q, float *scales, void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * Gradient of the gather: dx[t] = sum_j dxs[slot_row[t][j]] (fp32, j
 * ascending; zero for a token with every slot dropped).
 *   dxs [R][H] of in_dtype; dx [T][H] of out_dtype
 */
fp8_status fp8_moe_dispatch_grad(const void *dxs, int in_dtype, int64_t ld_dxs, int64_t R,
                                 const int32_t *slot_row, int64_t T, int64_t top_k, int64_t H,
                                 void *dx, int out_dtype, void *hip_stream);

/*
 * The experts' outputs weighted and summed back per token:
 *   out[t] = residual[t] + sum_j weights[t][j] ys[slot_row[t][j]]
 * (fp32, j ascending; dropped slots are not read).
 *   ys       [R][H] of in_dtype
 *   weights  [T][top_k] fp32, or NULL for ones
 *   residual [T][H] of out_dtype, or NULL; may be `out` itself
 *   out      [T][H] of out_dtype
 */
fp8_status fp8_moe_combine(const void *ys, int in_dtype, int64_t ld_ys, int64_t R,
                           const int32_t *slot_row, const float *weights, int64_t T,
                           int64_t top_k, int64_t H, const void *residual, int64_t ld_residual,
                           void *out, int out_dtype, void *hip_stream);

/*
 * Gradient of the weighted sum:
 *   dys[slot_row[t][j]] = weights[t][j] dout[t]
 *   dweights[t][j]      = sum_h dout[t][h] ys[slot_row[t][j]][h]  (0 if dropped)
 *   dout [T][H], ys [R][H] and dys [R][H] of dtype; dweights [T][top_k] fp32
 * dys or dweights may be NULL (not computed); without dweights ys is not read
 * and may be NULL.
 * weights NULL means ones.  Rows of dys that no slot names are left
 * untouched.  (The residual's gradient is dout itself.)
 */
fp8_status fp8_moe_combine_grad(const void *dout, int64_t ld_dout, const void *ys,
                                int64_t ld_ys, int dtype, int64_t R, const int32_t *slot_row,
                                const float *weights, int64_t T, int64_t top_k, int64_t H,
                                void *dys, float *dweights, void *hip_stream);

/* ---- norms before and after a block, with gate and residual scale ------- */

/*
 * Of a block's output y and the residual stream r, per token t over H:
 *   u  = y rstd_post w_post,  rstd_post = 1 / sqrt(mean(y^2) + eps)
 *        (u = y where post_norm is 0)
 *   r' = residual_scale r + branch_scale gate u
 *   n  = r' rstd_pre w_pre,   rstd_pre = 1 / sqrt(mean(r'^2) + eps)
 * n is computed from r' before r' is rounded to its type.
 *   y [T][H] of y_dtype; r [T][H] of r_dtype; (bf16, bf16), (bf16, f32) and
 *   (f32, f32) are supported
 *   w_post, w_pre [H] and gate [gate_rows][H] of param_dtype, each NULL for
 *   ones; token t takes gate row t / (T / gate_rows), so gate_rows divides T
 *   (1: one gate for all, T: one per token); it is ignored without a gate
 *   r_out [T][H] of r_dtype (may be r itself, where ldr = H)
 *   n [T][H] of y_dtype, or NULL (then rstd_pre is not written either)
 *   rstd_post, rstd_pre [T] fp32, or NULL: what the gradient needs
 * 1 <= H <= 32768 (FP8_ERR_SHAPE); 0 columns are a no-op.
 * The _quant_1x128 forms also write n quantized, q [T][H] E4M3 and scales
 * [T][ceil(H/128)], from the unrounded fp32 n, by the rules of
 * fp8_quant_act_1x128 (or its _pow2 form).
 */
fp8_status fp8_norm_residual(const void *y, int y_dtype, int64_t ldy, const void *r, int r_dtype,
                             int64_t ldr, const void *w_post, const void *gate,
                             const void *w_pre, int param_dtype, int64_t T, int64_t H,
                             int64_t gate_rows, int post_norm, float residual_scale,
                             float branch_scale, float eps, void *r_out, void *n,
                             float *rstd_post, float *rstd_pre, void *hip_stream);
fp8_status fp8_norm_residual_quant_1x128(const void *y, int y_dtype, int64_t ldy, const void *r,
                                         int r_dtype, int64_t ldr, const void *w_post,
                                         const void *gate, const void *w_pre, int param_dtype,
                                         int64_t T, int64_t H, int64_t gate_rows, int post_norm,
                                         float residual_scale, float branch_scale, float eps,
                                         void *r_out, void *n, void *q, float *scales,
                                         float *rstd_post, float *rstd_pre, void *hip_stream);
fp8_status fp8_norm_residual_quant_1x128_pow2(
    const void *y, int y_dtype, int64_t ldy, const void *r, int r_dtype, int64_t ldr,
    const void *w_post, const void *gate, const void *w_pre, int param_dtype, int64_t T,
    int64_t H, int64_t gate_rows, int post_norm, float residual_scale, float branch_scale,
    float eps, void *r_out, void *n, void *q, float *scales, float *rstd_post, float *rstd_pre,
    void *hip_stream);

/*
 * Its gradient, from dn (of n) and dr_out (of r'); either may be NULL (zero).
 *   dr      = residual_scale D, D the whole gradient of r'
 *   dy      the gradient of y
 *   dw_post [H], dw_pre [H], dgate [gate_rows][H] fp32, each may be NULL (not
 *           computed); dw_post needs post_norm, dgate a gate
 * dn, y and dy have y_dtype; dr_out, r_out and dr have r_dtype.  y, r_out,
 * rstd_post and rstd_pre are the forward's (rstd_post is not read where
 * post_norm is 0; r_out and rstd_pre are not read where dn is NULL).
 *   workspace  fp8_norm_residual_grad_workspace_bytes() bytes (asked for with
 *              gate_rows 1 where there is no gate), 16-byte aligned (NULL
 *              where that is 0)
 * With T = 0 the fp32 gradients are zeros.
 */
fp8_status fp8_norm_residual_grad(const void *dn, int64_t ld_dn, const void *dr_out,
                                  int64_t ld_dr_out, const void *y, int y_dtype, int64_t ldy,
                                  const void *r_out, int r_dtype, int64_t ld_r_out,
                                  const float *rstd_post, const float *rstd_pre,
                                  const void *w_post, const void *gate, const void *w_pre,
                                  int param_dtype, int64_t T, int64_t H, int64_t gate_rows,
                                  int post_norm, float residual_scale, float branch_scale,
                                  void *dy, void *dr, float *dw_post, float *dgate,
                                  float *dw_pre, void *workspace, size_t workspace_bytes,
                                  void *hip_stream);
size_t fp8_norm_residual_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows);

/* ---- products of a few rows with 4-bit weights --------------------------- */

/* How the groups of a 4-bit matrix are scaled. */
typedef enum {
    FP8_W4_F32_1X128 = 0, /* fp32, one per 128 channels of a row */
    FP8_W4_E8M0_1X32 = 1  /* E8M0 byte b = 2^(b - 127), one per 32 channels */
} fp8_w4_scale_kind;

/*
 * 4-bit weights: OCP E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign bit),
 * two a byte along K, the even channel in the low nibble.
 *   w_bf16 [N][K] bf16
 *   codes  [N][ceil(K/2)] bytes (an unpaired last high nibble is 0)
 *   scales FP8_W4_F32_1X128: fp32 [N][ceil(K/128)], fl32(amax / 6);
 *          FP8_W4_E8M0_1X32: bytes [N][ceil(K/32)], the smallest power of two
 *          from 2^-127 on that is at least amax / 6
 * code = E2M1 round to nearest even of fl32(w / s); an all-zero group has
 * scale 0 (fp32) or 2^-127 and codes 0.  A group that holds a NaN or an
 * infinity has scale NaN or infinity (fp32), or the NaN byte 255: products
 * with its row are NaN.  Weights of 1.75 * 2^127 and more (near the end of
 * bf16's range) round up to 2^128 with E8M0 scales, and that is infinite.
 */
fp8_status fp8_w4_quant_1x128(const void *w_bf16, int64_t N, int64_t K, void *codes,
                              float *scales, void *hip_stream);
fp8_status fp8_w4_quant_1x32(const void *w_bf16, int64_t N, int64_t K, void *codes,
                             void *scales_e8m0, void *hip_stream);

/*
 * y[m][n] = sum_k x[m][k] w[n][k], w as above.  Made for M of one to 16 rows
 * (decoding); any M is right, 16 rows at a pass over the weights.
 *   x_bf16 [M][K] bf16, used as it is (products are exact in fp32)
 *   y      [M][N] of out_dtype
 * K < 2^24 (FP8_ERR_SHAPE); K = 0 gives zeros.  A weight of 2^128 or more (E8M0
 * bytes 253 and 254 have some) is infinite and E8M0 byte 255 is NaN; a scale
 * that is not finite shows in its row's output alone.
 */
fp8_status fp8_w4_matvec(const void *x_bf16, int64_t ldx, const void *codes, const void *scales,
                         int scale_kind, int64_t M, int64_t N, int64_t K, void *y,
                         int out_dtype, void *hip_stream);

/*
 * The same per expert: row r of expert e (rows [off[e], off[e+1]) of
 * group_offsets [E+1], clamped as by fp8_block_grouped_gemm) times w[e].
 *   x_bf16 [R][K]; codes [E][N][ceil(K/2)]; scales [E][N][...]
 *   y [R][N]; rows outside every expert's range are left untouched
 * 1 <= E <= 65535 while R > 0.
 */
fp8_status fp8_w4_grouped_matvec(const void *x_bf16, int64_t ldx, const void *codes,
                                 const void *scales, int scale_kind,
                                 const int32_t *group_offsets, int64_t E, int64_t R, int64_t N,
                                 int64_t K, void *y, int out_dtype, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOE_H_ */

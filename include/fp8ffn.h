/*
 * fp8ffn — the operators inside a gated feed-forward block, dense or per
 * expert, for MI355X (gfx950).  C ABI, in the same library as fp8blk.h
 * (libfp8blk.so) and under its conventions: device pointers owned by the
 * caller, nothing allocated, freed or synchronized, work enqueued on
 * `hip_stream`, arguments validated before anything is enqueued, no C++
 * exception across the boundary, calls reentrant and thread-safe.
 *
 * The block, W_up = [Wg; Wu] [2 I][K] (the gate's rows first):
 *   [g | u] = x W_up^T,  a = act(g) u,  y = a W_down^T
 * with act(g) = g sigmoid(z), z = g (FP8_ACT_SILU) or z = 2 sqrt(2 / pi) (g +
 * 0.044715 g^3) (FP8_ACT_GELU_TANH: GELU in its tanh form).  A training step:
 *   forward   fp8_quant_act_1x128 (x, kept), fp8_block_gemm_gated_quant_1x128
 *             (a for the down projection, [g | u] kept in 8 bits),
 *             fp8_block_gemm
 *   backward  fp8_block_gemm_dgrad (da), fp8_gated_grad_quant (d[g | u] for
 *             both products that follow, a for the down weights),
 *             fp8_block_gemm_dgrad (dx), fp8_requant_act_128x1_t (the kept x),
 *             fp8_block_gemm_wgrad (twice)
 *
 * Conventions of this header:
 *   - E4M3 data, scales and the quantization rules are fp8blk.h's (the _pow2
 *     forms take and write power-of-two scales); type codes are
 *     fp8_out_dtype's.
 *   - Tensors are dense and row-major where no row stride (`ld...`, in
 *     elements) is given.
 *   - Outputs and workspaces must not overlap inputs or each other.
 *   - Activations and scales are FP32; an output is rounded to its type once,
 *     to nearest even.  The sigmoid s is off by at most 6e-7 + 9e-8 |z| (1 - s) of
 *     itself (GELU 6e-7 + 4.5e-7 |z| (1 - s)), and below 2^-126 it may be 0.
 *   - Products sum as in fp8_block_gemm or, for few rows or tiles, in FP32
 *     throughout: which depends on the sizes and on the workspace, never on the
 *     run, and results do not depend on the run.  fp8_block_gemm's matrix
 *     instruction drops what is below 2^-13 of the largest of eight products, so
 *     a row of a large call is less exact than in a small one, and codes of a
 *     quantized result flip: with channels 100 times the others 4096 rows were
 *     off by 0.0026 of their norm, with FP32 sums by 0.0017.
 *   - A workspace is one call's until that call has ended on its stream: calls
 *     (or replays of captured ones) that may run at the same time take one
 *     each.
 *   - NaN and infinities: products take finite operands (as fp8_block_gemm);
 *     elsewhere they propagate as the formulas have it, and a group that holds
 *     one is quantized so that it reads back as NaN (its scale is the largest
 *     magnitude, its codes are NaN).
 *   - No rows or no columns of a result is a valid no-op.
 *   - Limits (FP8_ERR_SHAPE): any one size below 2^31, a matrix below 2^40
 *     elements, and those a call states.
 */
#ifndef FP8FFN_H_
#define FP8FFN_H_

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP8_ACT_SILU = 0, FP8_ACT_GELU_TANH = 1 } fp8_activation;

/* ---- gated products -------------------------------------------------------- */

/*
 * Both projections, the activation and the product in one call:
 *   a_e4m3 [M][K] E4M3 with a_scales [M][K/128]; w_e4m3 [2 I][K] with w_scales
 *   [2 I / 128][K/128] (fp8_quant_weight_128x128 of W_up)
 *   out    [M][I] of out_dtype: a
 * K % 128 == 0, I % 128 == 0 and K < 2^24 (FP8_ERR_SHAPE), as fp8_block_gemm;
 * K = 0 is refused where there is something to compute.  a_e4m3, w_e4m3 and
 * out 16-byte aligned (FP8_ERR_ALIGN).
 *   activation  fp8_activation (FP8_ERR_DTYPE otherwise)
 *   workspace   optional (256-byte aligned): with
 *               fp8_gated_gemm_workspace_bytes() bytes the call takes the
 *               faster plan for few rows; with less (or NULL and 0) it runs
 *               without.
 */
fp8_status fp8_block_gemm_gated(const void *a_e4m3, const float *a_scales, const void *w_e4m3,
                                const float *w_scales, int activation, int64_t M, int64_t I,
                                int64_t K, void *out, int out_dtype, void *workspace,
                                size_t workspace_bytes, void *hip_stream);
fp8_status fp8_block_gemm_gated_pow2(const void *a_e4m3, const float *a_scales,
                                     const void *w_e4m3, const float *w_scales, int activation,
                                     int64_t M, int64_t I, int64_t K, void *out, int out_dtype,
                                     void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * The same with the result quantized 1x128 from its FP32 values:
 *   q [M][I] E4M3, scales [M][I/128]: a
 *   h [M][2 I] E4M3, h_scales [M][2 I / 128]: [g | u], the checkpoint that
 *   fp8_gated_grad... take; both NULL: not kept
 * q and h 16-byte aligned.
 */
fp8_status fp8_block_gemm_gated_quant_1x128(const void *a_e4m3, const float *a_scales,
                                            const void *w_e4m3, const float *w_scales,
                                            int activation, int64_t M, int64_t I, int64_t K,
                                            void *q, float *scales, void *h, float *h_scales,
                                            void *workspace, size_t workspace_bytes,
                                            void *hip_stream);
fp8_status fp8_block_gemm_gated_quant_1x128_pow2(const void *a_e4m3, const float *a_scales,
                                                 const void *w_e4m3, const float *w_scales,
                                                 int activation, int64_t M, int64_t I, int64_t K,
                                                 void *q, float *scales, void *h,
                                                 float *h_scales, void *workspace,
                                                 size_t workspace_bytes, void *hip_stream);
size_t fp8_gated_gemm_workspace_bytes(int64_t M, int64_t I, int64_t K);

/*
 * The same per expert, over expert-sorted rows (fp8_block_grouped_gemm's
 * a_e4m3 [T][K] and group_offsets [E+1], clamped as there): w_e4m3 [E][2 I][K],
 * w_scales [E][2 I / 128][K/128]; outputs have T rows, and rows outside every
 * expert's range are left untouched.  E = 0 is refused while T > 0.
 *   workspace   optional, as above, fp8_grouped_gated_gemm_workspace_bytes()
 */
fp8_status fp8_block_grouped_gemm_gated(const void *a_e4m3, const float *a_scales,
                                        const void *w_e4m3, const float *w_scales,
                                        const int32_t *group_offsets, int64_t E, int activation,
                                        int64_t T, int64_t I, int64_t K, void *out,
                                        int out_dtype, void *workspace,
                                        size_t workspace_bytes, void *hip_stream);
fp8_status fp8_block_grouped_gemm_gated_pow2(const void *a_e4m3, const float *a_scales,
                                             const void *w_e4m3, const float *w_scales,
                                             const int32_t *group_offsets, int64_t E,
                                             int activation, int64_t T, int64_t I, int64_t K,
                                             void *out, int out_dtype, void *workspace,
                                             size_t workspace_bytes, void *hip_stream);
fp8_status fp8_block_grouped_gemm_gated_quant_1x128(
    const void *a_e4m3, const float *a_scales, const void *w_e4m3, const float *w_scales,
    const int32_t *group_offsets, int64_t E, int activation, int64_t T, int64_t I, int64_t K,
    void *q, float *scales, void *h, float *h_scales, void *workspace, size_t workspace_bytes,
    void *hip_stream);
fp8_status fp8_block_grouped_gemm_gated_quant_1x128_pow2(
    const void *a_e4m3, const float *a_scales, const void *w_e4m3, const float *w_scales,
    const int32_t *group_offsets, int64_t E, int activation, int64_t T, int64_t I, int64_t K,
    void *q, float *scales, void *h, float *h_scales, void *workspace, size_t workspace_bytes,
    void *hip_stream);
size_t fp8_grouped_gated_gemm_workspace_bytes(int64_t T, int64_t E, int64_t I, int64_t K);

/* ---- gradient of the activation and the product ------------------------------ */

/*
 * dg = da u act'(g), du = da act(g), with act' = s + g z'(g) s (1 - s), s =
 * sigmoid(z):
 *   da [M][I] of da_dtype, rows ld_da elements apart
 *   h  [M][2 I], [g | u], rows ld_h elements apart: E4M3 with h_scales
 *      [M][2 I / 128] (I % 128 == 0, FP8_ERR_SHAPE), or, where h_scales is
 *      NULL, bf16 (as a plain product wrote it)
 *   dh [M][2 I] of dh_dtype: [dg | du]
 * I % 128 == 0 and M I / 128 <= 2^28 - 16 in all forms (FP8_ERR_SHAPE).
 * Pointers need the alignment of one element (q below 8 bytes).
 */
fp8_status fp8_gated_grad(const void *da, int da_dtype, int64_t ld_da, const void *h,
                          int64_t ld_h, const float *h_scales, int activation, int64_t M,
                          int64_t I, void *dh, int dh_dtype, void *hip_stream);

/*
 * The same with dh quantized from its FP32 values, each pair optional (both
 * NULL), at least one given (FP8_ERR_NULL):
 *   q [M][2 I], scales [M][2 I / 128]: 1x128, for the input gradient
 *   q_t [2 I][M], scales_t [2 I][ceil(M/128)]: 128x1 and transposed, for the
 *      weight gradient of W_up (as fp8_quant_act_128x1_t writes them)
 *   a_t [I][M], a_scales_t [I][ceil(M/128)]: a = act(g) u in the same form,
 *      for the weight gradient of W_down
 * All M rows count.  Rows of h and da that a grouped product left untouched
 * reach nothing but themselves in q; in q_t and a_t they share a group with
 * other rows, so they must hold zeros.
 */
fp8_status fp8_gated_grad_quant(const void *da, int da_dtype, int64_t ld_da, const void *h,
                                int64_t ld_h, const float *h_scales, int activation, int64_t M,
                                int64_t I, void *q, float *scales, void *q_t, float *scales_t,
                                void *a_t, float *a_scales_t, void *hip_stream);
fp8_status fp8_gated_grad_quant_pow2(const void *da, int da_dtype, int64_t ld_da, const void *h,
                                     int64_t ld_h, const float *h_scales, int activation,
                                     int64_t M, int64_t I, void *q, float *scales, void *q_t,
                                     float *scales_t, void *a_t, float *a_scales_t,
                                     void *hip_stream);

/* ---- 8-bit checkpoints --------------------------------------------------------- */

/*
 * 1x128 data read back: x[m][k] = code(q[m][k]) scales[m][k / 128], an FP32
 * product (rounded to bf16 where out_dtype says so).  q [M][K], scales
 * [M][ceil(K/128)], x [M][K]; any alignment, and any M, K with M ceil(K/8)
 * below 2^32 - 256 and ceil(M/128) ceil(K/128) below 2^23 (FP8_ERR_SHAPE; a
 * row is so below 2^30 values).
 */
fp8_status fp8_dequant_act_1x128(const void *q, const float *scales, int64_t M, int64_t K,
                                 void *x, int out_dtype, void *hip_stream);

/*
 * 1x128 data turned for a weight gradient: what fp8_quant_act_128x1_t (or its
 * _pow2 form) gives for the fp32 values that q and scales stand for.
 *   q [M][K], scales [M][ceil(K/128)]; q_t [K][M], scales_t [K][ceil(M/128)]
 * Any alignment, and M, K as fp8_dequant_act_1x128.
 */
fp8_status fp8_requant_act_128x1_t(const void *q, const float *scales, int64_t M, int64_t K,
                                   void *q_t, float *scales_t, void *hip_stream);
fp8_status fp8_requant_act_128x1_t_pow2(const void *q, const float *scales, int64_t M, int64_t K,
                                        void *q_t, float *scales_t, void *hip_stream);

/* ---- input gradient per expert --------------------------------------------------- */

/*
 * fp8_block_gemm_dgrad per expert: dx[r] = dy[r] W[e] for the rows r of expert
 * e (group_offsets [E+1], clamped as by fp8_block_grouped_gemm), the weights
 * read transposed from their forward layout.
 *   dy_e4m3 [T][N] with dy_scales [T][N/128]; w_e4m3 [E][N][K] with w_scales
 *   [E][N/128][K/128]; dx [T][K] of out_dtype, rows outside every expert's
 *   range left untouched
 * Requirements and errors as fp8_block_gemm_dgrad (N K < 2^32) and, for the
 * experts, fp8_block_grouped_gemm.  No host synchronization: the offsets stay
 * on the device.
 */
fp8_status fp8_block_grouped_gemm_dgrad(const void *dy_e4m3, const float *dy_scales,
                                        const void *w_e4m3, const float *w_scales,
                                        const int32_t *group_offsets, int64_t E, int64_t T,
                                        void *dx, int out_dtype, int64_t N, int64_t K,
                                        void *hip_stream);
fp8_status fp8_block_grouped_gemm_dgrad_pow2(const void *dy_e4m3, const float *dy_scales,
                                             const void *w_e4m3, const float *w_scales,
                                             const int32_t *group_offsets, int64_t E, int64_t T,
                                             void *dx, int out_dtype, int64_t N, int64_t K,
                                             void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8FFN_H_ */

// C ABI of the operators inside a gated feed-forward block
// (include/fp8ffn.h): argument validation, then dispatch to the launchers.
// Every check runs before anything is enqueued; on error nothing is written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8ffn.h"
#include "launch_ffn.hpp"

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
// A launch may not exceed 2^32 work-items: products have at most 512 threads
// to a tile of 128 x 128 outputs, so 2^22 tiles stay below it.
constexpr int64_t kMaxTiles = (int64_t)1 << 22;
constexpr int64_t kMaxWorkItems = (int64_t)1 << 32;
// inner dimension of a product: a tile's 256 operand rows have 32-bit offsets
constexpr int64_t kMaxInner = (int64_t)1 << 24;
constexpr int64_t kMaxExperts = (int64_t)1 << 20;

inline bool dim_ok(int64_t n) { return n >= 0 && n < kMaxDim; }
inline bool matrix_ok(int64_t rows, int64_t cols) {
    return dim_ok(rows) && dim_ok(cols) && rows * cols < kMaxElems;
}
inline bool stride_ok(int64_t rows, int64_t ld) {
    return ld >= 0 && ld < kMaxElems && (rows <= 1 || ld < kMaxElems / rows);
}
inline bool type_ok(int t) { return t == FP8_OUT_F32 || t == FP8_OUT_BF16; }
inline uintptr_t bytes_of(int t) { return t == FP8_OUT_BF16 ? 2 : 4; }
inline bool activation_ok(int a) { return a == FP8_ACT_SILU || a == FP8_ACT_GELU_TANH; }

// Sizes of a product with `rows` rows over E experts (1 for dense), `cols`
// columns and K inner values.
fp8_status check_product(int64_t rows, int64_t cols, int64_t K, int64_t E) {
    if (!matrix_ok(rows, K) || !matrix_ok(rows, cols) || !dim_ok(cols) || K >= kMaxInner)
        return FP8_ERR_SHAPE;
    if (cols % 128 != 0 || K % 128 != 0) return FP8_ERR_SHAPE;
    if (E < 0 || E >= kMaxExperts) return FP8_ERR_SHAPE;
    if (E > 0 && cols * K >= kMaxElems * 64 / E) return FP8_ERR_SHAPE;
    if (((rows + 127) / 128 + (E > 1 ? E : 1)) * (cols / 128) >= kMaxTiles) return FP8_ERR_SHAPE;
    return FP8_OK;
}

fp8_status check_operands(const void *a, const float *sa, const void *w, const float *sw) {
    if (!a || !sa || !w || !sw) return FP8_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(sa, 4) || !aligned(sw, 4))
        return FP8_ERR_ALIGN;
    return FP8_OK;
}

struct Experts {
    bool grouped;
    const int32_t *offsets;
    int64_t E;
};
constexpr Experts kDense = {false, nullptr, 1};

fp8_status gated(const void *a, const float *sa, const void *w, const float *sw,
                 const Experts &experts, int activation, int64_t M, int64_t I, int64_t K,
                 void *out, int out_dtype, void *q, float *scales, void *h, float *h_scales,
                 bool quant, void *ws, size_t ws_bytes, bool pow2, void *stream) {
    if (!activation_ok(activation) || !type_ok(out_dtype)) return FP8_ERR_DTYPE;
    if (I < 0 || I >= kMaxDim / 2 || I % 128 != 0) return FP8_ERR_SHAPE;
    fp8_status st = check_product(M, 2 * I, K, experts.E);
    if (st != FP8_OK) return st;
    if ((ws == nullptr) != (ws_bytes == 0) || !aligned(ws, 256)) return FP8_ERR_WORKSPACE;
    if (M == 0 || I == 0) return FP8_OK;
    if (K == 0 || experts.E == 0) return FP8_ERR_SHAPE;
    st = check_operands(a, sa, w, sw);
    if (st != FP8_OK) return st;
    if (experts.grouped && !experts.offsets) return FP8_ERR_NULL;
    if (quant ? !q || !scales || (h != nullptr) != (h_scales != nullptr) : !out)
        return FP8_ERR_NULL;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(h, 16) || !aligned(scales, 4) ||
        !aligned(h_scales, 4) || !aligned(experts.offsets, 4))
        return FP8_ERR_ALIGN;
    GatedGemm p = {};
    p.a = a; p.sa = sa; p.w = w; p.sw = sw;
    p.offsets = experts.offsets;
    p.E = experts.grouped ? experts.E : 0;
    p.M = M; p.K = K;
    p.to.out = out;
    p.to.q = static_cast<uint8_t *>(q);
    p.to.q_scales = scales;
    p.to.h = static_cast<uint8_t *>(h);
    p.to.h_scales = h_scales;
    p.to.I = I;
    p.to.bf16_out = out_dtype == FP8_OUT_BF16;
    p.to.gelu = activation == FP8_ACT_GELU_TANH;
    p.to.pow2 = pow2;
    p.workspace = ws;
    p.workspace_bytes = ws_bytes;
    clear_last_error();
    return from_hip(launch_gated_gemm(p, as_stream(stream)));
}

fp8_status gated_grad(const void *da, int da_dtype, int64_t ld_da, const void *h, int64_t ld_h,
                      const float *h_scales, int activation, int64_t M, int64_t I, void *dh,
                      int dh_dtype, bool quant, void *q, float *scales, void *q_t,
                      float *scales_t, void *a_t, float *a_scales_t, bool pow2, void *stream) {
    if (!activation_ok(activation) || !type_ok(da_dtype) || !type_ok(dh_dtype))
        return FP8_ERR_DTYPE;
    if (I < 0 || I >= kMaxDim / 2 || I % 128 != 0 || !matrix_ok(M, 2 * I)) return FP8_ERR_SHAPE;
    if (!stride_ok(M, ld_da) || !stride_ok(M, ld_h)) return FP8_ERR_SHAPE;
    // 16 threads to a row's 128 columns in workgroups of 256, or 512 to a tile of
    // 128 rows and columns
    if (M * (I / 128) > kMaxWorkItems / 16 - 16 ||
        (M + 127) / 128 * (I / 128) >= kMaxWorkItems / 512)
        return FP8_ERR_SHAPE;
    if (quant && ((q != nullptr) != (scales != nullptr) ||
                  (q_t != nullptr) != (scales_t != nullptr) ||
                  (a_t != nullptr) != (a_scales_t != nullptr)))
        return FP8_ERR_NULL;
    if (M == 0 || I == 0) return FP8_OK;
    if (!da || !h || (quant ? !q && !q_t && !a_t : !dh)) return FP8_ERR_NULL;
    if (!aligned(da, bytes_of(da_dtype)) || !aligned(h, h_scales ? 1 : 2) ||
        !aligned(h_scales, 4) || !aligned(dh, bytes_of(dh_dtype)) || !aligned(scales, 4) ||
        !aligned(scales_t, 4) || !aligned(a_scales_t, 4) || !aligned(q, 8))
        return FP8_ERR_ALIGN;
    GatedGrad p = {};
    p.da = da; p.ld_da = ld_da;
    p.h = h; p.ld_h = ld_h; p.h_scales = h_scales;
    p.M = M; p.I = I;
    p.da_bf16 = da_dtype == FP8_OUT_BF16;
    p.gelu = activation == FP8_ACT_GELU_TANH;
    p.pow2 = pow2;
    p.dh = dh;
    p.dh_bf16 = dh_dtype == FP8_OUT_BF16;
    p.q = static_cast<uint8_t *>(q);
    p.scales = scales;
    p.q_t = static_cast<uint8_t *>(q_t);
    p.scales_t = scales_t;
    p.a_t = static_cast<uint8_t *>(a_t);
    p.a_scales_t = a_scales_t;
    clear_last_error();
    return from_hip(launch_gated_grad(p, as_stream(stream)));
}

fp8_status check_stored(const void *q, const float *scales, int64_t M, int64_t K) {
    if (!matrix_ok(M, K)) return FP8_ERR_SHAPE;
    // one thread to 8 values, or 512 to a tile of 128 rows and columns (which also
    // keeps a row below 2^30 values: a span's byte offset in it has 32 bits)
    if (M * ((K + 7) / 8) >= kMaxWorkItems - 256 ||
        ((M + 127) / 128) * ((K + 127) / 128) >= kMaxWorkItems / 512)
        return FP8_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8_OK;
    if (!q || !scales) return FP8_ERR_NULL;
    return aligned(scales, 4) ? FP8_OK : FP8_ERR_ALIGN;
}

fp8_status requant_t(const void *q, const float *scales, int64_t M, int64_t K, void *q_t,
                     float *scales_t, bool pow2, void *stream) {
    const fp8_status st = check_stored(q, scales, M, K);
    if (st != FP8_OK || M == 0 || K == 0) return st;
    if (!q_t || !scales_t) return FP8_ERR_NULL;
    if (!aligned(scales_t, 4)) return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(
        launch_requant_act_t(q, scales, M, K, q_t, scales_t, pow2, as_stream(stream)));
}

fp8_status grouped_dgrad(const void *dy, const float *sdy, const void *w, const float *sw,
                         const int32_t *offsets, int64_t E, int64_t T, void *dx, int out_dtype,
                         int64_t N, int64_t K, bool pow2, void *stream) {
    if (!type_ok(out_dtype)) return FP8_ERR_DTYPE;
    fp8_status st = check_product(T, K, N, E);  // output T x K, inner dimension N
    if (st != FP8_OK) return st;
    // an expert's W is addressed through one buffer resource with 32-bit offsets
    if (N * K >= ((int64_t)1 << 32)) return FP8_ERR_SHAPE;
    if (T == 0 || K == 0) return FP8_OK;
    if (N == 0 || E == 0) return FP8_ERR_SHAPE;
    st = check_operands(dy, sdy, w, sw);
    if (st != FP8_OK) return st;
    if (!offsets || !dx) return FP8_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(dx, 16)) return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_grouped_gemm_dgrad(dy, sdy, w, sw, offsets, E, T, dx,
                                              out_dtype == FP8_OUT_BF16, N, K, pow2,
                                              as_stream(stream)));
}

}  // namespace

extern "C" {

size_t fp8_gated_gemm_workspace_bytes(int64_t M, int64_t I, int64_t K) {
    if (I < 0 || I >= kMaxDim / 2 || I % 128 != 0 || check_product(M, 2 * I, K, 1) != FP8_OK ||
        M == 0 || I == 0 || K == 0)
        return 0;
    return gated_gemm_workspace_bytes(M, 0, I, K);
}

size_t fp8_grouped_gated_gemm_workspace_bytes(int64_t T, int64_t E, int64_t I, int64_t K) {
    if (I < 0 || I >= kMaxDim / 2 || I % 128 != 0 || check_product(T, 2 * I, K, E) != FP8_OK ||
        T == 0 || I == 0 || K == 0 || E == 0)
        return 0;
    return gated_gemm_workspace_bytes(T, E, I, K);
}

fp8_status fp8_block_gemm_gated(const void *a_e4m3, const float *a_scales, const void *w_e4m3,
                                const float *w_scales, int activation, int64_t M, int64_t I,
                                int64_t K, void *out, int out_dtype, void *workspace,
                                size_t workspace_bytes, void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, kDense, activation, M, I, K, out, out_dtype,
                 nullptr, nullptr, nullptr, nullptr, false, workspace, workspace_bytes, false,
                 hip_stream);
}

fp8_status fp8_block_gemm_gated_pow2(const void *a_e4m3, const float *a_scales,
                                     const void *w_e4m3, const float *w_scales, int activation,
                                     int64_t M, int64_t I, int64_t K, void *out, int out_dtype,
                                     void *workspace, size_t workspace_bytes, void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, kDense, activation, M, I, K, out, out_dtype,
                 nullptr, nullptr, nullptr, nullptr, false, workspace, workspace_bytes, true,
                 hip_stream);
}

fp8_status fp8_block_gemm_gated_quant_1x128(const void *a_e4m3, const float *a_scales,
                                            const void *w_e4m3, const float *w_scales,
                                            int activation, int64_t M, int64_t I, int64_t K,
                                            void *q, float *scales, void *h, float *h_scales,
                                            void *workspace, size_t workspace_bytes,
                                            void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, kDense, activation, M, I, K, nullptr,
                 FP8_OUT_BF16, q, scales, h, h_scales, true, workspace, workspace_bytes, false,
                 hip_stream);
}

fp8_status fp8_block_gemm_gated_quant_1x128_pow2(const void *a_e4m3, const float *a_scales,
                                                 const void *w_e4m3, const float *w_scales,
                                                 int activation, int64_t M, int64_t I, int64_t K,
                                                 void *q, float *scales, void *h,
                                                 float *h_scales, void *workspace,
                                                 size_t workspace_bytes, void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, kDense, activation, M, I, K, nullptr,
                 FP8_OUT_BF16, q, scales, h, h_scales, true, workspace, workspace_bytes, true,
                 hip_stream);
}

fp8_status fp8_block_grouped_gemm_gated(const void *a_e4m3, const float *a_scales,
                                        const void *w_e4m3, const float *w_scales,
                                        const int32_t *group_offsets, int64_t E, int activation,
                                        int64_t T, int64_t I, int64_t K, void *out,
                                        int out_dtype, void *workspace, size_t workspace_bytes,
                                        void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, {true, group_offsets, E}, activation, T, I, K,
                 out, out_dtype, nullptr, nullptr, nullptr, nullptr, false, workspace,
                 workspace_bytes, false, hip_stream);
}

fp8_status fp8_block_grouped_gemm_gated_pow2(const void *a_e4m3, const float *a_scales,
                                             const void *w_e4m3, const float *w_scales,
                                             const int32_t *group_offsets, int64_t E,
                                             int activation, int64_t T, int64_t I, int64_t K,
                                             void *out, int out_dtype, void *workspace,
                                             size_t workspace_bytes, void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, {true, group_offsets, E}, activation, T, I, K,
                 out, out_dtype, nullptr, nullptr, nullptr, nullptr, false, workspace,
                 workspace_bytes, true, hip_stream);
}

fp8_status fp8_block_grouped_gemm_gated_quant_1x128(
    const void *a_e4m3, const float *a_scales, const void *w_e4m3, const float *w_scales,
    const int32_t *group_offsets, int64_t E, int activation, int64_t T, int64_t I, int64_t K,
    void *q, float *scales, void *h, float *h_scales, void *workspace, size_t workspace_bytes,
    void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, {true, group_offsets, E}, activation, T, I, K,
                 nullptr, FP8_OUT_BF16, q, scales, h, h_scales, true, workspace,
                 workspace_bytes, false, hip_stream);
}

fp8_status fp8_block_grouped_gemm_gated_quant_1x128_pow2(
    const void *a_e4m3, const float *a_scales, const void *w_e4m3, const float *w_scales,
    const int32_t *group_offsets, int64_t E, int activation, int64_t T, int64_t I, int64_t K,
    void *q, float *scales, void *h, float *h_scales, void *workspace, size_t workspace_bytes,
    void *hip_stream) {
    return gated(a_e4m3, a_scales, w_e4m3, w_scales, {true, group_offsets, E}, activation, T, I, K,
                 nullptr, FP8_OUT_BF16, q, scales, h, h_scales, true, workspace,
                 workspace_bytes, true, hip_stream);
}

fp8_status fp8_gated_grad(const void *da, int da_dtype, int64_t ld_da, const void *h,
                          int64_t ld_h, const float *h_scales, int activation, int64_t M,
                          int64_t I, void *dh, int dh_dtype, void *hip_stream) {
    return gated_grad(da, da_dtype, ld_da, h, ld_h, h_scales, activation, M, I, dh, dh_dtype,
                      false, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, false,
                      hip_stream);
}

fp8_status fp8_gated_grad_quant(const void *da, int da_dtype, int64_t ld_da, const void *h,
                                int64_t ld_h, const float *h_scales, int activation, int64_t M,
                                int64_t I, void *q, float *scales, void *q_t, float *scales_t,
                                void *a_t, float *a_scales_t, void *hip_stream) {
    return gated_grad(da, da_dtype, ld_da, h, ld_h, h_scales, activation, M, I, nullptr,
                      FP8_OUT_BF16, true, q, scales, q_t, scales_t, a_t, a_scales_t, false,
                      hip_stream);
}

fp8_status fp8_gated_grad_quant_pow2(const void *da, int da_dtype, int64_t ld_da, const void *h,
                                     int64_t ld_h, const float *h_scales, int activation,
                                     int64_t M, int64_t I, void *q, float *scales, void *q_t,
                                     float *scales_t, void *a_t, float *a_scales_t,
                                     void *hip_stream) {
    return gated_grad(da, da_dtype, ld_da, h, ld_h, h_scales, activation, M, I, nullptr,
                      FP8_OUT_BF16, true, q, scales, q_t, scales_t, a_t, a_scales_t, true,
                      hip_stream);
}

fp8_status fp8_dequant_act_1x128(const void *q, const float *scales, int64_t M, int64_t K,
                                 void *x, int out_dtype, void *hip_stream) {
    if (!type_ok(out_dtype)) return FP8_ERR_DTYPE;
    const fp8_status st = check_stored(q, scales, M, K);
    if (st != FP8_OK || M == 0 || K == 0) return st;
    if (!x) return FP8_ERR_NULL;
    if (!aligned(x, bytes_of(out_dtype))) return FP8_ERR_ALIGN;
    clear_last_error();
    return from_hip(launch_dequant_act(q, scales, M, K, x, out_dtype == FP8_OUT_BF16,
                                       as_stream(hip_stream)));
}

fp8_status fp8_requant_act_128x1_t(const void *q, const float *scales, int64_t M, int64_t K,
                                   void *q_t, float *scales_t, void *hip_stream) {
    return requant_t(q, scales, M, K, q_t, scales_t, false, hip_stream);
}

fp8_status fp8_requant_act_128x1_t_pow2(const void *q, const float *scales, int64_t M, int64_t K,
                                        void *q_t, float *scales_t, void *hip_stream) {
    return requant_t(q, scales, M, K, q_t, scales_t, true, hip_stream);
}

fp8_status fp8_block_grouped_gemm_dgrad(const void *dy_e4m3, const float *dy_scales,
                                        const void *w_e4m3, const float *w_scales,
                                        const int32_t *group_offsets, int64_t E, int64_t T,
                                        void *dx, int out_dtype, int64_t N, int64_t K,
                                        void *hip_stream) {
    return grouped_dgrad(dy_e4m3, dy_scales, w_e4m3, w_scales, group_offsets, E, T, dx, out_dtype,
                         N, K, false, hip_stream);
}

fp8_status fp8_block_grouped_gemm_dgrad_pow2(const void *dy_e4m3, const float *dy_scales,
                                             const void *w_e4m3, const float *w_scales,
                                             const int32_t *group_offsets, int64_t E, int64_t T,
                                             void *dx, int out_dtype, int64_t N, int64_t K,
                                             void *hip_stream) {
    return grouped_dgrad(dy_e4m3, dy_scales, w_e4m3, w_scales, group_offsets, E, T, dx, out_dtype,
                         N, K, true, hip_stream);
}

}  // extern "C"

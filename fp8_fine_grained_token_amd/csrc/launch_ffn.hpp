// Host-side launchers of the operators inside a gated feed-forward block
// (argument checking happens in abi_ffn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8blk {

// What a gated product writes, each part optional (NULL): a = act(g) u in
// bf16 or fp32, a quantized 1x128, [g | u] quantized 1x128.
struct GatedOut {
    void *out;  // [M][I]
    uint8_t *q;  // [M][I]
    float *q_scales;  // [M][I / 128]
    uint8_t *h;  // [M][2 I]
    float *h_scales;  // [M][2 I / 128]
    int64_t I;
    bool bf16_out, gelu, pow2;
};

// ---- gated products (gated.hip) ----
struct GatedGemm {
    const void *a;
    const float *sa;
    const void *w;
    const float *sw;
    const int32_t *offsets;  // grouped only
    int64_t E;               // 0: dense
    int64_t M, K;            // M = rows of all experts for grouped
    GatedOut to;
    void *workspace;
    size_t workspace_bytes;
};
hipError_t launch_gated_gemm(const GatedGemm &p, hipStream_t stream);
// Bytes that the split plan for this shape takes (0: none); E = 0 for dense.
size_t gated_gemm_workspace_bytes(int64_t M, int64_t E, int64_t I, int64_t K);

// ---- gradient of the activation and the product (gated_grad.hip) ----
struct GatedGrad {
    const void *da;  // [M][I], rows ld_da elements apart
    int64_t ld_da;
    const void *h;  // [M][2 I] E4M3 (h_scales given) or bf16
    int64_t ld_h;
    const float *h_scales;  // [M][2 I / 128]
    int64_t M, I;
    bool da_bf16, gelu, pow2;
    void *dh;  // [M][2 I] bf16 or fp32; the parts below are optional
    bool dh_bf16;
    uint8_t *q;  // [M][2 I]
    float *scales;
    uint8_t *q_t;  // [2 I][M]
    float *scales_t;
    uint8_t *a_t;  // [I][M]
    float *a_scales_t;
};
hipError_t launch_gated_grad(const GatedGrad &p, hipStream_t stream);

// ---- 8-bit checkpoints (gated_grad.hip) ----
hipError_t launch_dequant_act(const void *q, const float *scales, int64_t M, int64_t K, void *x,
                              bool bf16_out, hipStream_t stream);
hipError_t launch_requant_act_t(const void *q, const float *scales, int64_t M, int64_t K,
                                void *q_t, float *scales_t, bool pow2, hipStream_t stream);

// ---- input gradient per expert (gemm.hip) ----
// dx [T][Kx] = dy [T][N] W[e] [N][Kx], W in its forward layout.
hipError_t launch_grouped_gemm_dgrad(const void *dy, const float *sdy, const void *w,
                                     const float *sw, const int32_t *offsets, int64_t E,
                                     int64_t T, void *dx, bool bf16_out, int64_t N, int64_t Kx,
                                     bool pow2, hipStream_t stream);

}  // namespace fp8blk

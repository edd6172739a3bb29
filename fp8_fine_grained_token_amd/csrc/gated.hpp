// The activation of a gated feed-forward block and what is done with eight of
// its values at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch_ffn.hpp"
#include "vec.hpp"

namespace fp8blk {

// act(g) = g sigmoid(z): z = g for SiLU, and for GELU in its tanh form, since
// (1 + tanh(y)) / 2 = sigmoid(2 y), z = 2 sqrt(2 / pi) (g + 0.044715 g^3).
constexpr float kGelu1 = 1.5957691216057308f;             // 2 sqrt(2 / pi)
constexpr float kGelu3 = 1.5957691216057308f * 0.044715f;

__device__ __forceinline__ float sigmoid(float z) {
    // exp(-z) = inf gives 0 and exp(-z) = 0 gives 1: no case apart
    return __builtin_amdgcn_rcpf(1.0f + expf(-z));
}
template <bool kGelu>
__device__ __forceinline__ float gate_sigmoid(float g) {
    return sigmoid(kGelu ? g * __builtin_fmaf(kGelu3 * g, g, kGelu1) : g);
}

// a = act(g) u of eight columns.
__device__ __forceinline__ void gated8(const float (&g)[8], const float (&u)[8], bool gelu,
                                       float (&a)[8]) {
    if (gelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = g[i] * gate_sigmoid<true>(g[i]) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = g[i] * gate_sigmoid<false>(g[i]) * u[i];
    }
}

// Gradients of a = act(g) u at one column: act'(g) = s + g z' s (1 - s) with s
// = sigmoid(z).  Where s is 0 or 1 the second term is 0, whatever z' is (it
// may be infinite).
template <bool kGelu>
__device__ __forceinline__ void gated_grad(float g, float u, float da, float &dg, float &du,
                                           float &a) {
    const float s = gate_sigmoid<kGelu>(g);
    const float t = s * (1.0f - s);
    const float gz = kGelu ? g * __builtin_fmaf(3.0f * kGelu3 * g, g, kGelu1) : g;
    const float slope = t == 0.0f ? s : __builtin_fmaf(gz, t, s);
    const float act = g * s;
    a = act * u;
    dg = da * u * slope;
    du = da * act;
}

// Eight values of a 1x128 group that 16 lanes hold, quantized into row `q` (at
// column col) with the group's scale at `scale`; `live`: the row is one of the
// output's (every lane of the wave calls it).
__device__ __forceinline__ void put_quantized(const float (&f)[8], bool live, bool pow2, uint8_t *q,
                                              float *scale) {
    float s;
    const uint2 v = quantize8(f, group_max(f), live, pow2, s);
    if (live) {
        *reinterpret_cast<uint2 *>(q) = v;
        if ((threadIdx.x & 15) == 0) *scale = s;
    }
}

// What a gated product writes of one row's columns [n0 + c, n0 + c + 8), c = 8
// (lane % 16), from g and u there; 16 lanes hold the row's 128 columns, which
// are one scale group of a, of g and of u.
__device__ __forceinline__ void put_gated(const GatedOut &to, int64_t row, int64_t n0, bool live,
                                          const float (&g)[8], const float (&u)[8]) {
    const int c = 8 * (threadIdx.x & 15);
    float a[8];
    gated8(g, u, to.gelu, a);
    const int64_t GI = to.I >> 7, col = n0 + c, gb = n0 >> 7;
    if (to.out && live) {
        if (to.bf16_out) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = to_bf16x2(a[2 * i], a[2 * i + 1]);
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(to.out) + row * to.I + col) = v;
        } else {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(to.out) + row * to.I + col);
            d[0] = make_float4(a[0], a[1], a[2], a[3]);
            d[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
    if (to.q) put_quantized(a, live, to.pow2, to.q + row * to.I + col, to.q_scales + row * GI + gb);
    if (to.h) {
        put_quantized(g, live, to.pow2, to.h + row * 2 * to.I + col,
                      to.h_scales + row * 2 * GI + gb);
        put_quantized(u, live, to.pow2, to.h + (row * 2 + 1) * to.I + col,
                      to.h_scales + (row * 2 + 1) * GI + gb);
    }
}

}  // namespace fp8blk

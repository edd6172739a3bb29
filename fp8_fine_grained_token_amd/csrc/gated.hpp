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
    // exp(-z) = inf gives 0 and exp(-z) = 0 gives 1: no case apart.  2^h with h
    // = -z log2(e) rounded is off by |z| 2^-24 relatively, which a sigmoid near
    // 1 does not show and one near 0 may carry (expf, which carries h in two
    // parts, took the gradient's rows from 27 to 32 us and its tiles from 32 to
    // 35).
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
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
// = sigmoid(z).  From |g z'| = 128 on s is 0 or 1 and the second term 0, so g z'
// may stop at any larger value: a finite one, for an infinite g z'.  da meets the
// slope, of magnitude 1.13 at most, before u: da u may overflow where the gate
// is shut, and infinity times a slope of 0 is NaN.
constexpr float kFar = 0x1p64f;
template <bool kGelu>
__device__ __forceinline__ void gated_grad(float g, float u, float da, float &dg, float &du,
                                           float &a) {
    const float s = gate_sigmoid<kGelu>(g);
    const float gz = kGelu ? g * __builtin_fmaf(3.0f * kGelu3 * g, g, kGelu1) : g;
    const float t = s * (1.0f - s);
    const float slope = __builtin_fmaf(__builtin_amdgcn_fmed3f(gz, -kFar, kFar), t, s);
    const float act = g * s;
    a = act * u;
    dg = da * slope * u;
    du = da * act;
}

// fl32(x / s) from r = fl32(1 / s), by quot_fast's correction with the sign
// left in: the remainder is taken as q0 s - x, so that a zero keeps its sign
// through the last sum.  Unclamped: the conversion rounds before it looks for
// an overflow (448 to below 464 is 448), and a quotient by a normal amax / 448
// is at most 448 (1 + 2^-22).
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q0 = x * r;
    const float e = __builtin_fmaf(q0, s, -x);
    return __builtin_fmaf(-e, r, q0);
}

// How a group of largest magnitude `bits` is quantized (quantize8's rule; `any`
// is the general form of it, for groups of zeros, tiny and non-finite ones).
// With amax below 2^-60 values and scale are taken times 2^64, which is exact,
// so that the quotient's correction stays in range; where the scale is 0 all
// codes are 0, and in a group with a NaN or an infinity they are NaN.
struct GroupScale {
    static constexpr uint32_t kInf = 0x7F800000u, kTiny = 0x21800000u;  // 2^-60
    float scale;  // the group's
    float s, r;   // what values are divided by, and its reciprocal
    // whether the group is of the usual kind
    static __device__ __forceinline__ bool usual(uint32_t bits, bool pow2) {
        const uint32_t least = pow2 ? 1 : kTiny;
        return bits - least < kInf - least;
    }
    static __device__ __forceinline__ bool tiny(uint32_t bits, bool pow2) {
        return !pow2 && bits < kTiny;
    }
    __device__ __forceinline__ void set(uint32_t bits, bool pow2) {
        const float amax = __uint_as_float(bits);
        s = scale = pow2 ? scale_pow2(amax) : scale_fast(amax);
        r = 1.0f / s;
    }
    __device__ __forceinline__ void set_any(uint32_t bits, bool pow2) {
        const float amax = __uint_as_float(bits);
        scale = bits >= kInf ? amax : pow2 ? scale_pow2(amax) : amax / kE4M3Max;
        s = tiny(bits, pow2) ? scale * 0x1p64f : scale;
        r = s > 0.0f ? 1.0f / s : 0.0f;
    }
    static __device__ __forceinline__ float factor(uint32_t bits, bool pow2) {
        return tiny(bits, pow2) ? 0x1p64f : 1.0f;
    }
    // codes of a group that is not of the usual kind, from its quotients'
    __device__ __forceinline__ uint32_t codes(uint32_t quotients, uint32_t bits) const {
        return bits >= kInf ? 0x7F7F7F7Fu : bits == 0 || s == 0.0f ? 0u : quotients;
    }
};

// Eight values of a group that 16 lanes hold -> E4M3 bytes and the scale.
// `live`: the lane's group is asked for (every lane of the wave calls it).
__device__ __forceinline__ uint2 quantize_group(const float (&f)[8], bool live, bool pow2,
                                                float &scale) {
    const uint32_t bits = group_max(f);
    auto codes = [](const float (&x)[8], const GroupScale &q) {
        uint2 v = make_uint2(0, 0);
        v.x = cvt_pk_e4m3<false>(quotient(x[0], q.s, q.r), quotient(x[1], q.s, q.r), v.x);
        v.x = cvt_pk_e4m3<true>(quotient(x[2], q.s, q.r), quotient(x[3], q.s, q.r), v.x);
        v.y = cvt_pk_e4m3<false>(quotient(x[4], q.s, q.r), quotient(x[5], q.s, q.r), v.y);
        v.y = cvt_pk_e4m3<true>(quotient(x[6], q.s, q.r), quotient(x[7], q.s, q.r), v.y);
        return v;
    };
    GroupScale q;
    if (__all(!live || GroupScale::usual(bits, pow2))) {
        q.set(bits, pow2);
        scale = q.scale;
        return codes(f, q);
    }
    q.set_any(bits, pow2);
    scale = q.scale;
    // (a scale that is subnormal may be a third less than amax / 448: values stop
    // at 448 of it)
    const float by = GroupScale::factor(bits, pow2), most = kE4M3Max * q.s;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(f[i] * by, -most, most);
    uint2 v = codes(x, q);
    if (!GroupScale::usual(bits, pow2)) {  // else a usual group beside others
        v.x = q.codes(v.x, bits);
        v.y = q.codes(v.y, bits);
    }
    return v;
}

// Eight values of a 1x128 group that 16 lanes hold, quantized into row `q` (at
// their column) with the group's scale at `scale`; `live`: the row is one of
// the output's.
__device__ __forceinline__ void put_quantized(const float (&f)[8], bool live, bool pow2, uint8_t *q,
                                              float *scale) {
    float s;
    const uint2 v = quantize_group(f, live, pow2, s);
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

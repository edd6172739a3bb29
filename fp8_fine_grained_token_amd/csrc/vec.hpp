// Eight values of a row at a time, from bf16 or fp32 rows of any alignment.
//
// gfx950 reads and writes 16 bytes at any byte address, so a row of odd width
// or alignment needs no scalar path.  The last vector of a row is read as the
// row's last eight values (some of them its neighbour's): a load is then the
// same for every lane, and nothing but a store depends on where a row ends.
// Loads keep what they read as it is (Raw8) until it is used, so that many
// can be under way.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"

namespace fp8blk {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

struct Bf16 {
    uint16_t bits;
};

// Two fp32 -> two bf16 in one v_cvt_pk_bf16_f32: to nearest even, subnormals
// and NaN kept (the same bits as rounding by hand, over all 2^32 inputs, at a
// sixth of the instructions).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(Bf16 v) {
    return __uint_as_float((uint32_t)v.bits << 16);
}
__device__ __forceinline__ void from_float(float f, float &v) { v = f; }
__device__ __forceinline__ void from_float(float f, Bf16 &v) { v.bits = (uint16_t)to_bf16x2(f, f); }

// Vector v of a row of H values: values col .. col + 7, of which those from
// index lo up to hi are its own (none past the last vector; hi < 8 only in
// rows of fewer than eight values).
struct Span {
    int col, lo, hi;
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == 8; }
    __device__ __forceinline__ bool any() const { return lo < hi; }
    __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
};

template <bool kNarrow>
__device__ __forceinline__ Span row_span(int64_t v, int64_t H) {
    Span s;
    s.hi = kNarrow ? (int)H : 8;
    const int64_t most = H - s.hi;
    s.col = (int)(8 * v < most ? 8 * v : most);
    const int64_t over = 8 * v - s.col;
    s.lo = over < 8 ? (int)over : 8;
    return s;
}

template <typename T>
struct Raw8;
template <>
struct Raw8<Bf16> {
    u32x4 v;
};
template <>
struct Raw8<float> {
    u32x4 a, b;
};

// The eight values from p on; in rows of fewer than eight (kNarrow) those
// there are, the last one repeated.  A template parameter: as a branch it
// would put a wait after every load.  kOnce: values that are read this once
// and need no place in the caches.
template <bool kOnce>
__device__ __forceinline__ u32x4_any load16(const void *p) {
    const u32x4_any *v = static_cast<const u32x4_any *>(p);
    return kOnce ? __builtin_nontemporal_load(v) : *v;
}
template <bool kNarrow, bool kOnce = false>
__device__ __forceinline__ void load_raw(const Bf16 *p, int hi, Raw8<Bf16> &r) {
    if (!kNarrow) {
        r.v = load16<kOnce>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.v[i] = p[min(2 * i, hi - 1)].bits | (uint32_t)p[min(2 * i + 1, hi - 1)].bits << 16;
    }
}
template <bool kNarrow, bool kOnce = false>
__device__ __forceinline__ void load_raw(const float *p, int hi, Raw8<float> &r) {
    if (!kNarrow) {
        r.a = load16<kOnce>(p);
        r.b = load16<kOnce>(p + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.a[i] = __float_as_uint(p[min(i, hi - 1)]);
            r.b[i] = __float_as_uint(p[min(i + 4, hi - 1)]);
        }
    }
}
__device__ __forceinline__ void zero_raw(Raw8<Bf16> &r) { r.v = u32x4{0, 0, 0, 0}; }
__device__ __forceinline__ void zero_raw(Raw8<float> &r) { r.a = r.b = u32x4{0, 0, 0, 0}; }

__device__ __forceinline__ void unpack(const Raw8<Bf16> &r, float (&f)[8]) {
    unpack8(make_uint4(r.v.x, r.v.y, r.v.z, r.v.w), f);
}
__device__ __forceinline__ void unpack(const Raw8<float> &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(r.a[i]);
        f[i + 4] = __uint_as_float(r.b[i]);
    }
}
// The span's own values, zeros for the others.
template <typename T>
__device__ __forceinline__ void unpack_own(const Raw8<T> &r, const Span &s, float (&f)[8]) {
    unpack(r, f);
    if (!s.whole()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = s.has(i) ? f[i] : 0.0f;
    }
}

// Where a span begins in a row, by a 32-bit byte offset (rows are below 2^30
// bytes): next to a row address that a wave shares it is all a lane keeps.
template <typename T>
__device__ __forceinline__ T *span_at(T *row, const Span &s) {
    using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
    return reinterpret_cast<T *>(reinterpret_cast<Byte *>(row) +
                                 (uint32_t)s.col * (uint32_t)sizeof(T));
}

// The span's own values to a row.
__device__ __forceinline__ void store_span(Bf16 *row, const Span &s, const float (&f)[8]) {
    if (s.whole()) {
        u32x4_any v;
        v.x = to_bf16x2(f[0], f[1]);
        v.y = to_bf16x2(f[2], f[3]);
        v.z = to_bf16x2(f[4], f[5]);
        v.w = to_bf16x2(f[6], f[7]);
        *reinterpret_cast<u32x4_any *>(span_at(row, s)) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s.has(i)) from_float(f[i], span_at(row, s)[i]);
    }
}
__device__ __forceinline__ void store_span(float *row, const Span &s, const float (&f)[8]) {
    if (s.whole()) {
        u32x4_any a, b;
        a.x = __float_as_uint(f[0]); a.y = __float_as_uint(f[1]);
        a.z = __float_as_uint(f[2]); a.w = __float_as_uint(f[3]);
        b.x = __float_as_uint(f[4]); b.y = __float_as_uint(f[5]);
        b.z = __float_as_uint(f[6]); b.w = __float_as_uint(f[7]);
        *reinterpret_cast<u32x4_any *>(span_at(row, s)) = a;
        *reinterpret_cast<u32x4_any *>(span_at(row, s) + 4) = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s.has(i)) span_at(row, s)[i] = f[i];
    }
}

// The larger of two magnitudes, by their bits: so NaN, which fmaxf drops, is
// above infinity and infinity above every number.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float max_magnitude(float a, float b) {
    return __uint_as_float(max(magnitude(a), magnitude(b)));
}

// The same over the 16 lanes of a DPP row, in the steps of row16_max.
__device__ __forceinline__ uint32_t row16_max_bits(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true));
    return m;
}

// Largest magnitude of the 1x128 group that 16 lanes hold, as bits.
__device__ __forceinline__ uint32_t group_max(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(f[i]));
    return row16_max_bits(m);
}

// E4M3 bytes and scale of a lane's part of a 1x128 group of maximum `bits`
// (`used`: the lane holds any of it).  The usual groups take a path without
// branches and with one divide (the activation quantizer's); a wave with an
// all-zero, tiny or non-finite group takes the general one.  A group that
// holds a NaN or an infinity reads back as NaN: the scale is its maximum and
// the codes are E4M3's NaN.
__device__ __forceinline__ uint2 quantize8(const float (&f)[8], uint32_t bits, bool used, bool pow2,
                                           float &scale) {
    constexpr uint32_t kInf = 0x7F800000u, kTiny = 0x21800000u;  // 2^-60
    const float amax = __uint_as_float(bits);
    const uint32_t least = pow2 ? 1 : kTiny;
    if (__all(!used || bits - least < kInf - least)) {
        scale = pow2 ? scale_pow2(amax) : scale_fast(amax);
        const float r = 1.0f / scale;
        uint32_t lo = 0, hi = 0;
        lo = cvt_pk_e4m3<false>(quot_fast(f[0], scale, r), quot_fast(f[1], scale, r), lo);
        lo = cvt_pk_e4m3<true>(quot_fast(f[2], scale, r), quot_fast(f[3], scale, r), lo);
        hi = cvt_pk_e4m3<false>(quot_fast(f[4], scale, r), quot_fast(f[5], scale, r), hi);
        hi = cvt_pk_e4m3<true>(quot_fast(f[6], scale, r), quot_fast(f[7], scale, r), hi);
        return make_uint2(lo, hi);
    }
    scale = amax;
    if (bits >= kInf) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const QuotientCtx qc(amax, pow2);
    scale = qc.s;
    return quant8(f, qc);
}

// E4M3 bytes of the span's values of a 1x128 group.
__device__ __forceinline__ void store_e4m3(uint8_t *row, const Span &s, uint2 v) {
    if (s.whole()) {
        u32x2_any w;
        w.x = v.x;
        w.y = v.y;
        *reinterpret_cast<u32x2_any *>(span_at(row, s)) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s.has(i))
                span_at(row, s)[i] = (uint8_t)((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))) & 0xFF);
    }
}

// The number of threads that share a row of `vecs` vectors: a power of two
// from `least` to `most`, no more than needed.
inline int threads_per_row(int64_t vecs, int least, int most) {
    int t = least;
    while (t < most && t < vecs) t *= 2;
    return t;
}

}  // namespace fp8blk

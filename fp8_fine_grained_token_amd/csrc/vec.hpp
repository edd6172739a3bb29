// Eight values of a row at a time, from bf16 or fp32 rows of any alignment.
//
// gfx950 reads and writes 16 bytes at any byte address, so a row of odd
// width needs no scalar path: only the last vector of a row (n < 8 values)
// is taken value by value.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace fp8blk {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

struct Bf16 {
    uint16_t bits;
};

// fp32 -> bf16 bits to nearest even, NaN kept (its payload may vanish).
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    const uint32_t rounded = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    return f != f ? 0x7FC0u : rounded;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(Bf16 v) {
    return __uint_as_float((uint32_t)v.bits << 16);
}
__device__ __forceinline__ void from_float(float f, float &v) { v = f; }
__device__ __forceinline__ void from_float(float f, Bf16 &v) { v.bits = (uint16_t)to_bf16(f); }

// n in [0, 8] values at p, zeros past them.
__device__ __forceinline__ void load8(const Bf16 *p, int n, float (&f)[8]) {
    if (n == 8) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any *>(p);
        unpack8(make_uint4(v.x, v.y, v.z, v.w), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? to_float(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const float *p, int n, float (&f)[8]) {
    if (n == 8) {
        const u32x4_any a = *reinterpret_cast<const u32x4_any *>(p);
        const u32x4_any b = *reinterpret_cast<const u32x4_any *>(p + 4);
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void store8(Bf16 *p, int n, const float (&f)[8]) {
    if (n == 8) {
        u32x4_any v;
        v.x = to_bf16(f[0]) | (to_bf16(f[1]) << 16);
        v.y = to_bf16(f[2]) | (to_bf16(f[3]) << 16);
        v.z = to_bf16(f[4]) | (to_bf16(f[5]) << 16);
        v.w = to_bf16(f[6]) | (to_bf16(f[7]) << 16);
        *reinterpret_cast<u32x4_any *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) from_float(f[i], p[i]);
    }
}
__device__ __forceinline__ void store8(float *p, int n, const float (&f)[8]) {
    if (n == 8) {
        u32x4_any a, b;
        a.x = __float_as_uint(f[0]); a.y = __float_as_uint(f[1]);
        a.z = __float_as_uint(f[2]); a.w = __float_as_uint(f[3]);
        b.x = __float_as_uint(f[4]); b.y = __float_as_uint(f[5]);
        b.z = __float_as_uint(f[6]); b.w = __float_as_uint(f[7]);
        *reinterpret_cast<u32x4_any *>(p) = a;
        *reinterpret_cast<u32x4_any *>(p + 4) = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = f[i];
    }
}

// E4M3 bytes of one lane's n values of a 1x128 group.
__device__ __forceinline__ void store_e4m3(uint8_t *p, int n, uint2 v) {
    if (n == 8) {
        u32x2_any w;
        w.x = v.x;
        w.y = v.y;
        *reinterpret_cast<u32x2_any *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))) & 0xFF);
    }
}

// Values of a row that the 8-value vector v holds: min(8, H - 8 v), at least 0.
__device__ __forceinline__ int vec_count(int64_t H, int64_t v) {
    const int64_t left = H - 8 * v;
    return left >= 8 ? 8 : left > 0 ? (int)left : 0;
}

// The number of threads that share a row of `vecs` vectors: a power of two
// from `least` to `most`, no more than needed.
inline int threads_per_row(int64_t vecs, int least, int most) {
    int t = least;
    while (t < most && t < vecs) t *= 2;
    return t;
}

}  // namespace fp8blk

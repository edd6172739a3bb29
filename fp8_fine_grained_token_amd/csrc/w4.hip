// 4-bit weights (OCP E2M1 with group scales): the offline quantizer and the
// products of a few rows with them, dense and per expert (gfx950).
//
// A product of M <= 16 rows reads N K / 2 bytes of codes and N K / 32 bytes
// of scales and does at most 64 flops per byte of them: its floor is the
// weights' bytes at the rate of a large copy.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch_moe.hpp"
#include "vec.hpp"

namespace fp8blk {

namespace {

// ---- quantizer (offline) ---------------------------------------------------

// E2M1 code of |y| <= 6 (ties to the even code), without the sign.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
    const float a = fabsf(y);
    return (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
           (a > 5.0f);
}

// One wave per row and 128 channels, two channels a lane.
template <bool kE8m0>
__global__ __launch_bounds__(256) void w4_quant_kernel(const uint16_t *__restrict__ w, int64_t N,
                                                       int64_t K, uint8_t *__restrict__ codes,
                                                       void *__restrict__ scales) {
    const int64_t G = (K + 127) / 128, row_bytes = (K + 1) / 2;
    const int lane = threadIdx.x & 63;
    const int64_t units = N * G;
    for (int64_t u = blockIdx.x * 4ll + (threadIdx.x >> 6); u < units; u += gridDim.x * 4ll) {
        const int64_t n = u / G, g = u - u / G * G;
        const int64_t k = 128 * g + 2 * lane;
        const float a = k < K ? __uint_as_float((uint32_t)w[n * K + k] << 16) : 0.0f;
        const float b = k + 1 < K ? __uint_as_float((uint32_t)w[n * K + k + 1] << 16) : 0.0f;
        float amax = row16_max(fmaxf(fabsf(a), fabsf(b)));  // 16 lanes: 32 channels
        float qa = 0, qb = 0;
        if (kE8m0) {
            // smallest E with 6 * 2^E >= amax: amax = (1 + f) 2^(e - 127) and
            // 6 = 1.5 * 2^2, so E = e - 129, one more where 1 + f > 1.5
            const uint32_t bits = __float_as_uint(amax);
            int E = (int)(bits >> 23) - 129 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
            E = E < -127 ? -127 : E;
            // x / 2^E in two exact steps (2^-E itself can leave the range)
            const int h = -E / 2;
            const float r0 = __uint_as_float((uint32_t)(h + 127) << 23);
            const float r1 = __uint_as_float((uint32_t)(-E - h + 127) << 23);
            qa = a * r0 * r1;
            qb = b * r0 * r1;
            const int64_t group = k / 32;
            if ((lane & 15) == 0 && k < K)
                static_cast<uint8_t *>(scales)[n * ((K + 31) / 32) + group] = (uint8_t)(E + 127);
        } else {
            amax = fmaxf(amax, __shfl_xor(amax, 16));
            amax = fmaxf(amax, __shfl_xor(amax, 32));
            const float s = amax / 6.0f;
            if (s > 0) {
                qa = a / s;
                qb = b / s;
            }
            if (lane == 0) static_cast<float *>(scales)[u] = s;
        }
        if (k < K) {
            const bool zero = !(amax > 0);
            const uint32_t ca = e2m1_code(qa) | (zero ? 0u : (__float_as_uint(a) >> 31) << 3);
            uint32_t cb = e2m1_code(qb) | (zero ? 0u : (__float_as_uint(b) >> 31) << 3);
            if (k + 1 >= K) cb = 0;
            codes[n * row_bytes + k / 2] = (uint8_t)(ca | (cb << 4));
        }
    }
}

// ---- products -----------------------------------------------------------------

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7;
    const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126) << 23 | (m & 1) << 22);
    return c & 8 ? -v : v;
}

// One wave per output column, 16 rows of x at a time.
constexpr int kRows = 16;

template <bool kE8m0, typename Out>
__global__ __launch_bounds__(256) void w4_matvec_kernel(
    const Bf16 *__restrict__ x, int64_t ldx, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const int32_t *__restrict__ offsets, int64_t R, int64_t N,
    int64_t K, Out *__restrict__ y) {
    const int lane = threadIdx.x & 63;
    const int64_t n = blockIdx.x * 4ll + (threadIdx.x >> 6);
    if (n >= N) return;
    const int64_t e = blockIdx.y;
    int64_t r0 = 0, r1 = R;
    if (offsets) {
        // an expert's range starts no earlier than any before it ends
        int64_t low = 0;
        for (int64_t i = 0; i <= e; ++i) {
            const int64_t o = offsets[i];
            const int64_t c = o < 0 ? 0 : o > R ? R : o;
            low = c > low ? c : low;
        }
        const int64_t o = offsets[e + 1];
        r0 = low;
        r1 = o < low ? low : o > R ? R : o;
    }
    const int64_t row_bytes = (K + 1) / 2, row = e * N + n;
    const uint8_t *c = codes + row * row_bytes;
    for (int64_t m0 = r0; m0 < r1; m0 += kRows) {
        float acc[kRows] = {};
        const int rows = r1 - m0 < kRows ? (int)(r1 - m0) : kRows;
        for (int64_t b = lane; b < row_bytes; b += 64) {
            const int64_t k = 2 * b;
            float s;
            if (kE8m0) {
                const int E = static_cast<const uint8_t *>(scales)[row * ((K + 31) / 32) + k / 32];
                s = ldexpf(1.0f, E - 127);
            } else {
                s = static_cast<const float *>(scales)[row * ((K + 127) / 128) + k / 128];
            }
            const uint32_t pair = c[b];
            const float w0 = s * e2m1_value(pair & 15);
            const float w1 = k + 1 < K ? s * e2m1_value(pair >> 4) : 0.0f;
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                if (m >= rows) continue;
                const Bf16 *p = x + (m0 + m) * ldx + k;
                acc[m] = __builtin_fmaf(to_float(p[0]), w0, acc[m]);
                if (k + 1 < K) acc[m] = __builtin_fmaf(to_float(p[1]), w1, acc[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            for (int d = 32; d; d /= 2) acc[m] += __shfl_xor(acc[m], d);
            if (m < rows && lane == 0) from_float(acc[m], y[(m0 + m) * N + n]);
        }
    }
}

}  // namespace

hipError_t launch_w4_quant(const void *w, int64_t N, int64_t K, void *codes, void *scales,
                           bool e8m0, hipStream_t stream) {
    const int64_t units = N * ((K + 127) / 128);
    const int64_t blocks = (units + 3) / 4, most = (int64_t)1 << 20;
    auto *kernel = e8m0 ? w4_quant_kernel<true> : w4_quant_kernel<false>;
    kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(
        static_cast<const uint16_t *>(w), N, K, static_cast<uint8_t *>(codes), scales);
    return hipGetLastError();
}

hipError_t launch_w4_matvec(const void *x, int64_t ldx, const void *codes, const void *scales,
                            bool e8m0, const int32_t *offsets, int64_t E, int64_t R, int64_t N,
                            int64_t K, void *y, bool bf16_out, hipStream_t stream) {
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)E);
    auto go = [&](auto out, auto *kernel) {
        using Out = decltype(out);
        kernel<<<grid, 256, 0, stream>>>(static_cast<const Bf16 *>(x), ldx,
                                         static_cast<const uint8_t *>(codes), scales, offsets, R,
                                         N, K, static_cast<Out *>(y));
    };
    if (bf16_out)
        go(Bf16{}, e8m0 ? w4_matvec_kernel<true, Bf16> : w4_matvec_kernel<false, Bf16>);
    else
        go(float{}, e8m0 ? w4_matvec_kernel<true, float> : w4_matvec_kernel<false, float>);
    return hipGetLastError();
}

}  // namespace fp8blk

// Backward side of a gated feed-forward block: the gradient of a = act(g) u
// from a checkpoint of [g | u] (E4M3 with 1x128 scales, or bf16),
//   dg = da u act'(g), du = da act(g),
// as it is or quantized for the products that follow it, and 8-bit
// checkpoints read back or turned for a weight gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gated.hpp"
#include "launch_ffn.hpp"
#include "vec.hpp"

namespace fp8blk {

namespace {

// Four E4M3 bytes -> fp32 (exact).
__device__ __forceinline__ void e4m3x4(uint32_t w, float (&f)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = lo[0]; f[1] = lo[1]; f[2] = hi[0]; f[3] = hi[1];
}
__device__ __forceinline__ void e4m3x8(u32x2_any w, float s, float (&f)[8]) {
    float a[4], b[4];
    e4m3x4(w.x, a);
    e4m3x4(w.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i] * s;
        f[4 + i] = b[i] * s;
    }
}

template <bool kGelu>
__device__ __forceinline__ void grad8(const float (&g)[8], const float (&u)[8],
                                      const float (&da)[8], float (&dg)[8], float (&du)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a;
        gated_grad<kGelu>(g[i], u[i], da[i], dg[i], du[i], a);
    }
}

// g and u of one row's 8 columns as they are stored (u `I` values behind g, its
// scale `GI` behind g's), and as fp32.
template <bool kH8>
struct RawH;
template <>
struct RawH<true> {
    typedef uint8_t Value;
    u32x2_any g, u;
    float sg, su;
    __device__ __forceinline__ void load(const uint8_t *h, int64_t I, const float *s, int64_t GI) {
        g = *reinterpret_cast<const u32x2_any *>(h);
        u = *reinterpret_cast<const u32x2_any *>(h + I);
        sg = s[0];
        su = s[GI];
    }
    __device__ __forceinline__ void zero() {
        g.x = g.y = u.x = u.y = 0;
        sg = su = 0.0f;
    }
    __device__ __forceinline__ void get(float (&fg)[8], float (&fu)[8]) const {
        e4m3x8(g, sg, fg);
        e4m3x8(u, su, fu);
    }
};
template <>
struct RawH<false> {
    typedef Bf16 Value;
    Raw8<Bf16> g, u;
    __device__ __forceinline__ void load(const Bf16 *h, int64_t I, const float *, int64_t) {
        load_raw<false>(h, 8, g);
        load_raw<false>(h + I, 8, u);
    }
    __device__ __forceinline__ void zero() {
        zero_raw(g);
        zero_raw(u);
    }
    __device__ __forceinline__ void get(float (&fg)[8], float (&fu)[8]) const {
        unpack(g, fg);
        unpack(u, fu);
    }
};

// Row by row: 16 lanes to a row's 128 columns, 8 to a lane.  Bound by HBM: 4096
// x 2048 from E4M3 to bf16 15 us (4.6 TB/s), 8192 x 2048 to 1x128 26 us (3.9).
template <class Da, bool kH8, bool kGelu, bool kPow2>
__global__ __launch_bounds__(256) void gated_grad_rows_kernel(GatedGrad p) {
    const int64_t GI = p.I >> 7;
    const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const bool live = id < p.M * GI;
    const int64_t row = live ? id / GI : p.M - 1, gb = live ? id % GI : 0;
    const int64_t col = 128 * gb + 8 * (threadIdx.x & 15);
    Raw8<Da> da_raw;
    RawH<kH8> h_raw;
    load_raw<false>(static_cast<const Da *>(p.da) + row * p.ld_da + col, 8, da_raw);
    h_raw.load(static_cast<const typename RawH<kH8>::Value *>(p.h) + row * p.ld_h + col, p.I,
               p.h_scales + row * 2 * GI + gb, GI);
    float da[8], g[8], u[8], dg[8], du[8];
    unpack(da_raw, da);
    h_raw.get(g, u);
    grad8<kGelu>(g, u, da, dg, du);
    if (p.dh && live) {
        const Span s{(int)col, 0, 8};
        if (p.dh_bf16) {
            store_span(static_cast<Bf16 *>(p.dh) + row * 2 * p.I, s, dg);
            store_span(static_cast<Bf16 *>(p.dh) + (row * 2 + 1) * p.I, s, du);
        } else {
            store_span(static_cast<float *>(p.dh) + row * 2 * p.I, s, dg);
            store_span(static_cast<float *>(p.dh) + (row * 2 + 1) * p.I, s, du);
        }
    }
    if (p.q) {
        put_quantized(dg, live, kPow2, p.q + row * 2 * p.I + col, p.scales + row * 2 * GI + gb);
        put_quantized(du, live, kPow2, p.q + (row * 2 + 1) * p.I + col,
                      p.scales + (row * 2 + 1) * GI + gb);
    }
}

// Eight rows (tokens) of one column, quantized over the 128 rows that 16 lanes
// hold, to `d` of the transposed output (the first `count` of them, which may
// be none) and the group's scale.
template <bool kPow2>
__device__ __forceinline__ void put_turned(const float (&f)[8], uint8_t *d, float *scale,
                                           int count) {
    float s;
    const uint2 v = quantize_group(f, true, kPow2, s);
    if (count >= 8) {
        u32x2_any w;
        w.x = v.x;
        w.y = v.y;
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2_any *>(d));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) d[i] = (uint8_t)((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))) & 0xFF);
    }
    if ((threadIdx.x & 15) == 0) *scale = s;
}

// The gradient for the products that follow: a tile of 128 rows and 128
// columns (of g and of u), computed and quantized 1x128 by rows, 8 columns of
// four rows to a thread.  For the groups along the other direction a, dg and du
// go through one FP32 tile in LDS in turn and are read with a lane holding 8
// rows of 4 columns; dg and du wait in registers (64 values, no more fit beside
// the loads).
// 16-byte chunk c of row r is at c ^ (r / 8): the 16 lanes that read 8 rows
// each at one column are on different banks.
// 4096 x 2048 from E4M3 with all three outputs: 23-28 us, 2.7-3.4 TB/s, from
// bf16 29 us (3.2).  Bound by vector operations, about 65 for each value of a,
// which a CU's two tiles run nearly in step with their loads and stores.  With
// the gradient computed again for the columns, from what was loaded, 93
// operations: 25-30 us and 35.
constexpr int kTile = 128;
constexpr int kTileThreads = 512;

// Where column c of row r of a tile of T sits: 16-byte chunks of T.
template <class T>
__device__ __forceinline__ int tile_at(int r, int c) {
    constexpr int per = 16 / (int)sizeof(T), chunks = kTile / per;
    return (((c / per) ^ ((r >> 3) & (chunks - 1))) * per) + c % per;
}

__device__ __forceinline__ void read4(const float *p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
__device__ __forceinline__ void read4(const uint8_t *p, float (&f)[4]) {
    e4m3x4(*reinterpret_cast<const uint32_t *>(p), f);
}

__device__ __forceinline__ void write8(float (&row)[kTile], int r, int c, const float (&f)[8]) {
    *reinterpret_cast<float4 *>(&row[tile_at<float>(r, c)]) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(&row[tile_at<float>(r, c + 4)]) =
        make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void write8(uint8_t (&row)[kTile], int r, int c, u32x2_any v) {
    *reinterpret_cast<uint2 *>(&row[tile_at<uint8_t>(r, c)]) = make_uint2(v.x, v.y);
}

template <class Da, bool kH8, bool kGelu, bool kPow2>
__global__ __launch_bounds__(kTileThreads) void gated_grad_tile_kernel(GatedGrad p) {
    __shared__ __attribute__((aligned(16))) float tile[kTile][kTile];
    const int64_t GI = p.I >> 7;
    const int64_t m0 = (int64_t)blockIdx.x / GI * kTile, gb = (int64_t)blockIdx.x % GI;
    const int t = threadIdx.x;
    const int c8 = 8 * (t & 15), lr = t >> 4;
    const int64_t row0 = m0 + lr, col = kTile * gb + c8;
    const int rows = (int)min(p.M - row0, (int64_t)kTile);  // of this thread's, from its first
    Raw8<Da> da_raw[4];
    RawH<kH8> h_raw[4];
    // addresses go from row to row by sums: products of 64 bits take as long as
    // a tenth of the rest
    // (a row past the end is the last one again, and zeroed below)
    {
        const int64_t at = min(row0, p.M - 1);
        const Da *da = static_cast<const Da *>(p.da) + at * p.ld_da + col;
        const typename RawH<kH8>::Value *h =
            static_cast<const typename RawH<kH8>::Value *>(p.h) + at * p.ld_h + col;
        const float *s = p.h_scales + at * 2 * GI + gb;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            load_raw<false>(da, 8, da_raw[v]);
            h_raw[v].load(h, p.I, s, GI);
            const bool next = 32 * (v + 1) < rows;
            da += next ? 32 * p.ld_da : 0;
            h += next ? 32 * p.ld_h : 0;
            s += next ? 64 * GI : 0;
        }
    }
    uint8_t *q = p.q + row0 * 2 * p.I + col;
    float *scale = p.scales + row0 * 2 * GI + gb;
    float dg[4][8], du[4][8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int r = 32 * v + lr;
        const bool live = 32 * v < rows;
        if (!live) {  // zeros: their gradient is zero
            zero_raw(da_raw[v]);
            h_raw[v].zero();
        }
        float da[8], g[8], u[8], a[8];
        unpack(da_raw[v], da);
        h_raw[v].get(g, u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gated_grad<kGelu>(g[i], u[i], da[i], dg[v][i], du[v][i], a[i]);
        write8(tile[r], r, c8, a);
        if (p.q) {
            put_quantized(dg[v], live, kPow2, q, scale);
            put_quantized(du[v], live, kPow2, q + p.I, scale + GI);
            q += 64 * p.I;
            scale += 64 * GI;
        }
    }
    const int r0 = 8 * (t & 15), c0 = 4 * (t >> 4);
    const int count = (int)min(p.M - (m0 + r0), (int64_t)8);
    const int64_t GM = (p.M + 127) >> 7;
    // the tile's columns to rows k, k + 1, .. of a transposed output
    auto turn = [&](uint8_t *out, float *scales, int64_t k) {
        float f[4][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[4];
            read4(&tile[r0 + i][tile_at<float>(r0 + i, c0)], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j][i] = x[j];
        }
        uint8_t *d = out + k * p.M + m0 + r0;
        float *s = scales + k * GM + (m0 >> 7);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            put_turned<kPow2>(f[j], d, s, count);
            d += p.M;
            s += GM;
        }
    };
    auto hold = [&](const float (&f)[4][8]) {
        __syncthreads();  // the columns before are read
#pragma unroll
        for (int v = 0; v < 4; ++v) write8(tile[32 * v + lr], 32 * v + lr, c8, f[v]);
        __syncthreads();
    };
    const int64_t k = kTile * gb + c0;
    __syncthreads();
    if (p.a_t) turn(p.a_t, p.a_scales_t, k);
    if (!p.q_t) return;
    hold(dg);
    turn(p.q_t, p.scales_t, k);
    hold(du);
    turn(p.q_t, p.scales_t, p.I + k);
}

template <class Da, bool kH8, bool kGelu, bool kPow2>
hipError_t launch_grad(const GatedGrad &p, hipStream_t stream) {
    const int64_t GI = p.I >> 7;
    if (p.q_t || p.a_t) {
        const int64_t tiles = (p.M + kTile - 1) / kTile * GI;
        hipLaunchKernelGGL((gated_grad_tile_kernel<Da, kH8, kGelu, kPow2>), dim3((unsigned)tiles),
                           dim3(kTileThreads), 0, stream, p);
    } else {
        const int64_t blocks = (p.M * GI + 15) / 16;
        hipLaunchKernelGGL((gated_grad_rows_kernel<Da, kH8, kGelu, kPow2>), dim3((unsigned)blocks),
                           dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

template <class Da, bool kH8>
hipError_t launch_grad(const GatedGrad &p, hipStream_t stream) {
    if (p.gelu)
        return p.pow2 ? launch_grad<Da, kH8, true, true>(p, stream)
                      : launch_grad<Da, kH8, true, false>(p, stream);
    return p.pow2 ? launch_grad<Da, kH8, false, true>(p, stream)
                  : launch_grad<Da, kH8, false, false>(p, stream);
}

// ---- 8-bit checkpoints ----

// x = code scale: 8 values a thread, a row's last vector its last 8 values.
// Bound by HBM: 8192 x 4096 to bf16 21 us (4.7 TB/s).
template <class T, bool kNarrow>
__global__ __launch_bounds__(256) void dequant_act_kernel(const uint8_t *__restrict__ q,
                                                          const float *__restrict__ scales,
                                                          int64_t M, int64_t K, int64_t vecs,
                                                          T *__restrict__ x) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= M * vecs) return;
    const int64_t row = id / vecs, v = id % vecs;
    const Span s = row_span<kNarrow>(v, K);
    const uint8_t *src = q + row * K + s.col;
    u32x2_any w;
    if (!kNarrow) {
        w = *reinterpret_cast<const u32x2_any *>(src);
    } else {
        w.x = w.y = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w.x |= (uint32_t)src[min(i, s.hi - 1)] << (8 * i);
            w.y |= (uint32_t)src[min(i + 4, s.hi - 1)] << (8 * i);
        }
    }
    // the vector's own values are of one group
    const float scale = scales[row * ((K + 127) >> 7) + (v >> 4)];
    float f[8];
    e4m3x8(w, scale, f);
    store_span(x + row * K, s, f);
}

// 1x128 groups (128 columns of a row) to 128x1 groups (128 rows of a column),
// written transposed: 128 x 128 tiles through LDS, as in the gradient's, by
// workgroups that load the next tile while they work on one.  4096 x 7168:
// 15-20 us, 2.9-4.0 TB/s (the quantizer from bf16 to the same bytes 22); bound by
// HBM and the 128-byte pieces of a row of the result that a tile has.
constexpr int kTurnGrid = 2 * 256;  // two to a CU (three and four: 10% and 3% slower)

template <bool kPow2>
__global__ __launch_bounds__(kTileThreads) void requant_act_t_kernel(
    const uint8_t *__restrict__ q, const float *__restrict__ scales, int64_t M, int64_t K,
    int64_t GK, int64_t tiles, uint8_t *__restrict__ q_t, float *__restrict__ scales_t) {
    __shared__ __attribute__((aligned(16))) uint8_t tile[kTile][kTile];
    __shared__ float ss[kTile];
    const int t = threadIdx.x;
    const int lr = t >> 4, c = 8 * (t & 15);
    const int64_t GM = (M + 127) >> 7;
    u32x2_any raw[4];
    float scale = 0.0f;
    auto fetch = [&](int64_t id) {
        const int64_t m0 = id / GK * kTile, kb = id % GK, col = kTile * kb + c;
        const int rows = (int)min(M - m0, (int64_t)kTile);
        const uint8_t *src = q + (m0 + lr) * K + col;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            u32x2_any w;
            w.x = w.y = 0;
            if (32 * v + lr < rows) {
                if (col + 8 <= K) {
                    w = *reinterpret_cast<const u32x2_any *>(src);
                } else {
                    for (int i = 0; i < 8; ++i)
                        if (col + i < K) {
                            if (i < 4)
                                w.x |= (uint32_t)src[i] << (8 * i);
                            else
                                w.y |= (uint32_t)src[i] << (8 * (i - 4));
                        }
                }
            }
            raw[v] = w;
            src += 32 * K;
        }
        scale = t < rows ? scales[(m0 + t) * GK + kb] : 0.0f;
    };
    int64_t id = blockIdx.x;
    fetch(id);
    for (; id < tiles; id += gridDim.x) {
        const int64_t m0 = id / GK * kTile, kb = id % GK;
#pragma unroll
        for (int v = 0; v < 4; ++v) write8(tile[32 * v + lr], 32 * v + lr, c, raw[v]);
        if (t < kTile) ss[t] = scale;
        __syncthreads();
        if (id + gridDim.x < tiles) fetch(id + gridDim.x);
        const int r0 = 8 * (t & 15), c0 = 4 * (t >> 4);
        float f[4][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + i;
            float x[4];
            read4(&tile[r][tile_at<uint8_t>(r, c0)], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j][i] = x[j] * ss[r];
        }
        const int64_t k = kTile * kb + c0;
        const int count = (int)min(M - (m0 + r0), (int64_t)8);
        uint8_t *d = q_t + k * M + m0 + r0;
        float *s = scales_t + k * GM + (m0 >> 7);
        // 16 lanes share a column: whole groups of lanes leave together
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k + j < K) put_turned<kPow2>(f[j], d, s, count);
            d += M;
            s += GM;
        }
        __syncthreads();  // the tile's place is the next one's
    }
}

}  // namespace

hipError_t launch_gated_grad(const GatedGrad &p, hipStream_t stream) {
    if (p.da_bf16)
        return p.h_scales ? launch_grad<Bf16, true>(p, stream)
                          : launch_grad<Bf16, false>(p, stream);
    return p.h_scales ? launch_grad<float, true>(p, stream) : launch_grad<float, false>(p, stream);
}

hipError_t launch_dequant_act(const void *q, const float *scales, int64_t M, int64_t K, void *x,
                              bool bf16_out, hipStream_t stream) {
    const int64_t vecs = (K + 7) / 8;
    const dim3 grid((unsigned)((M * vecs + 255) / 256));
    const uint8_t *src = static_cast<const uint8_t *>(q);
    auto go = [&](auto kernel, auto *dst) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, src, scales, M, K, vecs, dst);
        return hipGetLastError();
    };
    if (bf16_out)
        return K < 8 ? go(dequant_act_kernel<Bf16, true>, static_cast<Bf16 *>(x))
                     : go(dequant_act_kernel<Bf16, false>, static_cast<Bf16 *>(x));
    return K < 8 ? go(dequant_act_kernel<float, true>, static_cast<float *>(x))
                 : go(dequant_act_kernel<float, false>, static_cast<float *>(x));
}

hipError_t launch_requant_act_t(const void *q, const float *scales, int64_t M, int64_t K,
                                void *q_t, float *scales_t, bool pow2, hipStream_t stream) {
    const int64_t GK = (K + 127) / 128, tiles = (M + kTile - 1) / kTile * GK;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < kTurnGrid ? tiles : kTurnGrid)),
                           dim3(kTileThreads), 0, stream, static_cast<const uint8_t *>(q), scales,
                           M, K, GK, tiles, static_cast<uint8_t *>(q_t), scales_t);
    };
    if (pow2)
        go(requant_act_t_kernel<true>);
    else
        go(requant_act_t_kernel<false>);
    return hipGetLastError();
}

}  // namespace fp8blk

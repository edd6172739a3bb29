// 4-bit weights (OCP E2M1 with group scales): the offline quantizer and the
// products of a few rows with them, dense and per expert (gfx950).
//
// A product of M <= 16 rows reads N K / 2 bytes of codes and N K / 32 bytes
// of scales and does at most 64 flops per byte of them: its floor is the
// weights' bytes at the rate of a large copy.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
//
// y = x w^T on the bf16 matrix cores: an E2M1 value times a power of two is a
// bf16 number, a product of two bf16 numbers is exact in FP32, and the sums
// are the matrix core's FP32 ones.  v_cvt_scalef32_pk_bf16_fp4 unpacks two
// codes an instruction and applies the E8M0 scale on the way (half a lane
// operation a weight, where the card's vector units have about three to
// spare at the rate the weights arrive); an FP32 group scale multiplies the
// group's 128-deep partial sum instead.
//
// A workgroup is eight waves.  A wave holds its part of x, kPer 128-channel
// blocks of 16 rows, in registers for the whole call and streams code rows
// past it, 16 bytes a lane: lane (c, q) of 16 x 4 reads channels 32 q ..
// 32 q + 31 of a block of the row of column c, which is the operand of four
// 16x16x32 products (each takes eight channels of every q, x alike).  The
// codes of the next tile are asked for, into the registers of the present
// ones, as soon as these are unpacked.  `split` waves share a column tile
// along K and their sums meet in LDS.
//
// Few rows leave matrix columns unused, so kSegs of 1, 2 or 4 puts as many
// stretches of K side by side: the 16 operand rows are then 16 / kSegs rows
// of x in kSegs stretches, the 16 columns 16 / kSegs output columns in the
// same stretches, and of the 16 x 16 products only those of equal stretches
// are added up.  That makes tiles of 8 or 4 columns, for outputs too narrow
// to fill the card with tiles of 16.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kBlockK = 128;  // channels of a block
constexpr int kHeld = 8;      // blocks of 16 rows of x a wave holds

struct W4Shape {
    int64_t ldx, N, K;
    int R, E;
    int blocks;      // 128-channel blocks of a row, the last one perhaps in part
    int split_log;   // log2 of the waves that share a column tile
    int chunks;      // passes over K of all stretches
    int steps;       // column tiles of a wave
    bool bf16_out;
};

__device__ __forceinline__ bf16x8 weights8(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The `which`-th expert that has rows, its first row and the end of its rows
// (r0 >= r1 where there are fewer): offsets clamped to [0, R], no range
// starting before an earlier one ends.  A grid over the experts with rows
// instead of all: one token sends 8 rows to 8 of 256 experts.
__device__ __forceinline__ void busy_expert(const int32_t *offsets, int E, int R, int which,
                                            int &e, int &r0, int &r1) {
    const int lane = threadIdx.x & 63;
    int low = 0, seen = 0;  // end of the ranges so far, experts with rows so far
    e = r0 = r1 = 0;
    for (int first = 0; first < E; first += 64) {
        const int i = first + lane;
        const int start = min(offsets[min(i, E)], R), stop = min(offsets[min(i + 1, E)], R);
        int up = max(start, low);  // running maximum: where expert i's rows begin
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(up, d);
            if (lane >= d) up = max(up, v);
        }
        const uint64_t busy = __ballot(i < E && stop > up);
        const int here = __popcll(busy);
        if (which < seen + here) {
            const uint64_t below = busy & ((1ull << lane) - 1);
            const uint64_t mine =
                __ballot(((busy >> lane) & 1) && __popcll(below) == which - seen);
            const int src = __ffsll((unsigned long long)mine) - 1;
            e = first + src;
            r0 = __shfl(up, src);
            r1 = __shfl(stop, src);
            break;
        }
        seen += here;
        low = max(__shfl(up, 63), low);
    }
    e = __builtin_amdgcn_readfirstlane(e);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
}

// The low 16 bytes of v moved down by `bytes` (0 to 16), zeros from above.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int bytes) {
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    const int s = 8 * (bytes & 7);
    const uint64_t low = lo >> s | hi << 1 << (63 - s), high = hi >> s;
    lo = bytes < 8 ? low : bytes < 16 ? high : 0;
    hi = bytes < 8 ? high : 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

template <bool kE8m0, int kSegs, int kPer, bool kChunked>
__global__ __launch_bounds__(64 * kWaves) void w4_matvec_kernel(
    const Bf16 *__restrict__ x, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const int32_t *__restrict__ offsets, W4Shape p,
    void *__restrict__ y) {
    constexpr int kCols = 16 / kSegs;  // rows of x and output columns of a tile
    __shared__ float sums[2][kWaves][16][17];
    __shared__ __attribute__((aligned(16))) uint16_t end_of_x[kCols][kBlockK];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = lane & 15, q = lane >> 4;
    const int col = c % kCols, seg = c / kCols;
    const int split = 1 << p.split_log, tiles_each = kWaves >> p.split_log;
    const int along = wave & (split - 1), sub = wave >> p.split_log;
    int e = 0, r0 = 0, r1 = p.R;
    if (offsets) busy_expert(offsets, p.E, p.R, blockIdx.y, e, r0, r1);

    const int64_t row_bytes = (p.K + 1) / 2, all_rows = p.E * p.N;
    const int groups = kE8m0 ? (int)((p.K + 31) / 32) : p.blocks;
    const int stretches = split * kSegs;
    const int64_t tile0 = (int64_t)blockIdx.x * p.steps * tiles_each + sub;
    const int full = (int)(p.K / kBlockK);  // whole blocks; one more, in part, if blocks > full

    for (int m0 = r0; m0 < r1; m0 += kCols) {
        const int rows = min(kCols, r1 - m0);
        const Bf16 *xrow = x + (int64_t)(m0 + min(col, rows - 1)) * p.ldx;
        bf16x8 held[kPer][4];
        u32x4 code[kPer];
        uint32_t scale[kPer];  // as loaded: E8M0 byte or FP32 bits

        // the first block of this lane's stretch in pass `chunk`
        auto first_block = [&](int chunk) {
            return (chunk * stretches + along * kSegs + seg) * kPer;
        };
        // x is zero past K: the block that K ends in is brought to LDS with
        // its zeros, once for these rows.
        if (p.blocks > full) {
            for (int i = threadIdx.x; i < kCols * kBlockK; i += 64 * kWaves) {
                const int m = i / kBlockK, k = i % kBlockK;
                const int64_t at = (int64_t)full * kBlockK + k;
                end_of_x[m][k] =
                    m < rows && at < p.K ? x[(int64_t)(m0 + m) * p.ldx + at].bits : (uint16_t)0;
            }
            __syncthreads();
        }
        // Lanes of rows past the last stay zero and idle: with one row the
        // loads touch a sixteenth of the lanes.
        auto load_x = [&](int chunk) {
            const int b0 = first_block(chunk);
            const Bf16 *from = xrow + (int64_t)b0 * kBlockK + 32 * q;
#pragma unroll
            for (int b = 0; b < kPer; ++b) {
                u32x4 v[4] = {};
                if (b0 + b < full && col < rows) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = *reinterpret_cast<const u32x4_any *>(from + b * kBlockK + 8 * i);
                }
                if (p.blocks > full && b0 + b == full) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = *reinterpret_cast<const u32x4 *>(&end_of_x[col][32 * q + 8 * i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) held[b][i] = __builtin_bit_cast(bf16x8, v[i]);
            }
        };
        // Where this lane's blocks of a tile begin.  Blocks past the row's last
        // one read that again (x is zero there); what lies past the end of a
        // row meets zeros of x as well.  Only the last block of the last rows
        // could reach past the end of all codes: there the 16 bytes begin
        // `back` bytes earlier, to be moved down before they are used.
        const uint8_t *from;
        const void *scale_from;
        int end, back, last, last_group;
        auto place = [&](int64_t tile, int chunk) {
            const int b0 = first_block(chunk);
            int64_t n = tile * kCols + col;
            n = n < p.N ? n : p.N - 1;  // a column past the end is not stored
            const int64_t row = e * p.N + n;
            const int64_t at = (int64_t)b0 * 64 + 16 * q;
            from = codes + row * row_bytes + at;
            last = p.blocks - 1 - b0;
            const int64_t left = (all_rows - row) * row_bytes - at - 64 * (int64_t)last;
            back = left < 16 ? 16 - (int)left : 0;
            end = 64 * last - back;
            if (kE8m0) {
                const int g = 4 * b0 + q;
                scale_from = static_cast<const uint8_t *>(scales) + row * groups + g;
                last_group = groups - 1 - g;
            } else {
                scale_from = static_cast<const float *>(scales) + row * groups + b0;
            }
        };
        auto load_weights = [&](int b) {
            code[b] = *reinterpret_cast<const u32x4_any *>(from + min(64 * b, end));
            if (kE8m0)
                scale[b] = static_cast<const uint8_t *>(scale_from)[min(4 * b, last_group)];
            else
                scale[b] = static_cast<const uint32_t *>(scale_from)[min(b, last)];
        };

        f32x4 acc = {0, 0, 0, 0};
        int buffer = 0;
        // One tile (of one pass): unpack, ask for the next one's codes, add up.
        auto products = [&](int cut, int cut_back, auto more) {
            if (__any(cut >= 0 && cut < kPer)) {
#pragma unroll
                for (int b = 0; b < kPer; ++b)
                    if (b == cut) code[b] = shift_down(code[b], cut_back);
            }
#pragma unroll
            for (int b = 0; b < kPer; ++b) {
                const float s = __uint_as_float(kE8m0 ? scale[b] << 23 : scale[b]);
                bf16x8 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = weights8(code[b][i], kE8m0 ? s : 1.0f);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (decltype(more)::value) load_weights(b);
                __builtin_amdgcn_sched_barrier(0);
                if (kE8m0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(held[b][i], w[i], acc, 0, 0,
                                                                      0);
                } else {
                    f32x4 part = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(held[b][i], w[i], part, 0,
                                                                       0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(s, part[r], acc[r]);
                }
            }
        };
        auto store = [&](int64_t tile) {
            // element (4 q + r, c) of the product: x row, output column
            float(*mine)[17] = sums[buffer][wave];
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[4 * q + r][c] = acc[r];
            __syncthreads();
            const int64_t first = tile - sub;
            for (int o = threadIdx.x; o < tiles_each * rows * kCols; o += 64 * kWaves) {
                const int which = o / (rows * kCols);
                const int m = o / kCols % rows, n = o % kCols;
                const int64_t at = (first + which) * kCols + n;
                if (at >= p.N) continue;
                float sum = 0;
                for (int w = 0; w < split; ++w)
#pragma unroll
                    for (int g = 0; g < kSegs; ++g)
                        sum += sums[buffer][which * split + w][m + g * kCols][n + g * kCols];
                const int64_t to = (int64_t)(m0 + m) * p.N + at;
                if (p.bf16_out) from_float(sum, static_cast<Bf16 *>(y)[to]);
                else static_cast<float *>(y)[to] = sum;
            }
            buffer ^= 1;
            acc = f32x4{0, 0, 0, 0};
        };

        place(tile0, 0);
#pragma unroll
        for (int b = 0; b < kPer; ++b) load_weights(b);
        load_x(0);
        const int64_t units = (int64_t)p.steps * p.chunks;
        int chunk = 0;
        int64_t tile = tile0;
        for (int64_t u = 1; u < units; ++u) {
            const int cut = back > 0 ? last : -1, cut_back = min(back, 16);
            const int64_t done = tile;
            if (kChunked) chunk = chunk + 1 < p.chunks ? chunk + 1 : 0;
            if (!kChunked || chunk == 0) tile += tiles_each;
            place(tile, chunk);
            products(cut, cut_back, std::true_type{});
            if (kChunked) load_x(chunk);
            if (!kChunked || chunk == 0) store(done);
        }
        products(back > 0 ? last : -1, min(back, 16), std::false_type{});
        store(tile);
        __syncthreads();  // the next rows begin with the first buffer again
    }
}

// Codes of fewer than 16 bytes in all (or none): the kernel above reads 16 at
// a time.  One thread a sum of at most 30 products.
template <bool kE8m0>
__global__ __launch_bounds__(256) void w4_few_codes_kernel(
    const Bf16 *__restrict__ x, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const int32_t *__restrict__ offsets, W4Shape p,
    void *__restrict__ y) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < p.R * p.N; i += gridDim.x * 256ll) {
        const int64_t m = i / p.N;
        int64_t row = i % p.N;
        if (offsets) {
            int e = 0, low = min(max(offsets[0], 0), p.R);  // the end of the ranges so far
            if (m < low) continue;
            for (; e < p.E; ++e) {
                low = max(low, min(offsets[e + 1], p.R));
                if (m < low) break;
            }
            if (e == p.E) continue;
            row += e * p.N;
        }
        float sum = 0;
        for (int64_t k = 0; k < p.K; ++k) {
            const uint32_t code = codes[row * ((p.K + 1) / 2) + k / 2] >> (4 * (k & 1));
            const float s = kE8m0 ? __uint_as_float((uint32_t)static_cast<const uint8_t *>(
                                                        scales)[row * ((p.K + 31) / 32) + k / 32]
                                                    << 23)
                                  : static_cast<const float *>(scales)[row];
            const bf16x2 w =
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code & 15, kE8m0 ? s : 1.0f, 0);
            const float value = kE8m0 ? (float)w[0] : s * (float)w[0];
            sum = __builtin_fmaf(to_float(x[m * p.ldx + k]), value, sum);
        }
        if (p.bf16_out) from_float(sum, static_cast<Bf16 *>(y)[i]);
        else static_cast<float *>(y)[i] = sum;
    }
}

// The kernel for `segs` stretches side by side of `per` blocks each (rounded
// up to one that is built; the blocks too many are read twice, times zero).
using MatvecKernel = void (*)(const Bf16 *, const uint8_t *, const void *, const int32_t *,
                              W4Shape, void *);
template <bool kE8m0>
MatvecKernel matvec_kernel(int segs, int &per, bool chunked) {
    if (chunked) return w4_matvec_kernel<kE8m0, 1, 8, true>;
    if (segs == 1) {
        if (per <= 1) return per = 1, w4_matvec_kernel<kE8m0, 1, 1, false>;
        if (per <= 2) return per = 2, w4_matvec_kernel<kE8m0, 1, 2, false>;
        if (per <= 4) return per = 4, w4_matvec_kernel<kE8m0, 1, 4, false>;
        if (per <= 6) return per = 6, w4_matvec_kernel<kE8m0, 1, 6, false>;
        if (per <= 7) return per = 7, w4_matvec_kernel<kE8m0, 1, 7, false>;
        return per = 8, w4_matvec_kernel<kE8m0, 1, 8, false>;
    }
    if (segs == 2) {
        if (per <= 1) return per = 1, w4_matvec_kernel<kE8m0, 2, 1, false>;
        if (per <= 2) return per = 2, w4_matvec_kernel<kE8m0, 2, 2, false>;
        return per = 4, w4_matvec_kernel<kE8m0, 2, 4, false>;
    }
    if (per <= 1) return per = 1, w4_matvec_kernel<kE8m0, 4, 1, false>;
    return per = 2, w4_matvec_kernel<kE8m0, 4, 2, false>;
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
    W4Shape p;
    p.ldx = ldx;
    p.N = N;
    p.K = K;
    p.R = (int)R;
    p.E = (int)E;
    p.blocks = (int)((K + kBlockK - 1) / kBlockK);
    p.bf16_out = bf16_out;
    const Bf16 *rows = static_cast<const Bf16 *>(x);
    const uint8_t *bytes = static_cast<const uint8_t *>(codes);
    if (K == 0 || E * N * ((K + 1) / 2) < 16) {
        const int64_t sums = R * N < (1 << 22) ? R * N : (1 << 22);
        auto *kernel = e8m0 ? w4_few_codes_kernel<true> : w4_few_codes_kernel<false>;
        kernel<<<(unsigned)((sums + 255) / 256), 256, 0, stream>>>(rows, bytes, scales, offsets, p,
                                                                   y);
        return hipGetLastError();
    }
    // Workgroups that can be busy: experts with rows times column tiles.
    // Stretches of K side by side (kSegs) and waves along K (split) both make
    // more and narrower tiles; they are taken as far as the card needs them.
    const int64_t active = offsets ? (E < R ? E : R) : 1;
    const int64_t want = 256;
    int segs = 1, split_log = 0;
    while ((1 << split_log) * kHeld < p.blocks && (1 << split_log) < kWaves) ++split_log;
    const bool chunked = p.blocks > kHeld * kWaves;
    auto groups = [&] {
        const int64_t tiles = (N + 16 / segs - 1) / (16 / segs), each = kWaves >> split_log;
        return (tiles + each - 1) / each * active;
    };
    while (groups() < want && (1 << split_log) < kWaves && (1 << split_log) < p.blocks)
        ++split_log;
    while (!chunked && groups() < want && segs < 4 && R <= 16 / (2 * segs) &&
           (segs << split_log) < p.blocks)
        segs *= 2;
    const int stretches = segs << split_log;
    p.split_log = split_log;
    int per = chunked ? kHeld : (p.blocks + stretches - 1) / stretches;
    const MatvecKernel kernel =
        e8m0 ? matvec_kernel<true>(segs, per, chunked) : matvec_kernel<false>(segs, per, chunked);
    p.chunks = (p.blocks + stretches * per - 1) / (stretches * per);
    const int64_t total = groups() / active;  // workgroups of an expert at one step each
    p.steps = 1;
    const int64_t target = offsets ? 1024 : 512;
    if (total * active > target) p.steps = (int)((total * active + target - 1) / target);
    const dim3 grid((unsigned)((total + p.steps - 1) / p.steps), (unsigned)active);
    kernel<<<grid, 64 * kWaves, 0, stream>>>(rows, bytes, scales, offsets, p, y);
    return hipGetLastError();
}

}  // namespace fp8blk

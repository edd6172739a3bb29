// 4-bit weights (OCP E2M1 with group scales): the offline quantizer and the
// products of a few rows with them, dense and per expert (gfx950).
//
// A product of M <= 16 rows reads N K / 2 bytes of codes and N K / 32 bytes
// of scales and does at most 64 flops per byte of them: its floor is the
// weights' bytes at the rate of a large copy.  More rows (of one expert) take a
// pass over its weights for each 16, most of them from HBM again: 64 rows by
// 7168 x 7168 read 42 MB for 29 and take 43 us (16 rows 13), 512 rows over 32
// experts of 4096 x 7168 847 MB for 511 and 227 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "launch_moe.hpp"
#include "vec.hpp"

namespace fp8blk {

namespace {

// ---- quantizer (offline) ---------------------------------------------------
//
// Run once for a model's weights: 2-byte loads and 1-byte stores a lane, 4096 x
// 7168 in 64 us (fp32 scales) and 56 us (E8M0), 1.2 and 1.3 TB/s.

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
        // maxima of bits keep NaN; 16 lanes: 32 channels
        float amax = __uint_as_float(row16_max_bits(max(magnitude(a), magnitude(b))));
        float qa = 0, qb = 0;
        if (kE8m0) {
            // smallest E with 6 * 2^E >= amax: amax = (1 + f) 2^(e - 127) and
            // 6 = 1.5 * 2^2, so E = e - 129, one more where 1 + f > 1.5
            const uint32_t bits = __float_as_uint(amax);
            int E = (int)(bits >> 23) - 129 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
            E = E < -127 ? -127 : E;
            if (bits >= 0x7F800000u) E = 128;  // E8M0's NaN
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
            amax = max_magnitude(amax, __shfl_xor(amax, 16));
            amax = max_magnitude(amax, __shfl_xor(amax, 32));
            const float s = amax / 6.0f;  // NaN or infinite with a weight that is
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
// blocks of 16 rows, in registers for the whole call and streams tiles of 16
// code rows (a stretch of 64 kPer bytes each) past it.  `split` waves share a
// column tile along K and their sums meet in LDS.
//
// A tile's bytes are read with neighbouring lanes on neighbouring addresses
// and brought into operand order by a trip through the wave's own part of
// LDS: lane (c, q) of 16 x 4 takes channels 32 q .. 32 q + 31 of a block of
// row c, the operand of four 16x16x32 products (each takes eight channels of
// every q, x alike).  Read in operand order, every lane would touch a cache
// line of its own and the 64 look-ups of a load, not HBM, were the bound (128
// rows over 32 experts of 4096 x 7168, 26 of them with rows: 131 us).  The next
// tile's loads are under way while a tile is multiplied.  That case takes 93 to
// 100 us (405 MB of codes and scales, 4.0 to 4.3 TB/s); one row with 18432 x 7168
// 19 us (70 MB, 3.7 TB/s), with 2048 x 7168 6.4 us, most of it the launch and
// one trip to HBM.
//
// Few rows leave matrix columns unused, so kSegs of 1, 2 or 4 puts as many
// stretches of K side by side: the 16 operand rows are then 16 / kSegs rows
// of x in kSegs stretches, the 16 columns 16 / kSegs output columns in the
// same stretches, and of the 16 x 16 products only those of equal stretches
// are added up.  That makes tiles of 8 or 4 columns, for outputs too narrow
// to fill the card with tiles of 16.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// v moved down by `bytes` (0 to 16), zeros from above.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int bytes) {
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    const int s = 8 * (bytes & 7);
    const uint64_t low = lo >> s | hi << 1 << (63 - s), high = hi >> s;
    lo = bytes < 8 ? low : bytes < 16 ? high : 0;
    hi = bytes < 8 ? high : 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// What a wave has written to its own LDS is read by its other lanes: the
// LDS keeps a wave's order, the compiler has to as well.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// How far before `at` a read of kBytes has to begin to end with the array,
// `left` bytes from `at` (0 where it ends inside).
template <int kBytes>
__device__ __forceinline__ int end_back(int64_t left) {
    return left >= kBytes ? 0 : (int)(kBytes - left);
}

template <bool kE8m0, int kSegs, int kPer, bool kChunked>
__global__ __launch_bounds__(64 * kWaves) void w4_matvec_kernel(
    const Bf16 *__restrict__ x, const uint8_t *__restrict__ codes,
    const uint8_t *__restrict__ scales, const int32_t *__restrict__ offsets, W4Shape p,
    void *__restrict__ y) {
    constexpr int kCols = 16 / kSegs;  // rows of x and output columns of a tile
    // A tile's scales: kPer words of each of the 16 code rows (four E8M0 bytes
    // or one FP32 number per block), kScaleLoads of them a lane.
    constexpr int kScaleLoads = (16 * kPer + 63) / 64;
    __shared__ float sums[2][kWaves][16][17];
    __shared__ __attribute__((aligned(16))) uint16_t end_of_x[16][kBlockK];
    __shared__ u32x4 lds_codes[kWaves][kPer < 4 ? 4 * 64 : kPer * 64];
    __shared__ uint32_t lds_scales[kWaves][kScaleLoads * 64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane & 15, q = lane >> 4;
    const int split = 1 << p.split_log, tiles_each = kWaves >> p.split_log;
    const int along = wave & (split - 1), sub = wave >> p.split_log;
    int e = 0, r0 = 0, r1 = p.R;
    if (offsets) busy_expert(offsets, p.E, p.R, blockIdx.y, e, r0, r1);

    const int64_t row_bytes = (p.K + 1) / 2;
    const int64_t scale_bytes = kE8m0 ? (p.K + 31) / 32 : 4 * (int64_t)p.blocks;
    const uint8_t *codes_end = codes + p.E * p.N * row_bytes;
    const uint8_t *scales_end = scales + p.E * p.N * scale_bytes;
    const int stretches = split * kSegs;
    const int64_t tile0 = (int64_t)blockIdx.x * p.steps * tiles_each + sub;
    const int full = (int)(p.K / kBlockK);  // whole blocks; one more, in part, if blocks > full
    u32x4 *my_codes = lds_codes[wave];
    uint32_t *my_scales = lds_scales[wave];

    // Operand row r is output column r % kCols in stretch r / kCols.
    auto first_block = [&](int r, int chunk) {
        return (chunk * stretches + along * kSegs + r / kCols) * kPer;
    };
    // A tile begins at column tile * kCols, or as many columns before the last
    // one as it has (columns it shares with the tile before it are not stored
    // again); a matrix of fewer columns reads its last one again.
    auto first_column = [&](int64_t tile) {
        const int64_t n = tile * kCols, most = p.N > kCols ? p.N - kCols : 0;
        return n < most ? n : most;
    };

    // Byte offsets of this lane's 16 bytes of each load within a tile (K below
    // 2^24 keeps them in 32 bits), and of its scale words.  A block past the
    // row's last takes the last one's scales.
    uint32_t code_at[kPer], scale_at[kScaleLoads];
    auto scale_word = [&](int j, int chunk) {
        return min(first_block(j / kPer, chunk) + j % kPer, p.blocks - 1);
    };
    auto place = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = 64 * i + lane, r = j / (4 * kPer);
            const int n = min(r % kCols, (int)(p.N < 16 ? p.N : 16) - 1);
            code_at[i] = n * (uint32_t)row_bytes + first_block(r, chunk) * 64u + j % (4 * kPer) * 16u;
        }
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) {
            const int j = min(64 * i + lane, 16 * kPer - 1), r = j / kPer;
            const int n = min(r % kCols, (int)(p.N < 16 ? p.N : 16) - 1);
            scale_at[i] = n * (uint32_t)scale_bytes + scale_word(j, chunk) * 4u;
        }
    };
    u32x4 code[kPer];
    uint32_t scale[kScaleLoads];
    // What lies past the end of a row (and in blocks past its last one) meets
    // zeros of x, so only a read past the end of the whole array is avoided:
    // it begins earlier and is moved down before it is used.  Scales are the
    // row's own in every case: another's need not be finite.
    auto near_end = [&](int64_t tile) {
        return (e * p.N + first_column(tile) + kCols) * row_bytes + 64ll * kPer * stretches * p.chunks
                   > p.E * p.N * row_bytes;
    };
    auto load_tile = [&](int64_t tile) {
        const int64_t row = e * p.N + first_column(tile);
        const uint8_t *from = codes + row * row_bytes, *scale_from = scales + row * scale_bytes;
        if (near_end(tile)) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint8_t *at = from + code_at[i];
                code[i] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_any *>(at - end_back<16>(codes_end - at)));
            }
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const uint8_t *at = scale_from + scale_at[i];
                scale[i] =
                    *reinterpret_cast<const u32_any *>(at - end_back<4>(scales_end - at));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                code[i] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_any *>(from + code_at[i]));
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i)
                scale[i] = *reinterpret_cast<const u32_any *>(scale_from + scale_at[i]);
        }
    };
    // Of a row's last word of E8M0 bytes, those that are not the next row's.
    const uint32_t own_bytes = scale_bytes % 4 ? (1u << 8 * (scale_bytes % 4)) - 1 : ~0u;
    // Loaded registers to the wave's LDS.
    auto keep_tile = [&](int64_t tile) {
        if (near_end(tile)) {
            const int64_t row = e * p.N + first_column(tile);
            const uint8_t *from = codes + row * row_bytes, *scale_from = scales + row * scale_bytes;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                code[i] = shift_down(
                    code[i], min(end_back<16>(codes_end - (from + code_at[i])), 16));
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const int back = end_back<4>(scales_end - (scale_from + scale_at[i]));
                scale[i] = back < 4 ? scale[i] >> (8 * back) : 0;
            }
        }
        wave_order();
#pragma unroll
        for (int i = 0; i < kPer; ++i) my_codes[64 * i + lane] = code[i];
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) my_scales[64 * i + lane] = scale[i];
        wave_order();
    };

    for (int m0 = r0; m0 < r1; m0 += kCols) {
        const int rows = min(kCols, r1 - m0);
        bf16x8 held[kPer][4];

        // x is zero past K: the block that K ends in is brought to LDS with
        // its zeros, once for these rows.
        if (p.blocks > full) {
            for (int i = threadIdx.x; i < 16 * kBlockK; i += 64 * kWaves) {
                const int m = i / kBlockK, k = i % kBlockK;
                const int64_t at = (int64_t)full * kBlockK + k;
                end_of_x[m][k] =
                    m < rows && at < p.K ? x[(int64_t)(m0 + m) * p.ldx + at].bits : (uint16_t)0;
            }
            __syncthreads();
        }
        // Also read along the rows, 16 lanes to the 256 bytes of a block, and
        // turned in the wave's LDS; rows past the last are zero and not read.
        auto load_x = [&](int chunk) {
            constexpr int kAtOnce = kPer < 4 ? kPer : 4;
            const Bf16 *from[4];
            int whole[4];  // blocks to read of row 4 i + q
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * i + q, m = r % kCols, first = first_block(r, chunk);
                from[i] = x + (int64_t)(m0 + m) * p.ldx + (int64_t)first * kBlockK + 8 * c;
                whole[i] = m < rows ? full - first : 0;
            }
#pragma unroll
            for (int b0 = 0; b0 < kPer; b0 += kAtOnce) {
                u32x4 v[kAtOnce][4];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (b0 + j >= kPer) continue;
                        v[j][i] = u32x4{0, 0, 0, 0};
                        if (b0 + j < whole[i])
                            v[j][i] = *reinterpret_cast<const u32x4_any *>(from[i] +
                                                                           (b0 + j) * kBlockK);
                    }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    if (b0 + j >= kPer) continue;
                    // unit u (16 bytes) of row r at u ^ r: all rows begin on the same banks
                    wave_order();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 4 * i + q;
                        my_codes[16 * r + (c ^ r)] = v[j][i];
                    }
                    wave_order();
                    const bool last = p.blocks > full && first_block(c, chunk) + b0 + j == full;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u32x4 t = my_codes[16 * c + ((4 * q + i) ^ c)];
                        if (last)
                            t = *reinterpret_cast<const u32x4 *>(
                                &end_of_x[c % kCols][32 * q + 8 * i]);
                        held[b0 + j][i] = __builtin_bit_cast(bf16x8, t);
                    }
                }
            }
        };

        f32x4 acc = {0, 0, 0, 0};
        int buffer = 0;
        auto products = [&](int chunk) {
#pragma unroll
            for (int b = 0; b < kPer; ++b) {
                const u32x4 code = my_codes[4 * kPer * c + 4 * b + q];
                uint32_t word = my_scales[kPer * c + b];
                if (kE8m0) word &= first_block(c, chunk) + b >= p.blocks - 1 ? own_bytes : ~0u;
                const float s = __uint_as_float(kE8m0 ? (word >> (8 * q) & 0xFF) << 23 : word);
                bf16x8 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = weights8(code[i], kE8m0 ? s : 1.0f);
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
                const int64_t at = first_column(first + which) + n;
                if (at >= p.N || at < (first + which) * kCols) continue;
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

        const int64_t units = (int64_t)p.steps * p.chunks;
        int chunk = 0;
        int64_t tile = tile0;
        // (keeps these loads here: taken out of the loop over rows, where there
        // is but one pass as a rule, they were spilled one by one)
        asm volatile("" : "+s"(tile));
        place(0);
        load_tile(tile);
        load_x(0);
        for (int64_t u = 0; u < units; ++u) {
            keep_tile(tile);
            const int64_t done = tile;
            const int done_chunk = chunk;
            if (u + 1 < units) {
                if (kChunked) {
                    chunk = chunk + 1 < p.chunks ? chunk + 1 : 0;
                    place(chunk);
                }
                if (!kChunked || chunk == 0) tile += tiles_each;
                load_tile(tile);
            }
            products(done_chunk);
            if (kChunked && u + 1 < units) load_x(chunk);
            if (!kChunked || chunk == 0 || u + 1 == units) store(done);
        }
        __syncthreads();  // the next rows begin with the first buffer again
    }
}

// Codes of fewer than 16 bytes in all, or E8M0 scales of fewer than 4: the
// kernel above reads as many at a time.  One thread a sum of at most 96
// products (or of none).
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
                                  : static_cast<const float *>(scales)[row * ((p.K + 127) / 128) + k / 128];
            const bf16x2 w =
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code & 15, kE8m0 ? s : 1.0f, 0);
            const float value = kE8m0 ? (float)w[0] : s * (float)w[0];
            sum = __builtin_fmaf(to_float(x[m * p.ldx + k]), value, sum);
        }
        if (p.bf16_out) from_float(sum, static_cast<Bf16 *>(y)[i]);
        else static_cast<float *>(y)[i] = sum;
    }
}

// The kernel for `segs` stretches side by side of `per` blocks each, rounded
// up to one that is built.  What the rounding (of K to the stretches, and to a
// build) leaves over are blocks past the row's end: the next rows' codes, read
// and multiplied by zeros, 1.0 to 2 times the row's own.  Of short rows the
// caches hold most of them (7168 in two stretches a wave: 8.2 MB from HBM for
// 7.8).  6 and 7 are built because 8 in their place costs what it reads more:
// one row by 18432 x 7168 19 us with 7, 22 with 8; by 18432 x 6144 16 with 6, 22
// with 8; 128 rows over 32 experts of 4096 x 7168 76 and 90.  3 and 5 are not
// built: those rows take 4 and 6.  Rows of more than 64 blocks (K past 8192) go
// in chunks of 64 and spill: one row by 7168 x 18432 (144 blocks, 192 read)
// takes 46 us, 121 MB from HBM for 70 and 31 MB of spills written.
using MatvecKernel = void (*)(const Bf16 *, const uint8_t *, const uint8_t *, const int32_t *,
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
    const uint8_t *scale_bytes = static_cast<const uint8_t *>(scales);
    if (K == 0 || E * N * ((K + 1) / 2) < 16 || E * N * ((K + 31) / 32) < 4) {
        const int64_t sums = R * N < (1 << 22) ? R * N : (1 << 22);
        auto *kernel = e8m0 ? w4_few_codes_kernel<true> : w4_few_codes_kernel<false>;
        kernel<<<(unsigned)((sums + 255) / 256), 256, 0, stream>>>(rows, bytes, scales, offsets, p,
                                                                   y);
        return hipGetLastError();
    }
    // Workgroups that can be busy: experts with rows times column tiles.
    // Stretches of K side by side (kSegs) and waves along K (split) both make
    // more and narrower tiles; they are taken as far as the card needs them
    // (one row: 2048 x 7168 8.2 us without, 6.6 with; 1037 x 1000 8.8 and 4.0).
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
    // Column tiles of a wave: x is read once for all of them and the next
    // tile's loads overlap the products, so dense grids stay at one workgroup a
    // CU (16 rows by 18432 x 7168: 21 us, with 512 workgroups 27, with 1024 32).
    // Experts differ in their rows and some have none, so theirs are dealt in
    // smaller pieces (128 rows over 32 experts of 4096 x 7168, 22 of them with
    // rows: 76 us with 1024 workgroups, with 512 122, with 2048 89).
    const int64_t target = offsets ? 1024 : 256;
    if (total * active > target) p.steps = (int)((total * active + target - 1) / target);
    const dim3 grid((unsigned)((total + p.steps - 1) / p.steps), (unsigned)active);
    kernel<<<grid, 64 * kWaves, 0, stream>>>(rows, bytes, scale_bytes, offsets, p, y);
    return hipGetLastError();
}

}  // namespace fp8blk

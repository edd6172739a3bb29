// Block-scaled FP8 GEMM and its grouped (MoE) variant for gfx950.
//
// What is computed (page "dssusan.co.kr qna 93378", passages on per-group
// scaling along the inner dimension K and on FP8-in / BF16-or-FP32-out GEMMs;
// page "kailasan.com recruit 147436", Figure 7 (b): partial sums are scaled
// and added into FP32 registers at a fixed K interval):
//   C[m][n] = sum_kb sa[m][kb] * sw[n/128][kb] * P_kb[m][n],
//   P_kb[m][n] = sum_{k in [128 kb, 128 kb + 128)} a[m][k] * w[n][k].
//
// On CDNA4 one V_MFMA_F32_16X16X128_F8F6F4 instruction computes P_kb for a
// 16x16 output tile inside the matrix core (exact FP8 products; measured on
// gfx950: each aligned group of 8 products is summed to 14 significant bits,
// truncated, and the groups are added in FP32 -- tests/test_mfma_accum_gpu.py),
// so the promotion interval is one instruction: the MFMA runs with a zero
// accumulator and the result is folded into FP32 accumulators in VGPRs with
// one FMA by sa*sw.  No copy to other registers is needed: the MFMA result
// already lands in the register file the FMAs read.
//
// Structure of one workgroup tile (BM x BN, K stepped 128 at a time):
//   - A (BM x 128 bytes) and W (BN x 128 bytes) tiles plus the weight
//     scales of the K block are staged in LDS by direct global->LDS copies
//     (weights with the nontemporal cache policy), issued one or more blocks
//     ahead of the MFMAs that use them (see tile_mainloop).  The tile's
//     activation scales are fetched eight K blocks at a time into a separate
//     double buffer.
//   - LDS rows are 128 bytes; 16-byte chunk j of row r is stored at chunk
//     j ^ key(r), so the MFMA operand reads (16 rows x 32 bytes per lane
//     group) are bank-conflict free.
//   - Waves are arranged (BM/WM) x (BN/WN); each owns a WM x WN sub-tile of
//     (WM/16) x (WN/16) MFMA tiles and their FP32 accumulators.
//   - blockIdx is remapped so that each XCD (hardware dispatches consecutive
//     workgroups round-robin over the 8 XCDs, each with its own L2) works on
//     a contiguous, compact range of output tiles.
//   - The output tile leaves through LDS in whole 128-byte lines.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "device_common.hpp"
#include "gemm_tile.hpp"
#include "launch.hpp"
#include "launch_ffn.hpp"

namespace fp8blk {

namespace {

template <class C, int OUT, bool kPow2, bool kTransW = false>
__global__ __launch_bounds__(C::kThreads) void dense_gemm_kernel(GemmParams p) {
    __shared__ TileLds<C> lds;
    const int logical = xcd_logical_tile();
    if (logical >= p.ntiles) return;
    const int per_split = p.tiles_m * p.tiles_n;
    const int ks = logical / per_split;
    const int t = logical - ks * per_split;
    // Grouped raster: runs of group_m M tiles sweep across N, so consecutive
    // logical tiles share W columns (and nearby ones share A rows).
    const int span = p.group_m * p.tiles_n;
    const int grp = t / span;
    const int first_m = grp * p.group_m;
    const int gm = min(p.tiles_m - first_m, p.group_m);
    const int in = t - grp * span;
    const int tm = first_m + in % gm;
    const int tn = in / gm;

    const int64_t row0 = (int64_t)tm * C::BM;
    const int64_t n0 = (int64_t)tn * C::BN;
    const int kb0 = ks * p.kb_per_split;
    const int kb1 = min(kb0 + p.kb_per_split, p.G);

    v4f acc[C::kTM][C::kTN];
    const TileOperands op =
        kTransW ? tile_operands_transw<C>(p.a, p.sa, p.w, p.sw, row0, p.M - row0, n0, p.N - n0,
                                          p.K, p.G, p.ldw, p.NB)
                : tile_operands<C>(p.a, p.sa, p.w, p.sw, row0, p.M - row0, n0, p.N - n0, p.K,
                                   p.G);
    const int wn = (threadIdx.x >> 6) % C::kWavesN;
    tile_mainloop<C, kPow2, kTransW>(op, p.K, p.G, kb0, kb1, (int)(n0 & 127) + wn * C::WN, lds,
                                     acc);
    // Partial sums are written and read back once, both with the
    // nontemporal policy (see splitk_reduce_kernel).
    if (OUT == kOutPartial)
        tile_store<C, kOutF32>(acc, lds, p.partial + (int64_t)ks * p.M * p.N, p.N, row0, p.M,
                               n0, p.N);
    else
        tile_store<C, OUT>(acc, lds, p.c, p.N, row0, p.M, n0, p.N);
}

// One 256-row tile of the dense GEMM at (row0, n0), full K.
template <class C, int OUT, bool kPow2, bool kTransW = false>
__device__ __forceinline__ void dense_tile(const GemmParams &p, TileLds<C> &lds, int64_t row0,
                                           int64_t n0) {
    v4f acc[C::kTM][C::kTN];
    const TileOperands op =
        kTransW ? tile_operands_transw<C>(p.a, p.sa, p.w, p.sw, row0, p.M - row0, n0, p.N - n0,
                                          p.K, p.G, p.ldw, p.NB)
                : tile_operands<C>(p.a, p.sa, p.w, p.sw, row0, p.M - row0, n0, p.N - n0, p.K,
                                   p.G);
    const int wn = (threadIdx.x >> 6) % C::kWavesN;
    tile_mainloop<C, kPow2, kTransW>(op, p.K, p.G, 0, p.G, (int)(n0 & 127) + wn * C::WN, lds,
                                     acc);
    tile_store<C, OUT>(acc, lds, p.c, p.N, row0, p.M, n0, p.N);
}

// Tile of a two-kind plan: slots [0, per1) of each XCD take its contiguous
// share of the CB tiles (columns [0, n_split)), the rest its share of the CN
// tiles (columns [n_split, N)).  The wide tiles are dispatched first; the
// LDS union holds either layout.
template <class CB, class CN, int OUT, bool kPow2, bool kTransW = false>
__device__ __forceinline__ void two_kind_tile(const GemmParams &p, TileLds<CB> &lds_b,
                                              TileLds<CN> &lds_n) {
    static_assert(CB::kThreads == CN::kThreads && CB::BM == CN::BM, "two-kind tiles");
    const int t1 = p.tiles_m * p.tn1, t2 = p.tiles_m * p.tn2;
    const int per1 = (t1 + kNumXcd - 1) / kNumXcd, per2 = (t2 + kNumXcd - 1) / kNumXcd;
    const int xcd = blockIdx.x % kNumXcd;
    const int slot = blockIdx.x / kNumXcd;
    int tm, tn;
    if (slot < per1) {
        const int t = xcd * per1 + slot;
        if (t >= t1) return;
        raster(t, p.tiles_m, p.tn1, p.group_m, tm, tn);
        dense_tile<CB, OUT, kPow2, kTransW>(p, lds_b, (int64_t)tm * CB::BM,
                                            (int64_t)tn * CB::BN);
    } else {
        const int t = xcd * per2 + (slot - per1);
        if (slot - per1 >= per2 || t >= t2) return;
        raster(t, p.tiles_m, p.tn2, p.group_m, tm, tn);
        dense_tile<CN, OUT, kPow2, kTransW>(p, lds_n, (int64_t)tm * CN::BM,
                                            p.n_split + (int64_t)tn * CN::BN);
    }
}

// Dense GEMM with two tile widths.  When 256 x 256 tiles alone would leave
// the last round of workgroups partly filled, columns [0, n_split) are
// covered by 256 x 256 tiles and [n_split, N) by 256 x 192 tiles, chosen so
// that each kind fills whole rounds (e.g. 4096 x 7168: 256 of each, one of
// each per CU instead of two 256 x 256 tiles on 192 CUs and one on the
// rest).  Each XCD takes a contiguous share of each kind, the wide tiles
// first; the LDS holds either layout.
template <int OUT, bool kPow2, bool kTransW = false>
__global__ __launch_bounds__(BigTile::kThreads) void dense_gemm_two_kind_kernel(GemmParams p) {
    __shared__ union DenseLds {
        TileLds<BigTile> big;
        TileLds<NarrowTile> narrow;
    } lds;
    two_kind_tile<BigTile, NarrowTile, OUT, kPow2, kTransW>(p, lds.big, lds.narrow);
}

// Wgrad with 128 x 256 tiles on columns [0, n_split) and 128 x 192 tiles on
// the rest (plan_row_scaled_two_kind); with power-of-two scales, 256 x 256 and
// 256 x 192 tiles.
template <class CW, class CN, int OUT, bool kPow2>
__global__ __launch_bounds__(CW::kThreads) void wgrad_two_kind_kernel(GemmParams p) {
    __shared__ union WgradLds {
        TileLds<CW> wide;
        TileLds<CN> narrow;
    } lds;
    two_kind_tile<CW, CN, OUT, kPow2>(p, lds.wide, lds.narrow);
}

// Split-K reduction: C = sum over splits in fixed order 0..S-1, then the
// output conversion.  Four elements per thread (M*N is a multiple of 128).
// The partials are loaded eight splits at a time before any is added, so
// their latencies overlap instead of adding up; only splits that exist are
// loaded (a uniform branch per load: re-reading the last split in the unused
// slots instead cost 0.8 us of a 15.7 us decode call).  The partials are
// stored and loaded with
// the nontemporal policy: on back-to-back decode-sized calls (256 x 2048 x
// 7168 over rotating operand sets) that took a call from 18.2 to 16.2 us,
// the streamed partials no longer displacing the next call's operands in the
// caches; either half alone gained at most 1.5%.
template <int OUT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float *__restrict__ partial,
                                                            void *__restrict__ c, int64_t MN,
                                                            int S) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= MN) return;
    auto load = [&](int k) {
        const v4f t =
            __builtin_nontemporal_load(reinterpret_cast<const v4f *>(partial + (int64_t)k * MN + i));
        return make_float4(t[0], t[1], t[2], t[3]);
    };
    float4 s = load(0);
    for (int k0 = 1; k0 < S; k0 += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < S) v[j] = load(k0 + j);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < S) {
                s.x += v[j].x; s.y += v[j].y; s.z += v[j].z; s.w += v[j].w;
            }
    }
    if (OUT == kOutBF16) {
        uint2 o;
        o.x = f32_to_bf16_bits(s.x) | (f32_to_bf16_bits(s.y) << 16);
        o.y = f32_to_bf16_bits(s.z) | (f32_to_bf16_bits(s.w) << 16);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(c) + i) = o;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(c) + i) = s;
    }
}

// Grouped GEMM: the tiles are found on the device (find_grouped_tile).
// kTransW: W [E][K][N] read transposed, the input gradient on the forward
// weights (see tile_operands_transw): 8192 rows over 32 experts, 2048 of 7168
// columns, 208 us at a steady clock (1.2 PFLOP/s; from idle up to 278 for some
// milliseconds), bound by the rows that fill up tiles, a tile's wait for its
// operands (matrix cores busy 38% of the time that a CU works) and two and a half
// rounds of tiles that run as three (CUs work 77% of the time).
template <class C, int OUT, bool kPow2, bool kTransW = false>
__global__ __launch_bounds__(C::kThreads) void grouped_gemm_kernel(GemmParams p) {
    __shared__ TileLds<C> lds;
    __shared__ int64_t info[4];
    find_grouped_tile<C::BM>(p.offsets, p.E, (int)p.M, p.tiles_n, info);
    const int64_t e = info[0];
    if (e < 0) return;
    const int64_t row0 = info[1], row_end = info[2];
    const int64_t n0 = info[3] * C::BN;

    const uint8_t *w = p.w + e * p.N * p.K;
    const float *sw = p.sw + e * (int64_t)p.NB * p.G;
    v4f acc[C::kTM][C::kTN];
    const TileOperands op =
        kTransW ? tile_operands_transw<C>(p.a, p.sa, w, sw, row0, row_end - row0, n0, p.N - n0,
                                          p.K, p.G, p.ldw, p.NB)
                : tile_operands<C>(p.a, p.sa, w, sw, row0, row_end - row0, n0, p.N - n0, p.K,
                                   p.G);
    const int wn = (threadIdx.x >> 6) % C::kWavesN;
    tile_mainloop<C, kPow2, kTransW>(op, p.K, p.G, 0, p.G, (int)(n0 & 127) + wn * C::WN, lds, acc);
    tile_store<C, OUT>(acc, lds, p.c, p.N, row0, row_end, n0, p.N);
}


// ---- Activation quantization fused into the GEMM ---------------------------
//
// The standalone quantizer reads 128 BF16 values per group from HBM, writes
// the FP8 bytes back, and the GEMM reads them again (page "why-be.co.kr
// as_center 36949", passage on that round trip and on fusing the FP8 cast
// with the transfer of activations from global memory).  This kernel takes
// the bf16 activations itself: each K block's bf16 A tile is copied to LDS,
// quantized there (the 1x128 rule of the standalone quantizer, with the same
// arithmetic, so the bytes and scales are identical) into the E4M3 tile the
// MFMAs read, and the scale goes straight into the promotion.  Optionally
// the workgroups of the first N tile also write the bytes and scales out.
//
// The cost moves from HBM to the VALU: every N tile quantizes its A tile
// again (N / 256 times in all), and A comes in at 2 bytes per element.  It
// pays where few N tiles share an A tile; where many do, the standalone
// quantizer plus the plain GEMM is faster.
//
// Tile 64 x 256 on 8 waves (2 x 4, wave tile 32 x 64).  Per K block each
// wave copies 8 bf16 rows (two 1 KiB copies) and a quarter of the W tile; it
// quantizes exactly the 8 rows it copied, so the bf16 tile needs no barrier.
// Pipeline: bf16 A, streamed from HBM, in three stages (copies two blocks
// ahead of their quantization, which runs one block ahead of the MFMAs); W,
// re-read by every M tile and mostly an L2 hit, in two stages (one block
// ahead); E4M3 A and its scales double buffered.
// When the tiles alone would not fill the CUs, K is split over workgroups
// as in the plain GEMM (partials in the caller's workspace, then the fixed-
// order reduction).
struct FusedCfg {
    static constexpr int BM = 64, BN = 256;
    static constexpr int kWavesM = 2, kWavesN = 4, kWaves = 8, kThreads = 512;
    static constexpr int WM = BM / kWavesM, WN = BN / kWavesN;
    static constexpr int kTM = WM / 16, kTN = WN / 16;
    static constexpr int kStagesW = 2, kStagesA = 3;
    static constexpr int kWLoads = BN / 8 / kWaves;            // 8 rows of 128 B per copy
    static constexpr int kALoads = BM * 256 / 1024 / kWaves;   // 4 rows of 256 B per copy
    static_assert(kALoads == 2, "each wave copies the 8 bf16 rows it quantizes");
    static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns in one weight-scale block");
};

struct __align__(4096) FusedLds {
    uint8_t w[FusedCfg::kStagesW][FusedCfg::BN * 128];
    uint8_t a16[FusedCfg::kStagesA][FusedCfg::BM * 256];
    uint8_t a8[2][FusedCfg::BM * 128];  // swizzled like Stage::a
    float sa[2][FusedCfg::BM];
    // weight scales in chunks of 8 K blocks, as in TileLds: buffer b holds
    // at word 8 nb + j the scale of column block nb for K block 8 c + j
    float swc[2][64];
};

template <int OUT>
__global__ __launch_bounds__(FusedCfg::kThreads) void fused_quant_gemm_kernel(GemmParams p) {
    using C = FusedCfg;
    __shared__ FusedLds L;
    const int logical = xcd_logical_tile();
    if (logical >= p.ntiles) return;
    const int per_split = p.tiles_m * p.tiles_n;
    const int ks = logical / per_split;
    int tm, tn;
    raster(logical - ks * per_split, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int64_t K = p.K;
    const int G = p.G;
    const int kb0 = ks * p.kb_per_split;
    const int kb1 = min(kb0 + p.kb_per_split, G);
    const int64_t row0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const int64_t ra = p.M - row0 < C::BM ? p.M - row0 : C::BM;
    const int64_t cw = p.N - n0 < C::BN ? p.N - n0 : C::BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / C::kWavesN, wn = wave % C::kWavesN;
    const int lr = lane & 15, lk = lane >> 4;
    const bool write_q = p.q_out != nullptr && tn == 0;

    const v4i rx = make_rsrc(p.x + row0 * K, (uint32_t)(ra * K * 2));
    const v4i rw = make_rsrc(p.w + n0 * K, (uint32_t)(cw * K));
    const int64_t nb0 = n0 >> 7, nbs = ((n0 + cw - 1) >> 7) - nb0 + 1;
    const v4i rsw = make_rsrc(p.sw + nb0 * G, (uint32_t)(nbs * G * 4));
    v4i rx0 = rx, rw0 = rw;  // empty views for blocks past the end
    rx0[2] = rw0[2] = 0;

    // W copy t of wave v fills W-stage rows 8 (v + 8 t) .. + 8 (as in
    // tile_mainloop: lane L -> physical chunk L % 8 of row L / 8, holding
    // logical chunk (L % 8) ^ key(row)).
    const uint32_t w_voff = (uint32_t)(8 * wave * K + (lane >> 3) * K +
                                       (((lane & 7) ^ ((lane >> 3) & 7) ^ (wave & 1)) << 4));
    const uint32_t w_rowstep = (uint32_t)(64 * K);
    // bf16 copy t of wave v: rows 4 (v + 8 t) + L / 16, 16-byte chunk L % 16
    // (1 KiB of the stage from byte 1024 (v + 8 t)).
    const uint32_t a_voff = (uint32_t)((4 * wave + (lane >> 4)) * 2 * K + (lane & 15) * 16);
    const uint32_t a_rowstep = (uint32_t)(32 * 2 * K);
    const uint32_t lds_w0 = lds_addr(&L.w[0][1024 * wave]);
    const uint32_t lds_a0 = lds_addr(&L.a16[0][1024 * wave]);
    const uint32_t lds_sw0 = lds_addr(&L.swc[0][0]);
    const uint32_t sw_voff = (uint32_t)((lane >> 3) * G * 4 + (lane & 7) * 4);

    // bf16 A of block k (this wave's 8 rows); the W tile of block k, and the
    // weight-scale chunk starting at block k if one does (at the split's
    // first block and every 8 blocks).  A and W of blocks past the split
    // read from empty views.  The loop's waits leave only the newest bf16
    // copies outstanding, so the chunk copies need no count of their own;
    // the prologue's wait counts the chunk that starts at the split's first
    // block.
    auto issue_a = [&](int k) {
        const bool in = k < kb1;
        const v4i &a_r = in ? rx : rx0;
        const int kc = in ? k : kb0;
        const uint32_t a_st = (uint32_t)((k % C::kStagesA) * sizeof(L.a16[0]));
#pragma unroll
        for (int t = 0; t < C::kALoads; ++t)
            copy16(a_r, a_voff + t * a_rowstep, (uint32_t)kc * 256u,
                   lds_a0 + a_st + 1024u * C::kWaves * t);
    };
    auto issue_w = [&](int k) {
        const bool in = k < kb1;
        const v4i &w_r = in ? rw : rw0;
        const int kc = in ? k : kb0;
        const uint32_t w_st = (uint32_t)((k % C::kStagesW) * sizeof(L.w[0]));
#pragma unroll
        for (int t = 0; t < C::kWLoads; ++t)
            copy16_nt(w_r, w_voff + t * w_rowstep, (uint32_t)kc * 128u,
                      lds_w0 + w_st + 1024u * C::kWaves * t);
        // (none past the split: such a copy would land in a buffer that the
        // split's last chunk may still occupy)
        if (in && (k == kb0 || (k & 7) == 0))
            copy4(rsw, sw_voff, (uint32_t)(k & ~7) * 4u,
                  lds_sw0 + (uint32_t)(((k >> 3) & 1) * sizeof(L.swc[0])));
    };

    // Quantize block kb from its bf16 stage (this wave's 8 rows) into E4M3
    // buffer kb % 2 and its scales; rows past M quantize to zero bytes.
    auto quant = [&](int kb) {
#pragma unroll
        for (int t = 0; t < C::kALoads; ++t) {
            const int r = 4 * (wave + C::kWaves * t) + (lane >> 4), j = lane & 15;
            const bool in = row0 + r < p.M;
            const uint4 v = *reinterpret_cast<const uint4 *>(
                &L.a16[kb % C::kStagesA][r * 256 + j * 16]);
            float f[8];
            unpack8(v, f);
            const float amax = row16_max(absmax8(f));
            float y[8], s;
            if (__all(!in || amax >= 0x1p-60f)) {
                s = in ? scale_fast(amax) : 1.0f;
                const float rc = 1.0f / s;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = quot_fast(f[i], s, rc);
            } else {
                const QuotientCtx qc(amax, false);
                s = qc.s;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = qc(f[i]);
            }
            if (!in) s = 0.0f;
            uint32_t lo = 0, hi = 0;
            lo = cvt_pk_e4m3<false>(y[0], y[1], lo);
            lo = cvt_pk_e4m3<true>(y[2], y[3], lo);
            hi = cvt_pk_e4m3<false>(y[4], y[5], hi);
            hi = cvt_pk_e4m3<true>(y[6], y[7], hi);
            const int chunk = (j >> 1) ^ swz_key(r);
            *reinterpret_cast<uint2 *>(&L.a8[kb & 1][r * 128 + chunk * 16 + (j & 1) * 8]) =
                make_uint2(lo, hi);
            if (j == 0) L.sa[kb & 1][r] = s;
            if (write_q && in) {
                *reinterpret_cast<uint2 *>(p.q_out + (row0 + r) * K + (int64_t)kb * 128 + 8 * j) =
                    make_uint2(lo, hi);
                if (j == 0) p.sa_out[(row0 + r) * G + kb] = s;
            }
        }
    };

    const int frag0 = lr * 128 + (((2 * lk) ^ swz_key(lr)) << 4);
    const int frag1 = lr * 128 + (((2 * lk + 1) ^ swz_key(lr)) << 4);
    const int col_off = (int)(n0 & 127) + wn * C::WN;
    v4f acc[C::kTM][C::kTN];
#pragma unroll
    for (int i = 0; i < C::kTM; ++i)
#pragma unroll
        for (int j = 0; j < C::kTN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // Block kb: W stage kb % 2, E4M3 A buffer kb % 2.  The MFMA takes the
    // weight fragment as its A operand, so lane L holds outputs n = 4 (L /
    // 16) + e, m = L % 16 of each 16 x 16 tile (see tile_mainloop).
    auto compute = [&](int kb) {
        const uint8_t *lw = L.w[kb % C::kStagesW] + wn * C::WN * 128;
        const uint8_t *la = L.a8[kb & 1] + wm * C::WM * 128;
        v8i wfr[C::kTN];
#pragma unroll
        for (int j = 0; j < C::kTN; ++j)
            wfr[j] = make_v8i(*reinterpret_cast<const uint4 *>(lw + j * 2048 + frag0),
                              *reinterpret_cast<const uint4 *>(lw + j * 2048 + frag1));
        const float swv = L.swc[(kb >> 3) & 1][(col_off >> 7) * 8 + (kb & 7)];
#pragma unroll
        for (int i = 0; i < C::kTM; ++i) {
            const v8i af = make_v8i(*reinterpret_cast<const uint4 *>(la + i * 2048 + frag0),
                                    *reinterpret_cast<const uint4 *>(la + i * 2048 + frag1));
            const float f = L.sa[kb & 1][wm * C::WM + 16 * i + lr] * swv;
            v4f pr[C::kTN];
#pragma unroll
            for (int j = 0; j < C::kTN; ++j) pr[j] = mfma_e4m3(wfr[j], af);
#pragma unroll
            for (int j = 0; j < C::kTN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(pr[j][e], f, acc[i][j][e]);
        }
    };

    // Prologue: bf16 A of block kb0, W and scales of block kb0, bf16 A of
    // blocks kb0 + 1 and kb0 + 2; block kb0's rows are quantized by the wave
    // that copied them (no barrier needed) once its two copies have landed.
    issue_a(kb0);
    issue_w(kb0);
    issue_a(kb0 + 1);
    issue_a(kb0 + 2);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::kWLoads + 1 + 2 * C::kALoads) : "memory");
    quant(kb0);
    for (int kb = kb0; kb < kb1; ++kb) {
        // Iteration kb - 1 issued W(kb), its scales, then bf16 A(kb + 2):
        // with only A(kb + 2) outstanding, W(kb) and the older A(kb + 1)
        // have landed.
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::kALoads) : "memory");
        __syncthreads();
        // W stage (kb + 1) % 2 was last read by block kb - 1 and bf16 stage
        // (kb + 3) % 3 held block kb's rows, quantized in the previous
        // iteration (every wave is past both)
        issue_w(kb + 1);
        issue_a(kb + 3);
        compute(kb);
        if (kb + 1 < kb1) quant(kb + 1);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (p.ksplit > 1)
        tile_store_buf<C, kOutF32, sizeof(L.w)>(acc, &L.w[0][0],
                                                 p.partial + (int64_t)ks * p.M * p.N, p.N, row0,
                                                 p.M, n0, p.N);
    else
        tile_store_buf<C, OUT, sizeof(L.w)>(acc, &L.w[0][0], p.c, p.N, row0, p.M, n0, p.N);
}

inline int round_up(int x, int m) { return (x + m - 1) / m * m; }

constexpr int kCUs = 256;

struct Plan {
    bool big;
    int ksplit;
    int kb_per_split;
    int tn1 = 0, tn2 = 0;  // two-kind plan (big only): 256-wide and 192-wide N tiles
};

// Two-kind plan for 256-row tiles: tn1 256-wide N tiles then tn2 192-wide
// ones, used when both kinds fill whole rounds of the CUs and the estimated
// time (a 256 x 192 tile costs ~0.85 of a 256 x 256 one: its copies are 7/8
// and its MFMAs 3/4) beats whole-width tiles.  Returns false if none does.
bool plan_two_kind(int64_t M, int64_t N, int &tn1, int &tn2) {
    const int64_t tm = (M + 255) / 256;
    const int64_t tn_big = (N + 255) / 256;
    const double base = (double)((tm * tn_big + kCUs - 1) / kCUs);
    double best = base;
    bool found = false;
    for (int64_t a = 0; a <= N / 256; ++a) {
        const int64_t rest = N - 256 * a;
        const int64_t b = (rest + 191) / 192;
        if (b == 0 || (tm * a) % kCUs != 0 || (tm * b) % kCUs != 0) continue;
        const double cost = (double)(tm * a / kCUs) + 0.85 * (double)(tm * b / kCUs);
        if (cost < best - 1e-9) {
            best = cost;
            tn1 = (int)a;
            tn2 = (int)b;
            found = true;
        }
    }
    return found;
}

// Wgrad column split: 128 x 256 tiles on columns [0, 256 a), 128 x 192
// tiles on the rest (the last one possibly ragged).  With 56 row tiles (7168
// rows) neither kind can fill whole rounds, so the split is chosen by
// modelling the dispatch: each XCD's 32 CUs take its share of wide tiles
// first, then its narrow ones, each tile going to the CU that is free first;
// a narrow tile costs kWgradNarrowCost of a wide one.  The busiest XCD (the
// first, whose shares are the largest) sets the finishing time.  A split is
// used when it finishes at least 3% before the wide tiles alone: for
// dW 7168 x 7168, a = 16 and b = 16 model at 6.46 wide-tile times against 7.
constexpr double kWgradNarrowCost = 0.82;
// The same model for the power-of-two Wgrad's 256 x 256 and 256 x 192 tiles,
// whose narrow tile costs ~0.85 of a wide one (as in plan_two_kind): for dW
// 7168 x 7168, a = 4 and b = 32 model at 3.55 wide-tile times against 4.
constexpr double kWgradPow2NarrowCost = 0.85;

// Finishing time of one XCD, in wide-tile times.  After the wide tiles, the
// 32 - rem CUs holding q of them are free at q, the rem CUs holding q + 1 at
// q + 1.  Each narrow tile goes to the CU free first, so the narrow tiles end
// level by level: all CUs of the first group at q + r, q + 2r, ..., those
// of the second at q + 1 + r, ..., merged in time order.
double xcd_finish(int64_t wide, int64_t narrow, double r) {
    constexpr int kCUsPerXcd = kCUs / kNumXcd;
    const int64_t q = wide / kCUsPerXcd, rem = wide % kCUsPerXcd;
    double end = (double)(q + (rem ? 1 : 0));
    int64_t left = narrow, k_lo = 1, k_hi = 1;
    while (left > 0) {
        const double t_lo = (double)q + (double)k_lo * r;
        const double t_hi = (double)(q + 1) + (double)k_hi * r;
        if (rem == 0 || t_lo <= t_hi) {
            left -= kCUsPerXcd - rem;
            end = t_lo > end ? t_lo : end;
            ++k_lo;
        } else {
            left -= rem;
            end = t_hi > end ? t_hi : end;
            ++k_hi;
        }
    }
    return end;
}

// CW: the wide tile, CN: the narrow one (same rows), r: the narrow tile's
// cost in wide-tile times.
template <class CW, class CN>
bool plan_row_scaled_two_kind(int64_t M, int64_t N, double r, int &tn1, int &tn2) {
    static_assert(CW::BM == CN::BM, "two-kind tiles");
    // the same shapes come back every training step (one cache per tile pair)
    thread_local int64_t last_m = -1, last_n = -1;
    thread_local int last_a = 0, last_b = 0;
    if (M == last_m && N == last_n) {
        tn1 = last_a;
        tn2 = last_b;
        return last_b > 0;
    }
    const int64_t tm = (M + CW::BM - 1) / CW::BM;
    const int64_t tn_wide = (N + CW::BN - 1) / CW::BN;
    const double base = xcd_finish((tm * tn_wide + kNumXcd - 1) / kNumXcd, 0, r);
    double best = 0.97 * base;
    int best_a = (int)tn_wide, best_b = 0;
    // a grid of at most one round of wide tiles finishes in one tile time
    // either way
    const int64_t a_end = tm * tn_wide > kCUs ? (N + CW::BN - 1) / CW::BN : 0;
    for (int64_t a = 0; a < a_end; ++a) {
        const int64_t rest = N - CW::BN * a;
        if (rest <= 0) break;
        const int64_t b = (rest + CN::BN - 1) / CN::BN;
        const double t = xcd_finish((tm * a + kNumXcd - 1) / kNumXcd,
                                    (tm * b + kNumXcd - 1) / kNumXcd, r);
        if (t < best) {
            best = t;
            best_a = (int)a;
            best_b = (int)b;
        }
    }
    last_m = M;
    last_n = N;
    last_a = tn1 = best_a;
    last_b = tn2 = best_b;
    return best_b > 0;
}

Plan plan_dense(int64_t M, int64_t N, int64_t K) {
    const int G = (int)(K / 128);
    const int64_t big_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (big_tiles >= kCUs) {
        Plan pl{true, 1, G};
        int a, b;
        if (plan_two_kind(M, N, a, b)) {
            pl.tn1 = a;
            pl.tn2 = b;
        }
        return pl;
    }
    const int64_t tiles = ((M + SmallTile::BM - 1) / SmallTile::BM) * ((N + SmallTile::BN - 1) / SmallTile::BN);
    int s = 1;
    // Split K only when the output tiles cannot fill the CUs and each split
    // keeps at least 4 K blocks.
    while (tiles * s * 2 <= kCUs && G / (s * 2) >= 4) s *= 2;
    const int per = (G + s - 1) / s;
    s = (G + per - 1) / per;
    return {false, s, per};
}

// With FP8BLK_LOG set in the environment (to anything but "" or "0"), every
// GEMM call prints the plan it launches, one line on stderr: the entry, the
// output and inner sizes, the tile shapes, the K splits and the grid.
bool plan_log_on() {
    static const bool on = [] {
        const char *v = getenv("FP8BLK_LOG");
        return v != nullptr && *v != 0 && strcmp(v, "0") != 0;
    }();
    return on;
}

}  // namespace

void log_plan(const char *entry, int64_t M, int64_t N, int64_t K, const char *tiles, int tn1,
              int tn2, int ksplit, int grid) {
    if (!plan_log_on()) return;
    if (tn2 > 0)
        fprintf(stderr,
                "fp8blk: %s M=%lld N=%lld K=%lld tiles=%s (%d + %d column tiles) ksplit=%d "
                "grid=%d\n",
                entry, (long long)M, (long long)N, (long long)K, tiles, tn1, tn2, ksplit, grid);
    else
        fprintf(stderr, "fp8blk: %s M=%lld N=%lld K=%lld tiles=%s ksplit=%d grid=%d\n", entry,
                (long long)M, (long long)N, (long long)K, tiles, ksplit, grid);
}

namespace {

// Plan of the dense GEMM family (forward and Dgrad) for the log line.
void log_dense_plan(const char *entry, const GemmParams &p, const Plan &pl) {
    if (!plan_log_on()) return;
    if (pl.big && pl.tn2 > 0) {
        const int tm = (int)((p.M + 255) / 256);
        const int grid = kNumXcd * ((tm * pl.tn1 + kNumXcd - 1) / kNumXcd +
                                    (tm * pl.tn2 + kNumXcd - 1) / kNumXcd);
        log_plan(entry, p.M, p.N, p.K, "256x256+256x192", pl.tn1, pl.tn2, 1, grid);
    } else if (pl.big) {
        const int t = (int)(((p.M + 255) / 256) * ((p.N + 255) / 256));
        log_plan(entry, p.M, p.N, p.K, "256x256", 0, 0, 1, round_up(t, kNumXcd));
    } else {
        const int t = (int)(((p.M + SmallTile::BM - 1) / SmallTile::BM) *
                            ((p.N + SmallTile::BN - 1) / SmallTile::BN));
        log_plan(entry, p.M, p.N, p.K, pl.ksplit > 1 ? "128x64 split-K + reduction" : "128x64", 0,
                 0, pl.ksplit, round_up(t * pl.ksplit, kNumXcd));
    }
}

template <class C, int OUT, bool kPow2, bool kTransW = false>
hipError_t launch_dense(const GemmParams &p0, hipStream_t stream) {
    GemmParams p = p0;
    p.tiles_m = (int)((p.M + C::BM - 1) / C::BM);
    p.tiles_n = (int)((p.N + C::BN - 1) / C::BN);
    p.ntiles = p.tiles_m * p.tiles_n * p.ksplit;
    const int grid = round_up(p.ntiles, kNumXcd);
    hipLaunchKernelGGL((dense_gemm_kernel<C, OUT, kPow2, kTransW>), dim3(grid),
                       dim3(C::kThreads), 0, stream, p);
    return hipGetLastError();
}

// Launches the planned dense GEMM for one output type and scale mode.
template <int OUT, bool kPow2>
hipError_t block_gemm(GemmParams p, const Plan &pl, void *c, hipStream_t stream) {
    if (pl.big && pl.tn2 > 0) {
        p.tiles_m = (int)((p.M + 255) / 256);
        p.tn1 = pl.tn1;
        p.tn2 = pl.tn2;
        p.n_split = (int64_t)pl.tn1 * BigTile::BN;
        const int per1 = (p.tiles_m * p.tn1 + kNumXcd - 1) / kNumXcd;
        const int per2 = (p.tiles_m * p.tn2 + kNumXcd - 1) / kNumXcd;
        const int grid = kNumXcd * (per1 + per2);
        hipLaunchKernelGGL((dense_gemm_two_kind_kernel<OUT, kPow2>), dim3(grid),
                           dim3(BigTile::kThreads), 0, stream, p);
        return hipGetLastError();
    }
    if (pl.big) return launch_dense<BigTile, OUT, kPow2>(p, stream);
    if (p.ksplit > 1) {
        hipError_t e = launch_dense<SmallTile, kOutPartial, kPow2>(p, stream);
        if (e != hipSuccess) return e;
        const int64_t MN = p.M * p.N;
        const int64_t blocks = (MN / 4 + 255) / 256;
        hipLaunchKernelGGL(splitk_reduce_kernel<OUT>, dim3((unsigned)blocks), dim3(256), 0, stream,
                           p.partial, c, MN, p.ksplit);
        return hipGetLastError();
    }
    return launch_dense<SmallTile, OUT, kPow2>(p, stream);
}

}  // namespace

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    const Plan pl = plan_dense(M, N, K);
    if (pl.ksplit <= 1) return 0;
    return (size_t)pl.ksplit * (size_t)M * (size_t)N * sizeof(float);
}

hipError_t launch_block_gemm(const void *a, const float *sa, const void *w, const float *sw,
                             void *c, bool bf16_out, int64_t M, int64_t N, int64_t K,
                             void *workspace, size_t workspace_bytes, bool pow2,
                             hipStream_t stream) {
    GemmParams p{};
    p.a = static_cast<const uint8_t *>(a);
    p.sa = sa;
    p.w = static_cast<const uint8_t *>(w);
    p.sw = sw;
    p.c = c;
    p.M = M;
    p.N = N;
    p.K = K;
    p.G = (int)(K / 128);
    p.NB = (int)(N / 128);
    p.group_m = 8;
    Plan pl = plan_dense(M, N, K);
    const size_t need = gemm_workspace_bytes(M, N, K);
    if (pl.ksplit > 1 && (workspace == nullptr || workspace_bytes < need)) pl = {false, 1, p.G};
    p.ksplit = pl.ksplit;
    p.kb_per_split = pl.kb_per_split;
    p.partial = static_cast<float *>(workspace);
    log_dense_plan(pow2 ? "block_gemm_pow2" : "block_gemm", p, pl);
    if (pow2)
        return bf16_out ? block_gemm<kOutBF16, true>(p, pl, c, stream)
                        : block_gemm<kOutF32, true>(p, pl, c, stream);
    return bf16_out ? block_gemm<kOutBF16, false>(p, pl, c, stream)
                    : block_gemm<kOutF32, false>(p, pl, c, stream);
}

namespace {

// Wgrad on the tile pair CW (wide) / CN (narrow): the two-kind plan when
// it beats wide tiles alone, else wide tiles.
template <class CW, class CN, bool kPow2>
hipError_t launch_wgrad(GemmParams &p, bool bf16_out, double narrow_cost, const char *entry,
                        const char *kinds, const char *wide, hipStream_t stream) {
    int tn1, tn2;
    if (plan_row_scaled_two_kind<CW, CN>(p.M, p.N, narrow_cost, tn1, tn2)) {
        p.tiles_m = (int)((p.M + CW::BM - 1) / CW::BM);
        p.tn1 = tn1;
        p.tn2 = tn2;
        p.n_split = (int64_t)tn1 * CW::BN;
        const int per1 = (p.tiles_m * tn1 + kNumXcd - 1) / kNumXcd;
        const int per2 = (p.tiles_m * tn2 + kNumXcd - 1) / kNumXcd;
        const dim3 grid((unsigned)(kNumXcd * (per1 + per2)));
        log_plan(entry, p.M, p.N, p.K, kinds, tn1, tn2, 1, (int)grid.x);
        if (bf16_out)
            hipLaunchKernelGGL((wgrad_two_kind_kernel<CW, CN, kOutBF16, kPow2>), grid,
                               dim3(CW::kThreads), 0, stream, p);
        else
            hipLaunchKernelGGL((wgrad_two_kind_kernel<CW, CN, kOutF32, kPow2>), grid,
                               dim3(CW::kThreads), 0, stream, p);
        return hipGetLastError();
    }
    log_plan(entry, p.M, p.N, p.K, wide, 0, 0, 1,
             round_up((int)(((p.M + CW::BM - 1) / CW::BM) * ((p.N + CW::BN - 1) / CW::BN)),
                      kNumXcd));
    return bf16_out ? launch_dense<CW, kOutBF16, kPow2>(p, stream)
                    : launch_dense<CW, kOutF32, kPow2>(p, stream);
}

}  // namespace

hipError_t launch_block_gemm_wgrad(const void *a, const float *sa, const void *b,
                                   const float *sb, void *c, bool bf16_out, int64_t M, int64_t N,
                                   int64_t K, bool pow2, hipStream_t stream) {
    GemmParams p{};
    p.a = static_cast<const uint8_t *>(a);
    p.sa = sa;
    p.w = static_cast<const uint8_t *>(b);
    p.sw = sb;
    p.c = c;
    p.M = M;
    p.N = N;
    p.K = K;
    p.G = (int)(K / 128);
    p.NB = (int)(N / 128);
    p.group_m = 8;
    p.ksplit = 1;
    p.kb_per_split = p.G;
    if (pow2)
        return launch_wgrad<WgradPow2Tile, WgradPow2NarrowTile, true>(
            p, bf16_out, kWgradPow2NarrowCost, "block_gemm_wgrad_pow2", "256x256+256x192",
            "256x256", stream);
    return launch_wgrad<WgradTile, WgradNarrowTile, false>(
        p, bf16_out, kWgradNarrowCost, "block_gemm_wgrad", "128x256+128x192", "128x256", stream);
}

namespace {

// Grouped GEMM over p's operands, W as it is or (kTransW) read transposed.
// `tile`: C's size, for the log.
template <class C, bool kTransW>
hipError_t launch_grouped(GemmParams &p, bool bf16_out, bool pow2, const char *entry,
                          const char *tile, hipStream_t stream) {
    p.G = (int)(p.K / 128);
    p.NB = (int)(p.N / 128);
    p.tiles_n = (int)((p.N + C::BN - 1) / C::BN);
    p.tiles_m = (int)((p.M + C::BM - 1) / C::BM) + p.E;  // worst-case M tiles over all experts
    p.ntiles = p.tiles_m * p.tiles_n;
    p.ksplit = 1;
    p.kb_per_split = p.G;
    const dim3 grid(round_up(p.ntiles, kNumXcd));
    log_plan(entry, p.M, p.N, p.K, tile, 0, 0, 1, (int)grid.x);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(C::kThreads), 0, stream, p);
        return hipGetLastError();
    };
    if (pow2)
        return bf16_out ? go(grouped_gemm_kernel<C, kOutBF16, true, kTransW>)
                        : go(grouped_gemm_kernel<C, kOutF32, true, kTransW>);
    return bf16_out ? go(grouped_gemm_kernel<C, kOutBF16, false, kTransW>)
                    : go(grouped_gemm_kernel<C, kOutF32, false, kTransW>);
}

}  // namespace

hipError_t launch_grouped_gemm(const void *a, const float *sa, const void *w, const float *sw,
                               const int32_t *offsets, int64_t E, int64_t T, void *c,
                               bool bf16_out, int64_t N, int64_t K, bool pow2,
                               hipStream_t stream) {
    GemmParams p{};
    p.a = static_cast<const uint8_t *>(a);
    p.sa = sa;
    p.w = static_cast<const uint8_t *>(w);
    p.sw = sw;
    p.c = c;
    p.offsets = offsets;
    p.M = T;
    p.N = N;
    p.K = K;
    p.E = (int)E;
    return launch_grouped<MidTile, false>(
        p, bf16_out, pow2, pow2 ? "block_grouped_gemm_pow2" : "block_grouped_gemm",
        "128x256 (tiles found on the device; grid sized for the worst case)", stream);
}

// Dgrad per expert: dY rows as the activations (inner dimension N), each
// expert's W read transposed from its forward layout.
//
// Tiles (us, against 128 x 256): the smallest that all run at once, 64 x 128
// (1037 rows over 10 experts, 1024 of 896 columns, 9.8 against 15.9; 1500 over
// 4, 2048 of 1024, 14.7 against 24.3; in more than a round 1024 over 4, 2048 of
// 2048, 25.8 against 24.6) or 128 x 128 (the latter 17.9; past a round 4096 over
// 16, 2048 of 1024, 33 against 26); else 64 x 256 for 64 rows an expert and less
// (2048 over 32, 4096 of 2048, 77 against 86; 256 over 32 of 7168 166 against
// 182; 1024 over those 199 against 195).
using GroupedHalfTile = TileCfg<64, 256, 2, 4, 3>;
using GroupedShortTile = TileCfg<128, 128, 2, 4, 4>;
using GroupedSmallTile = TileCfg<64, 128, 2, 4, 4>;
hipError_t launch_grouped_gemm_dgrad(const void *dy, const float *sdy, const void *w,
                                     const float *sw, const int32_t *offsets, int64_t E,
                                     int64_t T, void *dx, bool bf16_out, int64_t N, int64_t Kx,
                                     bool pow2, hipStream_t stream) {
    GemmParams p{};
    p.a = static_cast<const uint8_t *>(dy);
    p.sa = sdy;
    p.w = static_cast<const uint8_t *>(w);
    p.sw = sw;
    p.c = dx;
    p.offsets = offsets;
    p.M = T;
    p.N = Kx;
    p.K = N;
    p.ldw = Kx;
    p.E = (int)E;
    const char *entry = pow2 ? "block_grouped_gemm_dgrad_pow2" : "block_grouped_gemm_dgrad";
    // whether all tiles of this size, at most, run at once
    auto fit = [&](int rows, int cols) {
        return ((T + rows - 1) / rows + E) * ((Kx + cols - 1) / cols) <= kCUs;
    };
    if (fit(GroupedSmallTile::BM, GroupedSmallTile::BN))
        return launch_grouped<GroupedSmallTile, true>(p, bf16_out, pow2, entry,
                                                      "64x128 per expert", stream);
    if (fit(GroupedShortTile::BM, GroupedShortTile::BN))
        return launch_grouped<GroupedShortTile, true>(p, bf16_out, pow2, entry,
                                                      "128x128 per expert", stream);
    if (T <= 64 * E)
        return launch_grouped<GroupedHalfTile, true>(p, bf16_out, pow2, entry,
                                                     "64x256 per expert", stream);
    return launch_grouped<MidTile, true>(p, bf16_out, pow2, entry, "128x256 per expert", stream);
}

namespace {

// K splits of the fused GEMM: as for the plain GEMM's small tiles, doubled
// while the tiles times the splits still fit in the CUs and each split keeps
// at least 4 K blocks.
int fused_ksplit(int64_t M, int64_t N, int64_t K) {
    using C = FusedCfg;
    const int G = (int)(K / 128);
    const int64_t tiles = ((M + C::BM - 1) / C::BM) * ((N + C::BN - 1) / C::BN);
    int s = 1;
    while (tiles * s * 2 <= kCUs && G / (s * 2) >= 4) s *= 2;
    const int per = (G + s - 1) / s;
    return (G + per - 1) / per;
}

}  // namespace

size_t fused_quant_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    const int s = fused_ksplit(M, N, K);
    if (s <= 1) return 0;
    return (size_t)s * (size_t)M * (size_t)N * sizeof(float);
}

hipError_t launch_block_gemm_fused_quant(const void *x, const void *w, const float *sw, void *c,
                                         bool bf16_out, int64_t M, int64_t N, int64_t K,
                                         void *q_out, float *sa_out, void *workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
    using C = FusedCfg;
    GemmParams p{};
    p.x = static_cast<const uint16_t *>(x);
    p.w = static_cast<const uint8_t *>(w);
    p.sw = sw;
    p.c = c;
    p.q_out = static_cast<uint8_t *>(q_out);
    p.sa_out = sa_out;
    p.M = M;
    p.N = N;
    p.K = K;
    p.G = (int)(K / 128);
    p.NB = (int)(N / 128);
    p.tiles_m = (int)((M + C::BM - 1) / C::BM);
    p.tiles_n = (int)((N + C::BN - 1) / C::BN);
    int s = fused_ksplit(M, N, K);
    if (s > 1 && (workspace == nullptr || workspace_bytes < fused_quant_workspace_bytes(M, N, K)))
        s = 1;
    p.ksplit = s;
    p.kb_per_split = (p.G + s - 1) / s;
    p.partial = static_cast<float *>(workspace);
    p.ntiles = p.tiles_m * p.tiles_n * s;
    p.group_m = 8;
    const dim3 grid(round_up(p.ntiles, kNumXcd));
    log_plan("block_gemm_fused_quant", M, N, K,
             s > 1 ? "64x256 split-K + reduction" : "64x256", 0, 0, s, (int)grid.x);
    if (bf16_out)
        hipLaunchKernelGGL(fused_quant_gemm_kernel<kOutBF16>, grid, dim3(C::kThreads), 0, stream,
                           p);
    else
        hipLaunchKernelGGL(fused_quant_gemm_kernel<kOutF32>, grid, dim3(C::kThreads), 0, stream,
                           p);
    if (s > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t MN = M * N;
        const int64_t blocks = (MN / 4 + 255) / 256;
        if (bf16_out)
            hipLaunchKernelGGL(splitk_reduce_kernel<kOutBF16>, dim3((unsigned)blocks), dim3(256),
                               0, stream, p.partial, c, MN, s);
        else
            hipLaunchKernelGGL(splitk_reduce_kernel<kOutF32>, dim3((unsigned)blocks), dim3(256),
                               0, stream, p.partial, c, MN, s);
    }
    return hipGetLastError();
}

// Dgrad, dX [M][Kx] = dY [M][N] W [N][Kx]: the block GEMM with dY as the
// activations (inner dimension N) and W read transposed from its forward
// layout; the same plan as fp8_block_gemm for an M x Kx output over N
// (256 x 256 tiles, or 128 x 64 tiles with split-K for small M).
namespace {

// Launches the planned Dgrad (W read transposed) for one output type and
// scale mode: the forward GEMM's plans (see block_gemm).
template <int OUT, bool kPow2>
hipError_t dgrad_gemm(GemmParams p, const Plan &pl, void *dx, hipStream_t stream) {
    if (pl.big && pl.tn2 > 0) {
        // the forward GEMM's two tile widths
        p.tiles_m = (int)((p.M + 255) / 256);
        p.tn1 = pl.tn1;
        p.tn2 = pl.tn2;
        p.n_split = (int64_t)pl.tn1 * BigTile::BN;
        const int per1 = (p.tiles_m * p.tn1 + kNumXcd - 1) / kNumXcd;
        const int per2 = (p.tiles_m * p.tn2 + kNumXcd - 1) / kNumXcd;
        const int grid = kNumXcd * (per1 + per2);
        hipLaunchKernelGGL((dense_gemm_two_kind_kernel<OUT, kPow2, true>), dim3(grid),
                           dim3(BigTile::kThreads), 0, stream, p);
        return hipGetLastError();
    }
    if (pl.big) return launch_dense<BigTile, OUT, kPow2, true>(p, stream);
    if (p.ksplit > 1) {
        hipError_t e = launch_dense<SmallTile, kOutPartial, kPow2, true>(p, stream);
        if (e != hipSuccess) return e;
        const int64_t MN = p.M * p.N;
        const int64_t blocks = (MN / 4 + 255) / 256;
        hipLaunchKernelGGL(splitk_reduce_kernel<OUT>, dim3((unsigned)blocks), dim3(256), 0, stream,
                           p.partial, dx, MN, p.ksplit);
        return hipGetLastError();
    }
    return launch_dense<SmallTile, OUT, kPow2, true>(p, stream);
}

}  // namespace

hipError_t launch_block_gemm_dgrad(const void *dy, const float *sdy, const void *w,
                                   const float *sw, void *dx, bool bf16_out, int64_t M,
                                   int64_t N, int64_t Kx, void *workspace, size_t workspace_bytes,
                                   bool pow2, hipStream_t stream) {
    GemmParams p{};
    p.a = static_cast<const uint8_t *>(dy);
    p.sa = sdy;
    p.w = static_cast<const uint8_t *>(w);
    p.sw = sw;
    p.c = dx;
    p.M = M;
    p.N = Kx;
    p.K = N;
    p.G = (int)(N / 128);
    p.NB = (int)(Kx / 128);
    p.ldw = Kx;
    p.group_m = 8;
    Plan pl = plan_dense(M, Kx, N);
    const size_t need = gemm_workspace_bytes(M, Kx, N);
    if (pl.ksplit > 1 && (workspace == nullptr || workspace_bytes < need)) pl = {false, 1, p.G};
    p.ksplit = pl.ksplit;
    p.kb_per_split = pl.kb_per_split;
    p.partial = static_cast<float *>(workspace);
    log_dense_plan(pow2 ? "block_gemm_dgrad_pow2 (W read transposed)"
                        : "block_gemm_dgrad (W read transposed)",
                   p, pl);
    if (pow2)
        return bf16_out ? dgrad_gemm<kOutBF16, true>(p, pl, dx, stream)
                        : dgrad_gemm<kOutF32, true>(p, pl, dx, stream);
    return bf16_out ? dgrad_gemm<kOutBF16, false>(p, pl, dx, stream)
                    : dgrad_gemm<kOutF32, false>(p, pl, dx, stream);
}

}  // namespace fp8blk



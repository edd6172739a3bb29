// Norm of a block's output, gate, residual sum with its scales and norm of
// the new residual stream in one pass, and its gradient (gfx950).
//
//   forward   u = y rs1 w1,  r' = a r + b g u,  n = r' rs2 w2
//   gradient  A = dn w2,  rh = r' rs2,  D = dr' + rs2 (A - rh mean(A rh)),
//             dr = a D,  du = b g D,  B = du w1,  yh = y rs1,
//             dy = rs1 (B - yh mean(B yh)),
//             dw1 = sum_t du yh,  dw2 = sum_t dn rh,  dg = b sum_t D yh w1
//
// About 14 flops a value forward and 30 backward against 7 to 18 bytes: the
// bound is HBM.  A row stays in the registers of the threads that share it, so
// each tensor is read and written once (rows wider than kHeldForward and
// kHeldGrad are read again: forward y three times and r twice, gradient
// everything twice); a workgroup keeps the parameters of its columns over its
// rows, in registers for rows of up to 512 values and in LDS for the others,
// and has the next row's loads under way while a row's sums are waited for.
// The statistics are FP32 sums.
// 4096 rows of 7168 bf16 values that are not in the caches: forward with FP8
// result 206 MB in 50 us (4.1 TB/s; the two sums a row in series, not HBM, keep
// it from the 43 us of a copy), gradient 352 MB in 78 us and 5 us for the
// parameters' sums.  One row forward: 6 us, a launch and the chain of load, sum,
// sum, store.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch_moe.hpp"
#include "vec.hpp"

namespace fp8blk {

namespace {

constexpr int kSmallThreads = 256;  // workgroup where a row takes up to 64 threads

// Sum over the `tx` threads that share a row, in all of them, in a fixed
// order: a butterfly inside the wave and, for rows of several waves (tx =
// blockDim.x), the waves' sums from LDS.  `turn` alternates between two
// buffers, so one barrier a call is enough.
template <int kSums, bool kSmall>
__device__ __forceinline__ void row_sum(float (&v)[kSums], int tx, float *lds, int &turn) {
#pragma unroll
    for (int i = 0; i < kSums; ++i)
        for (int m = (kSmall ? tx : 64) / 2; m; m /= 2) v[i] += __shfl_xor(v[i], m);
    if (kSmall) return;
    float *part = lds + turn * 16 * kSums;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < kSums; ++i) part[(threadIdx.x >> 6) * kSums + i] = v[i];
    __syncthreads();
    // up to 16 waves: lane w takes wave w's sums
    const int w = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        v[i] = w < (int)blockDim.x / 64 ? part[w * kSums + i] : 0.0f;
#pragma unroll
        for (int m = 8; m; m /= 2) v[i] += __shfl_xor(v[i], m);
    }
}

template <typename T>
__device__ __forceinline__ const T *in_row(const void *p, int64_t row_at, const Span &s) {
    return span_at(static_cast<const T *>(p) + row_at, s);
}

// A parameter's values of a span (ones without one), zeros in columns that are
// not the span's own: the row's values are zero there, and an infinite
// parameter times them would put NaN into the sums.
template <bool kNarrow>
__device__ __forceinline__ void load_param(const void *p, bool bf16, int64_t at, const Span &s,
                                           float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    } else if (bf16) {
        Raw8<Bf16> r;
        load_raw<kNarrow>(in_row<Bf16>(p, at, s), s.hi, r);
        unpack_own(r, s, f);
    } else {
        Raw8<float> r;
        load_raw<kNarrow>(in_row<float>(p, at, s), s.hi, r);
        unpack_own(r, s, f);
    }
}

// How a kernel is built: y's and the stream's type, vectors of a row that a
// thread holds (lane, lane + tx, ...), the most threads of a workgroup, rows of
// up to 64 threads (kSmall: many to a workgroup, sums inside a wave) and rows
// of fewer than eight values.
template <typename Y_, typename S_, int kVecs_, int kThreads_, bool kSmall_, bool kNarrow_>
struct Build {
    using Y = Y_;
    using S = S_;
    static constexpr int vecs = kVecs_, threads = kThreads_;
    static constexpr bool small = kSmall_, narrow = kNarrow_;
    // Waves a SIMD should hold in the forward kernel: two workgroups of up to
    // 16 waves need eight (rows of 7168 values, 14 waves: with seven a second
    // workgroup did not fit, 57 us against 52 for 4096 rows).
    static constexpr int waves = kSmall_ || kVecs_ > 1 ? 4 : kThreads_ > 512 ? 8 : 6;
};

// Rows wider than this are not held in registers (beyond two vectors a thread
// the forward spills, beyond one the gradient).
constexpr int64_t kHeldForward = 16384, kHeldGrad = 8192;

// A parameter of a thread's columns, kept over its rows: in registers for
// short rows, in LDS (each thread its own 32 bytes a vector, no barrier) for
// the others, where two workgroups then fit a compute unit or the gradient
// stays clear of spills.
template <int kVecs, int kThreads, bool kSmall>
struct Kept {
    float f[kVecs][8];
    static constexpr int floats = 4;
    __device__ __forceinline__ explicit Kept(float4 *) {}
    __device__ __forceinline__ void put(int j, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = v[i];
    }
    __device__ __forceinline__ void get(int j, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[j][i];
    }
};
template <int kVecs, int kThreads>
struct Kept<kVecs, kThreads, false> {
    float4 *mine;
    static constexpr int floats = 8 * kThreads * kVecs;
    __device__ __forceinline__ explicit Kept(float4 *lds) : mine(lds + threadIdx.x) {}
    __device__ __forceinline__ void put(int j, const float (&v)[8]) {
        mine[2 * kThreads * j] = make_float4(v[0], v[1], v[2], v[3]);
        mine[2 * kThreads * j + kThreads] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void get(int j, float (&v)[8]) const {
        const float4 a = mine[2 * kThreads * j], b = mine[2 * kThreads * j + kThreads];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// Which row's threads these are: `member` counts workgroups, or rows' threads.
template <bool kSmall>
__device__ __forceinline__ int64_t member_of(int tx) {
    return kSmall ? blockIdx.x * (int64_t)(kSmallThreads / tx) + threadIdx.x / tx : blockIdx.x;
}

template <typename B, bool kQuant>
__global__ __launch_bounds__(B::threads, B::waves) void norm_kernel(NormArgs a, int tx,
                                                                    int64_t rows_each) {
    using Y = typename B::Y;
    using S = typename B::S;
    constexpr int kVecs = B::vecs;
    using Param = Kept<kVecs, B::threads, B::small>;
    __shared__ float lds[2 * 16];
    __shared__ float4 kept[2][Param::floats / 4];
    int turn = 0;
    const int lane = B::small ? threadIdx.x & (tx - 1) : threadIdx.x;
    const int64_t t0 = member_of<B::small>(tx) * rows_each;
    const int64_t t1 = t0 + rows_each < a.T ? t0 + rows_each : a.T;
    if (t0 >= t1) return;  // all threads of the row
    const float inv_h = 1.0f / (float)a.H;
    const int64_t per_gate = a.T / a.gate_rows, G = (a.H + kGroup - 1) / kGroup;
    const bool want_n = a.n || kQuant;

    Span span[kVecs];
    Raw8<Y> y_raw[kVecs];
    Raw8<S> r_raw[kVecs];
    auto load_row = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            load_raw<B::narrow>(in_row<Y>(a.y, t * a.ldy, span[j]), span[j].hi, y_raw[j]);
            load_raw<B::narrow>(in_row<S>(a.r, t * a.ldr, span[j]), span[j].hi, r_raw[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < kVecs; ++j) span[j] = row_span<B::narrow>(lane + j * tx, a.H);
    load_row(t0);
    Param q(kept[0]), w_pre(kept[1]);  // q = branch_scale gate w_post
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        float w[8];
        load_param<B::narrow>(want_n ? a.w_pre : nullptr, a.param_bf16, 0, span[j], w);
        w_pre.put(j, w);
    }
    int64_t gate_row = t0 / per_gate - 1, gate_end = (gate_row + 1) * per_gate;
    for (int64_t t = t0; t < t1; ++t) {
        float y[kVecs][8], s[kVecs][8];
        float sum[1] = {0};
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            unpack_own(y_raw[j], span[j], y[j]);
            unpack_own(r_raw[j], span[j], s[j]);
        }
        if (t + 1 < t1) load_row(t + 1);
        if (t == gate_end || t == t0) {
            ++gate_row;
            gate_end = (gate_row + 1) * per_gate;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float w[8], g[8];
                load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], g);
                load_param<B::narrow>(a.post ? a.w_post : nullptr, a.param_bf16, 0, span[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = a.branch_scale * g[i] * w[i];
                q.put(j, g);
            }
        }
        float rs1 = 1.0f;
        if (a.post) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(y[j][i], y[j][i], sum[0]);
            row_sum<1, B::small>(sum, tx, lds, turn);
            rs1 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
            if (a.rstd_post && lane == 0) a.rstd_post[t] = rs1;
        }
        sum[0] = 0;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w[8];
            q.get(j, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[j][i] = a.residual_scale * s[j][i] + w[i] * (y[j][i] * rs1);
                sum[0] = __builtin_fmaf(s[j][i], s[j][i], sum[0]);
            }
            store_span(static_cast<S *>(a.r_out) + t * a.H, span[j], s[j]);
        }
        if (!want_n) continue;
        row_sum<1, B::small>(sum, tx, lds, turn);
        const float rs2 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
        if (a.rstd_pre && lane == 0) a.rstd_pre[t] = rs2;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w[8];
            w_pre.get(j, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = s[j][i] * rs2 * w[i];
            if (a.n) store_span(static_cast<Y *>(a.n) + t * a.H, span[j], s[j]);
            if (kQuant) {
                float scale;
                const uint2 bytes = quantize8(s[j], group_max(s[j]), span[j].any(),
                                              a.pow2, scale);
                store_e4m3(static_cast<uint8_t *>(a.q) + t * a.H, span[j], bytes);
                if ((lane & 15) == 0 && span[j].any())
                    a.scales[t * G + (lane + (int64_t)j * tx) / 16] = scale;
            }
        }
    }
}

// Wide rows, one a workgroup: read once for y's sum, once for the new
// stream's, and once more (from L2) for the results.
template <typename Y, typename S, bool kQuant>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs a) {
    __shared__ float lds[2 * 16];
    int turn = 0;
    const float inv_h = 1.0f / (float)a.H;
    const int64_t per_gate = a.T / a.gate_rows, G = (a.H + kGroup - 1) / kGroup;
    const int vecs = (int)((a.H + 7) / 8), step = blockDim.x;
    const void *post_weights = a.post ? a.w_post : nullptr;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t gate_at = t / per_gate * a.H;
        float sum[1] = {0};
        // every thread takes every turn: the sums and 16-lane maxima need all
        auto row = [&](auto use) {
            for (int v0 = 0; v0 < vecs; v0 += step) {
                const Span span = row_span<false>(v0 + (int)threadIdx.x, a.H);
                Raw8<Y> y_raw;
                load_raw<false>(in_row<Y>(a.y, t * a.ldy, span), span.hi, y_raw);
                float y[8];
                unpack_own(y_raw, span, y);
                use(v0 + (int)threadIdx.x, span, y);
            }
        };
        float rs1 = 1.0f;
        if (a.post) {
            row([&](int, const Span &, const float(&y)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(y[i], y[i], sum[0]);
            });
            row_sum<1, false>(sum, 0, lds, turn);
            rs1 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
            if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rs1;
        }
        auto stream = [&](const Span &span, const float(&y)[8], float(&s)[8]) {
            Raw8<S> raw;
            load_raw<false>(in_row<S>(a.r, t * a.ldr, span), span.hi, raw);
            float w[8], g[8];
            load_param<false>(post_weights, a.param_bf16, 0, span, w);
            load_param<false>(a.gate, a.param_bf16, gate_at, span, g);
            unpack_own(raw, span, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = a.residual_scale * s[i] + a.branch_scale * g[i] * w[i] * (y[i] * rs1);
        };
        const bool want_n = a.n || kQuant;
        float rs2 = 1.0f;
        if (want_n) {
            sum[0] = 0;
            row([&](int, const Span &span, const float(&y)[8]) {
                float s[8];
                stream(span, y, s);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(s[i], s[i], sum[0]);
            });
            row_sum<1, false>(sum, 0, lds, turn);
            rs2 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
            if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = rs2;
        }
        row([&](int v, const Span &span, const float(&y)[8]) {
            float s[8], w[8];
            stream(span, y, s);
            store_span(static_cast<S *>(a.r_out) + t * a.H, span, s);
            if (!want_n) return;
            load_param<false>(a.w_pre, a.param_bf16, 0, span, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = s[i] * rs2 * w[i];
            if (a.n) store_span(static_cast<Y *>(a.n) + t * a.H, span, s);
            if (kQuant) {
                float scale;
                const uint2 bytes =
                    quantize8(s, group_max(s), span.any(), a.pow2, scale);
                store_e4m3(static_cast<uint8_t *>(a.q) + t * a.H, span, bytes);
                if ((threadIdx.x & 15) == 0 && span.any()) a.scales[t * G + v / 16] = scale;
            }
        });
    }
}

// ---- gradient ------------------------------------------------------------------
//
// Rows are dealt to members (a workgroup, or the tx threads of a short row)
// in runs that lie within one gate row, or that hold whole gate rows; a
// member sums its rows' parameter gradients in registers and writes one
// partial row for each, which a second kernel adds in a fixed order.
//
// Both means of a row come from one round of sums: with e = dr', q = b g w1,
//   c1 = sum A rh / H,  D = e + rs2 (A - rh c1),
//   c2 = sum q D yh / H = (sum q yh (e + rs2 A) - rs2 c1 sum q yh rh) / H.
// For wide rows a kernel of its own finds rs2 c1 and c2 of every row first
// (kGiven); the rest needs nothing of other columns, so a workgroup then takes
// a stretch of columns.
// Within a gate row, dg = b w1 sum D yh and its part of dw1 = b g sum D yh, so
// one running sum (of D yh) serves both until the gate row ends; where members
// share gate rows it is their partial row, and the factors come after the sums.
struct GradPlan {
    int64_t per_gate;   // rows of a gate row
    int64_t run;        // rows of a member
    int64_t chunks;     // members of a gate row (1 where a member holds whole ones)
    int64_t members;
};

GradPlan grad_plan(int64_t T, int64_t gate_rows, int64_t most) {
    GradPlan p;
    p.per_gate = T / gate_rows;
    const int64_t run = (T + most - 1) / most;
    if (run >= p.per_gate) {
        p.run = run / p.per_gate * p.per_gate;
        p.chunks = 1;
        p.members = (T + p.run - 1) / p.run;
    } else {
        p.run = run;
        p.chunks = (p.per_gate + run - 1) / run;
        p.members = gate_rows * p.chunks;
    }
    return p;
}

template <typename B, bool kGiven>
__global__ __launch_bounds__(B::threads) void norm_grad_kernel(NormArgs a, GradPlan p, int tx,
                                                               const float2 *given,
                                                               float *part_post, float *part_pre) {
    using Y = typename B::Y;
    using S = typename B::S;
    constexpr int kVecs = B::vecs;
    using Param = Kept<kVecs, B::threads, B::small>;
    __shared__ float lds[2 * 16 * 3];
    __shared__ float4 kept[2][Param::floats / 4];
    int turn = 0;
    const int lane = B::small ? threadIdx.x & (tx - 1) : threadIdx.x;
    const int64_t member = member_of<B::small>(tx);
    const int first_vec = kGiven ? blockIdx.y * tx : 0;
    if (member >= p.members) return;  // all threads of the row
    int64_t t0, t1;
    if (p.chunks == 1) {
        t0 = member * p.run;
        t1 = t0 + p.run < a.T ? t0 + p.run : a.T;
    } else {
        const int64_t first = member / p.chunks * p.per_gate, end = first + p.per_gate;
        t0 = first + member % p.chunks * p.run;
        t1 = t0 + p.run < end ? t0 + p.run : end;
    }
    const float inv_h = 1.0f / (float)a.H;

    Span span[kVecs];
    Raw8<Y> y_raw[kVecs], dn_raw[kVecs];
    float rs1_next = 1.0f, rs2_next = 0.0f;  // (read with the row: behind the stores they would wait for them)
    Raw8<S> r_raw[kVecs], e_raw[kVecs];
    float2 c_next = {0, 0};
    auto load_row = [&](int64_t t) {
        if (kGiven) c_next = given[t];
        if (a.dn) rs2_next = a.in_rstd_pre[t];
        if (a.post) rs1_next = a.in_rstd_post[t];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            load_raw<B::narrow>(in_row<Y>(a.y, t * a.ldy, span[j]), span[j].hi, y_raw[j]);
            if (a.dn) {
                load_raw<B::narrow>(in_row<Y>(a.dn, t * a.ld_dn, span[j]), span[j].hi, dn_raw[j]);
                load_raw<B::narrow>(in_row<S>(a.r, t * a.ldr, span[j]), span[j].hi, r_raw[j]);
            }
            if (a.dr_out)
                load_raw<B::narrow>(in_row<S>(a.dr_out, t * a.ld_dr_out, span[j]), span[j].hi,
                                    e_raw[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        span[j] = row_span<B::narrow>(first_vec + lane + j * tx, a.H);
        zero_raw(dn_raw[j]);
        zero_raw(r_raw[j]);
        zero_raw(e_raw[j]);
    }
    if (t0 < t1) load_row(t0);
    // q = b g w1, w2; sums of D yh (this gate row) and of dw2's terms; the
    // member's part of dw1 grows in its partial row, once a gate row
    Param q(kept[0]), w2(kept[1]);
    float acc[kVecs][8] = {}, acc2[kVecs][8] = {};
    const void *post_weights = a.post ? a.w_post : nullptr;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        float w[8];
        load_param<B::narrow>(a.dn ? a.w_pre : nullptr, a.param_bf16, 0, span[j], w);
        w2.put(j, w);
    }
    int64_t gate_row = 0, gate_end = 0;
    bool first_gate = true;
    auto begin_gate_row = [&](int64_t row) {
        gate_row = row;
        gate_end = (row + 1) * p.per_gate;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w1[8], g[8];
            load_param<B::narrow>(post_weights, a.param_bf16, 0, span[j], w1);
            load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = a.branch_scale * g[i] * w1[i];
            q.put(j, g);
        }
    };
    auto end_gate_row = [&] {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w[8];
            load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j][i] *= a.branch_scale;
            if (p.chunks > 1) {  // this member's only gate row
                if (a.dw_post || a.dgate) store_span(part_post + member * a.H, span[j], acc[j]);
                continue;
            }
            if (a.dw_post) {
                float *part = part_post + member * a.H, sum[8] = {};
                if (!first_gate) {
                    Raw8<float> r;
                    load_raw<B::narrow>(part + span[j].col, span[j].hi, r);
                    unpack(r, sum);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[i], acc[j][i], sum[i]);
                store_span(part, span[j], sum);
            }
            if (a.dgate) {
                load_param<B::narrow>(post_weights, a.param_bf16, 0, span[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j][i] *= w[i];
                store_span(a.dgate + gate_row * a.H, span[j], acc[j]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j][i] = 0;
        }
        first_gate = false;
    };
    if (t0 < t1) begin_gate_row(t0 / p.per_gate);
    for (int64_t t = t0; t < t1; ++t) {
        const float rs1 = rs1_next, rs2 = rs2_next;
        float c1 = c_next.x, c2 = c_next.y;
        float A[kVecs][8], rh[kVecs][8], yh[kVecs][8], e[kVecs][8];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            unpack_own(y_raw[j], span[j], yh[j]);
            unpack_own(dn_raw[j], span[j], A[j]);
            unpack_own(r_raw[j], span[j], rh[j]);
            unpack_own(e_raw[j], span[j], e[j]);
        }
        if (t + 1 < t1) load_row(t + 1);
        if (t == gate_end) {
            end_gate_row();
            begin_gate_row(gate_row + 1);
        }
        float sum[3] = {0, 0, 0};
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w[8], qv[8];
            w2.get(j, w);
            q.get(j, qv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                yh[j][i] *= rs1;
                rh[j][i] *= rs2;
                acc2[j][i] = __builtin_fmaf(A[j][i], rh[j][i], acc2[j][i]);
                A[j][i] *= w[i];
                sum[0] = __builtin_fmaf(A[j][i], rh[j][i], sum[0]);
                e[j][i] = __builtin_fmaf(rs2, A[j][i], e[j][i]);
                const float qy = qv[i] * yh[j][i];
                sum[1] = __builtin_fmaf(qy, e[j][i], sum[1]);
                sum[2] = __builtin_fmaf(qy, rh[j][i], sum[2]);
            }
        }
        if (!kGiven) {
            row_sum<3, B::small>(sum, tx, lds, turn);
            c1 = rs2 * sum[0] * inv_h;
            c2 = a.post ? (sum[1] - c1 * sum[2]) * inv_h : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float dr[8], dy[8], qv[8];
            q.get(j, qv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float D = __builtin_fmaf(-c1, rh[j][i], e[j][i]);
                dr[i] = a.residual_scale * D;
                acc[j][i] = __builtin_fmaf(D, yh[j][i], acc[j][i]);
                dy[i] = D * qv[i];
            }
            // (without the first norm y is not in dy at all, be it infinite)
            if (a.post)
#pragma unroll
                for (int i = 0; i < 8; ++i) dy[i] = rs1 * (dy[i] - yh[j][i] * c2);
            store_span(static_cast<S *>(a.dr) + t * a.H, span[j], dr);
            store_span(static_cast<Y *>(a.dy) + t * a.H, span[j], dy);
        }
    }
    end_gate_row();
    if (a.dw_pre)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) store_span(part_pre + member * a.H, span[j], acc2[j]);
}

// (rs2 c1, c2) of wide rows, one a workgroup.
template <typename Y, typename S>
__global__ __launch_bounds__(1024) void norm_grad_sums_kernel(NormArgs a, float2 *given) {
    __shared__ float lds[2 * 16 * 3];
    int turn = 0;
    const float inv_h = 1.0f / (float)a.H;
    const int64_t per_gate = a.T / a.gate_rows;
    const int vecs = (int)((a.H + 7) / 8);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float rs2 = a.dn ? a.in_rstd_pre[t] : 0.0f;
        const float rs1 = a.post ? a.in_rstd_post[t] : 1.0f;
        float sum[3] = {0, 0, 0};
        for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
            const Span span = row_span<false>(v, a.H);
            Raw8<Y> y_raw, dn_raw;
            Raw8<S> r_raw, e_raw;
            zero_raw(dn_raw);
            zero_raw(r_raw);
            zero_raw(e_raw);
            load_raw<false>(in_row<Y>(a.y, t * a.ldy, span), span.hi, y_raw);
            if (a.dn) {
                load_raw<false>(in_row<Y>(a.dn, t * a.ld_dn, span), span.hi, dn_raw);
                load_raw<false>(in_row<S>(a.r, t * a.ldr, span), span.hi, r_raw);
            }
            if (a.dr_out)
                load_raw<false>(in_row<S>(a.dr_out, t * a.ld_dr_out, span), span.hi, e_raw);
            float w1[8], w2[8], g[8], y[8], A[8], rh[8], e[8];
            load_param<false>(a.post ? a.w_post : nullptr, a.param_bf16, 0, span, w1);
            load_param<false>(a.dn ? a.w_pre : nullptr, a.param_bf16, 0, span, w2);
            load_param<false>(a.gate, a.param_bf16, t / per_gate * a.H, span, g);
            unpack_own(y_raw, span, y);
            unpack_own(dn_raw, span, A);
            unpack_own(r_raw, span, rh);
            unpack_own(e_raw, span, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                A[i] *= w2[i];
                rh[i] *= rs2;
                sum[0] = __builtin_fmaf(A[i], rh[i], sum[0]);
                e[i] = __builtin_fmaf(rs2, A[i], e[i]);
                const float qy = a.branch_scale * g[i] * w1[i] * (y[i] * rs1);
                sum[1] = __builtin_fmaf(qy, e[i], sum[1]);
                sum[2] = __builtin_fmaf(qy, rh[i], sum[2]);
            }
        }
        row_sum<3, false>(sum, 0, lds, turn);
        const float c1 = rs2 * sum[0] * inv_h;
        if (threadIdx.x == 0)
            given[t] = make_float2(c1, a.post ? (sum[1] - c1 * sum[2]) * inv_h : 0.0f);
    }
}

// Each group's `rows` partial rows added: out[group] = p * sum, and with a
// second output out2[group] = p2 * sum (p, p2 [H], ones without); with `each`
// [rows / each_rows][H] out = sum of each[row / each_rows] * row.  64 columns a
// workgroup, 16 threads a column, each every 16th row.
struct ReduceJob {
    const float *part;
    int rows, each_rows;
    int64_t groups;
    const void *each, *p, *p2;
    float *out, *out2;
};

struct ReduceJobs {
    ReduceJob job[3];
};

template <typename P>
__device__ __forceinline__ float param_at(const void *p, int64_t i) {
    return p ? to_float(static_cast<const P *>(p)[i]) : 1.0f;
}

template <typename P>
__global__ __launch_bounds__(1024) void reduce_rows_kernel(ReduceJobs jobs, int64_t H) {
    __shared__ float lds[16][64];
    const ReduceJob job = jobs.job[blockIdx.y];
    const int64_t tiles = (H + 63) / 64;
    for (int64_t i = blockIdx.x; i < job.groups * tiles; i += gridDim.x) {
        const int64_t group = i / tiles, h = i % tiles * 64 + (threadIdx.x & 63);
        const int part = threadIdx.x >> 6;
        float sum = 0;
        if (h < H) {
            const float *p = job.part + group * job.rows * H + h;
            if (job.each) {
                // row / each_rows by a product: exact, since rows are far below
                // 2^22 and row + 0.5 is half a row away from any multiple
                const float per = 1.0f / (float)job.each_rows;
                const P *each = static_cast<const P *>(job.each) + h;
#pragma unroll 8
                for (int r = part; r < job.rows; r += 16)
                    sum = __builtin_fmaf(to_float(each[(int)(((float)r + 0.5f) * per) * H]),
                                         p[r * H], sum);
            } else {
#pragma unroll 8
                for (int r = part; r < job.rows; r += 16) sum += p[r * H];
            }
        }
        lds[part][threadIdx.x & 63] = sum;
        __syncthreads();
        if (part == 0 && h < H) {
            sum = 0;
            for (int k = 0; k < 16; ++k) sum += lds[k][threadIdx.x & 63];
            job.out[group * H + h] = param_at<P>(job.p, h) * sum;
            if (job.out2)
                job.out2[group * H + h] = param_at<P>(job.p2, h) * sum;
        }
        __syncthreads();
    }
}

// How a row of H values is dealt: tx threads of kVecs vectors each.
struct RowSplit {
    bool small;
    int tx, vecs, block;
};

RowSplit row_split(int64_t H) {
    const int64_t vecs = (H + 7) / 8;
    RowSplit s;
    if (vecs <= 64) {
        s.small = true;
        s.tx = threads_per_row(vecs, 16, 64);
        s.vecs = 1;
        s.block = kSmallThreads;
        return s;
    }
    s.small = false;
    s.vecs = vecs <= 1024 ? 1 : 2;
    s.tx = s.block = (int)((((vecs + s.vecs - 1) / s.vecs) + 63) / 64 * 64);
    return s;
}

// f(Y{}, S{}) for the types at hand.
template <typename F>
void with_types(const NormArgs &a, F f) {
    if (a.y_bf16 && a.r_bf16) f(Bf16{}, Bf16{});
    else if (a.y_bf16) f(Bf16{}, float{});
    else f(float{}, float{});
}

// Members that share the rows: enough workgroups to keep the card's loads
// going, as few partial rows as that allows.  Times with the reduction, inputs
// not in the caches.  One workgroup a CU is enough for wide rows (4096 rows of
// 7168 values: 83 us, with two 86, with a half 95; 1024 rows 28, 36 and 32);
// shorter ones take two or four where there are rows enough for each (8192 rows
// of 2048 values: 57 us with one, 47 with two, 48 with four; of 1024 values 53,
// 40 and 32, with eight 38; but 1024 rows of 2048 16.1 with one, 17.6 with two).
int64_t grad_members(int64_t T, int64_t H) {
    const RowSplit s = row_split(H);
    if (s.small) return 512 * (kSmallThreads / s.tx);
    const int64_t most = H > 2048 ? 256 : H > 1024 ? 512 : 1024;
    return T / 4 < 256 ? 256 : T / 4 < most ? T / 4 : most;
}

}  // namespace

hipError_t launch_norm_residual(const NormArgs &a, hipStream_t stream) {
    const RowSplit s = row_split(a.H);
    const int64_t per = s.small ? kSmallThreads / s.tx : 1;
    int64_t blocks = (a.T + per - 1) / per;
    const int64_t most = s.small || s.block < 512 ? 2048 : 512;
    int64_t rows_each = 1;
    if (blocks > most) {
        rows_each = (a.T + most * per - 1) / (most * per);
        blocks = (a.T + rows_each * per - 1) / (rows_each * per);
    }
    with_types(a, [&](auto y, auto r) {
        using Y = decltype(y);
        using S = decltype(r);
        if (a.H > kHeldForward) {
            auto *kernel = a.q ? norm_wide_kernel<Y, S, true> : norm_wide_kernel<Y, S, false>;
            kernel<<<(unsigned)(a.T < 2048 ? a.T : 2048), 1024, 0, stream>>>(a);
            return;
        }
        auto go = [&](auto b) {
            using B = decltype(b);
            auto *kernel = a.q ? norm_kernel<B, true> : norm_kernel<B, false>;
            kernel<<<(unsigned)blocks, s.block, 0, stream>>>(a, s.tx, rows_each);
        };
        if (a.H < 8) go(Build<Y, S, 1, kSmallThreads, true, true>{});
        else if (s.small) go(Build<Y, S, 1, kSmallThreads, true, false>{});
        else if (s.vecs == 2) go(Build<Y, S, 2, 1024, false, false>{});
        else if (s.block <= 256) go(Build<Y, S, 1, 256, false, false>{});
        else if (s.block <= 512) go(Build<Y, S, 1, 512, false, false>{});
        else go(Build<Y, S, 1, 1024, false, false>{});
    });
    return hipGetLastError();
}

size_t norm_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows) {
    if (T == 0 || H == 0) return 0;
    const GradPlan p = grad_plan(T, gate_rows, grad_members(T, H));
    return ((size_t)2 * p.members * H + (H > kHeldGrad ? 2 * T : 0)) * sizeof(float);
}

hipError_t launch_norm_residual_grad(const NormArgs &a, hipStream_t stream) {
    const RowSplit s = row_split(a.H);
    const bool wide = a.H > kHeldGrad;
    GradPlan p = {1, 1, 1, 0};
    if (a.T > 0) p = grad_plan(a.T, a.gate_rows, grad_members(a.T, a.H));
    // wide rows' coefficients first: two floats a row, 16-byte aligned
    float2 *given = reinterpret_cast<float2 *>(a.workspace);
    float *part_post = a.workspace + (wide ? 2 * a.T : 0);
    float *part_pre = part_post + p.members * a.H;
    if (a.T > 0) {
        const int64_t per = s.small ? kSmallThreads / s.tx : 1;
        const unsigned blocks = (unsigned)((p.members + per - 1) / per);
        with_types(a, [&](auto y, auto r) {
            using Y = decltype(y);
            using S = decltype(r);
            auto go = [&](auto b) {
                norm_grad_kernel<decltype(b), false><<<blocks, s.block, 0, stream>>>(
                    a, p, s.tx, nullptr, part_post, part_pre);
            };
            if (wide) {
                const unsigned rows = (unsigned)(a.T < 2048 ? a.T : 2048);
                norm_grad_sums_kernel<Y, S><<<rows, 1024, 0, stream>>>(a, given);
                const dim3 grid(blocks, (unsigned)((a.H + 8 * 256 - 1) / (8 * 256)));
                norm_grad_kernel<Build<Y, S, 1, 256, false, false>, true>
                    <<<grid, 256, 0, stream>>>(a, p, 256, given, part_post, part_pre);
            } else if (a.H < 8) {
                go(Build<Y, S, 1, kSmallThreads, true, true>{});
            } else if (s.small) {
                go(Build<Y, S, 1, kSmallThreads, true, false>{});
            } else if (s.block <= 256) {
                go(Build<Y, S, 1, 256, false, false>{});
            } else if (s.block <= 512) {
                go(Build<Y, S, 1, 512, false, false>{});
            } else {
                go(Build<Y, S, 1, 1024, false, false>{});
            }
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    ReduceJobs jobs = {};
    int n = 0;
    auto add = [&](const float *part, int64_t rows, int64_t groups, const void *param,
                   float *out) -> ReduceJob & {
        jobs.job[n] = {part, (int)rows, 1, groups, nullptr, param, nullptr, out, nullptr};
        return jobs.job[n++];
    };
    const void *w_post = a.post ? a.w_post : nullptr;
    if (p.chunks == 1) {  // partial rows of dw_post; dgate is written, but for no tokens
        if (a.dw_post) add(part_post, p.members, 1, nullptr, a.dw_post);
        if (a.dgate && a.T == 0) add(part_post, 0, a.gate_rows, nullptr, a.dgate);
    } else if (a.dw_post && a.dgate && a.gate_rows == 1) {
        ReduceJob &both = add(part_post, p.members, 1, a.gate, a.dw_post);
        both.p2 = w_post;
        both.out2 = a.dgate;
    } else {
        if (a.dw_post && a.gate_rows == 1) {
            add(part_post, p.members, 1, a.gate, a.dw_post);
        } else if (a.dw_post) {
            ReduceJob &job = add(part_post, p.members, 1, nullptr, a.dw_post);
            job.each = a.gate;
            job.each_rows = (int)p.chunks;
        }
        if (a.dgate) add(part_post, p.chunks, a.gate_rows, w_post, a.dgate);
    }
    if (a.dw_pre) add(part_pre, p.members, 1, nullptr, a.dw_pre);
    if (n == 0) return hipSuccess;
    int64_t most = 1;
    for (int i = 0; i < n; ++i) most = jobs.job[i].groups > most ? jobs.job[i].groups : most;
    most *= (a.H + 63) / 64;
    const dim3 grid((unsigned)(most < (1 << 20) ? most : (1 << 20)), (unsigned)n);
    auto *kernel = a.param_bf16 ? reduce_rows_kernel<Bf16> : reduce_rows_kernel<float>;
    kernel<<<grid, 1024, 0, stream>>>(jobs, a.H);
    return hipGetLastError();
}

}  // namespace fp8blk

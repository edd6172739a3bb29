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
// bound is HBM.  A row stays in the registers of the threads that share it,
// so each tensor is read and written once; a workgroup keeps the parameters
// of its columns in registers over its rows and has the next row's loads
// under way while a row's sums are waited for.  The statistics are FP32 sums.
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
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        v[i] = 0;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) v[i] += part[w * kSums + i];
    }
}

// A parameter's values of a span (ones without one).
template <bool kNarrow>
__device__ __forceinline__ void load_param(const void *p, bool bf16, int64_t at, const Span &s,
                                           float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    } else if (bf16) {
        Raw8<Bf16> r;
        load_raw<kNarrow>(static_cast<const Bf16 *>(p) + at + s.col, s.hi, r);
        unpack(r, f);
    } else {
        Raw8<float> r;
        load_raw<kNarrow>(static_cast<const float *>(p) + at + s.col, s.hi, r);
        unpack(r, f);
    }
}

// How a kernel is built: y's and the stream's type, vectors of a row that a
// thread holds (lane, lane + tx, ...), rows of up to 64 threads (kSmall: many
// to a workgroup, sums inside a wave) and rows of fewer than eight values.
template <typename Y_, typename S_, int kVecs_, bool kSmall_, bool kNarrow_>
struct Build {
    using Y = Y_;
    using S = S_;
    static constexpr int vecs = kVecs_;
    static constexpr bool small = kSmall_, narrow = kNarrow_;
    static constexpr int threads = kSmall_ ? kSmallThreads : 1024;
};

// Which row's threads these are: `member` counts workgroups, or rows' threads.
template <bool kSmall>
__device__ __forceinline__ int64_t member_of(int tx) {
    return kSmall ? blockIdx.x * (int64_t)(kSmallThreads / tx) + threadIdx.x / tx : blockIdx.x;
}

template <typename B, bool kQuant>
__global__ __launch_bounds__(B::threads) void norm_kernel(NormArgs a, int tx, int64_t rows_each) {
    using Y = typename B::Y;
    using S = typename B::S;
    constexpr int kVecs = B::vecs;
    __shared__ float lds[2 * 16];
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
            load_raw<B::narrow>(static_cast<const Y *>(a.y) + t * a.ldy + span[j].col, span[j].hi,
                                y_raw[j]);
            load_raw<B::narrow>(static_cast<const S *>(a.r) + t * a.ldr + span[j].col, span[j].hi,
                                r_raw[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < kVecs; ++j) span[j] = row_span(lane + (int64_t)j * tx, a.H);
    load_row(t0);
    float q[kVecs][8], w_pre[kVecs][8];  // q = branch_scale gate w_post
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        load_param<B::narrow>(want_n ? a.w_pre : nullptr, a.param_bf16, 0, span[j], w_pre[j]);
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
                float w[8];
                load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], q[j]);
                load_param<B::narrow>(a.post ? a.w_post : nullptr, a.param_bf16, 0, span[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[j][i] = a.branch_scale * q[j][i] * w[i];
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
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[j][i] = a.residual_scale * s[j][i] + q[j][i] * (y[j][i] * rs1);
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
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = s[j][i] * rs2 * w_pre[j][i];
            if (a.n) store_span(static_cast<Y *>(a.n) + t * a.H, span[j], s[j]);
            if (kQuant) {
                const QuotientCtx qc(row16_max(absmax8(s[j])), a.pow2);
                store_e4m3(static_cast<uint8_t *>(a.q) + t * a.H, span[j], quant8(s[j], qc));
                if ((lane & 15) == 0 && span[j].any())
                    a.scales[t * G + (lane + (int64_t)j * tx) / 16] = qc.s;
            }
        }
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
// Within a gate row, dg = b w1 sum D yh and its part of dw1 = b g sum D yh, so
// one running sum (of D yh) serves both until the gate row ends.
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

template <typename B>
__global__ __launch_bounds__(B::threads) void norm_grad_kernel(NormArgs a, GradPlan p, int tx,
                                                               float *part_post, float *part_pre,
                                                               float *part_gate) {
    using Y = typename B::Y;
    using S = typename B::S;
    constexpr int kVecs = B::vecs;
    __shared__ float lds[2 * 16 * 3];
    int turn = 0;
    const int lane = B::small ? threadIdx.x & (tx - 1) : threadIdx.x;
    const int64_t member = member_of<B::small>(tx);
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
    auto load_row = [&](int64_t t) {
        if (a.dn) rs2_next = a.in_rstd_pre[t];
        if (a.post) rs1_next = a.in_rstd_post[t];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            load_raw<B::narrow>(static_cast<const Y *>(a.y) + t * a.ldy + span[j].col, span[j].hi,
                                y_raw[j]);
            if (a.dn) {
                load_raw<B::narrow>(static_cast<const Y *>(a.dn) + t * a.ld_dn + span[j].col,
                                    span[j].hi, dn_raw[j]);
                load_raw<B::narrow>(static_cast<const S *>(a.r) + t * a.ldr + span[j].col,
                                    span[j].hi, r_raw[j]);
            }
            if (a.dr_out)
                load_raw<B::narrow>(
                    static_cast<const S *>(a.dr_out) + t * a.ld_dr_out + span[j].col, span[j].hi,
                    e_raw[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        span[j] = row_span(lane + (int64_t)j * tx, a.H);
        zero_raw(dn_raw[j]);
        zero_raw(r_raw[j]);
        zero_raw(e_raw[j]);
    }
    if (t0 < t1) load_row(t0);
    // q = b g w1, w2; sums of D yh (this gate row) and of dw2's terms; the
    // member's part of dw1 grows in its partial row, once a gate row
    float q[kVecs][8], w2[kVecs][8];
    float acc[kVecs][8] = {}, acc2[kVecs][8] = {};
    const void *post_weights = a.post ? a.w_post : nullptr;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        load_param<B::narrow>(a.dn ? a.w_pre : nullptr, a.param_bf16, 0, span[j], w2[j]);
    int64_t gate_row = 0, gate_end = 0;
    bool first_gate = true;
    auto begin_gate_row = [&](int64_t row) {
        gate_row = row;
        gate_end = (row + 1) * p.per_gate;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w1[8];
            load_param<B::narrow>(post_weights, a.param_bf16, 0, span[j], w1);
            load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], q[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[j][i] = a.branch_scale * q[j][i] * w1[i];
        }
    };
    auto end_gate_row = [&] {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float w[8];
            load_param<B::narrow>(a.gate, a.param_bf16, gate_row * a.H, span[j], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j][i] *= a.branch_scale;
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
                store_span(p.chunks == 1 ? a.dgate + gate_row * a.H : part_gate + member * a.H,
                           span[j], acc[j]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j][i] = 0;
        }
        first_gate = false;
    };
    if (t0 < t1) begin_gate_row(t0 / p.per_gate);
    for (int64_t t = t0; t < t1; ++t) {
        const float rs1 = rs1_next, rs2 = rs2_next;
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
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                yh[j][i] *= rs1;
                rh[j][i] *= rs2;
                acc2[j][i] = __builtin_fmaf(A[j][i], rh[j][i], acc2[j][i]);
                A[j][i] *= w2[j][i];
                sum[0] = __builtin_fmaf(A[j][i], rh[j][i], sum[0]);
                e[j][i] = __builtin_fmaf(rs2, A[j][i], e[j][i]);
                const float qy = q[j][i] * yh[j][i];
                sum[1] = __builtin_fmaf(qy, e[j][i], sum[1]);
                sum[2] = __builtin_fmaf(qy, rh[j][i], sum[2]);
            }
        row_sum<3, B::small>(sum, tx, lds, turn);
        const float c1 = rs2 * sum[0] * inv_h;
        const float c2 = a.post ? (sum[1] - c1 * sum[2]) * inv_h : 0.0f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float dr[8], dy[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float D = __builtin_fmaf(-c1, rh[j][i], e[j][i]);
                dr[i] = a.residual_scale * D;
                acc[j][i] = __builtin_fmaf(D, yh[j][i], acc[j][i]);
                dy[i] = rs1 * (D * q[j][i] - yh[j][i] * c2);
            }
            store_span(static_cast<S *>(a.dr) + t * a.H, span[j], dr);
            store_span(static_cast<Y *>(a.dy) + t * a.H, span[j], dy);
        }
    }
    end_gate_row();
    if (a.dw_pre)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) store_span(part_pre + member * a.H, span[j], acc2[j]);
}

// out[group][h] = sum over the group's `rows` partial rows: 64 columns a
// workgroup, 16 threads a column, each every 16th row.
struct ReduceJob {
    const float *part;
    float *out;
    int64_t rows, groups;
};

struct ReduceJobs {
    ReduceJob job[3];
};

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
#pragma unroll 8
            for (int64_t r = part; r < job.rows; r += 16) sum += p[r * H];
        }
        lds[part][threadIdx.x & 63] = sum;
        __syncthreads();
        if (part == 0 && h < H) {
            sum = 0;
            for (int k = 0; k < 16; ++k) sum += lds[k][threadIdx.x & 63];
            job.out[group * H + h] = sum;
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
    s.vecs = 1;
    while (s.vecs * 1024 < vecs) s.vecs *= 2;
    s.tx = s.block = (int)((((vecs + s.vecs - 1) / s.vecs) + 63) / 64 * 64);
    return s;
}

// f(Build<...>{}) for the types and the split at hand.
template <typename Y, typename S, typename F>
void with_split(const RowSplit &s, int64_t H, F f) {
    if (H < 8) f(Build<Y, S, 1, true, true>{});
    else if (s.small) f(Build<Y, S, 1, true, false>{});
    else if (s.vecs == 1) f(Build<Y, S, 1, false, false>{});
    else if (s.vecs == 2) f(Build<Y, S, 2, false, false>{});
    else f(Build<Y, S, 4, false, false>{});
}

template <typename F>
void with_build(const NormArgs &a, const RowSplit &s, F f) {
    if (a.y_bf16 && a.r_bf16) with_split<Bf16, Bf16>(s, a.H, f);
    else if (a.y_bf16) with_split<Bf16, float>(s, a.H, f);
    else with_split<float, float>(s, a.H, f);
}

// Members that share the rows: enough workgroups to fill the card, as few
// partial rows as that allows.
int64_t grad_members(const RowSplit &s) {
    return s.small ? 512 * (kSmallThreads / s.tx) : s.block >= 512 ? 512 : 1024;
}

}  // namespace

hipError_t launch_norm_residual(const NormArgs &a, hipStream_t stream) {
    const RowSplit s = row_split(a.H);
    const int64_t per = s.small ? kSmallThreads / s.tx : 1;
    int64_t blocks = (a.T + per - 1) / per;
    const int64_t most = s.block >= 512 ? 512 : 2048;
    int64_t rows_each = 1;
    if (blocks > most) {
        rows_each = (a.T + most * per - 1) / (most * per);
        blocks = (a.T + rows_each * per - 1) / (rows_each * per);
    }
    with_build(a, s, [&](auto b) {
        using B = decltype(b);
        auto *kernel = a.q ? norm_kernel<B, true> : norm_kernel<B, false>;
        kernel<<<(unsigned)blocks, s.block, 0, stream>>>(a, s.tx, rows_each);
    });
    return hipGetLastError();
}

size_t norm_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows) {
    if (T == 0 || H == 0) return 0;
    const GradPlan p = grad_plan(T, gate_rows, grad_members(row_split(H)));
    return (size_t)(p.chunks > 1 ? 3 : 2) * p.members * H * sizeof(float);
}

hipError_t launch_norm_residual_grad(const NormArgs &a, hipStream_t stream) {
    const RowSplit s = row_split(a.H);
    GradPlan p = {1, 1, 1, 0};
    if (a.T > 0) p = grad_plan(a.T, a.gate_rows, grad_members(s));
    float *part_post = a.workspace, *part_pre = part_post + p.members * a.H;
    float *part_gate = part_pre + p.members * a.H;
    if (a.T > 0) {
        const int64_t per = s.small ? kSmallThreads / s.tx : 1;
        const int64_t blocks = (p.members + per - 1) / per;
        with_build(a, s, [&](auto b) {
            norm_grad_kernel<decltype(b)><<<(unsigned)blocks, s.block, 0, stream>>>(
                a, p, s.tx, part_post, part_pre, part_gate);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    ReduceJobs jobs = {};
    int n = 0;
    if (a.dw_post) jobs.job[n++] = {part_post, a.dw_post, p.members, 1};
    if (a.dw_pre) jobs.job[n++] = {part_pre, a.dw_pre, p.members, 1};
    if (a.dgate && (p.chunks > 1 || a.T == 0))
        jobs.job[n++] = {part_gate, a.dgate, a.T ? p.chunks : 0, a.gate_rows};
    if (n == 0) return hipSuccess;
    int64_t most = 1;
    for (int i = 0; i < n; ++i) most = jobs.job[i].groups > most ? jobs.job[i].groups : most;
    most *= (a.H + 63) / 64;
    const dim3 grid((unsigned)(most < (1 << 20) ? most : (1 << 20)), (unsigned)n);
    reduce_rows_kernel<<<grid, 1024, 0, stream>>>(jobs, a.H);
    return hipGetLastError();
}

}  // namespace fp8blk

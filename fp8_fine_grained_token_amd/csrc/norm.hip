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
// so each tensor is read and written once; the statistics are FP32 sums.
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

// n values of a parameter row from column 8 v on (ones without one).
__device__ __forceinline__ void load_param(const void *p, bool bf16, int64_t at, int n,
                                           float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? 1.0f : 0.0f;
    } else if (bf16) {
        load8(static_cast<const Bf16 *>(p) + at, n, f);
    } else {
        load8(static_cast<const float *>(p) + at, n, f);
    }
}

// A thread holds vectors lane, lane + tx, ... (kVecs of them) of its row.
template <typename Y, typename S, int kVecs, bool kSmall, bool kQuant>
__global__ void norm_kernel(NormArgs a, int tx, int64_t rows_each) {
    __shared__ float lds[2 * 16];
    int turn = 0;
    const int lane = kSmall ? threadIdx.x & (tx - 1) : threadIdx.x;
    const int64_t member = kSmall ? blockIdx.x * (int64_t)(kSmallThreads / tx) + threadIdx.x / tx
                                  : blockIdx.x;
    const int64_t t0 = member * rows_each;
    const float inv_h = 1.0f / (float)a.H;
    const int64_t per_gate = a.T / a.gate_rows;
    for (int64_t t = t0; t < t0 + rows_each; ++t) {
        if (t >= a.T) {
            if (kSmall) break;  // the sums stay inside a row's threads
            return;             // the whole workgroup
        }
        float y[kVecs][8], s[kVecs][8], w[8];
        float sum[1] = {0};
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
            load8(static_cast<const Y *>(a.y) + t * a.ldy + 8 * v, n, y[j]);
            load8(static_cast<const S *>(a.r) + t * a.ldr + 8 * v, n, s[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(y[j][i], y[j][i], sum[0]);
        }
        float rs1 = 1.0f;
        if (a.post) {
            row_sum<1, kSmall>(sum, tx, lds, turn);
            rs1 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
            if (a.rstd_post && lane == 0) a.rstd_post[t] = rs1;
        }
        sum[0] = 0;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
            if (a.post) {
                load_param(a.w_post, a.param_bf16, 8 * v, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[j][i] = y[j][i] * rs1 * w[i];
            }
            load_param(a.gate, a.param_bf16, t / per_gate * a.H + 8 * v, n, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[j][i] = a.residual_scale * s[j][i] + a.branch_scale * w[i] * y[j][i];
                sum[0] = __builtin_fmaf(s[j][i], s[j][i], sum[0]);
            }
            store8(static_cast<S *>(a.r_out) + t * a.H + 8 * v, n, s[j]);
        }
        if (!a.n && !kQuant) continue;
        row_sum<1, kSmall>(sum, tx, lds, turn);
        const float rs2 = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
        if (a.rstd_pre && lane == 0) a.rstd_pre[t] = rs2;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
            load_param(a.w_pre, a.param_bf16, 8 * v, n, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = s[j][i] * rs2 * w[i];
            if (a.n) store8(static_cast<Y *>(a.n) + t * a.H + 8 * v, n, s[j]);
            if (kQuant) {
                const int64_t G = (a.H + kGroup - 1) / kGroup;
                const QuotientCtx qc(row16_max(absmax8(s[j])), a.pow2);
                store_e4m3(static_cast<uint8_t *>(a.q) + t * a.H + 8 * v, n, quant8(s[j], qc));
                if ((lane & 15) == 0 && n > 0) a.scales[t * G + v / 16] = qc.s;
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
struct GradPlan {
    int64_t per_gate;   // rows of a gate row
    int64_t run;        // rows of a member
    int64_t chunks;     // members of a gate row (1 where a member holds whole ones)
    int64_t members;
};

constexpr int64_t kGradMembers = 512;

GradPlan grad_plan(int64_t T, int64_t gate_rows) {
    GradPlan p;
    p.per_gate = T / gate_rows;
    const int64_t run = (T + kGradMembers - 1) / kGradMembers;
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

template <typename Y, typename S, int kVecs, bool kSmall>
__global__ void norm_grad_kernel(NormArgs a, GradPlan p, int tx, float *part_post,
                                 float *part_pre, float *part_gate) {
    __shared__ float lds[2 * 16];
    int turn = 0;
    const int lane = kSmall ? threadIdx.x & (tx - 1) : threadIdx.x;
    const int64_t member = kSmall ? blockIdx.x * (int64_t)(kSmallThreads / tx) + threadIdx.x / tx
                                  : blockIdx.x;
    if (member >= p.members) return;
    int64_t t0, t1;
    if (p.chunks == 1) {
        t0 = member * p.run;
        t1 = t0 + p.run;
        if (t1 > a.T) t1 = a.T;
    } else {
        const int64_t first = member / p.chunks * p.per_gate;
        t0 = first + member % p.chunks * p.run;
        t1 = t0 + p.run;
        if (t1 > first + p.per_gate) t1 = first + p.per_gate;
    }
    const float inv_h = 1.0f / (float)a.H;
    float acc1[kVecs][8] = {}, acc2[kVecs][8] = {}, accg[kVecs][8] = {};
    for (int64_t t = t0; t < t1; ++t) {
        float d[kVecs][8], rh[kVecs][8], y[kVecs][8], w[8];
        float sum[1] = {0};
        const float rs2 = a.dn ? a.in_rstd_pre[t] : 0.0f;
        const float rs1 = a.post ? a.in_rstd_post[t] : 1.0f;
        const int64_t grow = t / p.per_gate * a.H;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
            load8(static_cast<const Y *>(a.y) + t * a.ldy + 8 * v, n, y[j]);
            if (a.dn) {
                load8(static_cast<const Y *>(a.dn) + t * a.ld_dn + 8 * v, n, d[j]);
                load8(static_cast<const S *>(a.r) + t * a.ldr + 8 * v, n, rh[j]);
                load_param(a.w_pre, a.param_bf16, 8 * v, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    rh[j][i] *= rs2;
                    acc2[j][i] = __builtin_fmaf(d[j][i], rh[j][i], acc2[j][i]);
                    d[j][i] *= w[i];
                    sum[0] = __builtin_fmaf(d[j][i], rh[j][i], sum[0]);
                }
            }
        }
        if (a.dn) row_sum<1, kSmall>(sum, tx, lds, turn);
        const float c1 = sum[0] * inv_h;
        sum[0] = 0;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
            float e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.dr_out) load8(static_cast<const S *>(a.dr_out) + t * a.ld_dr_out + 8 * v, n, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[j][i] = a.dn ? e[i] + rs2 * (d[j][i] - rh[j][i] * c1) : e[i];
                e[i] = a.residual_scale * d[j][i];
            }
            store8(static_cast<S *>(a.dr) + t * a.H + 8 * v, n, e);
            load_param(a.gate, a.param_bf16, grow + 8 * v, n, w);
            float w1[8];
            load_param(a.post ? a.w_post : nullptr, a.param_bf16, 8 * v, n, w1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[j][i] *= rs1;
                const float scaled = a.branch_scale * d[j][i];
                accg[j][i] = __builtin_fmaf(scaled * y[j][i], w1[i], accg[j][i]);
                const float du = scaled * w[i];
                acc1[j][i] = __builtin_fmaf(du, y[j][i], acc1[j][i]);
                d[j][i] = du * w1[i];
                sum[0] = __builtin_fmaf(d[j][i], y[j][i], sum[0]);
            }
        }
        float c2 = 0;
        if (a.post) {
            row_sum<1, kSmall>(sum, tx, lds, turn);
            c2 = sum[0] * inv_h;
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t v = lane + (int64_t)j * tx;
            const int n = vec_count(a.H, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[j][i] = rs1 * (d[j][i] - y[j][i] * c2);
            store8(static_cast<Y *>(a.dy) + t * a.H + 8 * v, n, d[j]);
        }
        // a gate row that ends here and lies whole in this member
        if (a.dgate && p.chunks == 1 && (t + 1) % p.per_gate == 0) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int64_t v = lane + (int64_t)j * tx;
                store8(a.dgate + grow + 8 * v, vec_count(a.H, v), accg[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) accg[j][i] = 0;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int64_t v = lane + (int64_t)j * tx;
        const int n = vec_count(a.H, v);
        const int64_t at = member * a.H + 8 * v;
        if (a.dw_post) store8(part_post + at, n, acc1[j]);
        if (a.dw_pre) store8(part_pre + at, n, acc2[j]);
        if (a.dgate && p.chunks > 1) store8(part_gate + at, n, accg[j]);
    }
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

// Calls f(Y{}, S{}, vecs, small) for the types and split at hand.
template <int N>
struct Count {
    static constexpr int value = N;
};

template <typename F>
void with_split(const RowSplit &s, F f) {
    if (s.small) f(Count<1>{}, Count<1>{});
    else if (s.vecs == 1) f(Count<1>{}, Count<0>{});
    else if (s.vecs == 2) f(Count<2>{}, Count<0>{});
    else f(Count<4>{}, Count<0>{});
}

template <typename F>
void with_types(const NormArgs &a, F f) {
    if (a.y_bf16 && a.r_bf16) f(Bf16{}, Bf16{});
    else if (a.y_bf16) f(Bf16{}, float{});
    else f(float{}, float{});
}

}  // namespace

hipError_t launch_norm_residual(const NormArgs &a, hipStream_t stream) {
    const RowSplit s = row_split(a.H);
    const int64_t per = s.small ? kSmallThreads / s.tx : 1;
    int64_t blocks = (a.T + per - 1) / per;
    const int64_t most = 2048;
    int64_t rows_each = 1;
    if (blocks > most) {
        rows_each = (a.T + most * per - 1) / (most * per);
        blocks = (a.T + rows_each * per - 1) / (rows_each * per);
    }
    with_types(a, [&](auto y, auto r) {
        with_split(s, [&](auto vecs, auto small) {
            using Y = decltype(y);
            using S = decltype(r);
            constexpr int V = decltype(vecs)::value;
            constexpr bool kSmall = decltype(small)::value;
            if (a.q)
                norm_kernel<Y, S, V, kSmall, true>
                    <<<(unsigned)blocks, s.block, 0, stream>>>(a, s.tx, rows_each);
            else
                norm_kernel<Y, S, V, kSmall, false>
                    <<<(unsigned)blocks, s.block, 0, stream>>>(a, s.tx, rows_each);
        });
    });
    return hipGetLastError();
}

size_t norm_grad_workspace_bytes(int64_t T, int64_t H, int64_t gate_rows) {
    if (T == 0) return 0;
    const GradPlan p = grad_plan(T, gate_rows);
    return (size_t)(p.chunks > 1 ? 3 : 2) * p.members * H * sizeof(float);
}

hipError_t launch_norm_residual_grad(const NormArgs &a, hipStream_t stream) {
    GradPlan p = {1, 1, 1, 0};
    if (a.T > 0) p = grad_plan(a.T, a.gate_rows);
    float *part_post = a.workspace, *part_pre = part_post + p.members * a.H;
    float *part_gate = part_pre + p.members * a.H;
    if (a.T > 0) {
        const RowSplit s = row_split(a.H);
        const int64_t per = s.small ? kSmallThreads / s.tx : 1;
        const int64_t blocks = (p.members + per - 1) / per;
        with_types(a, [&](auto y, auto r) {
            with_split(s, [&](auto vecs, auto small) {
                using Y = decltype(y);
                using S = decltype(r);
                norm_grad_kernel<Y, S, decltype(vecs)::value, decltype(small)::value>
                    <<<(unsigned)blocks, s.block, 0, stream>>>(a, p, s.tx, part_post, part_pre,
                                                               part_gate);
            });
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

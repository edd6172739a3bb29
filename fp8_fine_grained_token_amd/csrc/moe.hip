// Tokens sorted by expert and back (gfx950): a stable counting sort of the
// routed slots, the gather into expert order (as it is or quantized 1x128),
// the weighted sum back per token, and the gradients of both.
//
// Every kernel but the sort is a copy with a little arithmetic (at most 3
// flops a value): its floor is the bytes of the wide tensors at the rate of
// a large copy.  All of them work token by token, so that a token's row is
// read once however many experts it goes to, and nothing is summed by
// atomics: a token's slots are added in slot order by one thread.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch_moe.hpp"
#include "vec.hpp"

namespace fp8blk {

namespace {

// ---- sort ----------------------------------------------------------------
//
// A workgroup owns a run of kSortChunk slots (more when there are many), each
// of its waves an eighth of them.  It counts its slots per wave and expert in
// LDS; with the counts of the runs before it (several workgroups: written to
// the workspace by a first launch) and an exclusive prefix sum over the
// experts, every (wave, expert) has its first row.  A wave then takes its
// slots 64 at a time in order: the lanes that hold the same expert find each
// other by one ballot per bit of the expert's number, a lane's rank among
// them is the population count below it.  Order is by construction, so the
// sort is stable and the same in every run.
constexpr int kSortWaves = 8;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kSortChunk = 4096;      // slots of a workgroup
constexpr int64_t kSortMaxRuns = 512;  // more slots: longer runs

struct SortPlan {
    int64_t slots, run;  // run: slots of a workgroup, a multiple of kSortThreads
    int runs;
};

SortPlan sort_plan(int64_t slots) {
    SortPlan p;
    p.slots = slots;
    int64_t run = kSortChunk;
    if (slots > run * kSortMaxRuns) {
        run = (slots + kSortMaxRuns - 1) / kSortMaxRuns;
        run = (run + kSortThreads - 1) / kSortThreads * kSortThreads;
    }
    p.run = run;
    p.runs = (int)((slots + run - 1) / run);
    if (p.runs < 1) p.runs = 1;
    return p;
}

template <typename Id>
__device__ __forceinline__ int expert_of(const Id *ids, int64_t slot, int E) {
    const Id v = ids[slot];
    return v >= 0 && v < (Id)E ? (int)v : -1;
}

// Counts of this workgroup's slots, per wave and expert.
template <typename Id>
__device__ __forceinline__ void count_run(const Id *ids, int64_t first, int64_t last, int E,
                                          int32_t *mine) {
    for (int64_t s = first + (threadIdx.x & 63); s < last; s += 64) {
        const int e = expert_of(ids, s, E);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
}

template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const Id *__restrict__ ids,
                                                                  SortPlan p, int E,
                                                                  int32_t *__restrict__ counts) {
    __shared__ int32_t hist[kSortMaxExperts];
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int64_t each = p.run / kSortWaves;
    const int64_t first = (int64_t)blockIdx.x * p.run + (threadIdx.x >> 6) * each;
    const int64_t last = first + each < p.slots ? first + each : p.slots;
    count_run(ids, first, last, E, hist);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads)
        counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(
    const Id *__restrict__ ids, SortPlan p, int E, const int32_t *__restrict__ counts,
    int32_t *__restrict__ offsets, int32_t *__restrict__ slot_row,
    int32_t *__restrict__ row_slot) {
    __shared__ int32_t base[kSortWaves * kSortMaxExperts];
    __shared__ int32_t wave_total[kSortWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < kSortWaves * E; i += kSortThreads) base[i] = 0;
    __syncthreads();
    const int64_t each = p.run / kSortWaves;
    const int64_t first = (int64_t)blockIdx.x * p.run + wave * each;
    const int64_t last = first + each < p.slots ? first + each : p.slots;
    count_run(ids, first, last, E, base + wave * E);
    __syncthreads();

    // two experts a thread: `before` counts the runs before this one, `all`
    // every run
    constexpr int kPer = kSortMaxExperts / kSortThreads;
    int32_t all[kPer], before[kPer];
    int32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = (int)threadIdx.x * kPer + i;
        all[i] = before[i] = 0;
        if (e < E) {
            if (p.runs == 1) {
                for (int w = 0; w < kSortWaves; ++w) all[i] += base[w * E + e];
            } else {
                for (int b = 0; b < p.runs; ++b) {
                    const int32_t c = counts[(int64_t)b * E + e];
                    all[i] += c;
                    if (b < (int)blockIdx.x) before[i] += c;
                }
            }
        }
        sum += all[i];
    }
    int32_t up = sum;  // inclusive prefix sum over the wave
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t v = __shfl_up(up, d);
        if (lane >= d) up += v;
    }
    if (lane == 63) wave_total[wave] = up;
    __syncthreads();
    int32_t start = up - sum, total = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) start += wave_total[w];
        total += wave_total[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = (int)threadIdx.x * kPer + i;
        if (e < E) {
            if (blockIdx.x == 0) offsets[e] = start;
            int32_t row = start + before[i];
            for (int w = 0; w < kSortWaves; ++w) {
                const int32_t c = base[w * E + e];
                base[w * E + e] = row;
                row += c;
            }
        }
        start += all[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
    __syncthreads();

    int bits = 0;
    while ((1 << bits) < E) ++bits;
    int32_t *mine = base + wave * E;
    for (int64_t s0 = first; s0 < last; s0 += 64) {
        const int64_t s = s0 + lane;
        const int e = s < last ? expert_of(ids, s, E) : -1;
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const bool set = (e >> b) & 1;
            const uint64_t with = __ballot(set);
            same &= set ? with : ~with;
        }
        int32_t row = -1;
        if (e >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int leader = __ffsll((unsigned long long)same) - 1;
            int32_t old = 0;
            if (lane == leader) old = atomicAdd(&mine[e], (int32_t)__popcll(same));
            row = __shfl(old, leader) + rank;
            row_slot[row] = (int32_t)s;
        }
        if (s < last) slot_row[s] = row;
    }
    // rows past the kept slots
    const int64_t end = ((int64_t)blockIdx.x + 1) * p.run;
    for (int64_t r = (int64_t)blockIdx.x * p.run + threadIdx.x; r < end && r < p.slots;
         r += kSortThreads)
        if (r >= total) row_slot[r] = -1;
}

template <typename Id>
hipError_t sort_typed(const MoeRouting &r, hipStream_t stream) {
    const SortPlan p = sort_plan(r.T * r.k);
    const Id *ids = static_cast<const Id *>(r.ids);
    int32_t *counts = static_cast<int32_t *>(r.workspace);
    if (p.runs > 1) {
        sort_count_kernel<Id><<<p.runs, kSortThreads, 0, stream>>>(ids, p, (int)r.E, counts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    sort_place_kernel<Id><<<p.runs, kSortThreads, 0, stream>>>(ids, p, (int)r.E, counts,
                                                               r.offsets, r.slot_row, r.row_slot);
    return hipGetLastError();
}

// ---- gather ----------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;

// A workgroup of 256 threads takes 256 / tx tokens, tx (a power of two)
// threads to a row; the rows past the grid by strides.
struct RowShape {
    int64_t T;
    int tx_log;
};

inline int log2_of(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

inline unsigned row_blocks(int64_t T, int tx) {
    const int64_t per = kRowThreads / tx;
    const int64_t blocks = (T + per - 1) / per;
    return (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

__device__ __forceinline__ void copy_row(const GatherPlane &g, int64_t t, int64_t T, int64_t k,
                                         const int32_t *slot_row, int64_t R, int lane, int tx) {
    const uint8_t *src = static_cast<const uint8_t *>(g.src) + t * g.ld;
    uint8_t *dst = static_cast<uint8_t *>(g.dst);
    const int64_t vecs = (g.bytes + 15) / 16;
    for (int64_t v = lane; v < vecs; v += tx) {
        const int64_t at = 16 * v;
        if (at + 16 <= g.bytes) {
            const u32x4_any d = *reinterpret_cast<const u32x4_any *>(src + at);
            for (int64_t j = 0; j < k; ++j) {
                const int32_t row = slot_row[t * k + j];
                if (row >= 0 && row < R)
                    *reinterpret_cast<u32x4_any *>(dst + row * g.bytes + at) = d;
            }
        } else {
            for (int64_t j = 0; j < k; ++j) {
                const int32_t row = slot_row[t * k + j];
                if (row >= 0 && row < R)
                    for (int64_t i = at; i < g.bytes; ++i) dst[row * g.bytes + i] = src[i];
            }
        }
    }
}

__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(GatherPlane rows,
                                                               GatherPlane scales, RowShape shape,
                                                               const int32_t *__restrict__ slot_row,
                                                               int64_t k, int64_t R) {
    const int tx = 1 << shape.tx_log, lane = threadIdx.x & (tx - 1);
    const int64_t per = kRowThreads >> shape.tx_log;
    for (int64_t t = blockIdx.x * per + (threadIdx.x >> shape.tx_log); t < shape.T;
         t += gridDim.x * per) {
        copy_row(rows, t, shape.T, k, slot_row, R, lane, tx);
        if (scales.src) copy_row(scales, t, shape.T, k, slot_row, R, lane, tx);
    }
}

// Quantized: 16 lanes hold one 128-value group, eight values each, as in the
// activation quantizer; every lane of a wave takes the same number of turns,
// so the 16-lane maximum always has its lanes.
template <bool kPow2>
__global__ __launch_bounds__(kRowThreads) void dispatch_quant_kernel(
    const Bf16 *__restrict__ x, int64_t ldx, RowShape shape, int64_t H,
    const int32_t *__restrict__ slot_row, int64_t k, uint8_t *__restrict__ q,
    float *__restrict__ scales, int64_t R) {
    const int tx = 1 << shape.tx_log, lane = threadIdx.x & (tx - 1);
    const int64_t per = kRowThreads >> shape.tx_log;
    const int64_t G = (H + kGroup - 1) / kGroup, vecs = 16 * G;
    const int64_t rounds = (shape.T + per - 1) / per;
    for (int64_t b = blockIdx.x; b < rounds; b += gridDim.x) {
        const int64_t t = b * per + (threadIdx.x >> shape.tx_log);
        const bool in = t < shape.T;
        for (int64_t v0 = 0; v0 < vecs; v0 += tx) {
            const int64_t v = v0 + lane;
            const int n = in ? vec_count(H, v) : 0;
            float f[8];
            load8(x + t * ldx + 8 * v, n, f);
            const QuotientCtx qc(row16_max(absmax8(f)), kPow2);
            const uint2 bytes = quant8(f, qc);
            if (!in || v >= vecs) continue;
            for (int64_t j = 0; j < k; ++j) {
                const int32_t row = slot_row[t * k + j];
                if (row < 0 || row >= R) continue;
                store_e4m3(q + row * H + 8 * v, n, bytes);
                if ((lane & 15) == 0) scales[row * G + v / 16] = qc.s;
            }
        }
    }
}

// ---- weighted sum back, and the gradients -------------------------------------

template <typename In, typename Out>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(
    const In *__restrict__ ys, int64_t ld, int64_t R, const int32_t *__restrict__ slot_row,
    const float *__restrict__ weights, RowShape shape, int64_t k, int64_t H,
    const Out *residual, int64_t ld_residual, Out *out) {
    const int tx = 1 << shape.tx_log, lane = threadIdx.x & (tx - 1);
    const int64_t per = kRowThreads >> shape.tx_log;
    const int64_t vecs = (H + 7) / 8;
    for (int64_t t = blockIdx.x * per + (threadIdx.x >> shape.tx_log); t < shape.T;
         t += gridDim.x * per) {
        for (int64_t v = lane; v < vecs; v += tx) {
            const int n = vec_count(H, v);
            float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (residual) load8(residual + t * ld_residual + 8 * v, n, acc);
            for (int64_t j = 0; j < k; ++j) {
                const int32_t row = slot_row[t * k + j];
                if (row < 0 || row >= R) continue;
                const float w = weights ? weights[t * k + j] : 1.0f;
                float f[8];
                load8(ys + row * ld + 8 * v, n, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, f[i], acc[i]);
            }
            store8(out + t * H + 8 * v, n, acc);
        }
    }
}

// One token a workgroup: dys rows and the dot products, eight slots at a
// time (kBatch).
constexpr int kBatch = 8;

template <typename V>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(
    const V *__restrict__ dout, int64_t ld_dout, const V *__restrict__ ys, int64_t ld_ys,
    int64_t R, const int32_t *__restrict__ slot_row, const float *__restrict__ weights,
    int64_t T, int64_t k, int64_t H, V *__restrict__ dys, float *__restrict__ dweights) {
    __shared__ float part[kRowThreads / 64][kBatch];
    const int64_t vecs = (H + 7) / 8;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int64_t j0 = 0; j0 < k; j0 += kBatch) {
            float dot[kBatch] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int64_t v = threadIdx.x; v < vecs; v += kRowThreads) {
                const int n = vec_count(H, v);
                float d[8];
                load8(dout + t * ld_dout + 8 * v, n, d);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (j0 + b >= k) continue;
                    const int32_t row = slot_row[t * k + j0 + b];
                    if (row < 0 || row >= R) continue;
                    const float w = weights ? weights[t * k + j0 + b] : 1.0f;
                    float f[8];
                    if (dweights) {
                        load8(ys + row * ld_ys + 8 * v, n, f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[b] = __builtin_fmaf(d[i], f[i], dot[b]);
                    }
                    if (dys) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = w * d[i];
                        store8(dys + row * H + 8 * v, n, f);
                    }
                }
            }
            if (!dweights) continue;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
#pragma unroll
                for (int m = 32; m; m /= 2) dot[b] += __shfl_xor(dot[b], m);
                if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][b] = dot[b];
            }
            __syncthreads();
            if (threadIdx.x < kBatch && j0 + threadIdx.x < k) {
                float sum = 0;
                for (int w = 0; w < kRowThreads / 64; ++w) sum += part[w][threadIdx.x];
                dweights[t * k + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t slots, int64_t E) {
    const SortPlan p = sort_plan(slots);
    return p.runs > 1 ? (size_t)p.runs * E * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const MoeRouting &r, hipStream_t stream) {
    return r.wide_ids ? sort_typed<int64_t>(r, stream) : sort_typed<int32_t>(r, stream);
}

hipError_t launch_moe_dispatch(const GatherPlane &rows, const GatherPlane *scales,
                               const int32_t *slot_row, int64_t T, int64_t k, int64_t R,
                               hipStream_t stream) {
    const int tx = threads_per_row((rows.bytes + 15) / 16, 16, kRowThreads);
    const GatherPlane none = {nullptr, nullptr, 0, 0, 0};
    dispatch_kernel<<<row_blocks(T, tx), kRowThreads, 0, stream>>>(
        rows, scales ? *scales : none, RowShape{T, log2_of(tx)}, slot_row, k, R);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch_quant(const void *x, int64_t ldx, int64_t T, int64_t H,
                                     const int32_t *slot_row, int64_t k, void *q, float *scales,
                                     int64_t R, bool pow2, hipStream_t stream) {
    const int tx = threads_per_row((H + kGroup - 1) / kGroup * 16, 16, kRowThreads);
    auto *kernel = pow2 ? dispatch_quant_kernel<true> : dispatch_quant_kernel<false>;
    kernel<<<row_blocks(T, tx), kRowThreads, 0, stream>>>(
        static_cast<const Bf16 *>(x), ldx, RowShape{T, log2_of(tx)}, H, slot_row, k,
        static_cast<uint8_t *>(q), scales, R);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void *ys, bool ys_bf16, int64_t ld, int64_t R,
                              const int32_t *slot_row, const float *weights, int64_t T,
                              int64_t k, int64_t H, const void *residual, int64_t ld_residual,
                              void *out, bool out_bf16, hipStream_t stream) {
    const int tx = threads_per_row((H + 7) / 8, 16, kRowThreads);
    const RowShape shape{T, log2_of(tx)};
    auto go = [&](auto in, auto to) {
        using In = decltype(in);
        using Out = decltype(to);
        combine_kernel<In, Out><<<row_blocks(T, tx), kRowThreads, 0, stream>>>(
            static_cast<const In *>(ys), ld, R, slot_row, weights, shape, k, H,
            static_cast<const Out *>(residual), ld_residual, static_cast<Out *>(out));
    };
    if (ys_bf16) {
        if (out_bf16) go(Bf16{}, Bf16{}); else go(Bf16{}, float{});
    } else {
        if (out_bf16) go(float{}, Bf16{}); else go(float{}, float{});
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const void *dout, int64_t ld_dout, const void *ys,
                                   int64_t ld_ys, bool bf16, int64_t R, const int32_t *slot_row,
                                   const float *weights, int64_t T, int64_t k, int64_t H,
                                   void *dys, float *dweights, hipStream_t stream) {
    const unsigned blocks = (unsigned)(T < kMaxBlocks ? T : kMaxBlocks);
    auto go = [&](auto v) {
        using V = decltype(v);
        combine_grad_kernel<V><<<blocks, kRowThreads, 0, stream>>>(
            static_cast<const V *>(dout), ld_dout, static_cast<const V *>(ys), ld_ys, R, slot_row,
            weights, T, k, H, static_cast<V *>(dys), dweights);
    };
    if (bf16) go(Bf16{}); else go(float{});
    return hipGetLastError();
}

}  // namespace fp8blk

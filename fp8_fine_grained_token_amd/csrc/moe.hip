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
// experts, every (wave, expert) has its first row.  (Every workgroup adds the
// counts of all runs: 16 runs of 32768 slots are nothing; 512 runs, a million
// slots, take 52 us over 256 experts and 131 over 1024.)  A wave then takes its
// slots 64 at a time in order: the lanes that hold the same expert find each
// other by one ballot per bit of the expert's number, a lane's rank among
// them is the population count below it.  Order is by construction, so the
// sort is stable and the same in every run.  Latency bounds it: 32768 slots
// over 32 experts take 5 us for the counts and 7 us for the places, up to 4096
// slots 4 to 8 us in one launch.
constexpr int kSortWaves = 8;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kSortHeld = 4;  // slots a lane holds at a time
constexpr int kSortChunk = kSortThreads * kSortHeld;  // slots of a workgroup
constexpr int64_t kSortMaxRuns = 512;  // more slots: longer runs

struct SortPlan {
    int64_t slots, run;  // run: slots of a workgroup, a multiple of kSortThreads
    int runs;
};

SortPlan sort_plan(int64_t slots) {
    SortPlan p;
    p.slots = slots;
    // one workgroup, and one launch, for up to two chunks, dealt to all its waves
    int64_t run = kSortChunk;
    if (slots <= 2 * kSortChunk) run = (slots + kSortThreads - 1) / kSortThreads * kSortThreads;
    if (run == 0) run = kSortThreads;
    if (slots > run * kSortMaxRuns) {
        run = (slots + kSortMaxRuns - 1) / kSortMaxRuns;
        run = (run + kSortChunk - 1) / kSortChunk * kSortChunk;
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

// The experts of the kSortHeld * 64 slots from s0 on, 64 slots to each of a
// lane's values (-1 past `last` and for dropped slots); one wait for all.
template <typename Id>
__device__ __forceinline__ void hold_ids(const Id *ids, int64_t s0, int64_t last, int E,
                                         int (&e)[kSortHeld]) {
    Id v[kSortHeld];
#pragma unroll
    for (int i = 0; i < kSortHeld; ++i) {
        const int64_t s = s0 + 64 * i + (threadIdx.x & 63);
        v[i] = ids[s < last ? s : last - 1];
    }
#pragma unroll
    for (int i = 0; i < kSortHeld; ++i) {
        const int64_t s = s0 + 64 * i + (threadIdx.x & 63);
        e[i] = s < last && v[i] >= 0 && v[i] < (Id)E ? (int)v[i] : -1;
    }
}

// Adds a wave's slots to counts per expert.
template <typename Id>
__device__ __forceinline__ void count_run(const Id *ids, int64_t first, int64_t last, int E,
                                          int32_t *counts) {
    for (int64_t s0 = first; s0 < last; s0 += 64 * kSortHeld) {
        int e[kSortHeld];
        hold_ids(ids, s0, last, E, e);
#pragma unroll
        for (int i = 0; i < kSortHeld; ++i)
            if (e[i] >= 0) atomicAdd(&counts[e[i]], 1);
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
#pragma unroll 8
                for (int b = 0; b < p.runs; ++b) {
                    const int32_t c = counts[(int64_t)b * E + e];
                    all[i] += c;
                    before[i] += b < (int)blockIdx.x ? c : 0;
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
    for (int64_t s0 = first; s0 < last; s0 += 64 * kSortHeld) {
        int held[kSortHeld];
        hold_ids(ids, s0, last, E, held);
#pragma unroll
        for (int i = 0; i < kSortHeld; ++i) {
            const int e = held[i];
            const int64_t s = s0 + 64 * i + lane;
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

// ---- rows and their parts ---------------------------------------------------
//
// A row is taken in vectors of 16 bytes (the copies) or eight values (the
// rest), one a thread: tx threads (a power of two) to a row and 256 / tx rows
// to a workgroup, the workgroups of gridDim.y side by side along wide rows.
// A token's slots are read kBatch at a time, the row numbers of a batch in
// one go and then the rows, so that a wait covers a batch and not a slot.
// Where that leaves a thread with few loads (the gather reads a row once; four
// slots a token or fewer), it takes two or four vectors at a time, unless there
// are too few rows to give every thread work (kManyVecs).
//
// HBM bounds all of them once there are some thousand rows.  4096 tokens of
// 7168 bf16 values, eight slots each, not in the caches: quantized gather 301
// MB in 65 us (4.6 TB/s); gather of E4M3 rows 273 MB with their scales in 50 us;
// weighted sum 529 MB in 96 to 107 us (5.5 to 4.9 TB/s); its gradient 998 MB in
// 201 us (5.0 TB/s); a copy of 4 GiB runs at 4.8 TB/s.  For 256 tokens the
// weighted sum takes 8 us, for one token 3.3 us, the time of a launch that waits
// for two loads in a row.  A plane of fewer than 16 bytes a row (scales of up to
// 384 values) goes byte by byte: 4096 x 8 rows of 384 E4M3 values 18 us with
// scales, 5 without.
constexpr int kRowThreads = 256;
constexpr int kBatch = 8;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;
// Vectors from which a thread takes several: 8192 rows of 7168 values once
// each, quantized gather 63 -> 44 us, weighted sum 99 -> 50 us; weighted sum of
// four rows of 2048 values for 2048 tokens 10.0 -> 8.9 us.
constexpr int64_t kManyVecs = (int64_t)1 << 19;

struct RowShape {
    int64_t T;
    int tx_log;
};

inline int log2_of(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

// Threads and workgroups for T rows of `vecs` vectors.
struct RowGrid {
    RowShape shape;
    dim3 grid;
};

RowGrid row_grid(int64_t T, int64_t vecs, int least, int each = 1) {
    const int tx = threads_per_row((vecs + each - 1) / each, least, kRowThreads);
    const int64_t per = kRowThreads / tx, blocks = (T + per - 1) / per;
    const int64_t along = (vecs + tx * each - 1) / (tx * each);
    RowGrid g;
    g.shape = {T, log2_of(tx)};
    g.grid = dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks),
                  (unsigned)(along < 65535 ? along : 65535));
    return g;
}

// The rows of slots j0 .. of token t, -1 for a dropped slot (or none), and
// their weights.  A token has at least 16 lanes of a wave: lane b of each 16
// reads slot b and hands it round, so one load brings a batch.
template <int kCount>
struct Batch {
    static_assert(kCount <= 16, "a batch is read by 16 lanes");
    int32_t rows[kCount];
    float w[kCount];
    int32_t my_row;
    float my_w;
    __device__ __forceinline__ void load(const int32_t *slot_row, const float *weights, int64_t t,
                                         int64_t k, int64_t j0) {
        const int64_t lane = threadIdx.x & 15, j = j0 + lane < k ? j0 + lane : k - 1;
        my_w = 1.0f;
        if (weights) my_w = weights[t * k + j];
        my_row = slot_row[t * k + j];
    }
    __device__ __forceinline__ void share(int64_t k, int64_t j0, int64_t R) {
        const int64_t lane = threadIdx.x & 15;
        const int32_t row = j0 + lane < k && my_row >= 0 && my_row < R ? my_row : -1;
#pragma unroll
        for (int b = 0; b < kCount; ++b) {
            rows[b] = __shfl(row, b, 16);
            w[b] = __shfl(my_w, b, 16);
        }
    }
};

// ---- gather ----------------------------------------------------------------

enum GatherMode { kCopy, kQuant, kQuantPow2 };

// Quantizing rows of fewer than eight values or more (a copy does not ask),
// vectors a thread takes at a time.
template <int kMode, bool kNarrow, int kVecs>
struct Gather {
    static constexpr bool copy = kMode == kCopy, pow2 = kMode == kQuantPow2, narrow = kNarrow;
    static constexpr int vecs = kVecs;
};

struct GatherArgs {
    GatherPlane rows, scales;  // copy
    const Bf16 *x;             // quantize
    int64_t ldx, H;
    uint8_t *q;
    float *q_scales;
    int64_t k, R;
};

__device__ __forceinline__ int64_t plane_vecs(const GatherPlane &g) { return (g.bytes + 15) / 16; }

// Vectors v, v + step, ... of token t's row (16 bytes, the row's last 16 for
// its last vector) to the rows of its slots; get(j0, rows) gives a batch of
// them.
template <int kVecs, typename Rows>
__device__ __forceinline__ void copy_vecs(const GatherPlane &g, int64_t t, int64_t v, int64_t step,
                                          bool in, int64_t k, Rows get) {
    const bool wide = g.bytes >= 16;
    const uint8_t *src = static_cast<const uint8_t *>(g.src) + t * g.ld;
    int64_t at[kVecs];
    u32x4 d[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t from = 16 * (v + i * step), most = g.bytes - 16;
        at[i] = !wide ? 0 : from < most ? from : most;
        d[i] = u32x4{0, 0, 0, 0};
        if (wide) d[i] = *reinterpret_cast<const u32x4_any *>(src + at[i]);
    }
    for (int64_t j0 = 0; j0 < k; j0 += kBatch) {
        int32_t rows[kBatch];
        get(j0, rows);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (rows[b] < 0 || !in) continue;
            uint8_t *dst = static_cast<uint8_t *>(g.dst) + rows[b] * g.bytes;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (16 * (v + i * step) >= g.bytes) continue;
                if (wide) {
                    *reinterpret_cast<u32x4_any *>(dst + at[i]) = d[i];
                } else {
                    for (int c = 0; c < (int)g.bytes; ++c) dst[c] = src[c];
                }
            }
        }
    }
}

// The same quantized: 16 lanes hold one 128-value group, eight values each, as
// in the activation quantizer.  For all lanes of a wave or none: the 16-lane
// maximum needs its lanes.
template <typename M, typename Rows>
__device__ __forceinline__ void quant_vecs(const GatherArgs &a, int64_t t, int64_t v, int64_t step,
                                           bool in, Rows get) {
    const int64_t G = (a.H + kGroup - 1) / kGroup;
    Span s[M::vecs];
    Raw8<Bf16> raw[M::vecs];
    uint2 bytes[M::vecs];
    float scale[M::vecs];
#pragma unroll
    for (int i = 0; i < M::vecs; ++i) {
        s[i] = row_span<M::narrow>(v + i * step, a.H);
        load_raw<M::narrow>(a.x + t * a.ldx + s[i].col, s[i].hi, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < M::vecs; ++i) {
        float f[8];
        unpack_own(raw[i], s[i], f);
        bytes[i] = quantize8(f, group_max(f), s[i].any(), M::pow2, scale[i]);
    }
    for (int64_t j0 = 0; j0 < a.k; j0 += kBatch) {
        int32_t rows[kBatch];
        get(j0, rows);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (rows[b] < 0 || !in) continue;
#pragma unroll
            for (int i = 0; i < M::vecs; ++i) {
                if (!s[i].any()) continue;
                store_e4m3(a.q + rows[b] * a.H, s[i], bytes[i]);
                if ((threadIdx.x & 15) == 0)
                    a.q_scales[rows[b] * G + (v + i * step) / 16] = scale[i];
            }
        }
    }
}

template <typename M>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(GatherArgs a, RowShape shape,
                                                               const int32_t *__restrict__ slot_row) {
    const int tx = 1 << shape.tx_log, lane = threadIdx.x & (tx - 1);
    const int64_t per = kRowThreads >> shape.tx_log, rounds = (shape.T + per - 1) / per;
    for (int64_t b = blockIdx.x; b < rounds; b += gridDim.x) {
        const int64_t own = b * per + (threadIdx.x >> shape.tx_log);
        const bool in = own < shape.T;
        const int64_t t = in ? own : shape.T - 1;
        auto get = [&](int64_t j0, int32_t(&rows)[kBatch]) {
            Batch<kBatch> batch;
            batch.load(slot_row, nullptr, t, a.k, j0);
            batch.share(a.k, j0, a.R);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) rows[i] = batch.rows[i];
        };
        // every lane stays to the end: lanes hand each other row numbers
        const int64_t v0 = (int64_t)blockIdx.y * tx * M::vecs;
        const int64_t step = (int64_t)gridDim.y * tx * M::vecs;
        if (M::copy) {
            for (int64_t v = v0; v < plane_vecs(a.rows); v += step)
                copy_vecs<M::vecs>(a.rows, t, v + lane, tx, in, a.k, get);
            if (a.scales.src)
                for (int64_t v = v0; v < plane_vecs(a.scales); v += step)
                    copy_vecs<M::vecs>(a.scales, t, v + lane, tx, in, a.k, get);
        } else {
            for (int64_t v = v0; v < 16 * ((a.H + kGroup - 1) / kGroup); v += step)
                quant_vecs<M>(a, t, v + lane, tx, in, get);
        }
    }
}

// Sort and gather of few slots in one launch.  The row of slot (t, j) is the
// number of kept slots that come before it in the order (expert, slot): every
// workgroup of a token counts them for the token's own slots by going through
// all ids in L2, so there is no launch between the sort and the gather and
// nothing to wait for.  One more row of workgroups writes the offsets.  Worth
// it as long as the ids read in all stay few: 256 tokens of 7168 values to 8
// experts (2 million ids) 9.2 us against 11.6 in two launches (with the sort's),
// 512 of 2048 values 7.8 against 12.5; the crossing is near 512 tokens of 7168
// (8 million), 16.5 against 17.5.
constexpr int64_t kFewSlots = 4096, kFewReads = (int64_t)1 << 22;
// Ids a lane reads at a time (256 tokens: 10.9 us with one, 9.5 with four; 512
// tokens of 2048 values 11.4 and 8.2).
constexpr int kRound = 4;

template <typename M, typename Id>
__global__ __launch_bounds__(kRowThreads) void sort_dispatch_kernel(
    GatherArgs a, const Id *__restrict__ ids, int T, int E, int32_t *__restrict__ offsets,
    int32_t *__restrict__ slot_row, int32_t *__restrict__ row_slot) {
    constexpr int kWaves = kRowThreads / 64;
    __shared__ int32_t hist[kSortMaxExperts];
    __shared__ int32_t part[kWaves][kBatch];
    const int k = (int)a.k, slots = T * k;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if ((int)blockIdx.x == T) {
        if (blockIdx.y) return;
        for (int e = threadIdx.x; e < E; e += kRowThreads) hist[e] = 0;
        __syncthreads();
        for (int s = threadIdx.x; s < slots; s += kRowThreads) {
            const int e = expert_of(ids, s, E);
            if (e >= 0) atomicAdd(&hist[e], 1);
        }
        __syncthreads();
        constexpr int kPer = kSortMaxExperts / kRowThreads;
        int32_t sum = 0;
        for (int i = 0; i < kPer; ++i) {
            const int e = (int)threadIdx.x * kPer + i;
            sum += e < E ? hist[e] : 0;
        }
        int32_t up = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int32_t v = __shfl_up(up, d);
            if (lane >= d) up += v;
        }
        if (lane == 63) part[wave][0] = up;
        __syncthreads();
        int32_t start = up - sum, total = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) start += part[w][0];
            total += part[w][0];
        }
        for (int i = 0; i < kPer; ++i) {
            const int e = (int)threadIdx.x * kPer + i;
            if (e < E) {
                offsets[e] = start;
                start += hist[e];
            }
        }
        if (threadIdx.x == 0) offsets[E] = total;
        for (int r = total + threadIdx.x; r < slots; r += kRowThreads) row_slot[r] = -1;
        return;
    }
    const int t = blockIdx.x;
    auto get = [&](int64_t j0, int32_t(&rows)[kBatch]) {
        // key (expert, slot): below 1024 * 4096
        int key[kBatch], count[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int s = t * k + min((int)j0 + b, k - 1);
            const int e = (int)j0 + b < k ? expert_of(ids, s, E) : -1;
            key[b] = e < 0 ? -1 : e * slots + s;
            count[b] = 0;
        }
        for (int s0 = wave * 64; s0 < slots; s0 += kRound * kRowThreads) {
            Id id[kRound];  // one wait for all
#pragma unroll
            for (int i = 0; i < kRound; ++i)
                id[i] = ids[min(s0 + i * kRowThreads + lane, slots - 1)];
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
                const int s = s0 + i * kRowThreads + lane;
                const bool kept = s < slots && id[i] >= 0 && id[i] < (Id)E;
                const int other = kept ? (int)id[i] * slots + s : 0x7FFFFFFF;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) count[b] += __popcll(__ballot(other < key[b]));
            }
        }
        __syncthreads();  // the last batch's reads
        if (lane == 0)
#pragma unroll
            for (int b = 0; b < kBatch; ++b) part[wave][b] = count[b];
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            int row = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) row += part[w][b];
            rows[b] = key[b] < 0 ? -1 : row;
        }
        if (blockIdx.y == 0 && (int)threadIdx.x < kBatch && (int)j0 + (int)threadIdx.x < k) {
            int row = -1;
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if ((int)threadIdx.x == b) row = rows[b];
            const int s = t * k + (int)j0 + (int)threadIdx.x;
            slot_row[s] = row;
            if (row >= 0) row_slot[row] = s;
        }
    };
    // one vector a thread: the grid covers the row
    const int64_t v = (int64_t)blockIdx.y * kRowThreads + threadIdx.x;
    if (M::copy)
        copy_vecs<1>(a.rows, t, v, 0, true, a.k, get);  // past the row's end: counts only
    else
        quant_vecs<M>(a, t, v, 0, true, get);
}

// ---- weighted sum back, and the gradients -------------------------------------

// kCount slots of kVecs vectors at a time.
template <typename In, typename Out, int kCount, int kVecs, bool kNarrow, bool kOnce>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(
    const In *__restrict__ ys, int64_t ld, int64_t R, const int32_t *__restrict__ slot_row,
    const float *__restrict__ weights, RowShape shape, int64_t k, int64_t H,
    const Out *residual, int64_t ld_residual, Out *out) {
    const int tx = 1 << shape.tx_log, lane = threadIdx.x & (tx - 1);
    const int64_t per = kRowThreads >> shape.tx_log, rounds = (shape.T + per - 1) / per;
    const int64_t vecs = (H + 7) / 8;
    for (int64_t round = blockIdx.x; round < rounds; round += gridDim.x) {
        const int64_t own = round * per + (threadIdx.x >> shape.tx_log);
        const int64_t t = own < shape.T ? own : shape.T - 1;
        for (int64_t v0 = (int64_t)blockIdx.y * tx * kVecs; v0 < vecs;
             v0 += (int64_t)gridDim.y * tx * kVecs) {
            Span s[kVecs];
            float acc[kVecs][8] = {};
            Raw8<Out> first[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                s[i] = row_span<kNarrow>(v0 + lane + i * tx, H);
                zero_raw(first[i]);
                if (residual)
                    load_raw<kNarrow>(residual + t * ld_residual + s[i].col, s[i].hi, first[i]);
                if (k == 0) unpack(first[i], acc[i]);
            }
            for (int64_t j0 = 0; j0 < k; j0 += kCount) {
                Batch<kCount> batch;
                Raw8<In> raw[kVecs][kCount];
                batch.load(slot_row, weights, t, k, j0);
                batch.share(k, j0, R);
#pragma unroll
                for (int b = 0; b < kCount; ++b)
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        zero_raw(raw[i][b]);
                        if (batch.rows[b] >= 0)
                            load_raw<kNarrow, kOnce>(ys + (int64_t)batch.rows[b] * ld + s[i].col,
                                                     s[i].hi, raw[i][b]);
                    }
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    if (j0 == 0) unpack(first[i], acc[i]);
#pragma unroll
                    for (int b = 0; b < kCount; ++b) {
                        float f[8];
                        unpack(raw[i][b], f);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            acc[i][c] = batch.rows[b] < 0
                                            ? acc[i][c]
                                            : __builtin_fmaf(batch.w[b], f[c], acc[i][c]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (own < shape.T && s[i].any()) store_span(out + t * H, s[i], acc[i]);
        }
    }
}

// dys rows and the dot products: one token a workgroup, kCount slots of kVecs
// vectors at a time.  dout is read once for all of the token's slots, and a
// slot's dot product needs no second pass since its row is at hand for as long
// as dys is written.
template <typename V, int kThreads, int kCount, int kVecs, bool kNarrow, bool kOnce>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(
    const V *__restrict__ dout, int64_t ld_dout, const V *__restrict__ ys, int64_t ld_ys,
    int64_t R, const int32_t *__restrict__ slot_row, const float *__restrict__ weights,
    int64_t T, int64_t k, int64_t H, V *__restrict__ dys, float *__restrict__ dweights) {
    __shared__ float part[kThreads / 64][kCount];
    const int64_t vecs = (H + 7) / 8;
    const int waves = blockDim.x / 64;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int64_t j0 = 0; j0 < k; j0 += kCount) {
            Batch<kCount> batch;
            float dot[kCount] = {};
            batch.load(slot_row, weights, t, k, j0);
            batch.share(k, j0, R);
            const int32_t(&rows)[kCount] = batch.rows;
            const float(&w)[kCount] = batch.w;
            for (int64_t v = threadIdx.x; v < vecs; v += kVecs * blockDim.x) {
                Span s[kVecs];
                Raw8<V> raw[kVecs], y[kVecs][kCount];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    s[i] = row_span<kNarrow>(v + i * (int)blockDim.x, H);
                    load_raw<kNarrow>(dout + t * ld_dout + s[i].col, s[i].hi, raw[i]);
                    if (dweights) {
#pragma unroll
                        for (int b = 0; b < kCount; ++b) {
                            zero_raw(y[i][b]);
                            if (rows[b] >= 0)
                                load_raw<kNarrow, kOnce>(ys + (int64_t)rows[b] * ld_ys + s[i].col,
                                                  s[i].hi, y[i][b]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    float d[8];
                    unpack_own(raw[i], s[i], d);
                    if (dys) {
#pragma unroll
                        for (int b = 0; b < kCount; ++b) {
                            if (rows[b] < 0 || !s[i].any()) continue;
                            float g[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c) g[c] = w[b] * d[c];
                            store_span(dys + rows[b] * H, s[i], g);
                        }
                    }
                    if (dweights) {
#pragma unroll
                        for (int b = 0; b < kCount; ++b) {
                            float f[8];
                            unpack_own(y[i][b], s[i], f);
                            float sum = 0;
#pragma unroll
                            for (int c = 0; c < 8; ++c) sum = __builtin_fmaf(d[c], f[c], sum);
                            // (a dropped slot has no product, not one with zero)
                            dot[b] = rows[b] < 0 ? 0.0f : dot[b] + sum;
                        }
                    }
                }
            }
            if (!dweights) continue;
#pragma unroll
            for (int b = 0; b < kCount; ++b) {
#pragma unroll
                for (int m = 32; m; m /= 2) dot[b] += __shfl_xor(dot[b], m);
                if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][b] = dot[b];
            }
            __syncthreads();
            if (threadIdx.x < kCount && j0 + threadIdx.x < k) {
                float sum = 0;
                for (int i = 0; i < waves; ++i) sum += part[i][threadIdx.x];
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

namespace {

GatherArgs copy_args(const GatherPlane &rows, const GatherPlane *scales, int64_t k, int64_t R) {
    GatherArgs a = {};
    a.rows = rows;
    if (scales) a.scales = *scales;
    a.k = k;
    a.R = R;
    return a;
}

GatherArgs quant_args(const void *x, int64_t ldx, int64_t H, int64_t k, void *q, float *scales,
                      int64_t R) {
    GatherArgs a = {};
    a.x = static_cast<const Bf16 *>(x);
    a.ldx = ldx;
    a.H = H;
    a.q = static_cast<uint8_t *>(q);
    a.q_scales = scales;
    a.k = k;
    a.R = R;
    return a;
}

// go(Gather<...>{}) for quantizing rows of H values.
template <typename F>
auto with_quant(bool pow2, int64_t H, bool many, F go) {
    if (H < 8) return pow2 ? go(Gather<kQuantPow2, true, 1>{}) : go(Gather<kQuant, true, 1>{});
    if (many) return pow2 ? go(Gather<kQuantPow2, false, 4>{}) : go(Gather<kQuant, false, 4>{});
    return pow2 ? go(Gather<kQuantPow2, false, 1>{}) : go(Gather<kQuant, false, 1>{});
}

// Few slots: sort and gather in one launch, a workgroup for each token and
// stretch of its row.
template <typename M>
bool sort_dispatch_few(const MoeRouting &r, const GatherArgs &a, int64_t vecs,
                       hipStream_t stream) {
    const int64_t along = (vecs + kRowThreads - 1) / kRowThreads;
    if (r.T == 0 || r.T * r.k > kFewSlots || along > 65535) return false;
    if (r.T * along * (r.T * r.k) > kFewReads) return false;
    const dim3 grid((unsigned)r.T + 1, (unsigned)along);
    if (r.wide_ids)
        sort_dispatch_kernel<M, int64_t><<<grid, kRowThreads, 0, stream>>>(
            a, static_cast<const int64_t *>(r.ids), (int)r.T, (int)r.E, r.offsets, r.slot_row,
            r.row_slot);
    else
        sort_dispatch_kernel<M, int32_t><<<grid, kRowThreads, 0, stream>>>(
            a, static_cast<const int32_t *>(r.ids), (int)r.T, (int)r.E, r.offsets, r.slot_row,
            r.row_slot);
    return true;
}

}  // namespace

hipError_t launch_moe_dispatch(const GatherPlane &rows, const GatherPlane *scales,
                               const int32_t *slot_row, int64_t T, int64_t k, int64_t R,
                               hipStream_t stream) {
    const int64_t vecs = (rows.bytes + 15) / 16;
    const bool many = T * vecs >= kManyVecs;
    const RowGrid g = row_grid(T, vecs, 16, many ? 4 : 1);
    auto *kernel = many ? dispatch_kernel<Gather<kCopy, false, 4>>
                        : dispatch_kernel<Gather<kCopy, false, 1>>;
    kernel<<<g.grid, kRowThreads, 0, stream>>>(copy_args(rows, scales, k, R), g.shape, slot_row);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch_quant(const void *x, int64_t ldx, int64_t T, int64_t H,
                                     const int32_t *slot_row, int64_t k, void *q, float *scales,
                                     int64_t R, bool pow2, hipStream_t stream) {
    const int64_t vecs = (H + kGroup - 1) / kGroup * 16;
    with_quant(pow2, H, T * vecs >= kManyVecs, [&](auto m) {
        using M = decltype(m);
        const RowGrid g = row_grid(T, vecs, 16, M::vecs);
        dispatch_kernel<M><<<g.grid, kRowThreads, 0, stream>>>(
            quant_args(x, ldx, H, k, q, scales, R), g.shape, slot_row);
    });
    return hipGetLastError();
}

hipError_t launch_moe_sort_dispatch(const MoeRouting &r, const GatherPlane &rows,
                                    hipStream_t stream) {
    const int64_t R = r.T * r.k;
    if (sort_dispatch_few<Gather<kCopy, false, 1>>(r, copy_args(rows, nullptr, r.k, R), (rows.bytes + 15) / 16,
                                 stream))
        return hipGetLastError();
    const hipError_t e = launch_moe_sort(r, stream);
    return e != hipSuccess ? e
                           : launch_moe_dispatch(rows, nullptr, r.slot_row, r.T, r.k, R, stream);
}

hipError_t launch_moe_sort_dispatch_quant(const MoeRouting &r, const void *x, int64_t ldx,
                                          int64_t H, void *q, float *scales, bool pow2,
                                          hipStream_t stream) {
    const int64_t R = r.T * r.k, vecs = (H + kGroup - 1) / kGroup * 16;
    const GatherArgs a = quant_args(x, ldx, H, r.k, q, scales, R);
    if (with_quant(pow2, H, false,
                   [&](auto m) { return sort_dispatch_few<decltype(m)>(r, a, vecs, stream); }))
        return hipGetLastError();
    const hipError_t e = launch_moe_sort(r, stream);
    return e != hipSuccess ? e
                           : launch_moe_dispatch_quant(x, ldx, r.T, H, r.slot_row, r.k, q, scales,
                                                       R, pow2, stream);
}

namespace {

// Whether the kept rows are loaded as read once, without a place in the
// caches: from 96 MiB on, more than the caches keep until the next reader
// (8 rows of 7168 bf16 values a token; weighted sum for 4096 tokens: rows just
// written 160 us with the write, against 198; not in the caches 96 against 108;
// gradient for 2048 tokens 99 against 105; weighted sum for 512 tokens, 59 MB,
// just written 28 with the write both ways).
bool read_once(int64_t rows, int64_t row_bytes) { return rows * row_bytes >= 96 << 20; }

}  // namespace

hipError_t launch_moe_combine(const void *ys, bool ys_bf16, int64_t ld, int64_t R,
                              const int32_t *slot_row, const float *weights, int64_t T,
                              int64_t k, int64_t H, const void *residual, int64_t ld_residual,
                              void *out, bool out_bf16, hipStream_t stream) {
    const int64_t vecs = (H + 7) / 8;
    const bool once = read_once(T * k, H * (ys_bf16 ? 2 : 4));
    const int per = k > 4 || T * vecs < kManyVecs ? 1 : k > 2 ? 2 : 4;
    const RowGrid g = row_grid(T, vecs, 16, per);
    auto go = [&](auto in, auto to) {
        using In = decltype(in);
        using Out = decltype(to);
        auto *kernel = H < 8  ? combine_kernel<In, Out, kBatch, 1, true, false>
                       : once ? per == 4   ? combine_kernel<In, Out, 2, 4, false, true>
                                : per == 2 ? combine_kernel<In, Out, 4, 2, false, true>
                                           : combine_kernel<In, Out, kBatch, 1, false, true>
                       : per == 4 ? combine_kernel<In, Out, 2, 4, false, false>
                       : per == 2 ? combine_kernel<In, Out, 4, 2, false, false>
                                  : combine_kernel<In, Out, kBatch, 1, false, false>;
        kernel<<<g.grid, kRowThreads, 0, stream>>>(
            static_cast<const In *>(ys), ld, R, slot_row, weights, g.shape, k, H,
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
    const int64_t vecs = (H + 7) / 8;
    const bool once = read_once(T * k, H * (bf16 ? 2 : 4));
    // Few tokens do not fill the card: there a row has up to 512 threads
    // (one token of 7168 values to 8 experts: 10.5 us with 1024 threads and
    // four slots at a time).  Else a thread that would have four slots or
    // fewer to load takes two or four vectors, and the row the fewer threads
    // (4096 tokens of 2048 values: 4 slots 48 -> 29 us, 2 slots 22 -> 16).
    const bool few = T < 256;
    const int per = few ? 1 : k <= 2 ? 4 : k <= 4 ? 2 : 1;
    const int threads = threads_per_row((vecs + per - 1) / per, 64, few ? 512 : 256);
    auto go = [&](auto v) {
        using V = decltype(v);
        auto *kernel = H < 8  ? combine_grad_kernel<V, 256, 4, 1, true, false>
                       : few  ? combine_grad_kernel<V, 512, kBatch, 1, false, false>
                       : once ? per == 4   ? combine_grad_kernel<V, 256, 2, 4, false, true>
                                : per == 2 ? combine_grad_kernel<V, 256, 4, 2, false, true>
                                           : combine_grad_kernel<V, 256, kBatch, 1, false, true>
                       : per == 4 ? combine_grad_kernel<V, 256, 2, 4, false, false>
                       : per == 2 ? combine_grad_kernel<V, 256, 4, 2, false, false>
                                  : combine_grad_kernel<V, 256, kBatch, 1, false, false>;
        kernel<<<blocks, threads, 0, stream>>>(static_cast<const V *>(dout), ld_dout,
                                               static_cast<const V *>(ys), ld_ys, R, slot_row,
                                               weights, T, k, H, static_cast<V *>(dys), dweights);
    };
    if (bf16) go(Bf16{}); else go(float{});
    return hipGetLastError();
}

}  // namespace fp8blk

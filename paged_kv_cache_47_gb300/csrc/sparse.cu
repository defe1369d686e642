// Block means, scores and selection for sparse decode (include/pkv_sparse.h).
//
// block_means: a warp per (token, kv head) whose token filled its block; a
// lane adds D / 32 neighbouring elements over the block's rows, eight rows'
// loads at a time. Latency: 2.5 us for a step. A wave of prompts has a warp for
// every token though one in B has work: 16384 tokens of 8 heads (34 MB) 19 us.
//
// Scores. A warp takes one kv head and a run of a sequence's blocks. Lanes hold
// 8 neighbouring elements of a mean each, so a row is 16 lanes (D 128) and a
// load two rows; the q heads of the group sit in registers as fp32 pairs, two
// heads an instruction. Products of 16-bit elements are exact in fp32, so a
// fused multiply-add equals the product and the addition the definition names;
// fp32 caches use the two steps. The sums over lanes halve the heads a lane
// carries at each step, which leaves the order of the additions as defined:
// neighbours first. What is kept of a score is its key: its bits made
// monotonic, a NaN as +infinity, -0 as +0. Bound by instructions: at 8 heads a
// group 100 of a warp for each 512 bytes of means (32 of them the paired
// multiply-adds), 0.5 a cycle with the 16 warps that q's registers leave room
// for. 94 MB of means (8 contexts of up to 131072 tokens) take 31 us, 3 TB/s;
// 67 us without pairs and with loads held in registers. Half the heads at a time
// with 24 warps reads means twice: 45 us.
//
// Selection. The candidates taken are those above the top-th largest key and
// the first of its equals. One warp finds that key bit by bit, counting keys in
// registers; a CTA by digits of 11 bits, a histogram in shared memory each
// (the first digit begins at the highest bit in which the row's keys differ:
// above it scores are nearly all alike and the histogram's atomics would
// queue). Both end as soon as a threshold leaves exactly `top`. Threads hold
// neighbouring candidates, so two scans over them give each its place in
// ascending order.
//
// Short rows, or enough of them to fill the GPU: one kernel, a CTA for each
// (sequence, kv head), keys in shared memory; up to 256 candidates one warp
// selects alone, with no barrier: 12 us for 512 rows of 27 to 251 candidates, a
// chain of latencies (lengths, tables, means, scores, 20 bits, tables again).
// Few long rows: a first kernel scores even runs of blocks all over the GPU, a
// second one selects, a CTA a row: 11 us for 64 rows of up to 8192 candidates
// (16 bit by bit; CTAs of 1024 threads 17).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/pkv_sparse.h"
#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "rows_internal.h"

namespace {

using pkv::add2;
using pkv::fma2;
using pkv::launch_chained;
using pkv::mul2;
using pkv::Pair;
using pkv::pair_of;
using pkv::unpair;

constexpr int kRowMost = 512;        // threads of a CTA that scores and selects one row: 128, 256 or 512
constexpr int kScoreThreads = 256;
constexpr int kSelThreads = 512;
constexpr int kPerThread = 16;       // keys a thread holds
constexpr int kPerLane = 8;          // keys a lane holds where a warp selects alone
constexpr int kMeanThreads = 256;

template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half round_to<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// ---------------------------------------------------------------- means
struct MeansParams {
    const int64_t *slots;
    int64_t rows;                    // tokens * Hk
    int Hk, NB, B;
    const void *k;
    void *means;
    unsigned *err;
};

template <typename T, int D>
__global__ void __launch_bounds__(kMeanThreads) block_means_kernel(const MeansParams p) {
    constexpr int E = D / 32;        // elements a lane: 2 or 4
    struct alignas(E * sizeof(T)) Part { T e[E]; };
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kMeanThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kMeanThreads / 32) + (threadIdx.x >> 5); r < p.rows; r += step) {
        const int64_t tok = r / p.Hk;
        const int g = (int)(r - tok * p.Hk);
        const int64_t slot = p.slots[tok];
        if (slot < 0) continue;
        const int64_t blk = slot / p.B;
        if (blk >= p.NB) {
            if (lane == 0 && g == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
            continue;
        }
        if (slot - blk * p.B != p.B - 1) continue;
        const int64_t chunk = blk * p.Hk + g;
        const Part *src = reinterpret_cast<const Part *>(static_cast<const T *>(p.k) + chunk * p.B * D) + lane;
        float sum[E];
        for (int t0 = 0; t0 < p.B; t0 += 8) {
            Part x[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) x[t] = src[(t0 + t) * 32];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float v = pkv::Elem<T>::to_f32(x[t].e[i]);
                    sum[i] = t0 + t == 0 ? v : sum[i] + v;
                }
        }
        Part out;
        const float inv = 1.f / (float)p.B;      // a power of two: exact
#pragma unroll
        for (int i = 0; i < E; ++i) out.e[i] = round_to<T>(sum[i] * inv);
        reinterpret_cast<Part *>(static_cast<T *>(p.means) + chunk * D)[lane] = out;
    }
}

// ---------------------------------------------------------------- scores
struct SelectParams {
    const void *q, *means;
    const int32_t *tables, *lens;
    int S, Hq, Hk, G, M, NB, B;
    int top, first, last, W;
    uint32_t *keys;                  // [S][Hk][pitch], by candidate; NULL: in shared memory
    int pitch;
    int32_t *sel_tables, *sel_lens;
    unsigned *err;
};

__device__ __forceinline__ int clamp_len(const SelectParams &p, int s, bool report) {
    const int L = __ldg(p.lens + s);
    const int cap = p.M * p.B;
    if (L >= 0 && L <= cap) return L;
    if (report) atomicOr(p.err, PKV_DEVERR_CONTEXT);
    return L < 0 ? 0 : cap;
}

__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) x = INFINITY;
    const uint32_t b = __float_as_uint(x + 0.f);     // -0 becomes +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The neighbouring 8 elements of a row, as fp32.
template <typename T>
__device__ __forceinline__ void widen(const uint4 (&raw)[sizeof(T) / 2], float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(raw[0].x), x[1] = __uint_as_float(raw[0].y);
        x[2] = __uint_as_float(raw[0].z), x[3] = __uint_as_float(raw[0].w);
        x[4] = __uint_as_float(raw[1].x), x[5] = __uint_as_float(raw[1].y);
        x[6] = __uint_as_float(raw[1].z), x[7] = __uint_as_float(raw[1].w);
    } else {
        const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pkv::Elem<T>::unpack2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// The stream of means of one warp: loads of 16 bytes a lane, kLoads a stage,
// kStages stages in the warp's ring in shared memory. A lane reads back only
// what it copied itself, so nothing is shared and nothing waits but its own
// copies; the ring only lengthens what registers could hold in flight.
constexpr int kStages = 3;
constexpr int kStageBytes = 4096;
constexpr int kRingBytes = kStages * kStageBytes;

// Scores of blocks [lo, hi) of sequence s for kv head g, as keys by candidate
// (block - first). One warp. GP q heads at a time: a group of any size takes
// several passes.
template <typename T, int D, int GP>
__device__ __forceinline__ void score_blocks(const SelectParams &p, int s, int g, int lo, int hi,
                                             uint32_t *keys, uint32_t ring) {
    constexpr int LANES = D / 8;     // lanes of a row
    constexpr int ROWS = 32 / LANES; // rows of a load
    constexpr int V = sizeof(T) / 2; // 16-byte pieces of a lane's elements
    constexpr int LOADS = kStageBytes / (512 * V);
    constexpr int STAGE_ROWS = ROWS * LOADS;         // 8, 16 or 32
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const int32_t *row = p.tables + (int64_t)s * p.M;
    const T *means = static_cast<const T *>(p.means) + (int64_t)g * D + 8 * l;
    const int64_t pitch = (int64_t)p.Hk * D;
    const uint32_t mine = ring + lane * 16;
    const int stages = (hi - lo + STAGE_ROWS - 1) / STAGE_ROWS;
    // NV sums are carried at a time, of `JOINT` loads and GP heads. Slot v of a
    // lane holds sum v ^ swap: the sums over lanes below keep the lower half of
    // the slots and give the upper one at each step, and the lanes' orders
    // differ so that what one keeps the other gives. In the end a lane has one
    // sum: the load is told by its low bits, the head by those after them.
    constexpr int JOINT = LANES / GP < LOADS ? LANES / GP : LOADS;
    constexpr int NV = JOINT * GP;
    int swap = 0;
#pragma unroll
    for (int t = 0; (NV >> (t + 1)) > 0; ++t) swap |= (l >> t & 1) * (NV >> (t + 1));
    const int swap_head = swap % GP, swap_load = swap / GP;

    // block ids of 32 rows, and of the 32 after them; -1: none
    auto ids_from = [&](int r) {
        const int j = lo + r + lane;
        int id = j < hi ? __ldg(row + j) : -1;
        if (j < hi && (unsigned)id >= (unsigned)p.NB) {
            if (g == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
            id = -1;
        }
        return id;
    };
    for (int h0 = 0; h0 < p.G; h0 += GP) {
        int ids = ids_from(0), next_ids = ids_from(32);
        auto issue = [&](int k) {
            if (k < stages) {
                const int r0 = k * STAGE_ROWS;
                if (k && r0 % 32 == 0) {
                    ids = next_ids;
                    next_ids = ids_from(r0 + 32);
                }
                const uint32_t dst = mine + (k % kStages) * kStageBytes;
#pragma unroll
                for (int a = 0; a < LOADS; ++a) {
                    const int id = __shfl_sync(~0u, ids, r0 % 32 + a * ROWS + sub);
                    const T *src = means + (id < 0 ? 0 : id) * pitch;
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        pkv::cp_async_16(dst + (a * V + v) * 512, src + v * (16 / sizeof(T)), id >= 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) issue(k);
        Pair q[(GP + 1) / 2][8];
#pragma unroll
        for (int h = 0; h < GP; h += 2) {
            float x[2][8] = {};
#pragma unroll
            for (int e = 0; e < 2 && h + e < GP; ++e) {
                // past the group: its first head again, which changes no maximum
                const int hh = h0 + ((h + e) ^ swap_head), head = g * p.G + (hh < p.G ? hh : h0);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) +
                                                                   ((int64_t)s * p.Hq + head) * D + 8 * l);
                uint4 raw[V];
#pragma unroll
                for (int v = 0; v < V; ++v) raw[v] = __ldg(src + v);
                widen<T>(raw, x[e]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) q[h / 2][i] = pair_of(x[0][i], x[1][i]);
        }
        for (int k = 0; k < stages; ++k) {
            issue(k + kStages - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint32_t from = mine + (k % kStages) * kStageBytes;
            float best = 0.f;
#pragma unroll 1
            for (int a0 = 0; a0 < LOADS; a0 += JOINT) {
                float acc[NV + 1];
#pragma unroll
                for (int a = 0; a < JOINT; ++a) {
                    uint4 raw[V];
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        pkv::lds_u32x4(from + (a0 * V + v) * 512 + ((a ^ swap_load) * V * 512), raw[v].x, raw[v].y,
                                       raw[v].z, raw[v].w);
                    float x[8];
                    widen<T>(raw, x);
                    Pair sum[(GP + 1) / 2];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const Pair xx = pair_of(x[i], x[i]);
#pragma unroll
                        for (int h = 0; h < (GP + 1) / 2; ++h) {
                            if (i == 0) sum[h] = mul2(q[h][0], xx);
                            else if (sizeof(T) == 4) sum[h] = add2(sum[h], mul2(q[h][i], xx));
                            else sum[h] = fma2(q[h][i], xx, sum[h]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < GP; h += 2) unpair(sum[h / 2], acc[a * GP + h], acc[a * GP + h + 1]);
                }
                // over the lanes of the row, neighbours first
#pragma unroll
                for (int o = 1, keep = NV; o < LANES; o <<= 1) {
                    if (keep > 1) {
                        keep >>= 1;
#pragma unroll
                        for (int v = 0; v < keep; ++v)
                            acc[v] = __fadd_rn(acc[v], __shfl_xor_sync(~0u, acc[v + keep], o));
                    } else {
                        acc[0] = __fadd_rn(acc[0], __shfl_xor_sync(~0u, acc[0], o));
                    }
                }
                // the largest over the heads
                float top = acc[0] != acc[0] ? INFINITY : acc[0];
#pragma unroll
                for (int o = JOINT; o < NV; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                if (l / JOINT == a0 / JOINT) best = top;
            }
            // lane l has the score of load l / JOINT * JOINT + swap_load, if there is one
            const int j = lo + k * STAGE_ROWS + (l / JOINT * JOINT + swap_load) * ROWS + sub;
            if (l < LOADS && j < hi) {
                uint32_t *out = keys + (j - p.first);
                const uint32_t key = key_of(best);
                *out = h0 ? max(*out, key) : key;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
}

// Candidates of sequence s, 0 where all of them are taken.
__device__ __forceinline__ int candidates(const SelectParams &p, int s) {
    const int n = (clamp_len(p, s, false) + p.B - 1) / p.B, cand = n - p.first - p.last;
    return cand > p.top ? cand : 0;
}

// Few rows: the candidates of all sequences end to end, in even runs; a group
// of Hk warps takes a run, a warp each kv head, so that the heads' means of a
// block, which lie side by side, are read together.
template <typename T, int D, int GP>
__global__ void __launch_bounds__(kScoreThreads, 2) block_scores_kernel(const SelectParams p) {
    extern __shared__ __align__(128) uint8_t rings[];
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = pkv::smem_u32(rings) + warp * kRingBytes;
    long long total = 0;
    for (int s0 = 0; s0 < p.S; s0 += 32) {
        const int s = s0 + lane;
        total += __reduce_add_sync(~0u, s < p.S ? candidates(p, s) : 0);
    }
    const int64_t warps = (int64_t)gridDim.x * (kScoreThreads / 32);
    const int64_t groups = warps / p.Hk > 0 ? warps / p.Hk : 1;
    for (int64_t task = (int64_t)blockIdx.x * (kScoreThreads / 32) + warp; task < groups * p.Hk; task += warps) {
        const int g = (int)(task % p.Hk);
        long long at = task / p.Hk * total / groups;
        const long long end = (task / p.Hk + 1) * total / groups;
        // the sequence that holds `at`, then on to `end`
        long long before = 0;
        for (int s0 = 0; s0 < p.S && at < end; s0 += 32) {
            const int mine = s0 + lane < p.S ? candidates(p, s0 + lane) : 0;
            const int sum = __reduce_add_sync(~0u, mine);
            if (before + sum <= at) {
                before += sum;
                continue;
            }
            for (int i = 0; i < 32 && at < end; ++i) {
                const int c = __shfl_sync(~0u, mine, i);
                if (before + c > at) {
                    const int lo = (int)(at - before), hi = (int)min((long long)c, end - before);
                    score_blocks<T, D, GP>(p, s0 + i, g, p.first + lo, p.first + hi,
                                           p.keys + ((int64_t)(s0 + i) * p.Hk + g) * p.pitch, ring);
                    at = before + hi;
                }
                before += c;
            }
        }
    }
}

// ---------------------------------------------------------------- selection
// Exclusive prefix of `v` over the CTA's threads, and the total.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();                 // earlier readers of warp_sums are done
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = inc - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before;
}

// The entry of block j in a selection of kv head g.
__device__ __forceinline__ int32_t entry_of(const SelectParams &p, const int32_t *row, int j, int g) {
    const int id = __ldg(row + j);
    if ((unsigned)id < (unsigned)p.NB) return id * p.Hk + g;
    if (g == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    return -1;
}

// N keys from candidate `at` on (a multiple of 4); 0 past the last, below every key.
template <int N>
__device__ __forceinline__ void load_keys(uint32_t (&key)[N], const uint32_t *keys, int at, int cand) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (at + i < cand) v = *reinterpret_cast<const uint4 *>(keys + at + i);
        key[i] = v.x;
        key[i + 1] = at + i + 1 < cand ? v.y : 0u;
        key[i + 2] = at + i + 2 < cand ? v.z : 0u;
        key[i + 3] = at + i + 3 < cand ? v.w : 0u;
    }
}

// Which of N keys are taken; `tie`: those equal to the threshold.
template <int N>
__device__ __forceinline__ uint32_t compare_keys(const uint32_t (&key)[N], uint32_t threshold, uint32_t &tie) {
    uint32_t take = 0;
    tie = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        take |= (uint32_t)(key[i] > threshold) << i;
        tie |= (uint32_t)(key[i] == threshold) << i;
    }
    return take;
}

// Adds the first of the ties to `take`: those of rank below `ties`.
__device__ __forceinline__ uint32_t add_ties(uint32_t take, uint32_t tie, int rank, int ties) {
    for (; tie && rank < ties; tie &= tie - 1, ++rank) take |= tie & -tie;
    return take;
}

// One warp, up to 32 * kPerLane candidates: `top` < cand of them to out.
__device__ __forceinline__ void warp_select(const SelectParams &p, const uint32_t *keys, int cand,
                                            const int32_t *row, int g, int32_t *out) {
    if (p.top == 0) return;
    const int lane = threadIdx.x & 31;
    uint32_t key[kPerLane];
    load_keys(key, keys, lane * kPerLane, cand);
    uint32_t low = ~0u, high = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        high = max(high, key[i]);
        if (key[i]) low = min(low, key[i]);
    }
    low = __reduce_min_sync(~0u, low);
    high = __reduce_max_sync(~0u, high);
    const int bits = 32 - __clz(low ^ high);     // the keys differ in these
    uint32_t threshold = bits == 32 ? 0 : low >> bits << bits;
    int above = 0, ties = INT32_MAX;
    bool exact = false;
    for (int bit = bits - 1; bit >= 0 && !exact; --bit) {
        const uint32_t test = threshold | (1u << bit);
        int c = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) c += key[i] >= test;
        c = __reduce_add_sync(~0u, c);
        if (c >= p.top) threshold = test;
        else above = c;
        exact = c == p.top;          // these and no others: nothing equal is left out
    }
    if (!exact) ties = p.top - above;
    uint32_t tie;
    uint32_t take = compare_keys(key, threshold, tie);
    int rank = __popc(tie), mine = rank;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, rank, o);
        if (lane >= o) rank += x;
    }
    take = add_ties(take, tie, rank - mine, ties);
    int at = __popc(take);
    mine = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, at, o);
        if (lane >= o) at += x;
    }
    at -= mine;
    for (; take; take &= take - 1)
        out[at++] = entry_of(p, row, p.first + lane * kPerLane + __ffs(take) - 1, g);
}

// The whole CTA, any number of candidates.
constexpr int kDigitBits = 11;
template <int THREADS>
struct SelectShared {
    int sums[THREADS / 32];
    uint32_t lows[THREADS / 32], highs[THREADS / 32];
    int bins[1 << kDigitBits];
    int bin, above;
};

template <int THREADS>
__device__ __forceinline__ void block_select(const SelectParams &p, const uint32_t *keys, int cand,
                                             const int32_t *row, int g, int32_t *out,
                                             SelectShared<THREADS> &sh) {
    if (p.top == 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int per_pass = THREADS * kPerThread;
    constexpr int kBins = 1 << kDigitBits, PER = kBins / THREADS;
    uint32_t key[kPerThread];
    load_keys(key, keys, tid * kPerThread, cand);
    // smallest and largest key
    uint32_t low = ~0u, high = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        high = max(high, key[i]);
        if (key[i]) low = min(low, key[i]);
    }
    for (int j = per_pass + tid; j < cand; j += THREADS) {
        low = min(low, keys[j]);
        high = max(high, keys[j]);
    }
    low = __reduce_min_sync(~0u, low);
    high = __reduce_max_sync(~0u, high);
    if (lane == 0) {
        sh.lows[warp] = low;
        sh.highs[warp] = high;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        low = min(low, sh.lows[w]);
        high = max(high, sh.highs[w]);
    }
    // the top-th largest key: its bits from `shift` up are those of `threshold`,
    // `above` keys are larger in these bits
    int shift = 32 - __clz(low ^ high), above = 0, total;
    uint32_t threshold = shift == 32 ? 0 : low >> shift << shift;
    bool exact = false;
    while (shift > 0 && !exact) {
        const int next = max(0, shift - kDigitBits);
        const uint32_t prefix = shift == 32 ? 0 : threshold >> shift;
        auto digit_of = [&](uint32_t k, bool &in) {
            in = k != 0 && (shift == 32 || k >> shift == prefix);
            return (int)(k >> next) & ((1 << (shift - next)) - 1);
        };
#pragma unroll
        for (int i = 0; i < PER; ++i) sh.bins[tid * PER + i] = 0;
        __syncthreads();
        bool in;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int d = digit_of(key[i], in);
            if (in) atomicAdd(&sh.bins[d], 1);
        }
        for (int j = per_pass + tid; j < cand; j += THREADS) {
            const int d = digit_of(keys[j], in);
            if (in) atomicAdd(&sh.bins[d], 1);
        }
        __syncthreads();
        // thread t holds PER bins from the top down; keys in bins above them
        int c[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = sh.bins[kBins - 1 - (tid * PER + i)];
            sum += c[i];
        }
        int before = above + block_prefix<THREADS>(sum, sh.sums, total);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < p.top && before + c[i] >= p.top) {
                sh.bin = kBins - 1 - (tid * PER + i);
                sh.above = before;
            }
            before += c[i];
        }
        __syncthreads();
        const int d = sh.bin;
        above = sh.above;
        threshold |= (uint32_t)d << next;
        exact = above + sh.bins[d] == p.top;     // the whole bin: nothing equal is left out
        shift = next;
        __syncthreads();                         // before the bins are cleared
    }
    // exact: every key from the threshold's bin up; else those above it and the
    // first of its equals
    const int ties = p.top - above;
    int written = 0, tied = 0;
    for (int base = 0; base < cand; base += per_pass) {
        const int j0 = base + tid * kPerThread;
        if (base) load_keys(key, keys, j0, cand);
        uint32_t tie, take;
        if (exact) {
            take = compare_keys(key, threshold - 1, tie);
        } else {
            take = compare_keys(key, threshold, tie);
            const int rank = tied + block_prefix<THREADS>(__popc(tie), sh.sums, total);
            tied += total;
            take = add_ties(take, tie, rank, ties);
        }
        int at = written + block_prefix<THREADS>(__popc(take), sh.sums, total);
        written += total;
        for (; take; take &= take - 1)
            out[at++] = entry_of(p, row, p.first + j0 + __ffs(take) - 1, g);
    }
}

// What every row has besides its chosen candidates: the first and last blocks
// (or all blocks), and its length. Threads from `from` on.
__device__ __forceinline__ void write_rest(const SelectParams &p, int r, int L, int n, bool all,
                                           const int32_t *row, int g, int from) {
    int32_t *out = p.sel_tables + (int64_t)r * p.W;
    const int step = blockDim.x - from, t = threadIdx.x - from;
    if (t < 0) return;
    if (all) {
        for (int w = t; w < p.W; w += step) out[w] = w < n ? entry_of(p, row, w, g) : -1;
    } else {
        for (int w = t; w < p.first; w += step) out[w] = entry_of(p, row, w, g);
        for (int w = t; w < p.last; w += step) out[p.first + p.top + w] = entry_of(p, row, n - p.last + w, g);
    }
    const int count = all ? n : p.W;
    if (t == 0) p.sel_lens[r] = n ? (count - 1) * p.B + L - (n - 1) * p.B : 0;
}

// Selects from the keys of block_scores_kernel.
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const SelectParams p) {
    __shared__ SelectShared<kSelThreads> sh;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int s = blockIdx.x / p.Hk, g = blockIdx.x - s * p.Hk;
    const int L = clamp_len(p, s, g == 0 && threadIdx.x == 0);
    const int n = (L + p.B - 1) / p.B, cand = n - p.last - p.first;
    const bool all = cand <= p.top;
    const int32_t *row = p.tables + (int64_t)s * p.M;
    write_rest(p, blockIdx.x, L, n, all, row, g, 0);
    if (!all)
        block_select<kSelThreads>(p, p.keys + (int64_t)blockIdx.x * p.pitch, cand, row, g,
                                  p.sel_tables + (int64_t)blockIdx.x * p.W + p.first, sh);
}

// Scores and selects one row.
template <typename T, int D, int GP>
__global__ void __launch_bounds__(kRowMost, 1) block_rows_kernel(const SelectParams p) {
    extern __shared__ __align__(128) uint8_t rings[];       // then the row's keys
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int warps = blockDim.x / 32;
    uint32_t *row_keys = reinterpret_cast<uint32_t *>(rings + warps * kRingBytes);
    static_assert(sizeof(SelectShared<128>) <= 4 * kRingBytes && sizeof(SelectShared<kRowMost>) <= 8 * kRingBytes,
                  "it takes the rings' place");
    const int s = blockIdx.x / p.Hk, g = blockIdx.x - s * p.Hk, warp = threadIdx.x >> 5;
    const int L = clamp_len(p, s, g == 0 && threadIdx.x == 0);
    const int n = (L + p.B - 1) / p.B, cand = n - p.last - p.first;
    const bool all = cand <= p.top;
    const int32_t *row = p.tables + (int64_t)s * p.M;
    if (all) {
        write_rest(p, blockIdx.x, L, n, true, row, g, 0);
        return;
    }
    // even shares, in whole loads
    const int share = ((cand + warps - 1) / warps + 3) & ~3;
    const int lo = p.first + min(cand, warp * share), hi = p.first + min(cand, (warp + 1) * share);
    if (lo < hi) score_blocks<T, D, GP>(p, s, g, lo, hi, row_keys, pkv::smem_u32(rings) + warp * kRingBytes);
    __syncthreads();
    int32_t *out = p.sel_tables + (int64_t)blockIdx.x * p.W + p.first;
    if (cand <= 32 * kPerLane) {
        if (warp == 0) warp_select(p, row_keys, cand, row, g, out);
        else write_rest(p, blockIdx.x, L, n, false, row, g, 32);
    } else {
        write_rest(p, blockIdx.x, L, n, false, row, g, 0);
        // (the rings are used up: the selection's histogram takes their place)
        auto select = [&](auto threads) {
            constexpr int T = decltype(threads)::value;
            block_select<T>(p, row_keys, cand, row, g, out, *reinterpret_cast<SelectShared<T> *>(rings));
        };
        if (warps == 4) select(std::integral_constant<int, 128>());
        else if (warps == 8) select(std::integral_constant<int, 256>());
        else select(std::integral_constant<int, kRowMost>());
    }
}

// ---------------------------------------------------------------- host
bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Keys of a row, padded to whole 16-byte loads.
int key_pitch(int64_t M) { return (int)((M + 3) / 4 * 4); }

constexpr int kRowShort = 1024;                  // table columns up to which a CTA a row is always taken
constexpr size_t kRowKeyBytes = 64 << 10;        // keys of a row in shared memory, at most (128 threads)

// A CTA for each (sequence, kv head): its threads, or 0 for the two kernels that
// spread a row over the GPU. One SM against many: 144 rows of 512 to 1024 blocks
// take 15.5 us by rows and 20.7 spread, 24 rows 13.2 and 13.8, 8 rows 12.4 and
// 11.1, but 64 rows of 2048 to 4096 blocks 30 and 21; with rows for twice the
// SMs the spread form's second kernel and keys in memory cost more (800 rows of
// 512 to 1024: 49 and 62). Threads: an SM holds 512, in up to four CTAs (144 rows
// of 128 to 256 blocks: 9.9, 8.2 and 6.9 us with 128, 256 and 512; 480 rows:
// 12.7, 14.8 and 21.4), and short rows do not fill many warps (144 rows of 32
// to 64: 5.1, 5.4 and 5.5). These are rows of tables about as wide as the longest
// context. The lengths are on the device, so a wider table chooses by its width:
// 512 rows of 32 to 256 blocks take 10.5 us up to 2048 columns and 13.3 with 8192
// (keys in shared memory for all columns), 64 such rows 5.8 up to 1024 columns
// and 13.4 past them (the spread form).
int row_threads(int64_t rows, int M, int pitch, int sms) {
    if (M > kRowShort && (rows < 2 * sms || (size_t)pitch * 4 > kRowKeyBytes)) return 0;
    return rows <= sms && M > 128 && M <= kRowShort ? 512 : rows <= 2 * sms && M > 64 && M <= kRowShort ? 256 : 128;
}

// Shared memory above the default 48 KB: an attribute of each kernel on each
// device, set once (`ready`: devices done).
template <typename K>
cudaError_t allow_smem(K *kernel, size_t bytes, std::atomic<uint64_t> &ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <typename T, int D, int GP>
struct Launch {
    static cudaError_t rows(const SelectParams &p, int threads, cudaStream_t stream) {
        static std::atomic<uint64_t> ready{0};
        constexpr size_t most = kRowMost / 32 * (size_t)kRingBytes + kRowShort * 4;
        static_assert(4 * kRingBytes + kRowKeyBytes <= most, "four warps and the longest row");
        const cudaError_t e = allow_smem(block_rows_kernel<T, D, GP>, most, ready);
        if (e != cudaSuccess) return e;
        return launch_chained(block_rows_kernel<T, D, GP>, dim3((unsigned)(p.S * p.Hk)), threads,
                              threads / 32 * (size_t)kRingBytes + (size_t)p.pitch * 4, stream, p);
    }
    static cudaError_t runs(const SelectParams &p, int sms, cudaStream_t stream) {
        static std::atomic<uint64_t> ready{0};
        constexpr size_t ring = (size_t)kScoreThreads / 32 * kRingBytes;
        cudaError_t e = allow_smem(block_scores_kernel<T, D, GP>, ring, ready);
        if (e != cudaSuccess) return e;
        e = launch_chained(block_scores_kernel<T, D, GP>, dim3((unsigned)(2 * sms)), kScoreThreads, ring, stream, p);
        if (e != cudaSuccess) return e;
        return launch_chained(block_select_kernel, dim3((unsigned)(p.S * p.Hk)), kSelThreads, 0, stream, p);
    }
};

template <typename T, int D, int GP>
cudaError_t launch_select(const SelectParams &p, int threads, int sms, cudaStream_t stream) {
    return threads ? Launch<T, D, GP>::rows(p, threads, stream) : Launch<T, D, GP>::runs(p, sms, stream);
}

template <typename T, int D>
cudaError_t launch_select_d(const SelectParams &p, int threads, int sms, cudaStream_t stream) {
    // heads at a time: the registers of q are 8 a head
    auto *go = p.G == 1   ? &launch_select<T, D, 1>
               : p.G == 2 ? &launch_select<T, D, 2>
               : p.G <= 4 ? &launch_select<T, D, 4>
                          : &launch_select<T, D, 8>;
    return go(p, threads, sms, stream);
}

template <typename T>
cudaError_t launch_select_t(int D, const SelectParams &p, int threads, int sms, cudaStream_t stream) {
    return D == 64 ? launch_select_d<T, 64>(p, threads, sms, stream) : launch_select_d<T, 128>(p, threads, sms, stream);
}

size_t score_bytes(const pkv_cache_desc *c, int64_t S, int64_t M) {
    return (size_t)S * c->num_kv_heads * key_pitch(M) * 4;
}

// Workspace of the decode over a selection: 16-bit caches have a kernel for many
// short contexts, fp32 ones take the split-K decode.
size_t selection_decode_bytes(const pkv_cache_desc *c, int Hq) {
    const size_t n = c->dtype == PKV_F32 ? pkv_decode_workspace_bytes_ex(c, Hq, 0)
                                         : pkv::rows_workspace_bytes(Hq / c->num_kv_heads, c->head_dim);
    return (n + 15) / 16 * 16;
}

pkv_status check_batch(const pkv_cache_desc *c, int32_t S, int32_t M) {
    pkv_status st = pkv::check_cache_desc(c);
    if (st != PKV_OK) return st;
    if (S < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", S);
    if (M < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", M);
    if ((int64_t)c->num_blocks * c->num_kv_heads > INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is 2^31 or more");
    if ((int64_t)M * c->block_size > INT32_MAX || (int64_t)S * c->num_kv_heads > INT32_MAX / 64)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
    return PKV_OK;
}

pkv_status check_select(const pkv_cache_desc *c, int32_t S, int32_t Hq, int32_t M) {
    const pkv_status st = check_batch(c, S, M);
    if (st != PKV_OK) return st;
    if (Hq < 1 || Hq % c->num_kv_heads)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "num_q_heads %d is not a positive multiple of num_kv_heads %d", Hq,
                                   c->num_kv_heads);
    return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_block_means(const pkv_cache_desc *cache, const int64_t *slot_mapping,
                           int32_t num_tokens, const void *k_pool, void *k_means, void *stream) {
    pkv_status st = pkv::check_cache_desc(cache);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", num_tokens);
    if (num_tokens == 0) return PKV_OK;
    if (!slot_mapping || !k_pool || !k_means)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(slot_mapping, 8) || misaligned(k_pool, 16) || misaligned(k_means, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "k_pool and k_means must be 16-byte aligned (slot_mapping 8)");
    MeansParams p = {};
    if ((st = pkv::device_error_word(&p.err)) != PKV_OK) return st;
    p.slots = slot_mapping;
    p.rows = (int64_t)num_tokens * cache->num_kv_heads;
    p.Hk = cache->num_kv_heads;
    p.NB = cache->num_blocks;
    p.B = cache->block_size;
    p.k = k_pool;
    p.means = k_means;
    const bool d64 = cache->head_dim == 64;
    auto *kernel = cache->dtype == PKV_F32
                       ? (d64 ? &block_means_kernel<float, 64> : &block_means_kernel<float, 128>)
                   : cache->dtype == PKV_F16
                       ? (d64 ? &block_means_kernel<__half, 64> : &block_means_kernel<__half, 128>)
                       : (d64 ? &block_means_kernel<__nv_bfloat16, 64>
                              : &block_means_kernel<__nv_bfloat16, 128>);
    int64_t grid = (p.rows + kMeanThreads / 32 - 1) / (kMeanThreads / 32);
    if (grid > 16384) grid = 16384;
    const cudaError_t e = launch_chained(kernel, dim3((unsigned)grid), kMeanThreads, 0,
                                         static_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess)
        return pkv::set_last_error(PKV_ERR_CUDA, "block_means launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

size_t pkv_select_workspace_bytes(const pkv_cache_desc *cache, int32_t num_seqs,
                                  int32_t max_blocks_per_seq) {
    if (check_batch(cache, num_seqs, max_blocks_per_seq) != PKV_OK) return 0;
    const size_t n = score_bytes(cache, num_seqs, max_blocks_per_seq);
    return n ? n : 16;
}

pkv_status pkv_select_blocks(const pkv_cache_desc *cache, const void *q, int32_t num_seqs,
                             int32_t num_q_heads, const void *k_means,
                             const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *context_lens, const pkv_sparse_select *select,
                             int32_t *sel_tables, int32_t *sel_lens, void *workspace,
                             size_t workspace_bytes, void *stream) {
    pkv_status st = check_select(cache, num_seqs, num_q_heads, max_blocks_per_seq);
    if (st != PKV_OK) return st;
    if (!select) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "the selection is NULL");
    if (select->top_blocks < 0 || select->first_blocks < 0 || select->last_blocks < 1)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "selection %d, %d, %d (top >= 0, first >= 0, last >= 1)",
                                   select->top_blocks, select->first_blocks, select->last_blocks);
    const int64_t W = (int64_t)select->top_blocks + select->first_blocks + select->last_blocks;
    if (W > INT32_MAX / 64)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "a selection of %lld blocks", (long long)W);
    if (num_seqs == 0) return PKV_OK;
    if (!q || !k_means || !block_tables || !context_lens || !sel_tables || !sel_lens)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(q, 16) || misaligned(k_means, 16) || misaligned(block_tables, 4) ||
        misaligned(context_lens, 4) || misaligned(sel_tables, 4) || misaligned(sel_lens, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "q and k_means must be 16-byte aligned");
    const size_t need = score_bytes(cache, num_seqs, max_blocks_per_seq);
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    SelectParams p = {};
    if ((st = pkv::device_error_word(&p.err)) != PKV_OK) return st;
    p.q = q;
    p.means = k_means;
    p.tables = block_tables;
    p.lens = context_lens;
    p.S = num_seqs;
    p.Hq = num_q_heads;
    p.Hk = cache->num_kv_heads;
    p.G = num_q_heads / cache->num_kv_heads;
    p.M = max_blocks_per_seq;
    p.NB = cache->num_blocks;
    p.B = cache->block_size;
    p.top = select->top_blocks;
    p.first = select->first_blocks;
    p.last = select->last_blocks;
    p.W = (int)W;
    p.pitch = key_pitch(max_blocks_per_seq);
    p.keys = static_cast<uint32_t *>(workspace);
    p.sel_tables = sel_tables;
    p.sel_lens = sel_lens;
    int sms = 0;
    if ((st = pkv::device_sm_count(&sms)) != PKV_OK) return st;
    const int threads = row_threads((int64_t)num_seqs * p.Hk, max_blocks_per_seq, p.pitch, sms);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dtype == PKV_F32   ? launch_select_t<float>(cache->head_dim, p, threads, sms, s)
                          : cache->dtype == PKV_F16 ? launch_select_t<__half>(cache->head_dim, p, threads, sms, s)
                                                    : launch_select_t<__nv_bfloat16>(cache->head_dim, p, threads, sms, s);
    if (e != cudaSuccess)
        return pkv::set_last_error(PKV_ERR_CUDA, "block selection launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

size_t pkv_decode_sparse_workspace_bytes(const pkv_cache_desc *cache, int32_t num_seqs,
                                         int32_t num_q_heads, int32_t max_blocks_per_seq) {
    if (check_select(cache, num_seqs, num_q_heads, max_blocks_per_seq) != PKV_OK) return 0;
    const size_t dec = selection_decode_bytes(cache, num_q_heads);
    return dec ? dec + score_bytes(cache, num_seqs, max_blocks_per_seq) : 0;
}

pkv_status pkv_decode_attention_sparse(const pkv_cache_desc *cache, const void *q,
                                       int32_t num_seqs, int32_t num_q_heads, const void *k_pool,
                                       const void *v_pool, const void *k_means,
                                       const int32_t *block_tables, int32_t max_blocks_per_seq,
                                       const int32_t *context_lens, float scale,
                                       const pkv_sparse_select *select, int32_t *sel_tables,
                                       int32_t *sel_lens, void *out, int32_t out_dtype,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    pkv_status st = check_select(cache, num_seqs, num_q_heads, max_blocks_per_seq);
    if (st != PKV_OK) return st;
    // the decode's own checks come before anything is enqueued
    if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
    if (!isfinite(scale)) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "scale is not finite");
    if (num_seqs == 0) return PKV_OK;
    if (!k_pool || !v_pool || !out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(out, out_dtype == PKV_F32 ? 16 : 8))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "the pools must be 16-byte aligned, out to four of its elements");
    const size_t need = pkv_decode_sparse_workspace_bytes(cache, num_seqs, num_q_heads, max_blocks_per_seq);
    if (need == 0) return PKV_ERR_CUDA;      // the message is set
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    // what one launch of the decode holds: so many (sequence, kv head) contexts of W blocks
    const int64_t heads = num_q_heads / cache->num_kv_heads;
    const int64_t blocks = select ? (int64_t)select->top_blocks + select->first_blocks + select->last_blocks : 0;
    if (pkv::kRowsMaxSeqs * ((heads + 7) / 8) * (blocks * cache->block_size / 16 + 3) >= INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "selection too large for one launch");
    // [decode workspace][scores]: the decode's counters lie first, as it wants them
    const size_t dec = selection_decode_bytes(cache, num_q_heads);
    if ((st = pkv_select_blocks(cache, q, num_seqs, num_q_heads, k_means, block_tables,
                                max_blocks_per_seq, context_lens, select, sel_tables, sel_lens,
                                static_cast<uint8_t *>(workspace) + dec, workspace_bytes - dec,
                                stream)) != PKV_OK)
        return st;
    // each (sequence, kv head) is a sequence over a pool of one-head blocks
    pkv_cache_desc view = *cache;
    view.num_blocks = cache->num_blocks * cache->num_kv_heads;
    view.num_kv_heads = 1;
    const int S = num_seqs * cache->num_kv_heads, Hq = num_q_heads / cache->num_kv_heads;
    if (cache->dtype != PKV_F32)
        return pkv::decode_rows(&view, q, S, Hq, k_pool, v_pool, sel_tables, (int)blocks, sel_lens, scale, out,
                                out_dtype, workspace, static_cast<cudaStream_t>(stream));
    return pkv_decode_attention(&view, q, S, Hq, k_pool, v_pool, sel_tables, (int)blocks, sel_lens, scale, out,
                                out_dtype, workspace, dec, stream);
}

}  // extern "C"

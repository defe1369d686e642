// Block means, scores and selection for sparse decode (include/pkv_sparse.h).
//
// block_means: a warp per (token, kv head) whose token filled its block; a
// lane adds 4 (fp32: 2 x 2) neighbouring elements over the block's rows.
//
// block_scores: a warp takes one kv head and 64 of a sequence's blocks. Lanes
// hold 8 neighbouring elements of a mean each, so a row is 16 lanes (D 128),
// two rows a load; the q heads of the group sit in registers as fp32. Products
// of 16-bit elements are exact in fp32, so a fused multiply-add equals the
// product and the addition the definition names; fp32 caches use the two
// steps. The sums over lanes halve the heads a lane carries at each step,
// which leaves the order of the additions as defined: neighbours first.
// Bound by HBM on long contexts: each mean is read once.
//
// block_select: a CTA per (sequence, kv head). The key of a score is its bits
// made monotonic; the selected ones are those above the top-th largest key and
// the first of its equals. That key is found bit by bit, counting in registers
// (no shared-memory histogram: the high bits of scores are nearly all alike
// and its atomics would queue). Threads hold neighbouring blocks, so two scans
// over the threads give each selected block its place in ascending order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pkv_sparse.h"
#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"

namespace {

using pkv::launch_chained;

constexpr int kChunk = 64;           // blocks a warp scores
constexpr int kScoreThreads = 256;
constexpr int kSelThreads = 512;
constexpr int kPerThread = 16;       // keys a thread holds: 8192 blocks a pass
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
        if (slot < 0 || slot % p.B != p.B - 1) continue;
        const int64_t blk = slot / p.B;
        if (blk >= p.NB) {
            if (lane == 0 && g == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
            continue;
        }
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
    int chunks;                      // of kChunk blocks, a table row
    int top, first, last, W;
    float *scores;                   // [S][Hk][M]
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

// GP q heads at a time (a group of any size takes several passes)
template <typename T, int D, int GP>
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(const SelectParams p) {
    constexpr int LANES = D / 8;     // lanes of a row
    constexpr int ROWS = 32 / LANES; // rows of a load
    constexpr int AHEAD = 4;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const int64_t task = (int64_t)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
    const int g = (int)(task % p.Hk);
    const int64_t sc = task / p.Hk;
    const int chunk = (int)(sc % p.chunks), s = (int)(sc / p.chunks);
    if (s >= p.S) return;
    const int L = clamp_len(p, s, chunk == 0 && g == 0 && lane == 0);
    const int n = (L + p.B - 1) / p.B;
    // candidates of this chunk; nothing to score where all of them are taken
    const int lo = max(p.first, chunk * kChunk), hi = min(n - p.last, (chunk + 1) * kChunk);
    if (lo >= hi || n - p.last - p.first <= p.top) return;
    const int32_t *row = p.tables + (int64_t)s * p.M;
    float *out = p.scores + ((int64_t)s * p.Hk + g) * p.M;
    for (int h0 = 0; h0 < p.G; h0 += GP) {
        float q[GP][8];
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            // past the group: its first head again, which changes no maximum
            const int head = g * p.G + (h0 + h < p.G ? h0 + h : h0);
            const T *src = static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + head) * D + 8 * l;
#pragma unroll
            for (int i = 0; i < 8; ++i) q[h][i] = pkv::Elem<T>::to_f32(src[i]);
        }
        for (int j0 = lo; j0 < hi; j0 += ROWS * AHEAD) {
            uint4 x[AHEAD][sizeof(T) / 2];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int j = j0 + a * ROWS + sub;
                int id = j < hi ? __ldg(row + j) : -1;
                const bool ok = id >= 0 && id < p.NB;
                if (!ok && j < hi && l == 0 && g == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(p.means) + ((int64_t)(ok ? id : 0) * p.Hk + g) * D + 8 * l);
#pragma unroll
                for (int v = 0; v < (int)sizeof(T) / 2; ++v)
                    x[a][v] = ok ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int j = j0 + a * ROWS + sub;
                const T *m = reinterpret_cast<const T *>(x[a]);
                float acc[GP];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = pkv::Elem<T>::to_f32(m[i]);
#pragma unroll
                    for (int h = 0; h < GP; ++h) {
                        if (i == 0) acc[h] = __fmul_rn(q[h][0], v);
                        else if (sizeof(T) == 4) acc[h] = __fadd_rn(acc[h], __fmul_rn(q[h][i], v));
                        else acc[h] = fmaf(q[h][i], v, acc[h]);
                    }
                }
                // over the lanes of the row; a lane keeps half of its heads at
                // each step while it has more than one
#pragma unroll
                for (int o = 1, keep = GP; o < LANES; o <<= 1) {
                    if (keep > 1) {
                        keep >>= 1;
                        const bool up = l & o;
#pragma unroll
                        for (int h = 0; h < keep; ++h) {
                            const float give = up ? acc[h] : acc[h + keep];
                            const float mine = up ? acc[h + keep] : acc[h];
                            acc[h] = __fadd_rn(mine, __shfl_xor_sync(~0u, give, o));
                        }
                    } else {
                        acc[0] = __fadd_rn(acc[0], __shfl_xor_sync(~0u, acc[0], o));
                    }
                }
                // the largest over the heads: those this lane kept, then over the lanes
                constexpr int KEPT = GP > LANES ? GP / LANES : 1;
                float best = acc[0];
                bool nan = acc[0] != acc[0];
#pragma unroll
                for (int h = 1; h < KEPT; ++h) {
                    best = fmaxf(best, acc[h]);
                    nan |= acc[h] != acc[h];
                }
                if (nan) best = INFINITY;
#pragma unroll
                for (int o = 1; o < LANES && o < GP; o <<= 1)
                    best = fmaxf(best, __shfl_xor_sync(~0u, best, o));
                if (l == 0 && j < hi) out[j] = h0 ? fmaxf(out[j], best) : best;
            }
        }
    }
}

// ---------------------------------------------------------------- selection
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) x = INFINITY;
    const uint32_t b = __float_as_uint(x + 0.f);     // -0 becomes +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix of `v` over the CTA's threads, and the total.
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
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before;
}

__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const SelectParams p) {
    __shared__ int sums[kSelThreads / 32];
    __shared__ int counts[2][kSelThreads / 32];
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / p.Hk, g = blockIdx.x - s * p.Hk;
    const int L = clamp_len(p, s, false);
    const int n = (L + p.B - 1) / p.B;
    const int32_t *row = p.tables + (int64_t)s * p.M;
    int32_t *out = p.sel_tables + (int64_t)blockIdx.x * p.W;
    const float *score = p.scores + (int64_t)blockIdx.x * p.M;
    // candidates are [first, end); all blocks are listed where they are few
    const int first = p.first, end = n - p.last, cand = end - first;
    const bool all = cand <= p.top;

    uint32_t threshold = 0;          // the top-th largest key
    int ties = 0;                    // how many of its equals are taken, in order
    const int per_pass = kSelThreads * kPerThread;
    const bool one_pass = cand <= per_pass;
    uint32_t key[kPerThread];
    if (!all) {
        if (one_pass) {
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const int j = first + tid * kPerThread + i;
                key[i] = j < end ? key_of(__ldcg(score + j)) : 0u;   // below every real key
            }
        }
        // the largest key that at least `top` keys reach, bit by bit
        int above = 0;               // keys above the final threshold
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t test = threshold | (1u << bit);
            int c = 0;
            if (one_pass) {
#pragma unroll
                for (int i = 0; i < kPerThread; ++i) c += key[i] >= test;
            } else {
                for (int j = first + tid; j < end; j += kSelThreads) c += key_of(__ldcg(score + j)) >= test;
            }
            c = __reduce_add_sync(~0u, c);
            if (lane == 0) counts[bit & 1][warp] = c;
            __syncthreads();         // the other buffer is free: its readers came before
            c = 0;
#pragma unroll
            for (int w = 0; w < kSelThreads / 32; ++w) c += counts[bit & 1][w];
            if (c >= p.top) threshold = test;
            else above = c;
            if (c == p.top) {        // these and no others: nothing equal is left out
                above = -1;
                break;
            }
        }
        ties = above < 0 ? INT32_MAX : p.top - above;
        if (p.top == 0) ties = 0;
    }

    // walk the blocks in order; a thread holds neighbours
    int written = 0, tied = 0;       // over the passes before
    for (int base = 0; base < n; base += per_pass) {
        const int j0 = base + tid * kPerThread;
        uint32_t take = 0, tie = 0;  // a bit for each of the thread's blocks
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int j = j0 + i;
            if (j >= n) continue;
            if (all || j < first || j >= end) {
                take |= 1u << i;
            } else if (p.top > 0) {
                const uint32_t k = key_of(__ldcg(score + j));
                if (k > threshold) take |= 1u << i;
                else if (k == threshold) tie |= 1u << i;
            }
        }
        int total;
        int rank = tied + block_prefix(__popc(tie), sums, total);
        tied += total;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
            if (tie >> i & 1 && rank++ < ties) take |= 1u << i;
        int at = written + block_prefix(__popc(take), sums, total);
        written += total;
        for (; take; take &= take - 1) {
            const int id = __ldg(row + j0 + __ffs(take) - 1);
            const bool ok = id >= 0 && id < p.NB;
            if (!ok && g == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
            if (at < p.W) out[at] = ok ? id * p.Hk + g : -1;
            ++at;
        }
    }
    for (int w = written + tid; w < p.W; w += kSelThreads) out[w] = -1;
    if (tid == 0) p.sel_lens[blockIdx.x] = n ? (written - 1) * p.B + L - (n - 1) * p.B : 0;
}

// ---------------------------------------------------------------- host
bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

template <typename T, int D>
cudaError_t launch_scores(const SelectParams &p, cudaStream_t stream) {
    const int64_t tasks = (int64_t)p.S * p.chunks * p.Hk;
    const dim3 grid((unsigned)((tasks + kScoreThreads / 32 - 1) / (kScoreThreads / 32)));
    // heads at a time: the registers of q are 8 a head
    auto *kernel = p.G == 1   ? &block_scores_kernel<T, D, 1>
                   : p.G == 2 ? &block_scores_kernel<T, D, 2>
                   : p.G <= 4 ? &block_scores_kernel<T, D, 4>
                              : &block_scores_kernel<T, D, 8>;
    return launch_chained(kernel, grid, kScoreThreads, 0, stream, p);
}

template <typename T>
cudaError_t launch_scores_for(int D, const SelectParams &p, cudaStream_t stream) {
    return D == 64 ? launch_scores<T, 64>(p, stream) : launch_scores<T, 128>(p, stream);
}

size_t score_bytes(const pkv_cache_desc *c, int64_t S, int64_t M) {
    return (size_t)(((S * c->num_kv_heads * M * 4) + 15) / 16 * 16);
}

pkv_status check_select(const pkv_cache_desc *c, int32_t S, int32_t Hq, int32_t M) {
    pkv_status st = pkv::check_cache_desc(c);
    if (st != PKV_OK) return st;
    if (S < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", S);
    if (Hq < 1 || Hq % c->num_kv_heads)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "num_q_heads %d is not a positive multiple of num_kv_heads %d", Hq,
                                   c->num_kv_heads);
    if (M < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", M);
    if ((int64_t)c->num_blocks * c->num_kv_heads > INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is 2^31 or more");
    if ((int64_t)M * c->block_size > INT32_MAX || (int64_t)S * c->num_kv_heads > INT32_MAX / 64 ||
        (int64_t)S * c->num_kv_heads * ((M + kChunk - 1) / kChunk) / 8 >= INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
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
    if (pkv::check_cache_desc(cache) != PKV_OK || num_seqs < 0 || max_blocks_per_seq < 1) return 0;
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
    p.chunks = (max_blocks_per_seq + kChunk - 1) / kChunk;
    p.top = select->top_blocks;
    p.first = select->first_blocks;
    p.last = select->last_blocks;
    p.W = (int)W;
    p.scores = static_cast<float *>(workspace);
    p.sel_tables = sel_tables;
    p.sel_lens = sel_lens;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cache->dtype == PKV_F32   ? launch_scores_for<float>(cache->head_dim, p, s)
                    : cache->dtype == PKV_F16 ? launch_scores_for<__half>(cache->head_dim, p, s)
                                              : launch_scores_for<__nv_bfloat16>(cache->head_dim, p, s);
    if (e == cudaSuccess)
        e = launch_chained(block_select_kernel, dim3((unsigned)(num_seqs * p.Hk)), kSelThreads, 0, s, p);
    if (e != cudaSuccess)
        return pkv::set_last_error(PKV_ERR_CUDA, "block selection launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

size_t pkv_decode_sparse_workspace_bytes(const pkv_cache_desc *cache, int32_t num_seqs,
                                         int32_t num_q_heads, int32_t max_blocks_per_seq) {
    if (check_select(cache, num_seqs, num_q_heads, max_blocks_per_seq) != PKV_OK) return 0;
    const size_t dec = pkv_decode_workspace_bytes_ex(cache, num_q_heads, 0);
    return dec ? (dec + 15) / 16 * 16 + score_bytes(cache, num_seqs, max_blocks_per_seq) : 0;
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
    if (misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(out, out_dtype == PKV_F32 ? 4 : 2))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
    const size_t need = pkv_decode_sparse_workspace_bytes(cache, num_seqs, num_q_heads, max_blocks_per_seq);
    if (need == 0) return PKV_ERR_CUDA;      // the message is set
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    const int64_t heads = num_q_heads / cache->num_kv_heads;
    const int64_t tiles = select ? (((int64_t)select->top_blocks + select->first_blocks +
                                     select->last_blocks) * cache->block_size + 63) / 64 : 0;
    if (1024 * ((heads + 15) / 16) * tiles >= INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "selection too large for one launch");
    // [decode workspace][scores]: the decode's counters lie first, as it wants them
    const size_t dec = (pkv_decode_workspace_bytes_ex(cache, num_q_heads, 0) + 15) / 16 * 16;
    if ((st = pkv_select_blocks(cache, q, num_seqs, num_q_heads, k_means, block_tables,
                                max_blocks_per_seq, context_lens, select, sel_tables, sel_lens,
                                static_cast<uint8_t *>(workspace) + dec, workspace_bytes - dec,
                                stream)) != PKV_OK)
        return st;
    // each (sequence, kv head) is a sequence over a pool of one-head blocks
    pkv_cache_desc view = *cache;
    view.num_blocks = cache->num_blocks * cache->num_kv_heads;
    view.num_kv_heads = 1;
    return pkv_decode_attention(&view, q, num_seqs * cache->num_kv_heads,
                                num_q_heads / cache->num_kv_heads, k_pool, v_pool, sel_tables,
                                select->top_blocks + select->first_blocks + select->last_blocks,
                                sel_lens, scale, out, out_dtype, workspace, dec, stream);
}

}  // extern "C"

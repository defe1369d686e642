// Drafted tokens as trees: masks and positions, the branch that holds, and its
// rows moved together (include/pkv_tree.h).
//
// Ancestors. A CTA takes a sequence, a thread each drafted token, with its mask
// (itself, to begin with) and a pointer to its parent. Each round a token takes
// over the mask of the token it points to, and its pointer: after r rounds it
// knows the 2^r tokens above it, so a chain of 256 takes 8 rounds and not 256
// steps. Depth is the mask's population less one. Acceptance is the same walk
// with one more bit: whether all tokens passed so far hold; the path is then
// the mask of the deepest token that holds, and a token's place on it its own
// depth, so that nothing is walked one by one.
//
// Commit. A thread owns one 16-byte column of K and V of a sequence and moves
// the path's rows in order, eight loaded before any is stored. Path and
// places ascend, p_k >= k: a row that is written over at step k has place k,
// which later steps (p_j >= j > k) do not read. No thread reads what another
// writes.
//
// What bounds them: latency. A launch, two dependent loads, the rounds, a store.
// Masks and positions of 64 requests of 16 tokens take 3.5 us, the host's call (2.2
// replayed as a graph), of 997 requests of up to 256 tokens, three axes, 9.2: 6.6
// CTAs an SM and 8 rounds each. The commit is bound by HBM where it has work:
// append, accept, commit and blocks back for 199 requests of up to 64 tokens, 40 kv
// heads of 128, 330 MB, 57 us (5.8 TB/s, 0.86 of a copy); 64 requests of 16 tokens, 8
// kv heads 19, four calls of the host (10.4 as a graph).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv_tree.h"
#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "tree_internal.h"

namespace {

using pkv::launch_chained;
using pkv::TreeBatch;
using pkv::TreeSeq;

template <int W>
struct Walk {
    unsigned long long mask[2][64 * W][W];
    short up[2][64 * W];                 // token above the ones known, -1: none
    bool holds[2][64 * W];
};

// Each of the CTA's tokens i < n (a thread each) learns the tokens above it, and
// whether it and all of them hold.
template <int W, bool HOLDS>
__device__ __forceinline__ void walk_up(Walk<W> &sh, int n, int parent, unsigned long long (&m)[W], bool &holds) {
    const int i = threadIdx.x;
#pragma unroll
    for (int w = 0; w < W; ++w) m[w] = i / 64 == w ? 1ull << (i % 64) : 0;
    int up = i < n ? parent : -1;
    for (int b = 0; __syncthreads_or(up >= 0); b ^= 1) {
#pragma unroll
        for (int w = 0; w < W; ++w) sh.mask[b][i][w] = m[w];
        sh.up[b][i] = (short)up;
        if (HOLDS) sh.holds[b][i] = holds;
        __syncthreads();
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < W; ++w) m[w] |= sh.mask[b][up][w];
            if (HOLDS) holds = holds && sh.holds[b][up];
            up = sh.up[b][up];
        }
    }
}

// The token's parent, -1 for none and for a bad one (which is flagged).
__device__ __forceinline__ int load_parent(const int32_t *parents, int at, int i, unsigned *err, bool &bad) {
    bad = false;
    if (!parents) return i - 1;
    const int p = parents[at];
    if (p >= -1 && p < i) return p;
    atomicOr(err, PKV_DEVERR_TREE);
    bad = true;
    return -1;
}

template <int W>
__device__ __forceinline__ int population(const unsigned long long (&m)[W]) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n += __popcll(m[w]);
    return n;
}

struct PlanParams {
    TreeBatch b;
    const int32_t *parents, *deltas;
    uint64_t *masks;
    int32_t *positions;
    int axes;
};

template <int W>
__global__ void __launch_bounds__(64 * W) tree_plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ Walk<W> sh;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int s = blockIdx.x, i = threadIdx.x;
    const TreeSeq q = pkv::tree_seq(p.b, s, i == 0);
    const int at = q.o + i;
    bool bad, unused = true;
    const int parent = i < q.n ? load_parent(p.parents, at, i, p.b.err, bad) : -1;
    unsigned long long m[W];
    walk_up<W, false>(sh, q.n, parent, m, unused);
    if (i >= q.n) return;
    if (p.masks)
#pragma unroll
        for (int w = 0; w < W; ++w) p.masks[(size_t)at * W + w] = m[w];
    if (p.positions) {
        const int pos = q.L - q.n + (p.deltas ? p.deltas[s] : 0) + population<W>(m) - 1;
        for (int a = 0; a < p.axes; ++a) p.positions[(size_t)a * p.b.T + at] = pos;
    }
}

struct AcceptParams {
    TreeBatch b;
    const int32_t *parents, *tokens, *targets;
    int32_t *path, *counts, *next, *lens_out;
};

template <int W>
__global__ void __launch_bounds__(64 * W) tree_accept_kernel(const __grid_constant__ AcceptParams p) {
    __shared__ Walk<W> sh;
    __shared__ int best;
    __shared__ unsigned long long chosen[W];
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int s = blockIdx.x, i = threadIdx.x;
    const TreeSeq q = pkv::tree_seq(p.b, s, i == 0);
    const int at = q.o + i;
    bool holds = false, bad = false;
    int parent = -1;
    if (i < q.n) {
        parent = load_parent(p.parents, at, i, p.b.err, bad);
        holds = !bad && (parent < 0 || p.tokens[at] == p.targets[q.o + parent]);
    }
    if (i == 0) best = -1;
    unsigned long long m[W];
    walk_up<W, true>(sh, q.n, parent, m, holds);     // (its barrier orders `best` too)
    const int depth = population<W>(m) - 1;
    // the deepest that holds, of equals the first
    if (holds) atomicMax(&best, depth * 256 + 255 - i);
    __syncthreads();
    const int last = best < 0 ? -1 : 255 - best % 256, count = best < 0 ? 0 : best / 256 + 1;
    if (i == last)
#pragma unroll
        for (int w = 0; w < W; ++w) chosen[w] = m[w];
    __syncthreads();
    if (i < q.n) {
        if (i >= count) p.path[at] = -1;
        if (last >= 0 && (chosen[i / 64] >> (i % 64) & 1)) p.path[q.o + depth] = i;
    }
    if (i == 0) {
        p.counts[s] = count;
        p.next[s] = last < 0 ? -1 : p.targets[q.o + last];
        p.lens_out[s] = q.raw - q.n + count;
    }
}

struct CommitParams {
    TreeBatch b;
    const int32_t *path, *counts, *tables;
    uint4 *k, *v;
    int NB, Hk;
    int row, cols;                       // 16-byte vectors of a row, of a token's rows in one pool
};

constexpr int kCommitThreads = 256;
constexpr int kBatch = 8;                // rows loaded before any is stored

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const __grid_constant__ CommitParams p) {
    __shared__ long long src[PKV_TREE_MAX_TOKENS], dst[PKV_TREE_MAX_TOKENS];   // (block * Hk) * B + offset, -1: not moved
    __shared__ int good;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int s = blockIdx.x, tid = threadIdx.x;
    const bool tell = blockIdx.y == 0;
    const TreeSeq q = pkv::tree_seq(p.b, s, tell && tid == 0);
    int count = p.counts[s];
    if (count < 0 || count > q.n) {
        if (tell && tid == 0 && q.ok) atomicOr(p.b.err, PKV_DEVERR_TOKENS);
        count = 0;
    }
    if (count == 0) return;
    if (tid == 0) good = count;
    __syncthreads();
    if (tid < count) {
        const int at = p.path[q.o + tid], before = tid ? p.path[q.o + tid - 1] : -1;
        if (at < tid || at >= q.n || at <= before) atomicMin(&good, tid);
        src[tid] = -1;
        if (at != tid && at >= 0 && at < q.n) {
            const int32_t *row = p.tables + (int64_t)s * p.b.M;
            const int from = q.L - q.n + at, to = q.L - q.n + tid, off = (1 << p.b.lb) - 1;
            const int bf = row[from >> p.b.lb], bt = row[to >> p.b.lb];
            if ((unsigned)bf < (unsigned)p.NB && (unsigned)bt < (unsigned)p.NB) {
                src[tid] = ((int64_t)bf * p.Hk << p.b.lb) + (from & off);
                dst[tid] = ((int64_t)bt * p.Hk << p.b.lb) + (to & off);
            } else if (tell) {
                atomicOr(p.b.err, PKV_DEVERR_BLOCK_ID);
            }
        }
    }
    __syncthreads();
    if (tell && tid == 0 && good < count) atomicOr(p.b.err, PKV_DEVERR_TREE);
    count = good;
    for (int c = blockIdx.y * kCommitThreads + tid; c < 2 * p.cols; c += gridDim.y * kCommitThreads) {
        const int col = c < p.cols ? c : c - p.cols, head = col / p.row;
        uint4 *pool = (c < p.cols ? p.k : p.v) + (int64_t)(head << p.b.lb) * p.row + (col - head * p.row);
        for (int k0 = 0; k0 < count; k0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (k0 + j < count && src[k0 + j] >= 0) x[j] = pool[src[k0 + j] * p.row];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (k0 + j < count && src[k0 + j] >= 0) pool[dst[k0 + j] * p.row] = x[j];
        }
    }
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

pkv_status check_batch(int S, int T) {
    if (S < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", S);
    if (T < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", T);
    return PKV_OK;
}

pkv_status check_max_tree(int n) {
    if (n < 1 || n > PKV_TREE_MAX_TOKENS)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_tree %d (1..%d)", n, PKV_TREE_MAX_TOKENS);
    return PKV_OK;
}

pkv_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return PKV_OK;
    return pkv::set_last_error(PKV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

pkv_status pkv_tree_plan(int32_t num_seqs, int32_t num_tokens, const int32_t *parents,
                         const int32_t *token_offsets, const int32_t *context_lens,
                         const int32_t *position_deltas, uint64_t *masks, int32_t mask_words,
                         int32_t *positions, int32_t num_axes, void *stream) {
    pkv_status st = check_batch(num_seqs, num_tokens);
    if (st != PKV_OK) return st;
    if (mask_words < 1 || mask_words > PKV_TREE_MAX_TOKENS / 64)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "mask_words %d (1..%d)", mask_words, PKV_TREE_MAX_TOKENS / 64);
    if (num_axes < 1 || num_axes > PKV_TREE_MAX_AXES)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_axes %d (1..%d)", num_axes, PKV_TREE_MAX_AXES);
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!token_offsets || !context_lens)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(parents, 4) || misaligned(token_offsets, 4) || misaligned(context_lens, 4) ||
        misaligned(position_deltas, 4) || misaligned(masks, 8) || misaligned(positions, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    PlanParams p = {};
    if ((st = pkv::device_error_word(&p.b.err)) != PKV_OK) return st;
    p.b.offs = token_offsets;
    p.b.lens = context_lens;
    p.b.T = num_tokens;
    p.b.N = 64 * mask_words;
    p.b.cap = INT32_MAX;
    p.parents = parents;
    p.deltas = position_deltas;
    p.masks = masks;
    p.positions = positions;
    p.axes = num_axes;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)num_seqs);
    return launched(mask_words == 1   ? launch_chained(tree_plan_kernel<1>, grid, 64, 0, s, p)
                    : mask_words == 2 ? launch_chained(tree_plan_kernel<2>, grid, 128, 0, s, p)
                    : mask_words == 3 ? launch_chained(tree_plan_kernel<3>, grid, 192, 0, s, p)
                                      : launch_chained(tree_plan_kernel<4>, grid, 256, 0, s, p),
                    "tree_plan");
}

pkv_status pkv_tree_accept(int32_t num_seqs, int32_t num_tokens, int32_t max_tree,
                           const int32_t *parents, const int32_t *tokens, const int32_t *targets,
                           const int32_t *token_offsets, const int32_t *context_lens,
                           int32_t *path, int32_t *counts, int32_t *next_tokens,
                           int32_t *context_lens_out, void *stream) {
    pkv_status st = check_batch(num_seqs, num_tokens);
    if (st != PKV_OK || (st = check_max_tree(max_tree)) != PKV_OK) return st;
    if (num_seqs == 0) return PKV_OK;
    if (!token_offsets || !context_lens || !counts || !next_tokens || !context_lens_out ||
        (num_tokens > 0 && (!tokens || !targets || !path)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(parents, 4) || misaligned(tokens, 4) || misaligned(targets, 4) || misaligned(token_offsets, 4) ||
        misaligned(context_lens, 4) || misaligned(path, 4) || misaligned(counts, 4) || misaligned(next_tokens, 4) ||
        misaligned(context_lens_out, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    AcceptParams p = {};
    if ((st = pkv::device_error_word(&p.b.err)) != PKV_OK) return st;
    p.b.offs = token_offsets;
    p.b.lens = context_lens;
    p.b.T = num_tokens;
    p.b.N = max_tree;
    p.b.cap = INT32_MAX;
    p.parents = parents;
    p.tokens = tokens;
    p.targets = targets;
    p.path = path;
    p.counts = counts;
    p.next = next_tokens;
    p.lens_out = context_lens_out;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)num_seqs);
    return launched(max_tree <= 64    ? launch_chained(tree_accept_kernel<1>, grid, 64, 0, s, p)
                    : max_tree <= 128 ? launch_chained(tree_accept_kernel<2>, grid, 128, 0, s, p)
                    : max_tree <= 192 ? launch_chained(tree_accept_kernel<3>, grid, 192, 0, s, p)
                                      : launch_chained(tree_accept_kernel<4>, grid, 256, 0, s, p),
                    "tree_accept");
}

pkv_status pkv_tree_commit(const pkv_cache_desc *cache, int32_t num_seqs, int32_t num_tokens,
                           int32_t max_tree, const int32_t *path, const int32_t *counts,
                           const int32_t *token_offsets, const int32_t *context_lens,
                           const int32_t *block_tables, int32_t max_blocks_per_seq, void *k_pool,
                           void *v_pool, void *stream) {
    pkv_status st = pkv::check_cache_desc(cache);
    if (st != PKV_OK || (st = check_batch(num_seqs, num_tokens)) != PKV_OK ||
        (st = check_max_tree(max_tree)) != PKV_OK)
        return st;
    const int64_t capacity = (int64_t)max_blocks_per_seq * cache->block_size;
    if (max_blocks_per_seq < 1)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (capacity > INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "a table row of 2^31 tokens or more");
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!path || !counts || !token_offsets || !context_lens || !block_tables || !k_pool || !v_pool)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(path, 4) || misaligned(counts, 4) || misaligned(token_offsets, 4) || misaligned(context_lens, 4) ||
        misaligned(block_tables, 4) || misaligned(k_pool, 16) || misaligned(v_pool, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "pools must be 16-byte aligned, the others to their elements");
    const int row = cache->head_dim * (cache->dtype == PKV_F32 ? 4 : 2) / 16;
    if ((int64_t)cache->num_kv_heads * row > INT32_MAX / 4)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_kv_heads %d", cache->num_kv_heads);
    CommitParams p = {};
    if ((st = pkv::device_error_word(&p.b.err)) != PKV_OK) return st;
    p.b.offs = token_offsets;
    p.b.lens = context_lens;
    p.b.T = num_tokens;
    p.b.N = max_tree;
    p.b.M = max_blocks_per_seq;
    p.b.lb = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
    p.b.cap = (int)capacity;
    p.path = path;
    p.counts = counts;
    p.tables = block_tables;
    p.k = static_cast<uint4 *>(k_pool);
    p.v = static_cast<uint4 *>(v_pool);
    p.NB = cache->num_blocks;
    p.Hk = cache->num_kv_heads;
    p.row = row;
    p.cols = cache->num_kv_heads * row;
    int parts = (2 * p.cols + kCommitThreads - 1) / kCommitThreads;
    if (parts > 64) parts = 64;
    return launched(launch_chained(tree_commit_kernel, dim3((unsigned)num_seqs, (unsigned)parts), kCommitThreads, 0,
                                   static_cast<cudaStream_t>(stream), p),
                    "tree_commit");
}

}  // extern "C"

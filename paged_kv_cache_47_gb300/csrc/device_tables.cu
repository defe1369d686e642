// Block tables and slot maps on the device (include/pkv_tables.h).
//
// One launch per call. Every CTA scans all requests (counts of tokens and
// blocks, prefix sums over the threads), so each knows the totals, takes the
// same all-or-nothing decision and can place any token by itself; the CTAs
// share out the tokens (append, four a thread in a large step) or returned
// blocks (release). Lengths and the free count are written by one CTA, at once
// where they have buffers of their own; where they are updated in place every
// CTA has to have read them first, and the CTA that arrives last at a counter
// writes them. No CTA waits.
//
// What bounds it: latency. A step of 64 requests is one CTA (release: two) and a
// chain of launch, two dependent loads, a scan, a table load and a store; append
// and release together take 7.2 us, the host's time for two calls, and 5.2
// replayed as a graph (with the state updated in place 7.4 and 6.5: the counter).
// A prompt wave writes 12 bytes a token, which the CTAs stream out in order: 997
// requests, a fifth of them released and replaced by prompts of up to 2000
// tokens, 13.3 us for both calls, 11.4 as a graph (16.2 at one token a thread).
// Truncation is release from a length on: the same two CTAs and chain.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv_tables.h"
#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"

namespace {

using pkv::launch_chained;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kItemsPerCta = 2048;   // tokens (or blocks) one CTA is launched for
constexpr int kMaxCtas = 592;        // beyond, CTAs take several strides

enum { APPEND, RELEASE, TRUNCATE };

struct TablesParams {
    int NB, B, lb, S, M;       // B = 1 << lb
    const int32_t *add;        // append: new tokens; truncate: lengths kept
    const uint8_t *released;   // release: flags
    int32_t *tables;
    const int32_t *lens;
    int32_t *lens_out;
    int32_t *free_blocks;
    const int32_t *num_free;
    int32_t *num_free_out;
    int64_t *slots;
    int32_t *positions;
    int max_tokens;
    int32_t *offsets;
    bool in_place;             // lengths or free count are written over
    unsigned *arrived;         // zero between calls
    unsigned *err;
};

// Request s as the scan sees it. items: tokens (append) or blocks (release,
// truncate) to place; blocks: blocks taken or returned.
struct Req {
    int len, items, have, blocks;
    unsigned bad;              // PKV_DEVERR_* bits
};

template <int MODE>
__device__ __forceinline__ Req load_req(const TablesParams &p, int s) {
    Req r;
    r.len = p.lens[s];
    r.bad = 0;
    const int64_t cap = (int64_t)p.M * p.B;
    if (r.len < 0 || r.len > cap) r.bad = PKV_DEVERR_CONTEXT;
    r.have = r.bad ? 0 : (int)(((unsigned)r.len + p.B - 1) >> p.lb);
    if (MODE == RELEASE) {
        r.blocks = p.released[s] ? r.have : 0;
        r.items = r.blocks;
    } else if (MODE == TRUNCATE) {
        const int kept = p.add[s];
        if (kept < 0 || kept > r.len) r.bad |= PKV_DEVERR_CONTEXT;
        r.blocks = r.bad ? 0 : r.have - (int)(((unsigned)kept + p.B - 1) >> p.lb);
        r.items = r.blocks;
    } else {
        const int a = p.add[s];
        if (a < 0) r.bad |= PKV_DEVERR_TOKENS;
        else if (!r.bad && (int64_t)r.len + a > cap) r.bad |= PKV_DEVERR_CONTEXT;
        r.items = r.bad ? 0 : a;
        r.blocks = r.bad ? 0 : (int)(((unsigned)r.len + r.items + p.B - 1) >> p.lb) - r.have;
    }
    return r;
}

// Inclusive scan of two sums over the warp's lanes.
__device__ __forceinline__ void warp_scan(long long &a, long long &b, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
}

// Lengths and free count after the call.
template <int MODE>
__device__ __forceinline__ void write_state(const TablesParams &p, bool refused, int nf, long long blocks) {
    for (int s = threadIdx.x; s < p.S; s += kThreads) {
        const int len = p.lens[s];
        p.lens_out[s] = refused           ? len
                        : MODE == RELEASE ? (p.released[s] ? 0 : len)
                        : MODE == TRUNCATE ? p.add[s]
                                           : len + p.add[s];
    }
    if (threadIdx.x == 0) *p.num_free_out = refused ? nf : MODE != APPEND ? nf + (int)blocks : nf - (int)blocks;
}

// PER: items a thread places at a time, neighbours.
template <int MODE, int PER>
__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesParams p) {
    __shared__ long long first_item[kThreads + 1];   // items before thread t's requests
    __shared__ long long first_block[kThreads];
    __shared__ long long warp_items[kWarps], warp_blocks[kWarps];
    __shared__ unsigned warp_bad[kWarps];
    __shared__ int is_last;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // thread t owns requests [s0, s1): K neighbours
    const int K = (p.S + kThreads - 1) / kThreads;
    const int s0 = min(p.S, tid * K), s1 = min(p.S, s0 + K);
    long long items = 0, blocks = 0;
    unsigned bad = 0;
    for (int s = s0; s < s1; ++s) {
        const Req r = load_req<MODE>(p, s);
        items += r.items;
        blocks += r.blocks;
        bad |= r.bad;
    }
    const int nf = *p.num_free;
    const long long my_items = items, my_blocks = blocks;
    warp_scan(items, blocks, lane);
    bad = __reduce_or_sync(~0u, bad);
    if (lane == 31) {
        warp_items[warp] = items;
        warp_blocks[warp] = blocks;
        warp_bad[warp] = bad;
    }
    __syncthreads();
    long long item0 = items - my_items, block0 = blocks - my_blocks, total = 0, total_blocks = 0;
    bad = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            item0 += warp_items[w];
            block0 += warp_blocks[w];
        }
        total += warp_items[w];
        total_blocks += warp_blocks[w];
        bad |= warp_bad[w];
    }
    if (nf < 0 || nf > p.NB) bad |= PKV_DEVERR_NO_BLOCKS;
    if (MODE != APPEND) {
        if (nf + total_blocks > p.NB) bad |= PKV_DEVERR_NO_BLOCKS;
    } else {
        if (total_blocks > nf) bad |= PKV_DEVERR_NO_BLOCKS;
        if (total > p.max_tokens) bad |= PKV_DEVERR_TOKENS;
    }
    if (bad) total = 0;
    first_item[tid] = item0;
    first_block[tid] = block0;
    if (tid == kThreads - 1) first_item[kThreads] = total;
    const bool writer = blockIdx.x == gridDim.x - 1;     // the CTA with the fewest items
    if (writer) {
        if (tid == 0 && bad) atomicOr(p.err, bad);
        if (MODE == APPEND) {
            long long at = item0;
            for (int s = s0; s < s1; ++s) {
                p.offsets[s] = bad ? 0 : (int)at;
                at += load_req<MODE>(p, s).items;
            }
            if (tid == 0) p.offsets[p.S] = (int)total;
        }
        if (!p.in_place) write_state<MODE>(p, bad != 0, nf, total_blocks);
    }
    __syncthreads();

    const long long limit = MODE != APPEND ? total : (long long)p.max_tokens;
    for (long long i0 = ((long long)blockIdx.x * kThreads + tid) * PER; i0 < limit;
         i0 += (long long)gridDim.x * kThreads * PER) {
        // the last thread whose requests begin at or before item i0 holds it
        int t = 0, s = 0;
        long long at = 0, blk = 0;
        Req r = {};
        if (i0 < total) {
#pragma unroll
            for (int step = kThreads / 2; step; step >>= 1)
                if (first_item[t + step] <= i0) t += step;
            at = first_item[t];
            blk = first_block[t];
            s = t * K;
            r = load_req<MODE>(p, s);
        }
        int64_t slot[PER];
        int position[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const long long i = i0 + q;
            slot[q] = -1;                // past the last token: a buffer's unused end
            position[q] = 0;
            if (i >= total) continue;
            while (i >= at + r.items) {
                at += r.items;
                blk += r.blocks;
                r = load_req<MODE>(p, ++s);
            }
            const int k = (int)(i - at);
            if (MODE != APPEND) {
                const int id = p.tables[(int64_t)s * p.M + r.have - r.blocks + k];
                if (id < 0 || id >= p.NB) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                p.free_blocks[nf + i] = id;
            } else {
                const int pos = r.len + k, j = pos >> p.lb, off = pos & (p.B - 1);
                int32_t *entry = p.tables + (int64_t)s * p.M + j;
                const int id = j < r.have ? *entry : p.free_blocks[nf - 1 - blk - (j - r.have)];
                if (j >= r.have && off == 0) *entry = id;
                const bool ok = id >= 0 && id < p.NB;
                if (!ok) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                if (ok) slot[q] = (int64_t)id * p.B + off;
                position[q] = pos;
            }
        }
        if (MODE != APPEND) continue;
        if (PER == 4 && i0 + PER <= limit) {     // (the buffers are 16-byte aligned then)
            longlong2 *dst = reinterpret_cast<longlong2 *>(p.slots + i0);
            dst[0] = make_longlong2(slot[0], slot[PER > 1]);
            dst[1] = make_longlong2(slot[PER / 2], slot[PER - 1]);
            *reinterpret_cast<int4 *>(p.positions + i0) =
                make_int4(position[0], position[PER > 1], position[PER / 2], position[PER - 1]);
        } else {
            for (int q = 0; q < PER; ++q)
                if (i0 + q < limit) {
                    p.slots[i0 + q] = slot[q];
                    p.positions[i0 + q] = position[q];
                }
        }
    }
    if (!p.in_place) return;
    __syncthreads();                     // this CTA's reads are done
    if (gridDim.x > 1) {
        if (tid == 0) {
            __threadfence();
            is_last = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
            __threadfence();
        }
        __syncthreads();
        if (!is_last) return;
        if (tid == 0) *p.arrived = 0;
    }
    write_state<MODE>(p, bad != 0, nf, total_blocks);
}

template <int MODE>
pkv_status run(TablesParams &p, void *workspace, int64_t items, void *stream) {
    pkv_status st = pkv::device_error_word(&p.err);
    if (st != PKV_OK) return st;
    p.arrived = static_cast<unsigned *>(workspace);
    p.lb = p.B == 8 ? 3 : p.B == 16 ? 4 : 5;
    p.in_place = p.lens_out == p.lens || p.num_free_out == p.num_free;
    int64_t ctas = (items + kItemsPerCta - 1) / kItemsPerCta;
    ctas = ctas < 1 ? 1 : ctas > kMaxCtas ? kMaxCtas : ctas;
    // four tokens a thread once there are several CTAs
    const bool four = MODE == APPEND && ctas > 1 && reinterpret_cast<uintptr_t>(p.slots) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(p.positions) % 16 == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        four ? launch_chained(tables_kernel<MODE, 4>, dim3((unsigned)ctas), kThreads, 0, s, p)
             : launch_chained(tables_kernel<MODE, 1>, dim3((unsigned)ctas), kThreads, 0, s, p);
    if (e != cudaSuccess)
        return pkv::set_last_error(PKV_ERR_CUDA, "tables launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

pkv_status check(int NB, int B, int S, int M) {
    if (B != 8 && B != 16 && B != 32)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)", B);
    if (NB < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_blocks %d", NB);
    if (S < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", S);
    if (M < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", M);
    if ((int64_t)M * B > INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "a table row of 2^31 tokens or more");
    return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_tables_append(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                             const int32_t *new_tokens, int32_t *block_tables,
                             int32_t max_blocks_per_seq, const int32_t *context_lens,
                             int32_t *context_lens_out, const int32_t *free_blocks,
                             const int32_t *num_free, int32_t *num_free_out,
                             int64_t *slot_mapping, int32_t *positions, int32_t max_tokens,
                             int32_t *token_offsets, void *workspace, void *stream) {
    pkv_status st = check(num_blocks, block_size, num_seqs, max_blocks_per_seq);
    if (st != PKV_OK) return st;
    if (max_tokens < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_tokens %d", max_tokens);
    if ((num_seqs > 0 && (!new_tokens || !block_tables || !context_lens || !context_lens_out)) ||
        !free_blocks || !num_free || !num_free_out || !token_offsets ||
        (max_tokens > 0 && (!slot_mapping || !positions)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (!workspace) return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace is NULL");
    if (misaligned(new_tokens, 4) || misaligned(block_tables, 4) || misaligned(context_lens, 4) ||
        misaligned(context_lens_out, 4) || misaligned(free_blocks, 4) || misaligned(num_free, 4) ||
        misaligned(num_free_out, 4) || misaligned(positions, 4) || misaligned(token_offsets, 4) ||
        misaligned(slot_mapping, 8) || misaligned(workspace, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    TablesParams p = {};
    p.NB = num_blocks;
    p.B = block_size;
    p.S = num_seqs;
    p.M = max_blocks_per_seq;
    p.add = new_tokens;
    p.tables = block_tables;
    p.lens = context_lens;
    p.lens_out = context_lens_out;
    p.free_blocks = const_cast<int32_t *>(free_blocks);   // read only when appending
    p.num_free = num_free;
    p.num_free_out = num_free_out;
    p.slots = slot_mapping;
    p.positions = positions;
    p.max_tokens = max_tokens;
    p.offsets = token_offsets;
    return run<APPEND>(p, workspace, max_tokens, stream);
}

pkv_status pkv_tables_release(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                              const uint8_t *released, const int32_t *block_tables,
                              int32_t max_blocks_per_seq, const int32_t *context_lens,
                              int32_t *context_lens_out, int32_t *free_blocks,
                              const int32_t *num_free, int32_t *num_free_out, void *workspace,
                              void *stream) {
    pkv_status st = check(num_blocks, block_size, num_seqs, max_blocks_per_seq);
    if (st != PKV_OK) return st;
    if ((num_seqs > 0 && (!released || !block_tables || !context_lens || !context_lens_out)) ||
        !free_blocks || !num_free || !num_free_out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (!workspace) return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace is NULL");
    if (misaligned(block_tables, 4) || misaligned(context_lens, 4) ||
        misaligned(context_lens_out, 4) || misaligned(free_blocks, 4) || misaligned(num_free, 4) ||
        misaligned(num_free_out, 4) || misaligned(workspace, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    TablesParams p = {};
    p.NB = num_blocks;
    p.B = block_size;
    p.S = num_seqs;
    p.M = max_blocks_per_seq;
    p.released = released;
    p.tables = const_cast<int32_t *>(block_tables);       // read only when releasing
    p.lens = context_lens;
    p.lens_out = context_lens_out;
    p.free_blocks = free_blocks;
    p.num_free = num_free;
    p.num_free_out = num_free_out;
    // the blocks returned are at most the pool's; few requests finish in one
    // step, so the launch is sized for a quarter of the table and strides
    int64_t most = (int64_t)num_seqs * max_blocks_per_seq / 4;
    if (most > num_blocks) most = num_blocks;
    return run<RELEASE>(p, workspace, most, stream);
}

pkv_status pkv_tables_truncate(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                               const int32_t *kept_lens, const int32_t *block_tables,
                               int32_t max_blocks_per_seq, const int32_t *context_lens,
                               int32_t *context_lens_out, int32_t *free_blocks,
                               const int32_t *num_free, int32_t *num_free_out, void *workspace,
                               void *stream) {
    pkv_status st = check(num_blocks, block_size, num_seqs, max_blocks_per_seq);
    if (st != PKV_OK) return st;
    if ((num_seqs > 0 && (!kept_lens || !block_tables || !context_lens || !context_lens_out)) ||
        !free_blocks || !num_free || !num_free_out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (!workspace) return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace is NULL");
    if (misaligned(kept_lens, 4) || misaligned(block_tables, 4) || misaligned(context_lens, 4) ||
        misaligned(context_lens_out, 4) || misaligned(free_blocks, 4) || misaligned(num_free, 4) ||
        misaligned(num_free_out, 4) || misaligned(workspace, 4))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    if (num_seqs > 0 && kept_lens == context_lens_out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "kept_lens is also an output");
    TablesParams p = {};
    p.NB = num_blocks;
    p.B = block_size;
    p.S = num_seqs;
    p.M = max_blocks_per_seq;
    p.add = kept_lens;
    p.tables = const_cast<int32_t *>(block_tables);       // read only when truncating
    p.lens = context_lens;
    p.lens_out = context_lens_out;
    p.free_blocks = free_blocks;
    p.num_free = num_free;
    p.num_free_out = num_free_out;
    // a few blocks a request come back
    int64_t most = 4 * (int64_t)num_seqs;
    if (most > num_blocks) most = num_blocks;
    return run<TRUNCATE>(p, workspace, most, stream);
}

}  // extern "C"

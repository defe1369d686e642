// The work of a tree attention launch and the join of its pieces.
//
// A unit is (sequence, kv head, up to RC rows), a row one q head of one drafted
// token: row r of a sequence and kv head is head r % G of the kv head's group
// and drafted token r / G. A unit's context is cut into tiles; tiles of all
// units lie end to end, a sequence's units one after another, and worker c of C
// (a CTA, or one of two in a CTA) takes an even share of them. A unit that a
// share's border cuts leaves pieces in the workspace, normalised, with log2 of
// their denominators: slot 0 of a worker holds the piece of a unit that began in
// an earlier one, slot 1 the piece of a unit that goes on in the next. Once a CTA
// is done it counts its pieces in at each unit's counter, and where it counts the
// last one all its warps join the unit's pieces, in their order, so that equal
// inputs give equal bits. Nobody waits. (With a second kernel for the joins 64
// requests of 16 drafted tokens took 126 us and not 117, 32 trees 162 and not 153.)
// A join is one SM's reads: 8 pieces of 64 rows 5.2 us, 4 of 256 rows 8.4.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "pkv_internal.h"
#include "tree_internal.h"

namespace pkv {

constexpr int kTreeMaxSeqs = 1024;       // sequences of one launch
constexpr int kTreeMmaRows = 128;        // rows of a row tile on the tensor cores
constexpr int kTreeMmaTile = 64;         // tokens of a tile there

// A worker's piece of a unit cut between workers.
struct TreeCut {
    int parts, first;                    // pieces of the unit (0: none here), the worker it begins in
    int o, g, r0, nr;                    // first q row, kv head, first row and rows of the unit
    int due;                             // counts of it that are still to be made here

    // Counts n of `counts` a piece in; true for the last of all, which joins. What
    // the pieces' stores wrote comes before, through a fence and a barrier.
    __device__ __forceinline__ bool count(unsigned *counters, int n, int counts) const {
        if (atomic_add_acq_rel_gpu(counters + first, (unsigned)n) != (unsigned)(parts * counts - n)) return false;
        counters[first] = 0;
        return true;
    }
};

struct TreeParams {
    TreeBatch b;
    const int32_t *tables;
    const uint64_t *masks;               // [T][W] or NULL: chains
    int W;
    const void *q, *k, *v;
    void *out;
    float *lse_out;
    int out_dtype;
    int S, NB, Hk, Hq, G, RC, C;
    float scale_log2;
    unsigned *count;                     // [C] pieces counted in, of the unit that begins there; zero between calls
    float *ws_o, *ws_lse;                // [C][2][RC][D], [C][2][RC]
    unsigned long long wait_ns;          // bounded waits, as in DecodeParams
    int drop_arrival;
};

// 16-bit caches (tree_mma.cuh).
cudaError_t launch_tree_bf16(int D, const TreeParams &p, cudaStream_t s);
cudaError_t launch_tree_f16(int D, const TreeParams &p, cudaStream_t s);

__device__ __forceinline__ int tree_units(const TreeParams &p, int n) {
    return p.Hk * ((n * p.G + p.RC - 1) / p.RC);
}

// Where a worker is in the list: tile i of `tiles` of unit u of `units`
// of sequence s.
struct TreePlace {
    int s, u, i, tiles, units;
    TreeSeq q;

    template <int TILE>
    __device__ __forceinline__ void load(const TreeParams &p) {
        q = tree_seq(p.b, s, false);
        units = tree_units(p, q.n);
        tiles = (q.L + TILE - 1) / TILE;
    }
    // The next unit's first tile; there is one.
    template <int TILE>
    __device__ __forceinline__ void next_unit(const TreeParams &p) {
        i = 0;
        if (++u < units) return;
        u = 0;
        do {
            ++s;
            load<TILE>(p);
        } while (units == 0);
    }
};

struct TreeShare {
    int A, Z, NT, CT;                    // the worker's tiles [A, Z) of NT; workers with tiles
    int me;
};

// Tiles before each sequence, to prefix [kTreeMaxSeqs + 1]; returns all. scan
// [THREADS / 32]. All threads; the last barrier before others read is the caller's.
template <int TILE, int THREADS>
__device__ __forceinline__ int tree_tiles(const TreeParams &p, int *prefix, int *scan) {
    constexpr int K = (kTreeMaxSeqs + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n[K], sum = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int s = tid * K + k;
        n[k] = 0;
        if (s < p.S) {
            const TreeSeq q = tree_seq(p.b, s, blockIdx.x == 0);
            n[k] = tree_units(p, q.n) * ((q.L + TILE - 1) / TILE);
        }
        sum += n[k];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int s = tid * K + k;
        if (s <= kTreeMaxSeqs) prefix[s] = before;
        before += n[k];
    }
    if (tid == THREADS - 1) prefix[kTreeMaxSeqs] = total;
    __syncthreads();
    return total;
}

// The share of worker `me` of all, and the place of its first tile.
template <int TILE>
__device__ __forceinline__ TreeShare tree_share(const TreeParams &p, const int *prefix, int total, int me, int workers, TreePlace &at) {
    TreeShare r;
    r.me = me;
    r.NT = total;
    // two tiles each at least: half the pieces to join (one request of 1016 tokens
    // with 16 drafted 17.0 us; one tile each 19.7, four 17.5)
    r.CT = total < 2 * workers ? (total + 1) / 2 : workers;
    r.A = r.Z = 0;
    if (me < r.CT) {
        r.A = (int)((long long)me * total / r.CT);
        r.Z = (int)((long long)(me + 1) * total / r.CT);
        int lo = 0, hi = p.S - 1;        // the last sequence that begins at or before A
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= r.A) lo = mid;
            else hi = mid - 1;
        }
        at.s = lo;
        at.load<TILE>(p);
        const int x = r.A - prefix[lo];
        at.u = x / at.tiles;
        at.i = x - at.u * at.tiles;
    }
    return r;
}

// The worker that holds tile v of the list.
__device__ __forceinline__ int tree_owner(const TreeShare &sh, int v) {
    return (int)((((long long)v + 1) * sh.CT - 1) / sh.NT);
}
// What a worker has of a unit that begins at tile `first` of the list.
__device__ __forceinline__ TreeCut tree_cut(const TreeShare &sh, int first, int tiles, int o, int g, int r0, int nr) {
    const int a = tree_owner(sh, first);
    return {tree_owner(sh, first + tiles - 1) - a + 1, a, o, g, r0, nr, 0};
}

// Row rr (of sequence and kv head) as a row of q and out.
__device__ __forceinline__ size_t tree_row(const TreeParams &p, int o, int g, int rr) {
    const int i = rr / p.G;
    return (size_t)(o + i) * p.Hq + g * p.G + (rr - i * p.G);
}

// 32 bytes in one store: a whole sector of memory, where rows lie apart.
__device__ __forceinline__ void store_32(void *to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// E neighbouring outputs in this type.
template <int E>
__device__ __forceinline__ void tree_store(void *to, int dtype, size_t at, const float (&o)[E]) {
    static_assert(E % 4 == 0, "");
    if (dtype == PKV_F32) {
        if constexpr (E % 8 == 0) {
#pragma unroll
            for (int i = 0; i < E; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(o[i + j]);
                store_32(static_cast<float *>(to) + at + i, w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 4)
                *reinterpret_cast<float4 *>(static_cast<float *>(to) + at + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
        return;
    }
    float a, b;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E; i += 2)
        w[i / 2] = dtype == PKV_F16 ? Elem<__half>::pack2(o[i], o[i + 1], a, b)
                                          : Elem<__nv_bfloat16>::pack2(o[i], o[i + 1], a, b);
    uint16_t *dst = static_cast<uint16_t *>(to) + at;
    if constexpr (E % 16 == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 16) {
            const uint32_t x[8] = {w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3], w[i / 2 + 4], w[i / 2 + 5], w[i / 2 + 6], w[i / 2 + 7]};
            store_32(dst + i, x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4) *reinterpret_cast<uint2 *>(dst + i) = make_uint2(w[i / 2], w[i / 2 + 1]);
    }
}

// A unit's pieces joined by the CTA's warps, each R rows at a time and K pieces
// of them, whose elements are under way at once; four elements a lane.
template <int D, int WARPS, int R, int K>
__device__ __forceinline__ void tree_join(const TreeParams &p, const TreeCut &cut) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool mine = lane * 4 < D;
    for (int r0 = warp * R; r0 < cut.nr; r0 += WARPS * R) {
        // the first worker's piece is in its slot 1, the others' in slot 0
        auto piece = [&](int k, int r) { return (size_t)(2 * (cut.first + k) + (k == 0)) * p.RC + min(r0 + r, cut.nr - 1); };
        float mx[R], sum[R];
        float4 o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mx[r] = -INFINITY;
            sum[r] = 0.f;
            o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int k0 = 0; k0 < cut.parts; k0 += 32) {
            float f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) f[r] = k0 + lane < cut.parts ? __ldcg(p.ws_lse + piece(k0 + lane, r)) : -INFINITY;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float m = f[r];
#pragma unroll
                for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
                const float nm = fmaxf(mx[r], m), ref = nm == -INFINITY ? 0.f : nm;
                const float before = ex2_approx(mx[r] - ref);
                f[r] = ex2_approx(f[r] - ref);
                float s = f[r];
#pragma unroll
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
                sum[r] = sum[r] * before + s;
                mx[r] = nm;
                o[r].x *= before, o[r].y *= before, o[r].z *= before, o[r].w *= before;
            }
            const int here = min(32, cut.parts - k0);
#pragma unroll 1
            for (int j0 = 0; j0 < here; j0 += K) {
                float4 x[K][R];
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (mine && j0 + j < here)
                            x[j][r] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + piece(k0 + j0 + j, r) * D) + lane);
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float w = __shfl_sync(~0u, f[r], (j0 + j) & 31);
                        if (mine && j0 + j < here) {
                            o[r].x = fmaf(x[j][r].x, w, o[r].x);
                            o[r].y = fmaf(x[j][r].y, w, o[r].y);
                            o[r].z = fmaf(x[j][r].z, w, o[r].z);
                            o[r].w = fmaf(x[j][r].w, w, o[r].w);
                        }
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r0 + r >= cut.nr) break;
            const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
            const size_t row = tree_row(p, cut.o, cut.g, cut.r0 + r0 + r);
            if (mine) {
                const float x[4] = {o[r].x * inv, o[r].y * inv, o[r].z * inv, o[r].w * inv};
                tree_store<4>(p.out, p.out_dtype, row * D + lane * 4, x);
            }
            if (p.lse_out && lane == 0) p.lse_out[row] = sum[r] == 0.f ? -INFINITY : mx[r] + log2f(sum[r]);
        }
    }
}

// Counts the CTA's pieces in (cuts[N], shared memory; each `counts` times, less
// those that were counted before) and joins the units that are then complete. All
// threads, once the pieces are written.
template <int D, int WARPS, int R, int K, int N>
__device__ __forceinline__ void tree_join_cuts(const TreeParams &p, TreeCut (&cuts)[N]) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x < N && cuts[threadIdx.x].parts && cuts[threadIdx.x].due) {
        TreeCut &c = cuts[threadIdx.x];
        if (!c.count(p.count, c.due, c.due)) c.parts = 0;
    }
    __syncthreads();
    for (int i = 0; i < N; ++i)
        if (cuts[i].parts) tree_join<D, WARPS, R, K>(p, cuts[i]);
}

}  // namespace pkv

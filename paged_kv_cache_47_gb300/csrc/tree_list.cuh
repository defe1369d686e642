// The work of a tree attention launch and the join of its pieces.
//
// A unit is (sequence, kv head, up to RC rows), a row one q head of one drafted
// token: row r of a sequence and kv head is head r % G of the kv head's group
// and drafted token r / G. A unit's context is cut into tiles; tiles of all
// units lie end to end, a sequence's units one after another, and worker c of C
// (a CTA, or one of two in a CTA) takes an even share of them. A unit that a
// share's border cuts leaves pieces in the workspace, normalised, with log2 of
// their denominators: slot 0 of a worker holds the piece of a unit that began in
// an earlier one, slot 1 the piece of a unit that goes on in the next. The worker
// in which a unit begins writes down how many pieces it has, and a second kernel
// joins them, in order, so that equal inputs give equal bits.
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
constexpr int kTreeJoinWarps = 4;
constexpr int kTreeMmaRows = 128;        // rows of a row tile on the tensor cores
constexpr int kTreeMmaTile = 64;         // tokens of a tile there

// What the worker in which a cut unit begins writes down for the join.
struct TreeCut {
    int parts;                           // pieces (0: none to join)
    int o, g, r0, nr;                    // first q row, kv head, first row and rows of the unit
    int pad[3];
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
    float *ws_o, *ws_lse;                // [C][2][RC][D], [C][2][RC]
    TreeCut *cuts;                       // [C]
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
    r.CT = total < workers ? total : workers;
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

// Pieces of a unit that begins at tile `first` of the list, in this share.
__device__ __forceinline__ int tree_parts(const TreeShare &sh, int first, int tiles) {
    const long long last = first + tiles - 1;
    return (int)(((last + 1) * sh.CT - 1) / sh.NT) - sh.me + 1;
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

// The joins: CTA (c, y) takes rows y * warps.. of the unit cut that begins in
// worker c, a warp a row, four elements a lane. Denominators are asked for beside
// the record of the cut, and eight pieces' elements at once: two round trips of
// memory for few pieces.
template <int D>
__global__ void __launch_bounds__(32 * kTreeJoinWarps) tree_join_kernel(const __grid_constant__ TreeParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = __ldcg(&p.cuts[c].parts);
    const TreeCut cut = p.cuts[c];
    for (int r = blockIdx.y * kTreeJoinWarps + warp; r < p.RC; r += gridDim.y * kTreeJoinWarps) {
        // the first worker's piece is in its slot 1, the others' in slot 0
        const size_t at0 = (size_t)(2 * c + 1) * p.RC + r, step = (size_t)2 * p.RC;
        float l0 = c + lane < p.C ? __ldcg(p.ws_lse + at0 + lane * step - (lane ? p.RC : 0)) : -INFINITY;
        if (parts < 2 || r >= cut.nr) return;
        float mx = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < parts; k0 += 32) {
            const int k = k0 + lane;
            float l = -INFINITY;
            if (k < parts) l = k0 ? __ldcg(p.ws_lse + at0 + k * step - p.RC) : l0;
            float m = l;
#pragma unroll
            for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
            const float nm = fmaxf(mx, m), ref = nm == -INFINITY ? 0.f : nm;
            const float f0 = ex2_approx(mx - ref), f = ex2_approx(l - ref);
            float s = f;
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
            sum = sum * f0 + s;
            mx = nm;
            o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
            const int here = min(32, parts - k0);
            for (int j0 = 0; j0 < here; j0 += 8) {
                float4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int q = k0 + min(j0 + j, here - 1);
                    const size_t a = at0 + q * step - (q ? p.RC : 0);
                    if (lane * 4 < D) x[j] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + a * D) + lane);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = __shfl_sync(~0u, f, min(j0 + j, here - 1));
                    if (j0 + j < here && lane * 4 < D) {
                        o.x = fmaf(x[j].x, w, o.x);
                        o.y = fmaf(x[j].y, w, o.y);
                        o.z = fmaf(x[j].z, w, o.z);
                        o.w = fmaf(x[j].w, w, o.w);
                    }
                }
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const size_t row = tree_row(p, cut.o, cut.g, cut.r0 + r);
        if (lane * 4 < D) {
            const float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
            tree_store<4>(p.out, p.out_dtype, row * D + lane * 4, x);
        }
        if (p.lse_out && lane == 0) p.lse_out[row] = sum == 0.f ? -INFINITY : mx + log2f(sum);
    }
}

}  // namespace pkv

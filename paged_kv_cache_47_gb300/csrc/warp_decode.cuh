// The frame of a decode whose warps run alone: each warp takes a run of the
// batch's subtiles with its own copies, ring and softmax state; only at the end
// are the pieces of units cut between warps joined, in shared memory within a
// CTA and through the workspace between CTAs (by the CTA that arrives last;
// nobody waits). The subtiles' own work is the kernels'.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "pkv_internal.h"
#include "warp_split.h"

namespace pkv {

constexpr int kWdFewParts = 4;           // parts of a unit that one warp joins at once
constexpr int kWdHeads = 8;              // q heads of a unit (the n, or half the m, of the mma)
constexpr float kWdNone = 2e-38f;        // reference exponent of a head before its first finite
                                         // score: 0 to any score, and no score's own

// The work of one launch.
struct WdList {
    const int32_t *tables, *lens;
    int S, M, lb, U;                     // sequences, table columns, block size 1 << lb, units a sequence
    int tables_ready;
    unsigned *err;
};

// Where results go.
struct WdOut {
    void *out;                           // [S][Hq][D]
    int out_dtype;
    float *lse_out;                      // [S][Hq] or NULL
    int Hq, G, NC, GC;                   // q heads, per kv head; chunks of a group, heads of a chunk
    unsigned *cnt;                       // [C] arrivals, zero between calls
    float *ws_o, *ws_lse;                // [C][2][GC][D], [C][2][GC]

    // q heads and first q head of unit u of a sequence
    __device__ __forceinline__ int heads(int u) const { return min(GC, G - u % NC * GC); }
    __device__ __forceinline__ int first_head(int u) const { return u / NC * G + u % NC * GC; }
};

__device__ __forceinline__ float wd_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- the list
template <int W, int N>                  // N: sequences of one launch, at most
struct WdListShared {
    int prefix[N + 1];                   // places before a sequence, for one unit a sequence
    int len[N];
    uint16_t nonempty[N + 2];            // sequences with tokens before a sequence
    int scan[3][W];
};

// A warp's share of the list, places [a, z) of its CTA's [A, Z).
struct WdShare {
    int cost, NV, CT, A, Z, a, z;
};

using WdPlace = SplitPlace;

// Lengths, their prefixes, zeros for empty contexts, and this warp's share (a
// CTA without work gets an empty one: CT <= its index). SUB tokens a subtile.
// All threads of the CTA; waits for the preceding kernel.
template <int W, int SUB, int N>
__device__ __forceinline__ WdShare wd_share(const WdList &p, const WdOut &o, int D, int unit_cost,
                                            WdListShared<W, N> &sh) {
    constexpr int T = 32 * W;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!p.tables_ready) grid_dependency_wait();
    int longest = 0;
    WdShare r;
    {
        constexpr int K = (N + T - 1) / T;
        int n[K], sum = 0, some = 0;                 // subtiles; sequences that have any
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int s = tid * K + k;
            int L = s < p.S ? __ldg(p.lens + s) : 0;
            if (L < 0 || L > (p.M << p.lb)) {
                if (blockIdx.x == 0) atomicOr(p.err, PKV_DEVERR_CONTEXT);
                L = L < 0 ? 0 : p.M << p.lb;
            }
            if (s < N) sh.len[s] = L;
            n[k] = (L + SUB - 1) / SUB;
            sum += n[k];
            some += L > 0;
            longest = max(longest, n[k]);
        }
        int inc = sum, inc1 = some;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(~0u, inc, d), y = __shfl_up_sync(~0u, inc1, d);
            if (lane >= d) {
                inc += x;
                inc1 += y;
            }
        }
        longest = __reduce_max_sync(~0u, longest);
        if (lane == 31) {
            sh.scan[0][warp] = inc;
            sh.scan[1][warp] = inc1;
            sh.scan[2][warp] = longest;
        }
        __syncthreads();
        int before = inc - sum, before1 = inc1 - some, total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) {
                before += sh.scan[0][w];
                before1 += sh.scan[1][w];
            }
            total += sh.scan[0][w];
            longest = max(longest, sh.scan[2][w]);
        }
        r.cost = split_unit_cost(total * p.U, (int)gridDim.x, W, unit_cost);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int s = tid * K + k;
            if (s < N) {
                sh.prefix[s] = before + r.cost * before1;
                sh.nonempty[s] = (uint16_t)before1;
            }
            before += n[k];
            before1 += n[k] > 0;
        }
        if (tid == T - 1) {
            sh.prefix[N] = before + r.cost * before1;
            sh.nonempty[N] = (uint16_t)before1;
        }
        __syncthreads();
    }
    if (p.tables_ready) grid_dependency_wait();

    // empty contexts: zeros
    for (int s = blockIdx.x; s < p.S; s += gridDim.x)
        if (sh.len[s] == 0) {
            for (int e = tid; e < o.Hq * D; e += T)
                store_out(o.out, (size_t)s * o.Hq * D + e, o.out_dtype, 0.f);
            if (o.lse_out)
                for (int h = tid; h < o.Hq; h += T) o.lse_out[(size_t)s * o.Hq + h] = -INFINITY;
        }

    const int cta = blockIdx.x, units = sh.nonempty[N] * p.U;
    r.NV = sh.prefix[N] * p.U;
    r.A = r.Z = r.a = r.z = 0;
    if (split_units_alone(r.cost, units, longest, (int)gridDim.x, W)) {
        // a unit for each CTA
        r.CT = units;
        if (cta >= r.CT) return r;
        split_unit_share(sh.prefix, split_unit_sequence(sh.nonempty, p.S, p.U, cta), p.U, cta, r.A, r.Z);
    } else {
        r.CT = split_active_ctas(r.NV, (int)gridDim.x, W, r.cost);
        if (cta >= r.CT) return r;
        r.A = split_cta_cut(cta, r.NV, r.CT);
        r.Z = split_cta_cut(cta + 1, r.NV, r.CT);
    }
    r.a = split_warp_cut(warp, r.A, r.Z, W, r.cost);
    r.z = split_warp_cut(warp + 1, r.A, r.Z, W, r.cost);
    return r;
}

// The first subtile at or after place a.
template <int W, int N>
__device__ __forceinline__ WdPlace wd_place(const WdList &p, const WdListShared<W, N> &sh, int a, int cost) {
    const int lane = threadIdx.x & 31;
    const int s = split_sequence(p.S, [&](int lo, int n, int step) {
        return __popc(__ballot_sync(~0u, lane * step < n && sh.prefix[lo + lane * step] * p.U <= a));
    });
    return split_place(sh.prefix, s, p.U, a, cost);
}

// The next unit, if its first subtile lies before place z.
template <int W, int N>
__device__ __forceinline__ bool wd_next_unit(const WdList &p, const WdListShared<W, N> &sh, WdPlace &w, int z) {
    return split_next_unit(sh.prefix, sh.len, p.U, w, z);
}

// ---------------------------------------------------------------- rows of E = D / 32 elements a lane
template <int E>
__device__ __forceinline__ void wd_add_scaled(float (&o)[E], const float *src, float f) {
    if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
        o[2] = fmaf(v.z, f, o[2]);
        o[3] = fmaf(v.w, f, o[3]);
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
    }
}
template <int E>
__device__ __forceinline__ void wd_load(float (&o)[E], const float *src) {
    if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] = v.x, o[1] = v.y;
    }
}
template <int E>
__device__ __forceinline__ void wd_load_cg(float (&o)[E], const float *src) {
    if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
        o[0] = v.x, o[1] = v.y;
    }
}
template <int E>
__device__ __forceinline__ void wd_store_f32(float *dst, const float (&o)[E]) {
    if constexpr (E == 4) *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
    else *reinterpret_cast<float2 *>(dst) = make_float2(o[0], o[1]);
}
// E outputs in the output's type, element `at` on.
template <int E>
__device__ __forceinline__ void wd_store_row(const WdOut &p, size_t at, const float (&o)[E]) {
    if (p.out_dtype == PKV_F32) {
        wd_store_f32(static_cast<float *>(p.out) + at, o);
        return;
    }
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        float a, b;
        w[i / 2] = p.out_dtype == PKV_F16 ? Elem<__half>::pack2(o[i], o[i + 1], a, b)
                                          : Elem<__nv_bfloat16>::pack2(o[i], o[i + 1], a, b);
    }
    uint16_t *dst = static_cast<uint16_t *>(p.out) + at;
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(dst) = w[0];
}

// ---------------------------------------------------------------- joins
// What a warp leaves of a unit it does not hold whole: the unit's first
// subtile's place and its subtiles, sequence and unit. nu 0: none.
struct WdPiece {
    int tu, nu, s, u;
};

// A warp's piece in slot 0 belongs to a unit that began before its share, the
// one in slot 1 to a unit that goes on after it.
template <int W>
struct WdJoinShared {
    WdPiece piece[W][2];
    float lse[W][2][kWdHeads];           // log2 of the pieces' denominators
    int cut_tu[2], cut_nu[2], cut_s[2], cut_u[2];   // units cut at the CTA's start, end
    int join_first[2], join_n[2];        // of them, those to join here: parts
};

template <int W>
__device__ __forceinline__ void wd_join_init(WdJoinShared<W> &sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < 2) sh.piece[warp][lane].nu = 0;
    if (threadIdx.x < 2) sh.cut_nu[threadIdx.x] = sh.join_n[threadIdx.x] = 0;
}

// Joins what the CTA's warps left. slot0 + w * GC * D, slot1 + w * pitch: the
// normalised pieces [GC][D] of warp w. slot0 is written over. All threads.
template <int W, int D>
__device__ __forceinline__ void wd_join(const WdOut &p, const WdShare &share, WdJoinShared<W> &sh, float *slot0,
                                        const float *slot1, size_t pitch) {
    constexpr int E = D / 32;
    static_assert(W < 32 && W >= kWdHeads, "a lane for each possible start, a warp for each head");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
    __syncthreads();
    // A unit's pieces here: one that starts it (slot 1 of some warp, or slot 0
    // of warp 0 when it began in an earlier CTA), then slot 0 of the warps
    // after. A warp takes one head of one unit, a lane E elements.
    {
        const bool starts = lane <= W && sh.piece[lane ? lane - 1 : 0][lane ? 1 : 0].nu != 0;
        unsigned todo = __ballot_sync(~0u, starts);
        for (int k = 0; todo; ++k, todo &= todo - 1) {
            const int i = __ffs(todo) - 1, w = i ? i - 1 : 0, sl = i ? 1 : 0;
            const int h = (warp + W * kWdHeads - k * p.GC) % W;
            if (h >= p.GC) continue;
            const WdPiece pc = sh.piece[w][sl];
            if (h >= p.heads(pc.u)) continue;
            const bool next = lane > w && lane < W && sh.piece[lane % W][0].nu && sh.piece[lane % W][0].tu == pc.tu;
            const int more = __ffs(~(__ballot_sync(~0u, next) >> (w + 1))) - 1;      // pieces after the first
            float l = -INFINITY;
            if (lane <= more) l = lane ? sh.lse[w + lane][0][h] : sh.lse[w][sl][h];
            float mx = l;
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
            if (mx == -INFINITY) mx = 0.f;
            const float f = wd_ex2(l - mx);
            float sum = f;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
            float o[E] = {};
            for (int q0 = 0; q0 <= more; q0 += 4) {
                float x[4][E];                       // four loads under way at once
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int q = min(q0 + i, more);
                    const float *src = q == 0 && sl ? slot1 + w * pitch : slot0 + (size_t)(w + q) * p.GC * D;
                    wd_load(x[i], src + h * D + lane * E);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float fq = __shfl_sync(~0u, f, q0 + i);    // (0 past the last)
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = q0 + i <= more ? fmaf(x[i][e], fq, o[e]) : o[e];
                }
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= inv;
            const float lse = mx + log2f(sum);
            if (pc.tu >= share.A && pc.tu + pc.nu <= share.Z) {
                const size_t at = (size_t)pc.s * p.Hq + p.first_head(pc.u) + h;
                wd_store_row<E>(p, at * D + lane * E, o);
                if (p.lse_out && lane == 0) p.lse_out[at] = lse;
            } else {
                const int side = pc.tu < share.A ? 0 : 1;
                const size_t at = (size_t)(2 * cta + side) * p.GC + h;
                wd_store_f32(p.ws_o + at * D + lane * E, o);
                if (lane == 0) {
                    p.ws_lse[at] = lse;
                    if (h == 0) {
                        sh.cut_tu[side] = pc.tu;
                        sh.cut_nu[side] = pc.nu;
                        sh.cut_s[side] = pc.s;
                        sh.cut_u[side] = pc.u;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (!sh.cut_nu[0] && !sh.cut_nu[1]) return;

    // units cut between CTAs: count this CTA's part in; the last to come joins
    if (threadIdx.x < 2 && sh.cut_nu[threadIdx.x]) {
        const int side = threadIdx.x;
        const int first = split_owner(sh.cut_tu[side], share.NV, share.CT);
        const int n = split_owner(sh.cut_tu[side] + sh.cut_nu[side] - 1, share.NV, share.CT) - first + 1;
        // the parts' stores come before it for whoever counts later, and theirs
        // before the reads below
        const bool last = atomic_add_acq_rel_gpu(p.cnt + first, 1u) == (unsigned)n - 1;
        if (last) p.cnt[first] = 0;
        sh.join_n[side] = last ? n : 0;
        sh.join_first[side] = first;
    }
    __syncthreads();
    // few parts: a warp for each head of either unit, a lane for each part's denominator
    for (int task = warp; task < 2 * kWdHeads; task += W) {
        const int side = task & 1, h = task >> 1, n = sh.join_n[side];
        if (n == 0 || n > kWdFewParts || h >= p.heads(sh.cut_u[side])) continue;
        // the first CTA's part is its side 1, the others' their side 0
        const size_t at0 = (size_t)2 * sh.join_first[side] * p.GC + h;
        const size_t pitch_parts = 2 * (size_t)p.GC;
        float x[kWdFewParts][E], l = -INFINITY;
        if (lane < n) l = __ldcg(p.ws_lse + at0 + lane * pitch_parts + (lane ? 0 : p.GC));
#pragma unroll
        for (int k = 0; k < kWdFewParts; ++k) {
            const int part = min(k, n - 1);
            wd_load_cg(x[k], p.ws_o + (at0 + part * pitch_parts + (part ? 0 : p.GC)) * D + lane * E);
        }
        float mx = l;
#pragma unroll
        for (int d = kWdFewParts / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
        mx = __shfl_sync(~0u, mx, 0);
        if (mx == -INFINITY) mx = 0.f;
        const float f = wd_ex2(l - mx);              // (0 past the last)
        float sum = f;
#pragma unroll
        for (int d = kWdFewParts / 2; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        sum = __shfl_sync(~0u, sum, 0);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        float o[E] = {};
#pragma unroll
        for (int k = 0; k < kWdFewParts; ++k) {
            const float fk = __shfl_sync(~0u, f, k) * inv;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = k < n ? fmaf(x[k][e], fk, o[e]) : o[e];
        }
        const size_t at = (size_t)sh.cut_s[side] * p.Hq + p.first_head(sh.cut_u[side]) + h;
        wd_store_row<E>(p, at * D + lane * E, o);
        if (p.lse_out && lane == 0) p.lse_out[at] = mx + log2f(sum);
    }
    for (int side = 0; side < 2; ++side) {
        const int n = sh.join_n[side], first = sh.join_first[side];
        if (n <= kWdFewParts) continue;
        const int u = sh.cut_u[side], gca = p.heads(u);
        // the warps of a head take every ways-th part; they meet in slot0
        const int ways = W / gca, h = warp % gca, sub = warp / gca;
        float o[E] = {}, m = -3e38f, sum = 0.f;
        if (sub < ways) {
#pragma unroll 4
            for (int k = sub; k < n; k += ways) {
                const size_t at = (size_t)(2 * (first + k) + (k == 0)) * p.GC + h;
                const float l = __ldcg(p.ws_lse + at);
                float x[E];
                wd_load_cg(x, p.ws_o + at * D + lane * E);
                const float nm = fmaxf(m, l), f = wd_ex2(m - nm), fx = wd_ex2(l - nm);
                m = nm;
                sum = fmaf(sum, f, fx);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, x[e] * fx);
            }
            wd_store_f32(slot0 + (size_t)warp * D + lane * E, o);
            if (lane == 0) {
                sh.lse[warp][0][0] = m;
                sh.lse[warp][0][1] = sum;
            }
        }
        __syncthreads();
        if (sub == 0) {
            float mx = -3e38f, total = 0.f;
            for (int q = 0; q < ways; ++q) mx = fmaxf(mx, sh.lse[h + q * gca][0][0]);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = 0.f;
            for (int q = 0; q < ways; ++q) {
                const int w = h + q * gca;
                const float f = wd_ex2(sh.lse[w][0][0] - mx);
                total = fmaf(sh.lse[w][0][1], f, total);
                wd_add_scaled(o, slot0 + (size_t)w * D + lane * E, f);
            }
            const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= inv;
            const size_t at = (size_t)sh.cut_s[side] * p.Hq + p.first_head(u) + h;
            wd_store_row<E>(p, at * D + lane * E, o);
            if (p.lse_out && lane == 0) p.lse_out[at] = mx + log2f(total);
        }
        __syncthreads();
    }
}

}  // namespace pkv

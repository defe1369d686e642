// Decode attention over a 4-bit cache (include/pkv_q4.h).
//
// With value(c) = s c + m for each group y of 32 elements,
//   <q, k_t>  = sum_y s_ty <q_y, c_ty> + sum_y m_ty (sum of q over y)
//   sum_t p_t v_t[d] = sum_t (p_t s_ty) c_td + sum_t p_t m_ty          (d in y)
// so codes meet the matrix instructions as they are and the parameters enter
// per token and group, not per element.
//
// Codes as operands. A 4-bit code at bits 0..3 (or 4..7) of an fp16 whose other
// bits are zero is the subnormal number c 2^-24 (or c 2^-20), exactly: one AND
// makes two operands, with no bias to take off again and no conversion. Codes
// at bits 4..7 count 16 fold; q carries the 1/16 on the K side, the epilogue
// on the V side. mma.sync takes subnormals at full rate. (tcgen05 has no form
// that reads these rows: its 4-bit kinds want the contracted index along the
// row for both operands, and a V row holds one token.)
//
// Work. The batch's (sequence, kv head, up to 8 q heads) units, cut into
// subtiles of 16 tokens and laid end to end, are split evenly over the CTAs
// and in each CTA over its warps. A warp runs alone: its own ring of stages in
// shared memory filled by its own cp.async, its own softmax state; no barrier
// but the one before the CTA's pieces are joined. Pieces of a unit cut between
// warps are joined in shared memory, between CTAs through the workspace by the
// CTA that arrives last (nobody waits).
//
// Softmax in base 2 with a reference exponent that moves only when a score
// passes it by more than the fp16 weights can hold, or a V scale grows past
// its bound: most subtiles need one vote instead of a reduction over lanes and
// a rescale of the accumulators. The denominator is summed by the same product
// that weighs the minima (a row of ones), over the rounded weights, so a
// weight's rounding moves the average, not its normalisation. Weight times V
// scale is kept as an fp16 pair (22 bits): codes are positive, so an error
// there would not cancel against the minimum's share.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "q4_internal.h"
#include "q4_split.h"

namespace {

using pkv::launch_chained;

constexpr int kSub = 16;             // tokens of a subtile
constexpr int kHeads = 8;            // q heads of a unit (the n of the mma)
constexpr int kWarps = pkv::kQ4Warps;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSeqs = 1024;       // sequences of one launch
constexpr float kNone = -3e38f;      // reference exponent before the first score: finite, so
                                     // that a score of -infinity still has weight 0

struct Q4Params {
    const void *q;
    void *out;
    int out_dtype, act_f16;
    const int32_t *tables, *lens;
    int S, Hq, Hk, G, NC, GC, U, M, NB, lb;    // block size 1 << lb; U = Hk * NC units a sequence
    float scale_log2;
    const uint8_t *kc, *vc;
    const __half *kp, *vp;
    unsigned *cnt;                   // [C] arrivals, zero between calls
    float *ws_o, *ws_lse;            // [C][2][GC][D], [C][2][GC]
    int C;
    float *lse_out;
    int tables_ready;
    unsigned *err;
};

template <int D>
struct Cfg {
    static constexpr int NG = D / 32;
    static constexpr int kCodes = kSub * D / 2;          // bytes of a subtile's K (or V) codes
    static constexpr int kPar = kSub * 4 * NG;           // bytes of its K (or V) parameters
    static constexpr int kStage = 2 * kCodes + 2 * kPar;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t &a, uint32_t &b) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}

// A place in the flattened list of subtiles.
struct Cursor {
    int s, u, i, n;      // sequence, unit in it, subtile of the unit, subtiles of the unit
};

// Copies one warp's subtiles into its stages, ahead of their use.
template <int D>
struct Loader {
    using C = Cfg<D>;
    const Q4Params &p;
    const int *prefix, *len;         // shared memory: subtiles before a sequence, its length
    int lane;
    Cursor at;
    int32_t window, next_window;     // table entries: lane holds entry `base + lane` of each
    int base;

    __device__ __forceinline__ Loader(const Q4Params &p_, const int *prefix_, const int *len_, int lane_)
        : p(p_), prefix(prefix_), len(len_), lane(lane_) {}

    __device__ __forceinline__ int32_t entries(int s, int from) const {
        const int e = from + lane;
        return e < p.M ? __ldg(p.tables + (int64_t)s * p.M + e) : -1;
    }
    __device__ __forceinline__ void start(const Cursor &c) {
        at = c;
        base = ((at.i * kSub) >> p.lb) & ~31;
        window = entries(at.s, base);
        next_window = entries(at.s, base + 32);
    }
    // Next subtile; the sequence's table starts again with each unit.
    __device__ __forceinline__ void advance() {
        if (++at.i < at.n) {
            const int b = (at.i * kSub) >> p.lb;
            if (b >= base + 32) {
                base += 32;
                window = next_window;
                next_window = entries(at.s, base + 32);
            }
            return;
        }
        at.i = 0;
        if (++at.u == p.U) {
            at.u = 0;
            do ++at.s; while (at.s < p.S && prefix[at.s + 1] == prefix[at.s]);
            if (at.s >= p.S) return;             // the list's end
            at.n = prefix[at.s + 1] - prefix[at.s];
        }
        base = 0;
        window = entries(at.s, 0);
        next_window = entries(at.s, 32);
    }
    __device__ __forceinline__ void issue(uint32_t stage) {
        const int t0 = at.i * kSub, L = len[at.s], head = at.u / p.NC;
        const int B = 1 << p.lb;
        // block of the subtile's tokens 0..7 and 8..15 (one block unless B is 8)
        const int b0 = t0 >> p.lb, b1 = (t0 + 8) >> p.lb;
        int32_t id[2];
        id[0] = __shfl_sync(~0u, window, b0 - base);
        id[1] = __shfl_sync(~0u, window, b1 - base);
        bool ok[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ok[h] = id[h] >= 0 && id[h] < p.NB;
            if (!ok[h]) {
                if (lane == 0 && t0 + 8 * h < L) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                id[h] = 0;
            }
        }
        // codes: 16-byte pieces; each 128-byte line of shared memory has its
        // eight pieces exclusive-ored by a number of the line, so that the
        // fragment loads below meet 32 banks
#pragma unroll
        for (int j = 0; j < C::kCodes / 512; ++j) {
            const int c = lane + 32 * j, r = c / (D / 32), w = c % (D / 32);
            const int h = r >> 3;
            const int line = c >> 3;
            const int x = D == 128 ? (line & ~1) : ((line & 1) << 2 | (line & 2));
            const uint32_t dst = stage + line * 128 + (((c & 7) ^ x) << 4);
            const int off = (t0 + r) & (B - 1);
            const size_t src = (((size_t)id[h] * p.Hk + head) * B + off) * (D / 2) + w * 16;
            const bool live = ok[h] && t0 + r < L;
            pkv::cp_async_16(dst, p.kc + src, live);
            pkv::cp_async_16(dst + C::kCodes, p.vc + src, live);
        }
        // parameters: lanes 0..15 K (token-major), 16..31 V (tokens along the row)
        const uint32_t par = stage + 2 * C::kCodes;
        constexpr int kPieces = C::kPar / 16;            // 16 or 8
        const int l = lane & 15;
        if (l < kPieces) {
            if (lane < 16) {
                constexpr int kTok = 16 / (4 * C::NG);   // tokens of a piece: 1 or 2
                const int r = l * kTok, h = r >> 3, off = (t0 + r) & (B - 1);
                const __half *src = p.kp + (((size_t)id[h] * p.Hk + head) * B + off) * (2 * C::NG);
                const int live = ok[h] ? min(kTok, max(0, L - t0 - r)) : 0;
                pkv::cp_async_16_n(par + l * 16, src, live * 4 * C::NG);
            } else {
                const int row = l >> 1, h = l & 1, off = (t0 + 8 * h) & (B - 1);
                const __half *src = p.vp + (((size_t)id[h] * p.Hk + head) * (2 * C::NG) + row) * B + off;
                const int live = ok[h] ? min(8, max(0, L - t0 - 8 * h)) : 0;
                pkv::cp_async_16_n(par + C::kPar + l * 16, src, live * 2);
            }
        }
    }
};

// What a warp leaves of a unit it does not hold whole.
struct Piece {
    int tu, nu, s, u;     // the unit's first subtile and length in the list; its place; nu 0: none
};

template <int D, int NST>
__global__ void __launch_bounds__(kThreads, 1) decode_q4_kernel(const Q4Params p) {
    using C = Cfg<D>;
    constexpr int NG = C::NG;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int prefix[kMaxSeqs + 1], len[kMaxSeqs];
    __shared__ int scan[kWarps];
    __shared__ Piece piece[kWarps][2];
    __shared__ float piece_lse[kWarps][2][kHeads];
    __shared__ int merge_first[2], merge_n[2];
    uint8_t *ring_all = smem;
    float *heads_o = reinterpret_cast<float *>(smem + kWarps * NST * C::kStage);   // [warp][GC][D]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pkv::grid_dependents_launch();
    if (!p.tables_ready) pkv::grid_dependency_wait();

    // ---- lengths and their prefix of subtiles
    {
        constexpr int K = kMaxSeqs / kThreads;
        int n[K], sum = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int s = tid * K + k;
            int L = s < p.S ? __ldg(p.lens + s) : 0;
            if (L < 0 || L > (p.M << p.lb)) {
                if (blockIdx.x == 0) atomicOr(p.err, PKV_DEVERR_CONTEXT);
                L = L < 0 ? 0 : p.M << p.lb;
            }
            len[s] = L;
            n[k] = (L + kSub - 1) / kSub;
            sum += n[k];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) scan[warp] = inc;
        if (lane < 2) piece[warp][lane].nu = 0;
        __syncthreads();
        int before = inc - sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) before += scan[w];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            prefix[tid * K + k] = before;
            before += n[k];
        }
        if (tid == kThreads - 1) prefix[kMaxSeqs] = before;
        __syncthreads();
    }
    if (p.tables_ready) pkv::grid_dependency_wait();

    // empty contexts: zeros
    for (int s = blockIdx.x; s < p.S; s += gridDim.x)
        if (len[s] == 0) {
            for (int e = tid; e < p.Hq * D; e += kThreads)
                pkv::store_out(p.out, (size_t)s * p.Hq * D + e, p.out_dtype, 0.f);
            if (p.lse_out)
                for (int h = tid; h < p.Hq; h += kThreads) p.lse_out[(size_t)s * p.Hq + h] = -INFINITY;
        }

    // ---- this CTA's and this warp's part of the list
    const int NT = prefix[kMaxSeqs] * p.U;
    const int CT = pkv::q4_active_ctas(NT, (int)gridDim.x);
    const int cta = blockIdx.x;
    if (cta >= CT) return;
    const int A = pkv::q4_cta_cut(cta, NT, CT), Z = pkv::q4_cta_cut(cta + 1, NT, CT);
    const int a = pkv::q4_warp_cut(warp, A, Z), z = pkv::q4_warp_cut(warp + 1, A, Z);

    const uint32_t ring = pkv::smem_u32(ring_all) + warp * NST * C::kStage;
    const int g = lane >> 2, t = lane & 3;

    if (a < z) {
        Cursor c;
        {   // the sequence holding subtile a: the last whose units begin at or before it
            int lo = 0, hi = p.S - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] * p.U <= a) lo = mid;
                else hi = mid - 1;
            }
            // equal prefixes belong to empty sequences before it, not after
            c.s = lo;
            c.n = prefix[lo + 1] - prefix[lo];
            const int r = a - prefix[lo] * p.U;
            c.u = r / c.n;
            c.i = r - c.u * c.n;
        }
        Loader<D> ld(p, prefix, len, lane);
        ld.start(c);
        int to_issue = z - a;
#pragma unroll
        for (int st = 0; st < NST - 1; ++st) {
            if (to_issue > 0) {
                ld.issue(ring + st * C::kStage);
                if (--to_issue) ld.advance();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int stage = 0, fill = NST - 1;      // stage to use, stage to fill

        uint32_t qb[NG][2][2];              // q as B operands
        uint32_t qsum = 0;                  // sums of q over the groups, as a B operand
        float zs0 = 0.f, zs1 = 0.f;         // scores to log2 units, heads 2t and 2t + 1
        float me0 = kNone, me1 = kNone;     // reference exponents
        float room = 15.f;                  // largest score above the reference
        uint32_t sbound = 0;                // V scales so far stay at or below it (both halves)
        float acc[NG][2][4], accx[4];
        bool fresh = true;
        int tile = a;

        for (; tile < z; ++tile) {
            if (fresh) {
                fresh = false;
                // q of this unit: lane (g, t) holds elements 32 y + 8 t .. + 7 of head g
                const int gca = min(p.GC, p.G - (c.u % p.NC) * p.GC);
                const int h0 = (c.u / p.NC) * p.G + (c.u % p.NC) * p.GC;
                float x[NG][8], top = 0.f;
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    uint4 raw = make_uint4(0, 0, 0, 0);
                    if (g < gca)
                        raw = __ldg(reinterpret_cast<const uint4 *>(
                            static_cast<const uint16_t *>(p.q) +
                            ((size_t)c.s * p.Hq + h0 + g) * D + 32 * y + 8 * t));
                    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = p.act_f16 ? pkv::Elem<__half>::unpack2(w[i])
                                                   : pkv::Elem<__nv_bfloat16>::unpack2(w[i]);
                        x[y][2 * i] = f.x;
                        x[y][2 * i + 1] = f.y;
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                // a power of two that brings the head's largest element to
                // [2^14, 2^15): exact, and fp16 then holds q to 2^-25 of it
                const int ef = max((int)(__float_as_uint(top) >> 23), 15);
                const float up = __uint_as_float((uint32_t)(268 - ef) << 23);
                const float down = __uint_as_float((uint32_t)(ef - 14) << 23);
                float sum[NG];
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    sum[y] = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[y][i] *= up;
                        sum[y] += x[y][i];
                    }
                    sum[y] += __shfl_xor_sync(~0u, sum[y], 1);
                    sum[y] += __shfl_xor_sync(~0u, sum[y], 2);
                    sum[y] *= 0x1p-6f;               // at most 2^14
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        qb[y][k][0] = as_u32(__floats2half2_rn(x[y][2 * k], x[y][4 + 2 * k]));
                        qb[y][k][1] = as_u32(__floats2half2_rn(x[y][2 * k + 1] * 0.0625f,
                                                               x[y][4 + 2 * k + 1] * 0.0625f));
                    }
                }
                // sums as fp16 pairs: k = 0..NG-1 the high parts, then the low ones
                {
                    const int y = NG == 4 ? 2 * (t & 1) : 0;
                    float s0 = sum[0], s1 = sum[1];
                    if (NG == 4 && y == 2) {
                        s0 = sum[NG - 2];
                        s1 = sum[NG - 1];
                    }
                    __half2 hi = __floats2half2_rn(s0, s1);
                    const bool low = NG == 4 ? t >= 2 : t == 1;
                    if (low) {
                        const float2 f = __half22float2(hi);
                        hi = __floats2half2_rn(s0 - f.x, s1 - f.y);
                    }
                    qsum = NG == 2 && t >= 2 ? 0u : as_u32(hi);
                }
                const float zq = p.scale_log2 * 0x1p24f * down;
                zs0 = __shfl_sync(~0u, zq, 8 * t);
                zs1 = __shfl_sync(~0u, zq, 8 * t + 4);
                me0 = me1 = kNone;
                room = 15.f;
                sbound = 0x3c003c00u;                // 1
#pragma unroll
                for (int y = 0; y < NG; ++y)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[y][k][i] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) accx[i] = 0.f;
            }

            asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
            __syncwarp();
            // the stage used last is free now: fill it
            if (to_issue > 0) {
                ld.issue(ring + fill * C::kStage);
                if (--to_issue) ld.advance();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");

            const uint32_t sk = ring + stage * C::kStage, sv = sk + C::kCodes;
            const uint32_t pk = sv + C::kCodes, pv = pk + C::kPar;
            fill = stage;
            stage = stage + 1 == NST ? 0 : stage + 1;

            // ---- scores: rows g and g + 8 of the product are tokens r0 and r0 + 2,
            // so that after the transpose below lane t holds tokens 4t .. 4t + 3
            const int r0 = 4 * (g >> 1) + (g & 1);
            float sc[4];
            {
                uint32_t w[2][NG];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + 2 * h;
                    if constexpr (NG == 4) {
                        const int line = r >> 1, x = line & ~1;
                        pkv::lds_u32x4(sk + line * 128 + (((4 * (r & 1) + t) ^ x) << 4), w[h][0], w[h][1],
                                       w[h][2], w[h][3]);
                    } else {
                        const int line = r >> 2, x = (line & 1) << 2 | (line & 2);
                        lds64(sk + line * 128 + (((2 * (r & 3) + (t >> 1)) ^ x) << 4) + 8 * (t & 1), w[h][0],
                              w[h][1]);
                    }
                }
                float s0[NG], s1[NG];                // scales of tokens r0, r0 + 2
                uint32_t m0, m1;                     // minima of two groups
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t row = pk + (r0 + 2 * h) * 4 * NG;
                    uint32_t u[2];
                    if constexpr (NG == 4) lds64(row, u[0], u[1]);
                    else u[0] = pkv::lds_u32(row);
#pragma unroll
                    for (int y = 0; y < NG; y += 2) {
                        const float2 f = __half22float2(as_h2(u[y / 2]));
                        (h ? s1 : s0)[y] = f.x;
                        (h ? s1 : s0)[y + 1] = f.y;
                    }
                    uint32_t m = pkv::lds_u32(row + 2 * NG + (NG == 4 ? 4 * (t & 1) : 0));
                    if (NG == 2 && t >= 2) m = 0;
                    (h ? m1 : m0) = m;
                }
                float mn[4] = {0.f, 0.f, 0.f, 0.f};
                mma8(mn, m0, m1, qsum);
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[i] = mn[i] * 0x1p-18f;
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t wa = w[0][y], wb = w[1][y];
                    mma16(d, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u,
                          qb[y][0][0], qb[y][0][1]);
                    wa >>= 8;
                    wb >>= 8;
                    mma16(d, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u,
                          qb[y][1][0], qb[y][1][1]);
                    sc[0] = fmaf(d[0], s0[y], sc[0]);
                    sc[1] = fmaf(d[1], s0[y], sc[1]);
                    sc[2] = fmaf(d[2], s1[y], sc[2]);
                    sc[3] = fmaf(d[3], s1[y], sc[3]);
                }
            }
            sc[0] *= zs0;
            sc[1] *= zs1;
            sc[2] *= zs0;
            sc[3] *= zs1;
            const int left = len[c.s] - c.i * kSub;          // valid tokens from here on
            if (left < kSub) {
                if (r0 >= left) sc[0] = sc[1] = -INFINITY;
                if (r0 + 2 >= left) sc[2] = sc[3] = -INFINITY;
            }

            // ---- V scales of tokens 4t .. 4t + 3, and the reference exponent
            uint32_t vs[NG][2];
            __half2 big = __float2half2_rn(0.f);
#pragma unroll
            for (int y = 0; y < NG; ++y) {
                lds64(pv + y * 32 + t * 8, vs[y][0], vs[y][1]);
                big = __hmax2(big, __hmax2(as_h2(vs[y][0]), as_h2(vs[y][1])));
            }
            const float over = fmaxf(fmaxf(sc[0], sc[2]) - me0, fmaxf(sc[1], sc[3]) - me1);
            if (__any_sync(~0u, over > room || !__hble2(big, as_h2(sbound)))) {
                // raise the bound on V scales to this subtile's largest, the
                // reference to 7 (less where scales are large) below the top score
                float bs = fmaxf(__low2float(big), __high2float(big));
                float t0 = fmaxf(sc[0], sc[2]), t1 = fmaxf(sc[1], sc[3]);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    bs = fmaxf(bs, __shfl_xor_sync(~0u, bs, o));
                    if (o >= 4) {
                        t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, o));
                        t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, o));
                    }
                }
                bs = fminf(fmaxf(bs, __low2float(as_h2(sbound))), 65504.f);
                sbound = as_u32(__float2half2_rn(bs));
                // scales up to 2^e, e >= 0: weights up to 2^(15 - e)
                const int e = ((int)(__float_as_uint(bs) >> 23) - 127) + 1;
                room = 15.f - (float)e;
                const float n0 = fmaxf(me0, t0 - 7.f + (float)e), n1 = fmaxf(me1, t1 - 7.f + (float)e);
                const float f0 = ex2(me0 - n0), f1 = ex2(me1 - n1);
                me0 = n0;
                me1 = n1;
#pragma unroll
                for (int y = 0; y < NG; ++y)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        acc[y][k][0] *= f0;
                        acc[y][k][1] *= f1;
                        acc[y][k][2] *= f0;
                        acc[y][k][3] *= f1;
                    }
                accx[0] *= f0;
                accx[1] *= f1;
                accx[2] *= f0;
                accx[3] *= f1;
            }

            // ---- weights, transposed: lane (g, t) then has head g, tokens 4t .. 4t + 3
            const uint32_t p01 =
                transpose8(as_u32(__floats2half2_rn(ex2(sc[0] - me0), ex2(sc[1] - me1))));
            const uint32_t p23 =
                transpose8(as_u32(__floats2half2_rn(ex2(sc[2] - me0), ex2(sc[3] - me1))));

            // ---- V: rows of the product are d, its contracted index the tokens
            uint32_t v01[NG], v23[NG];
            {
                uint32_t w[4][NG / 2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * t + j;
                    if constexpr (NG == 4) {
                        const int line = r >> 1, x = line & ~1;
                        lds64(sv + line * 128 + (((4 * (r & 1) + (g >> 1)) ^ x) << 4) + 8 * (g & 1),
                              w[j][0], w[j][1]);
                    } else {
                        const int line = r >> 2, x = (line & 1) << 2 | (line & 2);
                        w[j][0] = pkv::lds_u32(sv + line * 128 + (((2 * (r & 3) + (g >> 2)) ^ x) << 4) +
                                               4 * (g & 3));
                    }
                }
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    const uint32_t sel = y & 1 ? 0x7632u : 0x5410u;
                    v01[y] = __byte_perm(w[0][y / 2], w[1][y / 2], sel);
                    v23[y] = __byte_perm(w[2][y / 2], w[3][y / 2], sel);
                }
            }
            {
                // minima as rows 0..NG-1, a row of ones as row 8
                uint32_t m01, m23;
                lds64(pv + (NG + (g & (NG - 1))) * 32 + t * 8, m01, m23);
                if (g >= NG) m01 = m23 = 0;
                const uint32_t one = g == 0 ? 0x3c003c00u : 0u;
                mma16(accx, m01, one, m23, one, p01, p23);
            }
#pragma unroll
            for (int y = 0; y < NG; ++y) {
                const __half2 h01 = __hmul2(as_h2(p01), as_h2(vs[y][0]));
                const __half2 h23 = __hmul2(as_h2(p23), as_h2(vs[y][1]));
                const uint32_t l01 = as_u32(__hfma2(as_h2(p01), as_h2(vs[y][0]), __hneg2(h01)));
                const uint32_t l23 = as_u32(__hfma2(as_h2(p23), as_h2(vs[y][1]), __hneg2(h23)));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t wa = v01[y] >> (8 * k), wb = v23[y] >> (8 * k);
                    const uint32_t a0 = wa & 0x000f000fu, a1 = wa & 0x00f000f0u;
                    const uint32_t a2 = wb & 0x000f000fu, a3 = wb & 0x00f000f0u;
                    mma16(acc[y][k], a0, a1, a2, a3, as_u32(h01), as_u32(h23));
                    mma16(acc[y][k], a0, a1, a2, a3, l01, l23);
                }
            }

            // ---- the unit's last subtile here: its output, or a piece
            if (c.i == c.n - 1 || tile == z - 1) {
                const int gca = min(p.GC, p.G - (c.u % p.NC) * p.GC);
                const int h0 = (c.u / p.NC) * p.G + (c.u % p.NC) * p.GC;
                const int tu = tile - c.i;
                const bool whole = tu >= a && c.i == c.n - 1;
                const int slot = tu < a ? 0 : 1;
                const float l0 = __shfl_sync(~0u, accx[2], t), l1 = __shfl_sync(~0u, accx[3], t);
                const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
                // a piece of a unit that goes on in the next warp lies in this
                // warp's ring, which is read to the end; the other has its own place
                float *po = slot ? reinterpret_cast<float *>(ring_all + warp * NST * C::kStage)
                                 : heads_o + (size_t)warp * p.GC * D;
                if (slot && !whole) __syncwarp();
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    const float x0 = __shfl_sync(~0u, accx[0], 4 * y + t);
                    const float x1 = __shfl_sync(~0u, accx[1], 4 * y + t);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {            // head 2t + e
                        const int h = 2 * t + e;
                        if (h >= gca) continue;
                        const float m = e ? x1 : x0, inv = e ? inv1 : inv0;
                        const float o0 = fmaf(acc[y][0][e], 0x1p24f, m) * inv;
                        const float o1 = fmaf(acc[y][0][2 + e], 0x1p20f, m) * inv;
                        const float o2 = fmaf(acc[y][1][e], 0x1p24f, m) * inv;
                        const float o3 = fmaf(acc[y][1][2 + e], 0x1p20f, m) * inv;
                        const int d = 32 * y + 4 * g;
                        if (whole) {
                            const size_t at = ((size_t)c.s * p.Hq + h0 + h) * D + d;
                            if (p.out_dtype == PKV_F32) {
                                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
                                    make_float4(o0, o1, o2, o3);
                            } else {
                                uint2 w;
                                if (p.out_dtype == PKV_F16) {
                                    w.x = as_u32(__floats2half2_rn(o0, o1));
                                    w.y = as_u32(__floats2half2_rn(o2, o3));
                                } else {
                                    float u0, u1;
                                    w.x = pkv::Elem<__nv_bfloat16>::pack2(o0, o1, u0, u1);
                                    w.y = pkv::Elem<__nv_bfloat16>::pack2(o2, o3, u0, u1);
                                }
                                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = w;
                            }
                        } else {
                            *reinterpret_cast<float4 *>(po + h * D + d) = make_float4(o0, o1, o2, o3);
                        }
                    }
                }
                if (g == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = 2 * t + e;
                        if (h >= gca) continue;
                        const float lse = (e ? me1 : me0) + log2f(e ? l1 : l0);
                        if (!whole) piece_lse[warp][slot][h] = lse;
                        else if (p.lse_out) p.lse_out[(size_t)c.s * p.Hq + h0 + h] = lse;
                    }
                }
                if (!whole && lane == 0) piece[warp][slot] = {tu, c.n, c.s, c.u};
                fresh = true;
            }
            if (++c.i == c.n) {
                c.i = 0;
                if (++c.u == p.U) {
                    c.u = 0;
                    do ++c.s; while (c.s < p.S && prefix[c.s + 1] == prefix[c.s]);
                    if (c.s < p.S) c.n = prefix[c.s + 1] - prefix[c.s];
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (tid < 2) merge_n[tid] = 0;
    __syncthreads();

    // ---- join the pieces of each unit cut between this CTA's warps. A unit's
    // pieces here: one that starts it (slot 1 of some warp, or slot 0 of warp 0
    // when it began in an earlier CTA), then slot 0 of the warps after
    bool open0 = false, open1 = false;       // units cut at this CTA's start, at its end
    for (int w = 0; w < kWarps; ++w) {
        for (int sl = w == 0 ? 0 : 1; sl < 2; ++sl) {
            const Piece pc = piece[w][sl];
            if (pc.nu == 0) continue;
            int last = w;
            while (last + 1 < kWarps && piece[last + 1][0].nu && piece[last + 1][0].tu == pc.tu) ++last;
            const int gca = min(p.GC, p.G - (pc.u % p.NC) * p.GC);
            const int h0 = (pc.u / p.NC) * p.G + (pc.u % p.NC) * p.GC;
            const bool done = pc.tu >= A && pc.tu + pc.nu <= Z;
            const int side = pc.tu < A ? 0 : 1;
            for (int e = tid; e < gca * D; e += kThreads) {
                const int h = e / D;
                float mx = piece_lse[w][sl][h];
                for (int k = w + 1; k <= last; ++k) mx = fmaxf(mx, piece_lse[k][0][h]);
                if (mx == -INFINITY) mx = 0.f;
                float sum = 0.f, o = 0.f;
                for (int k = w; k <= last; ++k) {
                    const int ks = k == w ? sl : 0;
                    const float f = ex2(piece_lse[k][ks][h] - mx);
                    const float *src = ks ? reinterpret_cast<const float *>(ring_all + k * NST * C::kStage)
                                          : heads_o + (size_t)k * p.GC * D;
                    sum += f;
                    o = fmaf(f, src[e], o);
                }
                o = sum == 0.f ? 0.f : o / sum;
                const float lse = mx + log2f(sum);
                if (done) {
                    pkv::store_out(p.out, ((size_t)pc.s * p.Hq + h0) * D + e, p.out_dtype, o);
                    if (p.lse_out && e % D == 0) p.lse_out[(size_t)pc.s * p.Hq + h0 + h] = lse;
                } else {
                    const size_t at = (size_t)(2 * cta + side) * p.GC;
                    p.ws_o[at * D + e] = o;
                    if (e % D == 0) p.ws_lse[at + h] = lse;
                }
            }
            open0 |= !done && side == 0;
            open1 |= !done && side == 1;
        }
    }
    if (!open0 && !open1) return;

    // ---- units cut between CTAs: count this CTA's part in; the last to come joins
    __syncthreads();
    if (tid == 0) {
        pkv::fence_acq_rel_gpu();
        for (int side = 0; side < 2; ++side) {
            if (!(side ? open1 : open0)) continue;
            const int edge = side == 0 ? A : Z - 1;      // a subtile of the unit in this CTA
            // its unit, from the pieces: slot 0 of warp 0, or the last piece
            Piece pc = {0, 0, 0, 0};
            if (side == 0) pc = piece[0][0];
            else
                for (int w = 0; w < kWarps; ++w)
                    for (int sl = 0; sl < 2; ++sl)
                        if (piece[w][sl].nu && piece[w][sl].tu <= edge &&
                            edge < piece[w][sl].tu + piece[w][sl].nu)
                            pc = piece[w][sl];
            const int first = pkv::q4_owner(pc.tu, NT, CT);
            const int n = pkv::q4_owner(pc.tu + pc.nu - 1, NT, CT) - first + 1;
            if (atomicAdd(p.cnt + first, 1u) == (unsigned)n - 1) {
                p.cnt[first] = 0;
                merge_first[side] = first;
                merge_n[side] = n;
                scan[2 * side] = pc.s;
                scan[2 * side + 1] = pc.u;
            }
        }
        pkv::fence_acq_rel_gpu();
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const int n = merge_n[side], first = merge_first[side];
        if (n == 0) continue;
        const int s = scan[2 * side], u = scan[2 * side + 1];
        const int gca = min(p.GC, p.G - (u % p.NC) * p.GC);
        const int h0 = (u / p.NC) * p.G + (u % p.NC) * p.GC;
        for (int e = tid; e < gca * D; e += kThreads) {
            const int h = e / D;
            // the first CTA's part is its side 1, the others' their side 0
            float mx = -INFINITY;
            for (int k = 0; k < n; ++k)
                mx = fmaxf(mx, __ldcg(p.ws_lse + (size_t)(2 * (first + k) + (k == 0)) * p.GC + h));
            if (mx == -INFINITY) mx = 0.f;
            float sum = 0.f, o = 0.f;
            for (int k = 0; k < n; ++k) {
                const size_t at = (size_t)(2 * (first + k) + (k == 0)) * p.GC;
                const float f = ex2(__ldcg(p.ws_lse + at + h) - mx);
                sum += f;
                o = fmaf(f, __ldcg(p.ws_o + at * D + e), o);
            }
            pkv::store_out(p.out, ((size_t)s * p.Hq + h0) * D + e, p.out_dtype,
                           sum == 0.f ? 0.f : o / sum);
            if (p.lse_out && e % D == 0) p.lse_out[(size_t)s * p.Hq + h0 + h] = mx + log2f(sum);
        }
    }
}

// Shared memory of a variant: the rings, then a piece's place for each warp.
template <int D, int NST>
size_t smem_bytes(int GC) {
    return (size_t)kWarps * (NST * Cfg<D>::kStage + GC * D * sizeof(float));
}

template <int D, int NST>
cudaError_t launch(const Q4Params &p, cudaStream_t stream) {
    // the attribute is per device and idempotent; set once for each
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(decode_q4_kernel<D, NST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<D, NST>(NST == 4 ? 4 : kHeads));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(decode_q4_kernel<D, NST>, dim3((unsigned)p.C), kThreads, smem_bytes<D, NST>(p.GC),
                          stream, p);
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// workspace: [PKV_MAX_DECODE_CTAS] arrival counters (a fixed region, whatever
// the launch), then [C][2][GC][D] outputs, then [C][2][GC] log2 denominators
constexpr size_t kCounterBytes = PKV_MAX_DECODE_CTAS * sizeof(unsigned);
size_t workspace_for(int C, int GC, int D) {
    return kCounterBytes + (size_t)C * 2 * GC * (D + 1) * sizeof(float);
}

}  // namespace

extern "C" {

size_t pkv_decode_q4_workspace_bytes(const pkv_q4cache_desc *cache, int32_t num_q_heads,
                                     int32_t num_ctas) {
    if (pkv::check_q4cache(cache) != PKV_OK) return 0;
    if (num_q_heads < 1 || num_q_heads % cache->num_kv_heads || num_ctas < 0 ||
        num_ctas > PKV_MAX_DECODE_CTAS)
        return 0;
    int C = num_ctas;
    if (C == 0 && pkv::device_sm_count(&C) != PKV_OK) return 0;
    const int G = num_q_heads / cache->num_kv_heads;
    return workspace_for(C, G < kHeads ? G : kHeads, cache->head_dim);
}

pkv_status pkv_decode_attention_q4(const pkv_q4cache_desc *cache, const void *q, int32_t num_seqs,
                                   int32_t num_q_heads, const pkv_q4cache_pools *pools,
                                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                                   const int32_t *context_lens, float scale, void *out,
                                   int32_t out_dtype, void *workspace, size_t workspace_bytes,
                                   void *stream, const pkv_decode_options *o) {
    pkv_status st = pkv::check_q4cache(cache);
    if (st != PKV_OK) return st;
    const int Hk = cache->num_kv_heads, D = cache->head_dim, M = max_blocks_per_seq;
    if (num_q_heads < 1 || num_q_heads % Hk)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "num_q_heads %d is not a positive multiple of num_kv_heads %d",
                                   num_q_heads, Hk);
    if (num_seqs < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", num_seqs);
    if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
    if (M < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", M);
    if (!isfinite(scale)) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "scale is not finite");
    int C = o ? o->num_ctas : 0;
    if (o) {
        if (o->consumer < 0 || o->consumer > 2)
            return pkv::set_last_error(PKV_ERR_INVALID_ARG, "consumer %d", o->consumer);
        if (o->consumer == 1)
            return pkv::set_last_error(PKV_ERR_UNSUPPORTED,
                                       "4-bit caches use the tensor-core math (consumer 1 given)");
        if (C < 0 || C > PKV_MAX_DECODE_CTAS)
            return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_ctas %d outside [0, %d]", C,
                                       PKV_MAX_DECODE_CTAS);
        if (o->pending_tail < 0)
            return pkv::set_last_error(PKV_ERR_INVALID_ARG, "pending_tail %d is negative",
                                       o->pending_tail);
        if (o->pending_tail > 0 && !o->tables_ready)
            return pkv::set_last_error(PKV_ERR_INVALID_ARG, "pending_tail needs tables_ready");
    }
    if (num_seqs == 0) return PKV_OK;
    if (!q || !block_tables || !context_lens || !out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if ((st = pkv::check_q4pools(pools)) != PKV_OK) return st;
    const int oes = out_dtype == PKV_F32 ? 4 : 2;
    if (misaligned(q, 16) || misaligned(out, 4 * oes) || misaligned(block_tables, 4) ||
        misaligned(context_lens, 4) || (o && misaligned(o->lse_out, 4)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "q must be 16-byte aligned, out to four of its elements");
    const int G = num_q_heads / Hk, GC = G < kHeads ? G : kHeads, NC = (G + GC - 1) / GC;
    // flattened subtile counts, times the CTAs, are taken in 64 bits; the list itself in 32
    const int64_t tokens = (int64_t)M * cache->block_size;
    const int64_t seqs = num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs;
    if (tokens > INT32_MAX / 2 ||
        seqs * Hk * NC * ((tokens + kSub - 1) / kSub) >= (int64_t)INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
    if (C == 0 && (st = pkv::device_sm_count(&C)) != PKV_OK) return st;
    const size_t need = workspace_for(C, GC, D);
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    Q4Params p = {};
    if ((st = pkv::device_error_word(&p.err)) != PKV_OK) return st;
    p.out_dtype = out_dtype;
    p.act_f16 = cache->act_dtype == PKV_F16;
    p.Hq = num_q_heads;
    p.Hk = Hk;
    p.G = G;
    p.NC = NC;
    p.GC = GC;
    p.U = Hk * NC;
    p.M = M;
    p.NB = cache->num_blocks;
    p.lb = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.kc = static_cast<const uint8_t *>(pools->k_codes);
    p.vc = static_cast<const uint8_t *>(pools->v_codes);
    p.kp = static_cast<const __half *>(pools->k_params);
    p.vp = static_cast<const __half *>(pools->v_params);
    p.cnt = static_cast<unsigned *>(workspace);
    p.ws_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    p.ws_lse = p.ws_o + (size_t)C * 2 * GC * D;
    p.C = C;
    p.tables_ready = o && o->tables_ready;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int s0 = 0; s0 < num_seqs; s0 += kMaxSeqs) {
        p.S = num_seqs - s0 < kMaxSeqs ? num_seqs - s0 : kMaxSeqs;
        p.q = static_cast<const uint16_t *>(q) + (size_t)s0 * num_q_heads * D;
        p.out = static_cast<uint8_t *>(out) + (size_t)s0 * num_q_heads * D * oes;
        p.tables = block_tables + (size_t)s0 * M;
        p.lens = context_lens + s0;
        p.lse_out = o && o->lse_out ? static_cast<float *>(o->lse_out) + (size_t)s0 * num_q_heads : nullptr;
        cudaError_t e;
        if (s0 == 0 && o && o->timing_events[0] &&
            (e = pkv::record_event(static_cast<cudaEvent_t>(o->timing_events[0]), s)) != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "cudaEventRecord: %s", cudaGetErrorString(e));
        // up to 4 heads a unit leave room for a fourth stage
        if (D == 128) e = GC <= 4 ? launch<128, 4>(p, s) : launch<128, 3>(p, s);
        else e = GC <= 4 ? launch<64, 4>(p, s) : launch<64, 3>(p, s);
        if (e != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "decode_q4 launch: %s", cudaGetErrorString(e));
        if (s0 == 0 && o && o->timing_events[1] &&
            (e = pkv::record_event(static_cast<cudaEvent_t>(o->timing_events[1]), s)) != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "cudaEventRecord: %s", cudaGetErrorString(e));
    }
    return PKV_OK;
}

}  // extern "C"

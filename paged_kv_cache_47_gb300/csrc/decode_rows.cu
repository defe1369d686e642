// Decode attention over many short contexts of a 16-bit cache: what the
// block-sparse decode is once its blocks are chosen (a table and a length for
// each sequence and kv head).
//
// The split-K kernel feeds all of a CTA's math warps from producer warps, tile
// by tile; each unit's end stops them all for a combine. Contexts of a few
// hundred tokens are mostly ends: 512 contexts of 592 tokens took 69 us there,
// 3.0 times their bytes' time. Here warps run alone (warp_decode.cuh): a
// subtile is 16 tokens of one unit, copied by the warp's own cp.async into its
// own ring, and no warp waits for another until the end.
//
// Products. S = Q K^T with the unit's (up to 8) q heads as rows 0..7 of the
// m16n8k16's m: then a lane's scores are already where the next product wants
// its weights, and rows 8..15 carry the weights' low parts: O = [P_hi; P_lo] V
// costs nothing more than P_hi V, and weights keep 16 (bf16) or 22 (fp16) bits.
// bf16's half a step, 2^-17, is 2^-8 of the one that a bf16 output has; a third
// part in a product of its own took 0.7 us of 51 and 1 of 74 (the two cases
// below with their selections). Softmax in base 2 in
// fp32, with a reference exponent that moves only when a score passes what the
// type holds: fp16 weights stand as high as they can, the top one at 2^10 to
// 2^15, so that a light token keeps its bits down to 2^-35 of the top. The
// denominator sums the weights as they enter the product.
//
// What bounds it: HBM, 4 D bytes a token. 10 warps keep two subtiles each in
// flight or in use, 160 KB an SM, and the pieces that they leave fit beside the
// rings: 12 warps whose pieces went through memory took 5 us more, as a join
// waits for such loads twice. 512 contexts of 592 tokens (155 MB) take 33 us and
// 64 of 4096 with 8 heads each (135 MB) 31; from the first copy to the last the
// stream runs at the memory's rate, the list and the first table entries before
// it (4 us) and the joins after it (5) are what is left. A unit counted as two
// subtiles evens the warps' ends out by 0.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "rows_internal.h"
#include "warp_decode.cuh"

namespace {

using pkv::launch_chained;
using pkv::wd_ex2;

constexpr int kSub = 16;             // tokens of a subtile
constexpr int kHeads = pkv::kWdHeads;
constexpr int kWarps = 10;
constexpr int kThreads = 32 * kWarps;
// Contexts of one launch. The longer list costs its scan and the L1 that it
// takes, half a microsecond, and is taken where it saves a second launch.
constexpr int kFewSeqs = 1024, kMaxSeqs = pkv::kRowsMaxSeqs;
constexpr int kUnitCost = 2;         // what a unit costs a warp besides its subtiles, in subtiles
constexpr float kNone = pkv::kWdNone;
// Exponent that a reference gives the top score, and the largest that needs no new one.
template <typename T> constexpr float kTop = 0.f;
template <> constexpr float kTop<__half> = 10.f;
template <typename T> constexpr float kRoom = 8.f;
template <> constexpr float kRoom<__half> = 15.f;

struct RowsParams {
    pkv::WdList list;
    pkv::WdOut o;
    const void *q;
    const uint8_t *k, *v;
    int Hk, NB;
    uint32_t chunk_bytes;            // of one (block, kv head) chunk, K or V
    float scale_log2;
    int C;
};

template <int D>
struct Cfg {
    static constexpr int kRow = 2 * D;                   // bytes of a row
    static constexpr int kHalf = kSub * kRow;            // K or V of a subtile
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kRing = kStages * kStage;       // 16 KB
    static constexpr int kPieces = kHalf / 512;          // 16-byte pieces a lane copies, K or V
};

// A row's 16-byte pieces are exclusive-ored by the row modulo 8: the fragment
// loads' eight rows then lie in 32 banks. Lane's piece j of a subtile:
template <int D>
__device__ __forceinline__ uint32_t piece_dst(int lane, int j) {
    constexpr int PPR = Cfg<D>::kRow / 16;               // pieces a row: 16 or 8
    const int c = lane + 32 * j, r = c / PPR, w = c % PPR;
    return r * Cfg<D>::kRow + ((w ^ (r & 7)) << 4);
}

// A context's last subtile, or one with a block id outside the pool: what is
// not there becomes zeros.
template <int D, int LB>
__device__ __noinline__ void issue_ragged(const RowsParams &p, uint32_t stage, int32_t window, int at, int off,
                                          int head, int left, int lane) {
    using C = Cfg<D>;
    constexpr int B = 1 << LB;
#pragma unroll 1
    for (int j = 0; j < C::kPieces; ++j) {
        const int c = lane + 32 * j, r = c / (C::kRow / 16), w = c % (C::kRow / 16);
        int id = __shfl_sync(~0u, window, at + ((off + r) >> LB));
        const bool ok = (unsigned)id < (unsigned)p.NB;
        if (!ok && r < left) atomicOr(p.list.err, PKV_DEVERR_BLOCK_ID);
        if (!ok) id = 0;
        const size_t src = ((size_t)id * p.Hk + head) * p.chunk_bytes + ((off + r) & (B - 1)) * C::kRow + w * 16;
        const uint32_t dst = stage + piece_dst<D>(lane, j);
        pkv::cp_async_16(dst, p.k + src, ok && r < left);
        pkv::cp_async_16(dst + C::kHalf, p.v + src, ok && r < left);
    }
}

// Copies one warp's subtiles into its stages, ahead of their use.
template <int D, int LB>
struct Loader {
    using C = Cfg<D>;
    const RowsParams &p;
    const int *len;
    int lane, cost;                  // cost: places before a unit's first subtile
    int s, u, head, t0, left;
    int32_t window, next_window;     // table entries: lane holds entry `base + lane` of each
    int base;

    __device__ __forceinline__ Loader(const RowsParams &p_, const int *len_, int lane_, int cost_)
        : p(p_), len(len_), lane(lane_), cost(cost_) {}

    __device__ __forceinline__ int32_t entries(int from) const {
        const int e = from + lane;
        return e < p.list.M ? __ldg(p.list.tables + (int64_t)s * p.list.M + e) : -1;
    }
    __device__ __forceinline__ void windows() {
        base = (t0 >> LB) & ~31;
        window = entries(base);
        next_window = entries(base + 32);
    }
    __device__ __forceinline__ void start(const pkv::WdPlace &at) {
        s = at.s;
        u = at.u;
        head = u / p.o.NC;
        t0 = at.i * kSub;
        left = len[s] - t0;
        windows();
    }
    // Next subtile; returns the places passed over.
    __device__ __forceinline__ int advance() {
        t0 += kSub;
        left -= kSub;
        if (left > 0) {
            if ((t0 >> LB) >= base + 32) {
                base += 32;
                window = next_window;
                next_window = entries(base + 32);
            }
            return 0;
        }
        if (++u == p.list.U) {
            u = 0;
            do ++s; while (s < p.list.S - 1 && len[s] == 0);
        }
        head = u / p.o.NC;
        t0 = 0;
        left = len[s];
        windows();
        return cost;
    }
    __device__ __forceinline__ void issue(uint32_t stage) {
        // the block of tokens 0..7, and of 8..15 (the same unless blocks hold 8)
        const int at = (t0 >> LB) - base, off = LB == 5 ? t0 & 16 : 0;
        const int id0 = __shfl_sync(~0u, window, at);
        const int id1 = LB == 3 ? __shfl_sync(~0u, window, at + 1) : id0;
        if (left < kSub || (unsigned)id0 >= (unsigned)p.NB || (LB == 3 && (unsigned)id1 >= (unsigned)p.NB)) {
            issue_ragged<D, LB>(p, stage, window, at, off, head, left, lane);
            return;
        }
        const uint64_t src0 = (uint64_t)(uint32_t)(id0 * p.Hk + head) * p.chunk_bytes +
                              (uint32_t)(off * C::kRow + lane * 16);
        const uint64_t src1 = LB == 3 ? (uint64_t)(uint32_t)(id1 * p.Hk + head) * p.chunk_bytes + lane * 16
                                      : src0 + C::kHalf / 2;
#pragma unroll
        for (int j = 0; j < C::kPieces; ++j) {
            const uint32_t dst = stage + piece_dst<D>(lane, j);
            const uint64_t src = (j < C::kPieces / 2 ? src0 : src1) + j % (C::kPieces / 2) * 512;
            pkv::cp_async_16(dst, p.k + src, true);
            pkv::cp_async_16(dst + C::kHalf, p.v + src, true);
        }
    }
};

template <typename T, int D, int LB, int N>
__global__ void __launch_bounds__(kThreads, 1) decode_rows_kernel(const __grid_constant__ RowsParams p) {
    using C = Cfg<D>;
    using E = pkv::Elem<T>;
    using Mma = pkv::MmaOp<T>;
    extern __shared__ __align__(1024) uint8_t rings[];
    __shared__ pkv::WdListShared<kWarps, N> list;
    __shared__ pkv::WdJoinShared<kWarps> join;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // pieces of units that began before a warp's share: [warps][GC][D] behind the rings
    float *heads_o = reinterpret_cast<float *>(rings + kWarps * Cfg<D>::kRing);
    pkv::grid_dependents_launch();
    pkv::wd_join_init(join);
    const pkv::WdShare share = pkv::wd_share<kWarps, kSub>(p.list, p.o, D, kUnitCost, list);
    if ((int)blockIdx.x >= share.CT) return;
    const int a = share.a, z = share.z;
    const uint32_t ring = pkv::smem_u32(rings) + warp * C::kRing, ring_end = ring + C::kRing;
    const int g = lane >> 2, t = lane & 3;

    if (a < z) {
        pkv::WdPlace at = pkv::wd_place(p.list, list, a, share.cost);
        Loader<D, LB> ld(p, list.len, lane, share.cost);
        ld.start(at);
        int rem = z - (at.tu + at.i);        // places from the next subtile to copy on
#pragma unroll
        for (int st = 0; st < C::kStages; ++st) {
            if (rem > 0) {
                ld.issue(ring + st * C::kStage);
                if (--rem > 0) rem -= ld.advance();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        uint32_t stage = ring;
        // this lane's rows of the fragment loads: K's four matrices are tokens
        // 0..7 and 8..15 by two neighbouring pieces, V's tokens by pieces
        // (a stage begins at a multiple of the row, so pieces are exclusive-ored
        // into the whole address)
        const int k_row = (lane & 7) + ((lane >> 4) << 3), v_row = lane & 15;
        const uint32_t k_at = k_row * C::kRow + ((((lane >> 3) & 1) ^ (k_row & 7)) << 4);
        const uint32_t v_at = C::kHalf + v_row * C::kRow + (((lane >> 4) ^ (v_row & 7)) << 4);

        while (true) {
            // ---- a unit, or the part of it that lies here: `count` subtiles
            const int n = at.nv - share.cost;
            const int count = min(n, z - at.tu) - at.i;
            if (count <= 0) break;
            const int gca = p.o.heads(at.u), h0 = p.o.first_head(at.u);
            int left = list.len[at.s] - at.i * kSub;
            // q as A operands: rows 0..7 are the heads, rows 8..15 nothing
            uint32_t qa[D / 16][2];
            {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(
                    static_cast<const uint16_t *>(p.q) + ((size_t)at.s * p.o.Hq + h0 + (g < gca ? g : 0)) * D) + t;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qa[k][0] = g < gca ? __ldg(src + 8 * k) : 0u;
                    qa[k][1] = g < gca ? __ldg(src + 8 * k + 4) : 0u;
                }
            }
            float mu = kNone, room = -INFINITY, l = 0.f;     // of head g
            float acc[D / 8][4];             // head g: high parts' products, low parts'
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

            for (int it = 0; it < count; ++it) {
                asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
                __syncwarp();
                // ---- scores of head g: tokens 2t, 2t + 1 and 8 + 2t, 9 + 2t
                float s0[4] = {}, s1[4] = {};
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t b0, b1, b2, b3;
                    pkv::ldsm_x4((stage + k_at) ^ (k << 5), b0, b1, b2, b3);
                    Mma::run(s0, qa[k][0], 0u, qa[k][1], 0u, b0, b1);
                    Mma::run(s1, qa[k][0], 0u, qa[k][1], 0u, b2, b3);
                }
                float e[4] = {fmaf(s0[0], p.scale_log2, -mu), fmaf(s0[1], p.scale_log2, -mu),
                              fmaf(s1[0], p.scale_log2, -mu), fmaf(s1[1], p.scale_log2, -mu)};
                if (left < kSub) {
                    if (2 * t >= left) e[0] = -INFINITY;
                    if (2 * t + 1 >= left) e[1] = -INFINITY;
                    if (2 * t + 8 >= left) e[2] = -INFINITY;
                    if (2 * t + 9 >= left) e[3] = -INFINITY;
                }
                left -= kSub;
                float top = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                if (__any_sync(~0u, top > room)) {
                    top += mu;
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const bool none = mu == kNone;
                    float nm = mu;
                    if (top > -INFINITY) nm = none ? top - kTop<T> : fmaxf(mu, top - kTop<T>);
                    const float f = none ? 1.f : wd_ex2(mu - nm);
                    // a head that has had no score but -infinity keeps none,
                    // and the next subtile asks again
                    room = __any_sync(~0u, nm == kNone) ? -INFINITY : kRoom<T>;
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = e[i] + mu - nm;
                    mu = nm;
                    l *= f;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j][i] *= f;
                }
                // ---- weights: high parts in rows 0..7, low parts in rows 8..15
                float w[4], r0, r1, r2, r3, x0, x1, x2, x3;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = wd_ex2(e[i]);
                const uint32_t a0 = E::pack2(w[0], w[1], r0, r1), a2 = E::pack2(w[2], w[3], r2, r3);
                const uint32_t a1 = E::pack2(w[0] - r0, w[1] - r1, x0, x1), a3 = E::pack2(w[2] - r2, w[3] - r3, x2, x3);
                l += ((r0 + x0) + (r1 + x1)) + ((r2 + x2) + (r3 + x3));
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t b0, b1, b2, b3;
                    pkv::ldsm_x4_t((stage + v_at) ^ (j << 5), b0, b1, b2, b3);
                    Mma::run(acc[2 * j], a0, a1, a2, a3, b0, b1);
                    Mma::run(acc[2 * j + 1], a0, a1, a2, a3, b2, b3);
                }
                // ---- the stage is used up: fill it
                __syncwarp();
                if (rem > 0) {
                    ld.issue(stage);
                    if (--rem > 0) rem -= ld.advance();
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                stage += C::kStage;
                if (stage == ring_end) stage = ring;
            }

            // ---- the unit's output, or a piece of it
            const bool whole = at.i == 0 && count == n;
            const int slot = at.i ? 0 : 1;           // i > 0: it began before this warp's part
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // a piece of a unit that goes on in the next warp lies in this
            // warp's ring, which is read to the end
            float *po = slot ? reinterpret_cast<float *>(rings + warp * C::kRing)
                             : heads_o + (size_t)warp * p.o.GC * D;
            if (slot && !whole) __syncwarp();
            if (g < gca) {
                const size_t row = (size_t)at.s * p.o.Hq + h0 + g;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const float o[2] = {(acc[j][0] + acc[j][2]) * inv, (acc[j][1] + acc[j][3]) * inv};
                    if (whole) pkv::wd_store_row<2>(p.o, row * D + 8 * j + 2 * t, o);
                    else pkv::wd_store_f32(po + g * D + 8 * j + 2 * t, o);
                }
                const float lse = mu + log2f(l);
                if (t == 0) {
                    if (!whole) join.lse[warp][slot][g] = lse;
                    else if (p.o.lse_out) p.o.lse_out[row] = lse;
                }
            }
            if (!whole && lane == 0) join.piece[warp][slot] = {at.tu, n, at.s, at.u};
            if (!pkv::wd_next_unit(p.list, list, at, z)) break;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    pkv::wd_join<kWarps, D>(p.o, share, join, heads_o, reinterpret_cast<const float *>(rings), C::kRing / 4);
}

template <typename T, int D, int LB, int N>
cudaError_t launch_list(const RowsParams &p, cudaStream_t stream) {
    // the attribute is per device and idempotent; set once for each
    static std::atomic<uint64_t> ready{0};
    constexpr int ring = kWarps * Cfg<D>::kRing, most = ring + kWarps * kHeads * D * 4;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(decode_rows_kernel<T, D, LB, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(decode_rows_kernel<T, D, LB, N>, dim3((unsigned)p.C), kThreads, ring + kWarps * p.o.GC * D * 4, stream, p);
}

template <typename T, int D, int LB>
cudaError_t launch(const RowsParams &p, cudaStream_t stream) {
    return p.list.S <= kFewSeqs ? launch_list<T, D, LB, kFewSeqs>(p, stream) : launch_list<T, D, LB, kMaxSeqs>(p, stream);
}

template <typename T>
cudaError_t launch_for(int D, const RowsParams &p, cudaStream_t stream) {
    const int lb = p.list.lb;
    auto *go = D == 128 ? (lb == 3 ? &launch<T, 128, 3> : lb == 4 ? &launch<T, 128, 4> : &launch<T, 128, 5>)
                        : (lb == 3 ? &launch<T, 64, 3> : lb == 4 ? &launch<T, 64, 4> : &launch<T, 64, 5>);
    return go(p, stream);
}

// workspace: [PKV_MAX_DECODE_CTAS] arrival counters (a fixed region, whatever
// the launch), then [C][2][GC][D] outputs and [C][2][GC] log2 denominators of
// units cut between CTAs
constexpr size_t kCounterBytes = PKV_MAX_DECODE_CTAS * sizeof(unsigned);

}  // namespace

namespace pkv {

size_t rows_workspace_bytes(int heads, int D) {
    int C = 0;
    if (device_sm_count(&C) != PKV_OK) return 0;
    const int GC = heads < kHeads ? heads : kHeads;
    return kCounterBytes + (size_t)C * GC * (2 * D + 2) * sizeof(float);
}

pkv_status decode_rows(const pkv_cache_desc *cache, const void *q, int S, int Hq, const void *k_pool,
                       const void *v_pool, const int32_t *tables, int M, const int32_t *lens, float scale,
                       void *out, int out_dtype, void *ws, cudaStream_t stream) {
    const int Hk = cache->num_kv_heads, D = cache->head_dim, B = cache->block_size;
    const int G = Hq / Hk, GC = G < kHeads ? G : kHeads, NC = (G + GC - 1) / GC;
    const int64_t tokens = (int64_t)M * B, seqs = S < kMaxSeqs ? S : kMaxSeqs;
    // the list's places fit 32 bits; products with the CTAs are taken in 64
    if (tokens > INT32_MAX / 2 || seqs * Hk * NC * ((tokens + kSub - 1) / kSub + kUnitCost) >= (int64_t)INT32_MAX)
        return set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
    RowsParams p = {};
    pkv_status st = device_error_word(&p.list.err);
    if (st != PKV_OK) return st;
    if ((st = device_sm_count(&p.C)) != PKV_OK) return st;
    p.list.M = M;
    p.list.lb = B == 8 ? 3 : B == 16 ? 4 : 5;
    p.list.U = Hk * NC;
    p.o.out_dtype = out_dtype;
    p.o.Hq = Hq;
    p.o.G = G;
    p.o.NC = NC;
    p.o.GC = GC;
    p.o.cnt = static_cast<unsigned *>(ws);
    p.o.ws_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kCounterBytes);
    p.o.ws_lse = p.o.ws_o + (size_t)p.C * 2 * GC * D;
    p.k = static_cast<const uint8_t *>(k_pool);
    p.v = static_cast<const uint8_t *>(v_pool);
    p.Hk = Hk;
    p.NB = cache->num_blocks;
    p.chunk_bytes = (uint32_t)(B * D * 2);
    p.scale_log2 = scale * 1.4426950408889634f;
    const int oes = out_dtype == PKV_F32 ? 4 : 2;
    for (int s0 = 0; s0 < S; s0 += kMaxSeqs) {
        p.list.S = S - s0 < kMaxSeqs ? S - s0 : kMaxSeqs;
        p.list.tables = tables + (size_t)s0 * M;
        p.list.lens = lens + s0;
        p.q = static_cast<const uint16_t *>(q) + (size_t)s0 * Hq * D;
        p.o.out = static_cast<uint8_t *>(out) + (size_t)s0 * Hq * D * oes;
        const cudaError_t e = cache->dtype == PKV_F16 ? launch_for<__half>(D, p, stream)
                                                      : launch_for<__nv_bfloat16>(D, p, stream);
        if (e != cudaSuccess)
            return set_last_error(PKV_ERR_CUDA, "decode_rows launch: %s", cudaGetErrorString(e));
    }
    return PKV_OK;
}

}  // namespace pkv

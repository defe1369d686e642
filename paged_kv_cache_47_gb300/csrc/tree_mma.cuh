// Tree attention over 16-bit caches on the 5th-generation tensor cores.
//
// Products. A unit's rows (a q head of a drafted token each) are the M of
// tcgen05.mma, 128 at a time: S[128 rows][64 tokens] = Q K^T, Q and K from
// shared memory as they were copied, and O[128 rows][D] += P V, P from tensor
// memory, V from shared memory read along its tokens. A thread owns a row: the
// softmax's maximum and sum need no other thread. K and V are read once for
// all rows of a kv head, so up to 128 rows (or 256, in two row tiles that share
// each K and V) cost the memory what one row does.
//
// P enters as two parts, hi (fp16: the nearest; bf16: the upper half of the fp32
// value, which takes fewer steps) and lo = the nearest to the rest, so weights keep
// 16 (bf16) or 22 (fp16) bits: with hi alone a 16-bit
// output's error against 64 bits is half as large again, as weights are then
// rounded as outputs are. The parts lie where their scores lay: 16 scores become
// 8 words of hi and 8 of lo.
//
// Roles. A CTA holds two groups, each four warps of softmax and one that issues
// its products, with 256 columns of tensor memory: two S of 64 columns (the next
// tile's scores are made while this one's become weights) and O. Units of one row
// tile: each group is a worker with its own share of the list, its own warps that
// copy K, V and q through cp.async (whose 16-byte pieces serve blocks of 8 to 32
// tokens), and its own rings; nothing is shared but the tensor cores. Units of
// two row tiles: one worker, each tile of K and V for both groups.
//
// The softmax's reference exponent moves only when a score passes what the type
// holds; only then are the outputs rescaled, by one read and write of them.
//
// What a row does not see has weight zero; as zero times infinity is not zero,
// tiles with drafted tokens are looked through for V that are not finite, and
// such a tile's second product is done on the CUDA cores, over what has weight.
//
// What bounds it. Up to 128 rows: a group's softmax, 1900 cycles a tile of 64 tokens
// of 128 elements, and the memory, which gives a worker a tile in 2860, with 5 to 8
// us of list and first copies before and 8 of pieces and joins behind. 64 requests
// of 512 to 4096 tokens, 16 drafted, 32 q and 8 kv heads, bf16: 115 to 121 us, 5.2
// to 5.4 TB/s (0.76 to 0.80 of a copy); 128 of 128 to 2048, one q head a kv head,
// fp16: 503 to 562 us, 5.1 to 5.7 TB/s. 256 rows: softmax (1700), products (1800) and
// shared memory (1500) near one another, 2500 measured, and the power limit: 8
// contexts of 32768 to 131072 tokens, up to 26 drafted, 8 q heads a kv head, bf16:
// 655 to 732 us, 0.61 to 0.69 PFLOP/s, 0.92 to 1.03 with the weights' low parts.
//
// Barriers. Each is waited for phase after phase by the same role, and no phase
// can complete before the one waited for has been seen: a parity names it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "tree_list.cuh"

namespace {

using pkv::launch_chained;
using pkv::TreeParams;
using pkv::TreePlace;
using pkv::TreeShare;

constexpr int kTile = pkv::kTreeMmaTile, kRowTile = pkv::kTreeMmaRows;
constexpr int kGroups = 2, kGroupThreads = 128, kGroupWarps = 4;
constexpr int kSoftmaxThreads = kGroups * kGroupThreads;
constexpr int kThreads = kSoftmaxThreads + 8 * 32;     // and K, issue, V and q: two warps each
constexpr int kMetas = 16;                     // more than the tiles between the first copy and the softmax
constexpr uint32_t kColumns = 512;             // tensor memory: each group two S, then O
constexpr float kNone = 2e-38f;                // reference exponent before a row's first finite score

// Exponent that a reference gives the top score, and the largest that needs no new one.
template <typename T> constexpr float kTop = 0.f;
template <> constexpr float kTop<__half> = 10.f;
template <typename T> constexpr float kRoom = 8.f;
template <> constexpr float kRoom<__half> = 15.f;

// A tile as its groups see it.
struct Tile {
    int o, n, L, g;          // first q row, drafted tokens, context, kv head
    int r0, nr;              // the unit's first row and rows
    int t0;                  // first token
    int left;                // tiles of the segment after it
    int seg;                 // the worker's segments before it
    int whole, slot;         // whole unit, or slot of the piece
    int pad;
};

// Rows of a unit at most: 64 and 128 take one row tile, 256 two.
template <int D, int ROWS>
struct Cfg {
    static constexpr bool kTwo = ROWS > kRowTile;            // two row tiles: one worker for both groups
    static constexpr int kWorkers = kTwo ? 1 : 2;
    static constexpr int kCopyWarps = kTwo ? 2 : 1;          // of K, and of V, for a worker
    static constexpr int kPlanes = D / 64;                   // of 64 elements, 128 bytes a row
    static constexpr int kPlane = kTile * 128;
    static constexpr int kSlot = kPlanes * kPlane;           // K or V of a tile
    static constexpr int kQPlane = (kTwo ? kRowTile : ROWS) * 128;
    static constexpr int kQTile = kPlanes * kQPlane;         // q of a row tile
    static constexpr int kQ = (kTwo ? 2 : 1) * kQTile;       // q of a unit
    // Units of up to 64 rows: group 1 has them in rows 64..127 of its products, so
    // that the groups' softmax warps run on schedulers of their own (a warp reaches
    // a quarter of tensor memory's lanes). The other rows hold anything.
    static constexpr int kShift = ROWS == 64 ? 64 : 0;
    // rings of K and of V: with q 224 KB (D 64: 208, 160 and 192)
    static constexpr int kK = kTwo ? (D == 128 ? 4 : 10) : D == 128 ? (ROWS == 64 ? 3 : 2) : ROWS == 64 ? 6 : 4;
    static constexpr int kV = kTwo ? (D == 128 ? 6 : 10) : D == 128 ? 3 : ROWS == 64 ? 6 : 4;
    static constexpr int kWorker = kQ + (kK + kV) * kSlot;   // bytes of a worker
    static constexpr int kBytes = kWorkers * kWorker;
    static_assert(kBytes <= 224 * 1024 && kK + 4 < kMetas, "");
};

constexpr int kMostSlots = 10;
struct Rings {
    uint64_t full_k[kMostSlots], free_k[kMostSlots], full_v[kMostSlots], free_v[kMostSlots], free_q;
    Tile tiles[kMetas];
};
struct Control {
    Rings rings[2];
    uint64_t s[kGroups][2], p[kGroups][2], o[kGroups][2], meet[kGroups];
    int odd[kGroups][2];             // tile (+ 1) last found to have V that are not finite, by turns
    int skip[kGroups][2];            // by S: the weights are used up already
    int4 which[kGroups][2];          // by S: the worker's tile (-1: no more), segment, first token's place
                                     // among the drafted ones, tiles of the segment after it
    pkv::TreeCut cuts[4];            // the workers' pieces of cut units
    int last[kGroups];               // 1: the group counted its first unit's last piece
    uint32_t tmem;
};

template <typename T>
constexpr uint32_t idesc(int N, bool b_mn, bool negate) {
    constexpr uint32_t f = sizeof(T) == 2 && !std::is_same<T, __half>::value ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((negate ? 1u : 0u) << 13) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(accumulate)
        : "memory");
}
// A from tensor memory: lane = row, 8 columns = 16 elements along K.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"(accumulate)
        : "memory");
}

#define PKV_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define PKV_M8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
#define PKV_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of this thread's lane; valid after tm_wait on them.
__device__ __forceinline__ void tm_load(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
        "%23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : PKV_R8(r, 0), PKV_R8(r, 8), PKV_R8(r, 16), PKV_R8(r, 24)
        : "r"(at));
}
__device__ __forceinline__ void tm_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PKV_M8(r, 0), PKV_M8(r, 8), PKV_M8(r, 16), PKV_M8(r, 24) : : "memory");
}
__device__ __forceinline__ uint32_t tm_load1(uint32_t at) {
    uint32_t x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x) : : "memory");
    return x;
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::PKV_W8(r, 0),
        PKV_W8(r, 8), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float f32(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ bool warp_wait(const TreeParams &p, uint64_t &bar, uint32_t parity) {
    return __all_sync(~0u, pkv::mbar_wait(pkv::smem_u32(&bar), parity & 1, p.b.err, p.wait_ns));
}
// Whether the phase has completed, the same for the whole warp.
__device__ __forceinline__ bool ready(uint64_t &bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(pkv::smem_u32(&bar)), "r"(parity & 1)
        : "memory");
    return __all_sync(~0u, ok != 0);
}

// A place in a ring of N slots: the slot, and how often it was used.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) slot = 0, turn ^= 1;
    }
};

// A segment: the tiles of one unit that lie in the worker's share.
struct Segment {
    int n, i0, g, r0, nr;
    bool whole;
};
__device__ __forceinline__ Segment segment(const TreeParams &p, const TreePlace &at, int left) {
    Segment x;
    x.n = min(at.tiles - at.i, left);
    x.i0 = at.i;
    const int chunks = at.units / p.Hk;
    x.g = at.u / chunks;
    x.r0 = (at.u - x.g * chunks) * p.RC;
    x.nr = min(p.RC, at.q.n * p.G - x.r0);
    x.whole = x.n == at.tiles;
    return x;
}

// Copies of K, or of V, into a ring of their own; a tile's tokens shared out to the warps.
template <int D, int ROWS, int LB, bool V>
struct Producer {
    using C = Cfg<D, ROWS>;
    static constexpr int kRows = kTile / C::kCopyWarps;
    static constexpr int E = kRows >> LB;                    // blocks of a warp's tokens of a tile
    static constexpr int kAhead = 32 / E;                    // tiles whose entries a warp holds
    static constexpr int kPieces = kRows * C::kPlanes * 8 / 32;    // 16-byte pieces a lane copies of a tile
    static constexpr int kRing = V ? C::kV : C::kK;
    const TreeParams &p;
    Rings &rings;
    pkv::TreeCut *cuts;                                      // the worker's pieces
    uint32_t base;                                           // the ring
    int lane, pw;
    int32_t window, next_window;
    int from;                                                // tile that the window begins at

    __device__ __forceinline__ int32_t entries(int s, int tile) const {
        const int e = (tile + lane / E) * (kTile >> LB) + pw * E + lane % E;
        return e < p.b.M ? __ldg(p.tables + (int64_t)s * p.b.M + e) : -1;
    }

    // Lane's destination of its piece j of the warp's rows, of which piece 0's is
    // at lane_at: rows are 128 bytes and their pieces exclusive-ored by the row
    // modulo 8, so later pieces differ by a constant and a constant's bits.
    static __device__ __forceinline__ uint32_t lane_at(int pw, int lane) {
        if (D == 128) return pw * kRows * 128 + (lane >> 3 & 1) * C::kPlane + (lane >> 4) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
        return pw * kRows * 128 + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
    }
    static __device__ __forceinline__ uint32_t piece(uint32_t at, int j) {
        return D == 128 ? (at ^ ((2 * j & 6) << 4)) + j * 256 : (at ^ ((4 * j & 4) << 4)) + j * 512;
    }

    // The warp's rows of a tile, left of them in the context. What is past it, or
    // in a block whose id lies outside the pool, becomes zeros: all that a product
    // reads (16 tokens at a time) of V, as zero weights want them.
    __device__ __forceinline__ void copy(uint32_t slot, int32_t ids, int at, int g, int left) const {
        const uint8_t *src = static_cast<const uint8_t *>(V ? p.v : p.k) + lane * 16;
        uint32_t to = slot + lane_at(pw, lane);
        left -= pw * kRows;
        const int rows = min(kRows, V ? (left + 15) & ~15 : left), row = lane / (C::kPlanes * 8);
        constexpr int PB = kPieces / E, PR = 32 / (C::kPlanes * 8);    // pieces of a block, rows of a piece
#pragma unroll 1
        for (int k = 0; k << LB < rows; ++k) {
            const int id = __shfl_sync(~0u, ids, at + k);
            const bool ok = (unsigned)id < (unsigned)p.NB;
            if (!ok && !V && lane == 0) atomicOr(p.b.err, PKV_DEVERR_BLOCK_ID);
            const int here = ok ? left - (k << LB) - row : 0;          // rows from this lane's first on
            const uint8_t *block = src + (((size_t)(ok ? id : 0) * p.Hk + g) << LB) * (2 * D);
#pragma unroll
            for (int j = 0; j < PB; ++j) pkv::cp_async_16(piece(to, j), block + j * 512, j * PR < here);
            to += 128 << LB;
        }
    }

    __device__ __forceinline__ void run(const TreeShare &share, TreePlace at) {
        const int count = share.Z - share.A;
        const bool first_thread = pw == 0 && lane == 0;
        int32_t first = count > 0 ? entries(at.s, at.i) : 0;
        Ring<kRing> r;
        for (int t = 0, seg = 0; t < count; ++seg) {
            const Segment x = segment(p, at, count - t);
            if (!V && first_thread && !x.whole) {
                pkv::TreeCut &c = cuts[x.i0 ? 0 : 1];
                c = pkv::tree_cut(share, share.A + t - x.i0, at.tiles, at.q.o, x.g, x.r0, x.nr);
                // pieces of units that began elsewhere are counted as soon as they are
                // written, by each group that has rows of them: the others at the end
                if (!x.i0) c.due = C::kTwo && x.nr > kRowTile ? 2 : 1;
            }
            window = first;
            from = x.i0;
            next_window = x.n > kAhead ? entries(at.s, x.i0 + kAhead) : 0;
            const pkv::TreeSeq q = at.q;
            const int s = at.s;
            if (t + x.n < count) {                           // the next unit's first entries, ahead of time
                at.next_unit<kTile>(p);
                first = entries(at.s, 0);
            }
            for (int k = 0; k < x.n; ++k, ++t) {
                const int i = x.i0 + k;
                if (i == from + kAhead) {
                    window = next_window;
                    from = i;
                    next_window = x.n - k > kAhead ? entries(s, i + kAhead) : 0;
                }
                if (!warp_wait(p, (V ? rings.free_v : rings.free_k)[r.slot], r.turn ^ 1)) return;
                uint64_t &full = (V ? rings.full_v : rings.full_k)[r.slot];
                if (!V && first_thread) {
                    rings.tiles[t % kMetas] = {q.o, q.n, q.L, x.g, x.r0, x.nr, i * kTile, x.n - 1 - k, seg, x.whole, x.i0 ? 0 : 1, 0};
                    pkv::mbar_arrive(pkv::smem_u32(&full));
                }
                copy(base + r.slot * C::kSlot, window, (i - from) * E, x.g, q.L - i * kTile);
                if (V || !p.drop_arrival || share.me || !first_thread || t)
                    pkv::cp_async_arrive_noinc(pkv::smem_u32(&full));
                r.next();
            }
        }
    }
};

// A warp copies a worker's q rows, each unit's with its first tile here, and
// counts in every K tile's barrier once its copies so far have landed: a tile
// that is there has its q there. (Rows past the unit's hold anything: no other
// row depends on them.)
template <int D, int ROWS>
__device__ __forceinline__ void copy_q(const TreeParams &p, Rings &rings, uint32_t to, const TreeShare &share, TreePlace at) {
    using C = Cfg<D, ROWS>;
    constexpr int R = C::kPlanes * 8;
    const int count = share.Z - share.A, lane = threadIdx.x & 31;
    const uint8_t *q = static_cast<const uint8_t *>(p.q);
    Ring<C::kK> r;
    for (int t = 0, seg = 0; t < count; ++seg) {
        const Segment x = segment(p, at, count - t);
        const int o = at.q.o;
        if (t + x.n < count) at.next_unit<kTile>(p);
        for (int k = 0; k < x.n; ++k, ++t) {
            if (k == 0) {
                if (!warp_wait(p, rings.free_q, seg + 1)) return;
#pragma unroll 4
                for (int j = lane; j < x.nr * R; j += 32) {
                    const int row = j / R, w = j % R, y = row % kRowTile;
                    pkv::cp_async_16(to + (row / kRowTile) * C::kQTile + (w >> 3) * C::kQPlane + y * 128 + (((w & 7) ^ (y & 7)) << 4),
                                     q + pkv::tree_row(p, o, x.g, x.r0 + row) * (2 * D) + w * 16, true);
                }
            }
            if (!warp_wait(p, rings.free_k[r.slot], r.turn ^ 1)) return;
            pkv::cp_async_arrive_noinc(pkv::smem_u32(&rings.full_k[r.slot]));
            r.next();
        }
    }
}

// ---------------------------------------------------------------- the products
// One warp issues a group's products, each as soon as it may: S of a tile at most
// two ahead of the weights (its columns are those weights'), P V once the weights
// are there. Waits for data, for the softmax and for products go by looking, so
// that none holds up another.
template <typename T, int D, int ROWS>
struct Issuer {
    using C = Cfg<D, ROWS>;
    static constexpr uint32_t kPv = idesc<T>(D, true, false);
    const TreeParams &p;
    Control &ctl;
    Rings &rings;
    uint32_t base, tmem;                     // the worker's shared memory; tensor memory of the group, lane 0
    int w, count;

    __device__ __forceinline__ void issue_s(int slot, int buf, uint32_t desc) const {
        const uint64_t dq = pkv::sdesc_sw128(base + (C::kTwo ? w * C::kQTile : 0) - w * C::kShift * 128, 16, 1024);
        const uint64_t dk = pkv::sdesc_sw128(base + C::kQ + slot * C::kSlot, 16, 1024);
        pkv::fence_proxy_async_smem();
        pkv::tc_fence_after();
#pragma unroll C::kTwo ? 8 : 1
        for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + kTile * buf, dq + (k / 4) * (C::kQPlane >> 4) + (k % 4) * 2, dk + (k / 4) * (C::kPlane >> 4) + (k % 4) * 2, desc, k);
        pkv::tc_commit(pkv::smem_u32(&ctl.s[w][buf]));
        pkv::tc_commit(pkv::smem_u32(&rings.free_k[slot]));
    }

    __device__ __forceinline__ void issue_pv(int ntok, int slot, int buf, bool accumulate) const {
        // K step k: 16 tokens, 16 rows of 128 bytes; planes of 64 elements along N
        const uint64_t dv = pkv::sdesc_sw128(base + C::kQ + (C::kK + slot) * C::kSlot, C::kPlane, 1024);
        pkv::fence_proxy_async_smem();
        pkv::tc_fence_after();
#pragma unroll C::kTwo ? 4 : 1
        for (int k = 0; k < kTile / 16; ++k)
            if (16 * k < ntok) {
                const uint32_t a = tmem + kTile * buf + 16 * k;
                mma_ts(tmem + 2 * kTile, a, dv + 128 * k, kPv, accumulate || k);
                mma_ts(tmem + 2 * kTile, a + 8, dv + 128 * k, kPv, 1);
            }
        pkv::tc_commit(pkv::smem_u32(&ctl.o[w][buf]));
        pkv::tc_commit(pkv::smem_u32(&rings.free_v[slot]));
    }

    __device__ __forceinline__ void run() const {
        const uint32_t desc = idesc<T>(kTile, false, p.scale_log2 < 0.f);
        Ring<C::kK> k;
        Ring<C::kV> v;
        int tk = 0, tv = 0;                  // the worker's tiles whose S was begun, whose P V was
        int us = 0, up = 0, od = 0;          // the group's products: S begun; P V begun; P V done
        int seg_p = -1;
        uint64_t since = 0;                  // no progress since (0: some)
        while (tk < count || tv < count) {
            bool moved = false;
            while (od < up && ready(ctl.o[w][od & 1], od >> 1)) ++od;
            // ---- S of the next tile: its columns are those of the last but one (a group
            // without rows runs no further ahead than the tiles' records last)
            if (tk < count && us < od + 2 && tk < tv + kMetas - C::kK && ready(rings.full_k[k.slot], k.turn)) {
                const Tile &m = rings.tiles[tk % kMetas];
                const bool none = C::kTwo && m.nr <= w * kRowTile;   // the unit has no rows for this group
                if (pkv::elect_one()) {
                    if (none) {
                        pkv::mbar_arrive(pkv::smem_u32(&rings.free_k[k.slot]));
                        if (m.left == 0) pkv::mbar_arrive(pkv::smem_u32(&rings.free_q));
                    } else {
                        issue_s(k.slot, us & 1, desc);
                        if (m.left == 0) pkv::tc_commit(pkv::smem_u32(&rings.free_q));
                        ctl.which[w][us & 1] = make_int4(tk, m.seg, m.t0 - (m.L - m.n), m.left);
                        pkv::mbar_arrive(pkv::smem_u32(&ctl.s[w][us & 1]));
                    }
                }
                __syncwarp();
                us += !none;
                ++tk;
                k.next();
                moved = true;
            }
            // ---- P V of the next product
            if (tv < tk) {
                const Tile &m = rings.tiles[tv % kMetas];
                const bool none = C::kTwo && m.nr <= w * kRowTile;
                if ((none || ready(ctl.p[w][up & 1], up >> 1)) && ready(rings.full_v[v.slot], v.turn)) {
                    const bool skip = !none && *reinterpret_cast<volatile int *>(&ctl.skip[w][up & 1]) != 0;
                    if (pkv::elect_one()) {
                        if (none || skip) {
                            if (skip) pkv::mbar_arrive(pkv::smem_u32(&ctl.o[w][up & 1]));
                            pkv::mbar_arrive(pkv::smem_u32(&rings.free_v[v.slot]));
                        } else {
                            issue_pv(m.L - m.t0, v.slot, up & 1, m.seg == seg_p);
                        }
                    }
                    __syncwarp();
                    seg_p = m.seg;
                    up += !none;
                    ++tv;
                    v.next();
                    moved = true;
                }
            }
            if (moved) {
                since = 0;
            } else {
                const uint64_t now = pkv::globaltimer_ns();
                if (since == 0) since = now;
                else if (__any_sync(~0u, now - since > p.wait_ns)) {
                    if (pkv::elect_one()) atomicOr(p.b.err, PKV_DEVERR_TIMEOUT);
                    break;
                }
            }
        }
        // nothing more comes: the softmax leaves
        if (tv >= count) {
            if (pkv::elect_one()) {
                ctl.which[w][us & 1].x = -1;
                pkv::mbar_arrive(pkv::smem_u32(&ctl.s[w][us & 1]));
                pkv::mbar_arrive(pkv::smem_u32(&ctl.s[w][us & 1]));
            }
            __syncwarp();
        }
        while (od < up && warp_wait(p, ctl.o[w][od & 1], od >> 1)) ++od;      // its products are done
    }
};

// ---------------------------------------------------------------- the softmax
// Four warps, a thread a row.
template <typename T, int D, int ROWS>
struct Softmax {
    using C = Cfg<D, ROWS>;
    using El = pkv::Elem<T>;
    const TreeParams &p;
    Control &ctl;
    Rings &rings;
    uint32_t base, tm;                                       // the worker's shared memory; tensor memory of the group, this lane quarter
    int w, thread, row;                                      // group, thread of it, row of the unit (or none)
    float scale, mu, room, l;
    bool have_o;
    uint32_t mask[2];                                        // the row's first mask words

    __device__ __forceinline__ uint32_t O() const { return tm + 2 * kTile; }
    // The warp has done what the barrier counts; what it did to tensor memory is ordered.
    __device__ __forceinline__ void arrive(uint64_t &bar) const {
        pkv::tc_fence_before();
        __syncwarp();
        if ((thread & 31) == 0) pkv::mbar_arrive(pkv::smem_u32(&bar));
    }
    __device__ __forceinline__ bool wait(uint64_t &bar, uint32_t parity) const {
        const bool ok = warp_wait(p, bar, parity);
        pkv::tc_fence_after();
        return ok;
    }

    // Outputs of product u are in.
    __device__ __forceinline__ bool wait_o(int u) const { return wait(ctl.o[w][u & 1], u >> 1); }

    __device__ __forceinline__ const uint32_t *mask_row(const Tile &m, int i) const {
        return reinterpret_cast<const uint32_t *>(p.masks + (size_t)(m.o + i) * p.W);
    }
    // Bits of the 32 tokens from drafted token d0 on (before: d0 < 0) that token i sees.
    __device__ __forceinline__ uint32_t word(const Tile &m, int i, int k) const {
        if (32 * k >= m.n) return 0;
        uint32_t x;
        if (p.masks) x = k == 0 ? mask[0] : k == 1 ? mask[1] : __ldg(mask_row(m, i) + k);
        else x = i >= 32 * k + 31 ? ~0u : i < 32 * k ? 0u : (2u << (i - 32 * k)) - 1;
        return m.n - 32 * k >= 32 ? x : x & ((1u << (m.n - 32 * k)) - 1);
    }
    __device__ __forceinline__ uint32_t sees(const Tile &m, int i, int d0) const {
        if (d0 <= -32) return ~0u;
        if (d0 < 0) return (word(m, i, 0) << -d0) | ((1u << -d0) - 1);
        return __funnelshift_r(word(m, i, d0 >> 5), word(m, i, (d0 >> 5) + 1), d0 & 31);
    }

    __device__ __forceinline__ void scale_o(float f) const {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t x[16];
            pkv::tmem_ld16(O() + c, x);
            pkv::tmem_ld_wait(x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(f32(x[i]) * f);
            tm_store16(O() + c, x);
        }
    }

    // Whether any V of the tile's drafted tokens is not finite (told through *odd).
    __device__ __forceinline__ void look_through(uint32_t slot, const Tile &m, int tag, volatile int *odd) const {
        const int a = max(0, m.L - m.n - m.t0), z = min(kTile, m.L - m.t0);
        constexpr int R = C::kPlanes * 8;
        constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
        constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
        uint32_t any = 0;
        for (int x = a * R + thread; x < z * R; x += kGroupThreads) {
            // (the order of a row's pieces says nothing here)
            uint32_t y[4];
            pkv::lds_u32x4(slot + (x % R >> 3) * C::kPlane + (x / R) * 128 + (x % 8 << 4), y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= ((y[i] & kExp) + kOne) & 0x80008000u;     // the exponent is all ones
        }
        if (any) *odd = tag;
    }

    // O += P V of a tile on the CUDA cores, over what has weight.
    __device__ __forceinline__ void slow_pv(uint32_t P, uint32_t slot, int ntok) const {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            if (have_o) {
                pkv::tmem_ld16(O() + c, o);
                pkv::tmem_ld_wait(o);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0;
            }
#pragma unroll 1
            for (int t = 0; t < ntok; ++t) {                 // weight of token t: hi and lo words of a pair
                const uint32_t pair = P + (t & ~15) + (t & 15) / 2;
                const float2 hi = El::unpack2(tm_load1(pair)), lo = El::unpack2(tm_load1(pair + 8));
                const float pt = t & 1 ? hi.y + lo.y : hi.x + lo.x;
                if (pt != 0.f) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t y[4];
                        pkv::lds_u32x4(slot + (c >> 6) * C::kPlane + t * 128 + ((((c & 63) / 8 + k) ^ (t & 7)) << 4), y[0], y[1], y[2], y[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = El::unpack2(y[e]);
                            o[8 * k + 2 * e] = __float_as_uint(fmaf(pt, v.x, f32(o[8 * k + 2 * e])));
                            o[8 * k + 2 * e + 1] = __float_as_uint(fmaf(pt, v.y, f32(o[8 * k + 2 * e + 1])));
                        }
                    }
                }
                __syncwarp();
            }
            tm_store16(O() + c, o);
        }
        tm_store_wait();
    }

    // Scores at `at` to weights: maximum, reference, and the parts in the scores'
    // place. d0: the first token's place among the drafted ones; u: the product.
    template <bool MASKED>
    __device__ __forceinline__ bool weights(uint32_t at, const Tile &m, int i, int d0, int u) {
        uint32_t bits[2];
        bits[0] = MASKED ? sees(m, i, d0) : ~0u;
        bits[1] = MASKED ? sees(m, i, d0 + 32) : ~0u;
        float a4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // (rolled: longer code is fetched more slowly than it runs)
#pragma unroll 1
        for (int c = 0; c < kTile; c += 32) {
            uint32_t x[32];
            tm_load(at + c, x);
            const uint32_t seen = c ? bits[1] : bits[0];
            tm_wait(x);
#pragma unroll
            for (int j = 0; j < 32; j += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = j + 2 * e;
                    a4[e] = fmaxf(fmaxf(a4[e], MASKED && !(seen >> k & 1) ? -INFINITY : f32(x[k])),
                                  MASKED && !(seen >> (k + 1) & 1) ? -INFINITY : f32(x[k + 1]));
                }
        }
        const float top = fmaxf(fmaxf(a4[0], a4[1]), fmaxf(a4[2], a4[3])) * scale;    // (scale is not negative; NaN stays out)
        if (__any_sync(~0u, top > room)) {
            const bool none = mu == kNone;
            const float nm = top > room ? top - kTop<T> : mu;
            const float f = none || nm == mu ? 1.f : pkv::ex2_approx(mu - nm);
            if (have_o) {                                    // the last product's outputs are in
                if (!wait_o(u - 1)) return false;
                scale_o(f);
            }
            l *= f;
            mu = nm;
            if (mu != kNone) room = mu + kRoom<T>;
        }
        const pkv::Pair s2 = pkv::pair_of(scale, scale), m2 = pkv::pair_of(-mu, -mu), minus = pkv::pair_of(-1.f, -1.f);
        pkv::Pair sum = 0;
#pragma unroll 1
        for (int c = 0; c < kTile; c += 16) {
            uint32_t x[16], y[16];
            pkv::tmem_ld16(at + c, x);
            const uint32_t seen = (c < 32 ? bits[0] : bits[1]) >> (c & 16);
            pkv::tmem_ld_wait(x);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float a, b, ra, rb, la, lb;
                pkv::unpair(pkv::fma2(pkv::pair_of(f32(x[j]), f32(x[j + 1])), s2, m2), a, b);
                a = pkv::ex2_approx(a);
                b = pkv::ex2_approx(b);
                if (MASKED) {
                    a = seen >> j & 1 ? a : 0.f;
                    b = seen >> (j + 1) & 1 ? b : 0.f;
                }
                const pkv::Pair ab = pkv::pair_of(a, b);
                sum = pkv::add2(sum, ab);
                if constexpr (std::is_same<T, __half>::value) {
                    y[j / 2] = El::pack2(a, b, ra, rb);
                } else {                                     // (the upper halves, not rounded: fewer steps, and the rest in lo)
                    y[j / 2] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                    ra = f32(__float_as_uint(a) & 0xffff0000u);
                    rb = f32(__float_as_uint(b) & 0xffff0000u);
                }
                pkv::unpair(pkv::fma2(pkv::pair_of(ra, rb), minus, ab), la, lb);
                y[8 + j / 2] = El::pack2(la, lb, ra, rb);
            }
            tm_store16(at + c, y);
        }
        float a, b;
        pkv::unpair(sum, a, b);
        l += a + b;
        tm_store_wait();
        return true;
    }

    // The rows' outputs, or a piece.
    __device__ __forceinline__ void finish(const Tile &m, int me, int r0, int nr) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool mine = row < nr;                          // (of a live warp: row >= 0)
        const size_t at = m.whole ? pkv::tree_row(p, m.o, m.g, m.r0 + r0 + (mine ? row : 0))
                                  : (size_t)(2 * me + m.slot) * p.RC + r0 + row;
        void *to = m.whole ? p.out : p.ws_o;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t x[32];
            float y[32];
            tm_load(O() + c, x);
            tm_wait(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = inv == 0.f ? 0.f : f32(x[i]) * inv;
            if (mine) pkv::tree_store<32>(to, m.whole ? p.out_dtype : PKV_F32, at * D + c, y);
            __syncwarp();
        }
        if (mine) {
            const float lse = l == 0.f ? -INFINITY : mu + log2f(l);
            if (!m.whole) p.ws_lse[at] = lse;
            else if (p.lse_out) p.lse_out[at] = lse;
        }
        __syncwarp();
    }

    __device__ __forceinline__ bool run(int me) {
        int seg = -1, i = 0, r0 = 0, nr = 0;
        uint32_t met = 0;                                    // uses of that barrier
        for (int u = 0;; ++u) {
            const int buf = u & 1;
            if (!wait(ctl.s[w][buf], u >> 1)) return false;
            const int4 it = ctl.which[w][buf];
            const int t = it.x, d0 = it.z;
            if (t < 0) return true;
            const Tile &m = rings.tiles[t % kMetas];         // stays until the weights are there
            if (it.y != seg) {
                seg = it.y;
                mu = kNone;
                room = -INFINITY;
                l = 0.f;
                have_o = false;
                r0 = C::kTwo ? w * kRowTile : 0;
                nr = min(kRowTile, m.nr - r0);
                i = (m.r0 + r0 + max(0, min(row, nr - 1))) / p.G;
                if (p.masks) {                               // asked for now, needed at the unit's end
                    const uint2 two = __ldg(reinterpret_cast<const uint2 *>(mask_row(m, i)));
                    mask[0] = two.x;
                    mask[1] = two.y;
                }
            }
            const bool live = row >= 0 && (row & ~31) < nr;           // warps without rows only keep the meetings
            const uint32_t at = tm + kTile * buf;
            bool odd = false;
            if (d0 + kTile > 0) {                            // drafted tokens among them, or the context's end
                if (live && !weights<true>(at, m, i, d0, u)) return false;
                const uint32_t slot = base + C::kQ + (C::kK + t % C::kV) * C::kSlot;
                if (!wait(rings.full_v[t % C::kV], t / C::kV)) return false;
                volatile int *flag = &ctl.odd[w][met & 1];   // (written again two meetings later)
                look_through(slot, m, t + 1, flag);
                arrive(ctl.meet[w]);
                if (!wait(ctl.meet[w], met++)) return false;
                odd = *flag == t + 1;
                if (odd) {
                    if (have_o && !wait_o(u - 1)) return false;
                    if (live) slow_pv(at, slot, min(kTile, m.L - m.t0));
                }
            } else {
                if (live && !weights<false>(at, m, i, d0, u)) return false;
            }
            if (thread == 0) ctl.skip[w][buf] = odd;
            Tile end;
            if (it.w == 0) end = m;
            arrive(ctl.p[w][buf]);
            have_o = true;
            if (it.w == 0) {
                if (!wait_o(u)) return false;
                if (live) finish(end, me, r0, nr);
                if (!end.whole && end.slot == 0) {
                    // a piece of a unit that began elsewhere, which that worker will join:
                    // this one is hardly ever the last
                    __threadfence();
                    arrive(ctl.meet[w]);
                    if (!wait(ctl.meet[w], met++)) return false;
                    if (thread == 0) {
                        pkv::TreeCut &c = ctl.cuts[C::kTwo ? 0 : 2 * w];
                        if (c.count(p.count, 1, C::kTwo && end.nr > kRowTile ? 2 : 1)) ctl.last[w] = 1;
                    }
                }
            }
        }
    }
};

template <typename T, int D, int ROWS, int LB>
__global__ void __launch_bounds__(kThreads, 1) tree_mma_kernel(const __grid_constant__ TreeParams p) {
    using C = Cfg<D, ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Control ctl;
    const int tid = threadIdx.x, warp = tid >> 5;
    pkv::grid_dependents_launch();
    if (warp == 0) pkv::tmem_alloc(pkv::smem_u32(&ctl.tmem), kColumns);
    if (tid == 32) {
        auto init = [](uint64_t &bar, int n) { pkv::mbar_init(pkv::smem_u32(&bar), n); };
        constexpr int users = C::kTwo ? 2 : 1;
        for (int i = 0; i < C::kWorkers; ++i) {
            for (int b = 0; b < kMostSlots; ++b) {
                init(ctl.rings[i].full_k[b], 32 * (C::kCopyWarps + 1) + 1);      // copies, q's, and the tile's record
                init(ctl.rings[i].full_v[b], 32 * C::kCopyWarps);
                init(ctl.rings[i].free_k[b], users);
                init(ctl.rings[i].free_v[b], users);
            }
            init(ctl.rings[i].free_q, users);
        }
        for (int i = 0; i < kGroups; ++i) {
            for (int b = 0; b < 2; ++b) {
                init(ctl.s[i][b], 2);                        // the products, and which they are
                init(ctl.p[i][b], kGroupWarps);
                init(ctl.o[i][b], 1);
                ctl.odd[i][b] = 0;
            }
            init(ctl.meet[i], kGroupWarps);
        }
        pkv::fence_mbarrier_init();
    }
    pkv::tc_fence_before();
    pkv::grid_dependency_wait();
    if (tid < 4) ctl.cuts[tid].parts = ctl.cuts[tid].due = 0;
    if (tid < kGroups) ctl.last[tid] = 0;
    int *prefix = reinterpret_cast<int *>(smem) + kThreads / 32;
    const int total = pkv::tree_tiles<kTile, kThreads>(p, prefix, reinterpret_cast<int *>(smem));
    // softmax warps, then by twos (worker or half of its copies): K, issue, V, q
    // (so that the issuing warps share no scheduler with the softmax of rows 0..63)
    const int x = warp - kSoftmaxThreads / 32, role = x < 0 ? -1 : x / 2, which = x < 0 ? tid / kGroupThreads : x & 1;
    const int worker = C::kTwo ? 0 : which;
    TreePlace at;
    const TreeShare share = pkv::tree_share<kTile>(p, prefix, total, worker * gridDim.x + blockIdx.x, C::kWorkers * gridDim.x, at);
    __syncthreads();
    pkv::tc_fence_after();
    const uint32_t base = pkv::smem_u32(smem) + worker * C::kWorker, tmem = ctl.tmem;
    Rings &rings = ctl.rings[worker];
    if (role < 0) {
        Softmax<T, D, ROWS> sm{p, ctl, rings, base, tmem + 256 * which + ((uint32_t)(warp & 3) << 21), which, tid % kGroupThreads,
                               tid % kGroupThreads - which * C::kShift,
                               fabsf(p.scale_log2)};
        sm.run(share.me);
    } else {
        const int lane = tid & 31, part = C::kTwo ? which : 0;
        if (role == 0) {
            Producer<D, ROWS, LB, false> pr{p, rings, ctl.cuts + 2 * worker, base + C::kQ, lane, part, 0, 0, 0};
            pr.run(share, at);
        } else if (role == 1) {
            Issuer<T, D, ROWS> is{p, ctl, rings, base, tmem + 256 * which, which, share.Z - share.A};
            is.run();
        } else if (role == 2) {
            Producer<D, ROWS, LB, true> pr{p, rings, ctl.cuts + 2 * worker, base + C::kQ + C::kK * C::kSlot, lane, part, 0, 0, 0};
            pr.run(share, at);
        } else if (!C::kTwo || which == 0) {
            copy_q<D, ROWS>(p, rings, base, share, at);
        }
        pkv::cp_async_wait_all();
    }
    pkv::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        pkv::tc_fence_after();
        pkv::tmem_dealloc(tmem, kColumns);
    }
    __syncthreads();
    if (tid < C::kWorkers && !(C::kTwo ? ctl.last[0] | ctl.last[1] : ctl.last[tid])) ctl.cuts[2 * tid].parts = 0;
    pkv::tree_join_cuts<D, kThreads / 32, 4, 4>(p, ctl.cuts);
}

template <typename T, int D, int ROWS, int LB>
cudaError_t launch_one(const TreeParams &p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    constexpr int bytes = Cfg<D, ROWS>::kBytes;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(tree_mma_kernel<T, D, ROWS, LB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(tree_mma_kernel<T, D, ROWS, LB>, dim3((unsigned)(p.C / Cfg<D, ROWS>::kWorkers)), kThreads, bytes, stream, p);
}

template <typename T, int D, int ROWS>
cudaError_t launch_b(const TreeParams &p, cudaStream_t s) {
    return p.b.lb == 3 ? launch_one<T, D, ROWS, 3>(p, s) : p.b.lb == 4 ? launch_one<T, D, ROWS, 4>(p, s) : launch_one<T, D, ROWS, 5>(p, s);
}

template <typename T>
cudaError_t launch_rows(int D, const TreeParams &p, cudaStream_t s) {
    if (D == 128)
        return p.RC <= 64 ? launch_b<T, 128, 64>(p, s) : p.RC <= 128 ? launch_b<T, 128, 128>(p, s) : launch_b<T, 128, 256>(p, s);
    return p.RC <= 64 ? launch_b<T, 64, 64>(p, s) : p.RC <= 128 ? launch_b<T, 64, 128>(p, s) : launch_b<T, 64, 256>(p, s);
}

}  // namespace

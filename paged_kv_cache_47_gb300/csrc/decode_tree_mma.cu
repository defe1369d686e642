// Tree attention over 16-bit caches on the 5th-generation tensor cores.
//
// Products. A unit's rows (a q head of a drafted token each) are the M of
// tcgen05.mma, 128 at a time: S[128 rows][128 tokens] = Q K^T, Q and K from
// shared memory as they were copied, and O[128 rows][D] += P V, P from tensor
// memory, V from shared memory read along its tokens. A thread owns a row: the
// softmax's maximum and sum need no other thread. K and V are read once for
// all rows of a kv head, so up to 128 rows (or 256, in two tiles that share
// each K and V) cost the memory what one row does.
//
// P enters as two parts, hi = the type's nearest and lo = the rest's, so
// weights keep 16 (bf16) or 22 (fp16) bits: with hi alone a bf16 output's error
// against 64 bits grows by half (weights are rounded like the outputs). The
// parts lie where their scores lay: 32 scores become 16 words of hi and 16 of lo.
//
// Roles. Four warps copy K, V (tiles of 128 tokens, a ring of half-tiles) and q
// rows through cp.async, whose 16-byte pieces serve blocks of 8 to 32 tokens
// as well as long runs. Two groups of four warps each take a tile through both
// products; a group's chain (product, softmax, product) is long, so units of up
// to 128 rows give their tiles to the groups in turn and join the two states,
// which lie in the same lanes of tensor memory, at the end. Units of more rows
// give each group its own 128 rows, and every tile.
//
// The softmax's reference exponent moves only when a score passes what the type
// holds; only then are the outputs rescaled, by one read and write of them.
//
// What a row does not see has weight zero; as zero times infinity is not zero,
// tiles with drafted tokens are looked through for V that are not finite, and
// such a tile's second product is done on the CUDA cores, over what has weight.
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

constexpr int kTile = pkv::kTreeMmaTile;       // 128 tokens
constexpr int kGroups = 2, kGroupThreads = 128;
constexpr int kProducers = 128;
constexpr int kThreads = kGroups * kGroupThreads + kProducers;
constexpr int kMetas = 16;                     // more than the tiles a ring holds
constexpr uint32_t kColumns = 512;             // tensor memory: each group 128 of S, then O
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
    int at, left;            // tiles of the segment before and after it
    int seg;                 // the CTA's segments before it
    int whole, slot;         // whole unit, or slot of the piece
};

template <int D, int RT>
struct Cfg {
    static constexpr int kPlanes = D / 64;                   // of 64 elements, 128 bytes a row
    static constexpr int kPlane = kTile * 128;
    static constexpr int kSlot = kPlanes * kPlane;           // K or V of a tile; 128 rows of q
    static constexpr int kQ = RT * kSlot;
    static constexpr int kQBufs = RT == 1 ? 2 : 1;
    static constexpr int kSlots = D == 128 ? 5 : 12;         // the ring's; with q 224 KB
    static constexpr int kRing = kQBufs * kQ;                // where it begins
    static constexpr int kBytes = kRing + kSlots * kSlot;
};

struct Control {
    uint64_t full[16], empty[16], full_q[2], free_q[2];
    uint64_t s[kGroups], o[kGroups], p[kGroups], state[kGroups], taken[kGroups];
    Tile tiles[kMetas];
    int odd[kGroups][2];     // tile (+ 1) last found to have V that are not finite, by turns
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
__device__ __forceinline__ void tm_store(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
        "%23, %24, %25, %26, %27, %28, %29, %30, %31};" ::PKV_W8(r, 0),
        PKV_W8(r, 8), PKV_W8(r, 16), PKV_W8(r, 24), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_store2(uint32_t at, uint32_t a, uint32_t b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tm_load2(uint32_t at, uint32_t &a, uint32_t &b) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(a), "+r"(b) : : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float f32(uint32_t x) { return __uint_as_float(x); }

// ---------------------------------------------------------------- copies
template <typename T, int D, int RT, int LB>
struct Producer {
    using C = Cfg<D, RT>;
    static constexpr int E = 32 >> LB;                       // blocks of a warp's 32 tokens of a tile
    static constexpr int kAhead = 32 / E;                    // tiles whose entries a warp holds
    static constexpr int kPieces = 32 * C::kPlanes * 8 / 32; // 16-byte pieces a lane copies of 32 rows
    const TreeParams &p;
    Control *ctl;
    uint32_t base;                                           // shared memory
    int tid, lane, pw;
    int32_t window, next_window;
    int from;                                                // tile that the window begins at

    __device__ __forceinline__ int32_t entries(int s, int tile) const {
        const int e = (tile + lane / E) * (kTile >> LB) + pw * E + lane % E;
        return e < p.b.M ? __ldg(p.tables + (int64_t)s * p.b.M + e) : -1;
    }

    // Lane's destination of its piece j of the warp's rows.
    static __device__ __forceinline__ uint32_t piece(int pw, int lane, int j) {
        if (D == 128) {
            const int r = pw * 32 + 2 * j + (lane >> 4), w = lane & 15;
            return (w >> 3) * C::kPlane + r * 128 + (((w & 7) ^ (r & 7)) << 4);
        }
        const int r = pw * 32 + 4 * j + (lane >> 3), w = lane & 7;
        return r * 128 + ((w ^ (r & 7)) << 4);
    }

    // A context's last tile, or one with a block id outside the pool.
    static __device__ __noinline__ void ragged(const TreeParams &p, const uint8_t *pool, uint32_t slot, int32_t ids, int at, int g,
                                               int left, int pw, bool tell) {
        const int lane = threadIdx.x & 31;
        constexpr int R = C::kPlanes * 8;                    // pieces of a row
#pragma unroll 1
        for (int j = 0; j < kPieces; ++j) {
            const int r = (lane + 32 * j) / R, w = (lane + 32 * j) % R;
            int id = __shfl_sync(~0u, ids, at + (r >> LB));
            const bool in = pw * 32 + r < left, ok = (unsigned)id < (unsigned)p.NB;
            if (in && !ok && tell) atomicOr(p.b.err, PKV_DEVERR_BLOCK_ID);
            const size_t src = ((((size_t)(ok ? id : 0) * p.Hk + g) << LB) + (r & ((1 << LB) - 1))) * (2 * D) + w * 16;
            pkv::cp_async_16(slot + piece(pw, lane, j), pool + src, in && ok);
        }
    }

    __device__ __forceinline__ void copy(const void *pool, uint32_t slot, int32_t ids, int at, int g, int left, bool tell) const {
        int id[E];
        bool ok = left >= kTile;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            id[k] = __shfl_sync(~0u, ids, at + k);
            ok = ok && (unsigned)id[k] < (unsigned)p.NB;
        }
        const uint8_t *src = static_cast<const uint8_t *>(pool);
        if (!ok) {
            ragged(p, src, slot, ids, at, g, left, pw, tell);
            return;
        }
        constexpr int PB = kPieces / E;                      // pieces of a block
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const uint8_t *block = src + (((size_t)(uint32_t)id[k] * p.Hk + g) << LB) * (2 * D) + lane * 16;
#pragma unroll
            for (int j = 0; j < PB; ++j) pkv::cp_async_16(slot + piece(pw, lane, k * PB + j), block + j * 512, true);
        }
    }

    // The unit's q rows, and zeros up to whole tiles of 128.
    __device__ __forceinline__ void copy_q(uint32_t to, int o, int g, int r0, int nr) const {
        constexpr int R = C::kPlanes * 8;
        const uint8_t *q = static_cast<const uint8_t *>(p.q);
#pragma unroll 4
        for (int j = 0; j < RT * kTile * R / kProducers; ++j) {
            const int x = tid + j * kProducers, row = x / R, w = x % R, r = row % kTile;
            const bool in = row < nr;
            const size_t src = in ? pkv::tree_row(p, o, g, r0 + row) * (2 * D) + w * 16 : 0;
            pkv::cp_async_16(to + (row / kTile) * C::kSlot + (w >> 3) * C::kPlane + r * 128 + (((w & 7) ^ (r & 7)) << 4),
                             q + src, in);
        }
    }

    __device__ __forceinline__ bool wait(uint64_t &bar, uint32_t parity) const {
        return __all_sync(~0u, pkv::mbar_wait(pkv::smem_u32(&bar), parity, p.b.err, p.wait_ns));
    }

    __device__ __forceinline__ void run(const TreeShare &share, TreePlace at) {
        const int count = share.Z - share.A;
        int use = 0;
        int32_t first = count > 0 ? entries(at.s, at.i) : 0;
        for (int t = 0, seg = 0; t < count; ++seg) {
            const int n = min(at.tiles - at.i, count - t), i0 = at.i;
            const int chunks = at.units / p.Hk, g = at.u / chunks, r0 = (at.u - g * chunks) * p.RC;
            const int nr = min(p.RC, at.q.n * p.G - r0);
            const bool whole = n == at.tiles;
            if (!whole && i0 == 0 && tid == 0)
                p.cuts[blockIdx.x] = {pkv::tree_parts(share, share.A + t, at.tiles), at.q.o, g, r0, nr, {}};
            window = first;
            from = i0;
            next_window = n > kAhead ? entries(at.s, i0 + kAhead) : 0;
            const pkv::TreeSeq q = at.q;
            const int s = at.s;
            if (t + n < count) {                             // the next unit's first entries, ahead of time
                at.next_unit<kTile>(p);
                first = entries(at.s, 0);
            }
            for (int k = 0; k < n; ++k, ++t) {
                const int i = i0 + k, t0 = i * kTile;
                if (i == from + kAhead) {
                    window = next_window;
                    from = i;
                    next_window = n - k > kAhead ? entries(s, i + kAhead) : 0;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v, ++use) {
                    const int slot = use % C::kSlots;
                    if (!wait(ctl->empty[slot], (use / C::kSlots & 1) ^ 1)) return;
                    if (tid == 0) {
                        if (v == 0)
                            ctl->tiles[t % kMetas] = {q.o, q.n, q.L, g, r0, nr, t0, k, n - 1 - k, seg, whole, i0 ? 0 : 1};
                        pkv::mbar_arrive(pkv::smem_u32(&ctl->full[slot]));
                    }
                    copy(v ? p.v : p.k, base + C::kRing + slot * C::kSlot, window, (i - from) * E, g, q.L - t0, v == 0);
                    if (!(p.drop_arrival && blockIdx.x == 0 && tid == 0 && use == 0))
                        pkv::cp_async_arrive_noinc(pkv::smem_u32(&ctl->full[slot]));
                    else
                        pkv::cp_async_wait_all();
                }
                if (k == 0) {
                    const int buf = seg % C::kQBufs;
                    if (!wait(ctl->free_q[buf], (seg / C::kQBufs & 1) ^ 1)) return;
                    copy_q(base + buf * C::kQ, q.o, g, r0, nr);
                    pkv::cp_async_arrive_noinc(pkv::smem_u32(&ctl->full_q[buf]));
                }
            }
        }
    }
};

// ---------------------------------------------------------------- the products and the softmax
template <typename T, int D, int RT>
struct Group {
    using C = Cfg<D, RT>;
    using El = pkv::Elem<T>;
    static constexpr uint32_t kPv = idesc<T>(D, true, false);
    const TreeParams &p;
    Control *ctl;
    uint32_t base, S, O, other_S, other_O;                   // shared memory; tensor memory of this lane quarter
    uint32_t mS, mO;                                         // the same as the products take it
    int w, row, lane, warp;                                  // group, row of the tile, lane, warp of the group
    uint32_t qk;
    float scale, mu, room, l;
    bool have_o, o_due;
    uint32_t n_s, n_o, n_p, n_state, n_seen, n_taken;        // uses of the barriers

    __device__ __forceinline__ bool wait(uint64_t &bar, uint32_t parity) const {
        return __all_sync(~0u, pkv::mbar_wait(pkv::smem_u32(&bar), parity & 1, p.b.err, p.wait_ns));
    }
    // The group's four warps meet; what they did to tensor memory is ordered.
    __device__ __forceinline__ void arrive(uint64_t &bar) const {
        pkv::tc_fence_before();
        __syncwarp();
        if (lane == 0) pkv::mbar_arrive(pkv::smem_u32(&bar));
    }
    __device__ __forceinline__ bool meet() {
        arrive(ctl->p[w]);
        const bool ok = wait(ctl->p[w], n_p++);
        pkv::tc_fence_after();
        return ok;
    }
    __device__ __forceinline__ bool wait_o() {
        if (!o_due) return true;
        const bool ok = wait(ctl->o[w], n_o++);
        o_due = false;
        pkv::tc_fence_after();
        return ok;
    }

    // Bits of the 32 tokens from drafted token d0 on (before: d0 < 0) that token i sees.
    __device__ __forceinline__ uint32_t word(const Tile &m, int i, int k) const {
        if (32 * k >= m.n) return 0;
        uint32_t x;
        if (p.masks) x = __ldg(reinterpret_cast<const uint32_t *>(p.masks + (size_t)(m.o + i) * p.W) + k);
        else x = i >= 32 * k + 31 ? ~0u : i < 32 * k ? 0u : (2u << (i - 32 * k)) - 1;
        return m.n - 32 * k >= 32 ? x : x & ((1u << (m.n - 32 * k)) - 1);
    }
    __device__ __forceinline__ uint32_t sees(const Tile &m, int i, int d0) const {
        if (d0 <= -32) return ~0u;
        if (d0 < 0) return (word(m, i, 0) << -d0) | ((1u << -d0) - 1);
        return __funnelshift_r(word(m, i, d0 >> 5), word(m, i, (d0 >> 5) + 1), d0 & 31);
    }

    __device__ __forceinline__ void scale_o(float f) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t x[32];
            tm_load(O + c, x);
            tm_wait(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(f32(x[i]) * f);
            tm_store(O + c, x);
        }
    }

    // Whether any of the tile's V of drafted tokens is not finite (told through ctl->odd).
    __device__ __forceinline__ void look_through(uint32_t slot, const Tile &m, int t, volatile int *odd) const {
        const int a = max(0, m.L - m.n - m.t0), z = min(kTile, m.L - m.t0);
        constexpr int R = C::kPlanes * 8;
        constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
        constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
        uint32_t any = 0;
        for (int x = a * R + row; x < z * R; x += kGroupThreads) {
            // (the order of a row's pieces says nothing here)
            uint32_t y[4];
            pkv::lds_u32x4(slot + (x % R >> 3) * C::kPlane + (x / R) * 128 + (x % 8 << 4), y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= ((y[i] & kExp) + kOne) & 0x80008000u;     // the exponent is all ones
        }
        if (any) *odd = t + 1;
    }

    // O += P V of a tile on the CUDA cores, over what has weight.
    static __device__ __noinline__ void slow_pv(uint32_t S, uint32_t O, uint32_t slot, int ntok, bool have_o) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (have_o) {
                tm_load(O + c, o);
                tm_wait(o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0;
            }
#pragma unroll 1
            for (int t0 = 0; t0 < ntok; t0 += 32) {
                uint32_t x[32];
                tm_load(S + t0, x);
                tm_wait(x);
                const int most = min(32, ntok - t0);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 hi = El::unpack2(x[j / 2]), lo = El::unpack2(x[16 + j / 2]);
                    const float pj = j % 2 ? hi.y + lo.y : hi.x + lo.x;
                    if (pj == 0.f || j >= most) continue;
                    const int r = t0 + j;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t y[4];
                        pkv::lds_u32x4(slot + (c >> 6) * C::kPlane + r * 128 + ((((c & 63) / 8 + k) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = El::unpack2(y[e]);
                            o[8 * k + 2 * e] = __float_as_uint(fmaf(pj, v.x, f32(o[8 * k + 2 * e])));
                            o[8 * k + 2 * e + 1] = __float_as_uint(fmaf(pj, v.y, f32(o[8 * k + 2 * e + 1])));
                        }
                    }
                }
                __syncwarp();
            }
            tm_store(O + c, o);
        }
        tm_store_wait();
    }

    // Scores to weights: maximum, reference, and the parts in the scores' place.
    template <bool MASKED>
    __device__ __forceinline__ void softmax(const Tile &m, int i) {
        const int d0 = m.t0 - (m.L - m.n);
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kTile; c += 64) {
            uint32_t x[2][32];
            tm_load(S + c, x[0]);
            tm_load(S + c + 32, x[1]);
            tm_wait(x[0]);
            tm_wait(x[1]);
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t bits = MASKED ? sees(m, i, d0 + c + 32 * h) : ~0u;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    a = fmaxf(a, MASKED && !(bits >> j & 1) ? -INFINITY : f32(x[h][j]));
                    b = fmaxf(b, MASKED && !(bits >> (j + 1) & 1) ? -INFINITY : f32(x[h][j + 1]));
                }
            }
            top = fmaxf(top, fmaxf(a, b));
        }
        top *= scale;                                        // (not negative; 0 times -infinity stays below)
        if (__any_sync(~0u, top > room)) {
            const bool none = mu == kNone;
            const float nm = top > room ? top - kTop<T> : mu;
            const float f = none || nm == mu ? 1.f : pkv::ex2_approx(mu - nm);
            if (have_o) scale_o(f);
            l *= f;
            mu = nm;
            if (mu != kNone) room = mu + kRoom<T>;
        }
        const pkv::Pair s2 = pkv::pair_of(scale, scale), m2 = pkv::pair_of(-mu, -mu), minus = pkv::pair_of(-1.f, -1.f);
        pkv::Pair sum = 0;
#pragma unroll 1
        for (int c = 0; c < kTile; c += 64) {
            uint32_t x[2][32];
            tm_load(S + c, x[0]);
            tm_load(S + c + 32, x[1]);
            tm_wait(x[0]);
            tm_wait(x[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t bits = MASKED ? sees(m, i, d0 + c + 32 * h) : ~0u;
                uint32_t y[32];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    float a, b, ra, rb, la, lb;
                    pkv::unpair(pkv::fma2(pkv::pair_of(f32(x[h][j]), f32(x[h][j + 1])), s2, m2), a, b);
                    a = pkv::ex2_approx(a);
                    b = pkv::ex2_approx(b);
                    if (MASKED) {
                        a = bits >> j & 1 ? a : 0.f;
                        b = bits >> (j + 1) & 1 ? b : 0.f;
                    }
                    const pkv::Pair ab = pkv::pair_of(a, b);
                    sum = pkv::add2(sum, ab);
                    y[j / 2] = El::pack2(a, b, ra, rb);
                    pkv::unpair(pkv::fma2(pkv::pair_of(ra, rb), minus, ab), la, lb);
                    y[16 + j / 2] = El::pack2(la, lb, ra, rb);
                }
                tm_store(S + c + 32 * h, y);
            }
        }
        tm_store_wait();
        float a, b;
        pkv::unpair(sum, a, b);
        l += a + b;
    }

    // The rows' outputs, or a piece: this group's state, and the other's (two: RT 1 and more than one tile).
    __device__ __forceinline__ void finish(const Tile &m, int r0, int nr, bool two) {
        float m1 = kNone, l1 = 0.f, f0 = 1.f, f1 = 0.f;
        if (two) {
            uint32_t a, b;
            tm_load2(other_S, a, b);
            m1 = f32(a);
            l1 = f32(b);
            // a state without a weight has no reference of its own
            const float top = l == 0.f ? m1 : l1 == 0.f ? mu : fmaxf(mu, m1);
            f0 = l == 0.f ? 0.f : pkv::ex2_approx(mu - top);
            f1 = l1 == 0.f ? 0.f : pkv::ex2_approx(m1 - top);
            l = l * f0 + l1 * f1;
            mu = top;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f0 *= inv;
        f1 *= inv;
        const bool mine = row < nr;
        const size_t at = m.whole ? pkv::tree_row(p, m.o, m.g, m.r0 + r0 + (mine ? row : 0))
                                  : (size_t)(2 * blockIdx.x + m.slot) * p.RC + r0 + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t x[32];
            float y[32];
            tm_load(O + c, x);
            tm_wait(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = l == 0.f ? 0.f : f32(x[i]) * f0;
            if (two) {
                tm_load(other_O + c, x);
                tm_wait(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = f1 == 0.f ? y[i] : fmaf(f32(x[i]), f1, y[i]);
            }
            if (mine && m.whole) {
                pkv::tree_store<32>(p, at * D + c, y);
            } else if (mine) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4 *>(p.ws_o + at * D + c + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
            __syncwarp();
        }
        if (mine) {
            const float lse = l == 0.f ? -INFINITY : mu + log2f(l);
            if (!m.whole) p.ws_lse[at] = lse;
            else if (p.lse_out) p.lse_out[at] = lse;
        }
        __syncwarp();
    }

    __device__ __forceinline__ bool run(int count) {
        int seg = -1;
        n_s = n_o = n_p = n_state = n_seen = n_taken = 0;
        o_due = false;
        bool shown = false;                                  // a state the other group has not taken yet
        int i = 0, r0 = 0, nr = 0;
        for (int t = RT == 1 ? w : 0; t < count; t += RT == 1 ? kGroups : 1) {
            const int uk = 2 * t, sk = uk % C::kSlots, uv = uk + 1, sv = uv % C::kSlots;
            if (!wait(ctl->full[sk], uk / C::kSlots)) return false;
            const Tile m = ctl->tiles[t % kMetas];
            if (m.seg != seg) {
                seg = m.seg;
                mu = kNone;
                room = -INFINITY;
                l = 0.f;
                have_o = false;
                r0 = RT == 1 ? 0 : w * kTile;
                nr = min(kTile, m.nr - r0);
                i = (m.r0 + r0 + max(0, min(row, nr - 1))) / p.G;
                if (!wait(ctl->full_q[seg % C::kQBufs], seg / C::kQBufs)) return false;
            }
            if (RT == 2 && nr <= 0) {                        // the unit has no rows for this group
                if (!wait(ctl->full[sv], uv / C::kSlots)) return false;
                if (row == 0) {
                    pkv::mbar_arrive(pkv::smem_u32(&ctl->empty[sk]));
                    pkv::mbar_arrive(pkv::smem_u32(&ctl->empty[sv]));
                    if (m.left == 0) pkv::mbar_arrive(pkv::smem_u32(&ctl->free_q[seg % C::kQBufs]));
                }
                continue;
            }
            // the scores' columns are free once the last tile's weights are used, and
            // the state that lay there is taken
            if (!wait_o()) return false;
            if (shown) {
                if (!wait(ctl->taken[w], n_taken++)) return false;
                pkv::tc_fence_after();
                shown = false;
            }
            if (warp == 0) {
                const uint64_t dq = pkv::sdesc_sw128(base + (seg % C::kQBufs) * C::kQ + (RT == 1 ? 0 : w * C::kSlot), 16, 1024);
                const uint64_t dk = pkv::sdesc_sw128(base + C::kRing + sk * C::kSlot, 16, 1024);
                if (pkv::elect_one()) {
                    pkv::fence_proxy_async_smem();
                    pkv::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t step = (k / 4) * (C::kPlane >> 4) + (k % 4) * 2;
                        mma_ss(mS, dq + step, dk + step, qk, k);
                    }
                    pkv::tc_commit(pkv::smem_u32(&ctl->s[w]));
                    pkv::tc_commit(pkv::smem_u32(&ctl->empty[sk]));
                }
                __syncwarp();
            }
            if (!wait(ctl->s[w], n_s++)) return false;
            pkv::tc_fence_after();
            if (RT == 2 && m.left == 0 && row == 0) pkv::mbar_arrive(pkv::smem_u32(&ctl->free_q[seg % C::kQBufs]));
            const bool masked = m.t0 + kTile > m.L - m.n;
            const uint32_t slot = base + C::kRing + sv * C::kSlot;
            bool odd = false;
            if (masked) {
                softmax<true>(m, i);
                if (!wait(ctl->full[sv], uv / C::kSlots)) return false;
                volatile int *flag = &ctl->odd[w][n_p & 1];  // (written again two meetings later)
                look_through(slot, m, t, flag);
                if (!meet()) return false;
                odd = *flag == t + 1;
            } else {
                softmax<false>(m, i);
                arrive(ctl->p[w]);
                ++n_p;
            }
            if (odd) {
                slow_pv(S, O, slot, min(kTile, m.L - m.t0), have_o);
                if (!meet()) return false;
                if (row == 0) pkv::mbar_arrive(pkv::smem_u32(&ctl->empty[sv]));
            } else {
                if (warp == 0) {
                    if (!masked) {
                        if (!wait(ctl->full[sv], uv / C::kSlots) || !wait(ctl->p[w], n_p - 1)) return false;
                    }
                    // K step k: 16 tokens, 16 rows of 128 bytes; planes of 64 elements along N
                    const uint64_t dv = pkv::sdesc_sw128(slot, C::kPlane, 1024);
                    const int steps = min(kTile / 16, (m.L - m.t0 + 15) / 16);
                    if (pkv::elect_one()) {
                        pkv::fence_proxy_async_smem();
                        pkv::tc_fence_after();
                        for (int k = 0; k < steps; ++k) {
                            const uint32_t a = mS + (k / 2) * 32 + (k % 2) * 8;
                            mma_ts(mO, a, dv + 128 * k, kPv, have_o || k);
                            mma_ts(mO, a + 16, dv + 128 * k, kPv, 1);
                        }
                        pkv::tc_commit(pkv::smem_u32(&ctl->o[w]));
                        pkv::tc_commit(pkv::smem_u32(&ctl->empty[sv]));
                    }
                    __syncwarp();
                }
                o_due = true;
            }
            have_o = true;
            if (m.left == 0) {
                if (!wait_o()) return false;
                const bool two = RT == 1 && m.at > 0;
                if (two) {
                    if (!wait(ctl->state[w ^ 1], n_seen++)) return false;
                    pkv::tc_fence_after();
                }
                finish(m, r0, nr, two);
                if (two) arrive(ctl->taken[w ^ 1]);
                if (RT == 1 && row == 0) pkv::mbar_arrive(pkv::smem_u32(&ctl->free_q[seg % C::kQBufs]));
            } else if (RT == 1 && m.left == 1) {             // the other group has the last tile
                if (!wait_o()) return false;
                tm_store2(S, __float_as_uint(mu), __float_as_uint(l));
                tm_store_wait();
                arrive(ctl->state[w]);
                shown = true;
            }
        }
        return wait_o();
    }
};

template <typename T, int D, int RT, int LB>
__global__ void __launch_bounds__(kThreads, 1) tree_mma_kernel(const __grid_constant__ TreeParams p) {
    using C = Cfg<D, RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Control ctl;
    __shared__ int scan[kThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5;
    pkv::grid_dependents_launch();
    if (warp == 0) pkv::tmem_alloc(pkv::smem_u32(&ctl.tmem), kColumns);
    if (tid == 32) {
        auto init = [](uint64_t &bar, int n) { pkv::mbar_init(pkv::smem_u32(&bar), n); };
        for (int i = 0; i < C::kSlots; ++i) {
            init(ctl.full[i], kProducers + 1);               // copies, and the tile's record
            init(ctl.empty[i], RT);
        }
        for (int i = 0; i < 2; ++i) {
            init(ctl.full_q[i], kProducers);
            init(ctl.free_q[i], RT);
        }
        for (int i = 0; i < kGroups; ++i) {
            init(ctl.s[i], 1);
            init(ctl.o[i], 1);
            init(ctl.p[i], 4);
            init(ctl.state[i], 4);
            init(ctl.taken[i], 4);
            ctl.odd[i][0] = ctl.odd[i][1] = 0;
        }
        pkv::fence_mbarrier_init();
    }
    pkv::tc_fence_before();
    pkv::grid_dependency_wait();
    if (tid == 0) p.cuts[blockIdx.x].parts = 0;
    TreePlace at;
    const TreeShare share = pkv::tree_share<kTile, kThreads>(p, reinterpret_cast<int *>(smem), scan, at);
    __syncthreads();
    pkv::tc_fence_after();
    const uint32_t base = pkv::smem_u32(smem), tmem = ctl.tmem;
    if (tid >= kGroups * kGroupThreads) {
        const int x = tid - kGroups * kGroupThreads;
        Producer<T, D, RT, LB> pr{p, &ctl, base, x, x & 31, x >> 5, 0, 0, 0};
        pr.run(share, at);
        pkv::cp_async_wait_all();
    } else {
        const int w = tid / kGroupThreads;
        const uint32_t quarter = (uint32_t)(warp & 3) << 21;
        Group<T, D, RT> gr{p, &ctl, base};
        gr.S = tmem + quarter + 256 * w;
        gr.O = gr.S + 128;
        gr.other_S = tmem + quarter + 256 * (w ^ 1);
        gr.other_O = gr.other_S + 128;
        gr.mS = tmem + 256 * w;
        gr.mO = gr.mS + 128;
        gr.w = w;
        gr.row = tid % kGroupThreads;
        gr.lane = tid & 31;
        gr.warp = warp & 3;
        gr.qk = idesc<T>(128, false, p.scale_log2 < 0.f);
        gr.scale = fabsf(p.scale_log2);
        gr.run(share.Z - share.A);
    }
    pkv::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        pkv::tc_fence_after();
        pkv::tmem_dealloc(tmem, kColumns);
    }
}

template <typename T, int D, int RT, int LB>
cudaError_t launch_one(const TreeParams &p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    constexpr int bytes = Cfg<D, RT>::kBytes;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(tree_mma_kernel<T, D, RT, LB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(tree_mma_kernel<T, D, RT, LB>, dim3((unsigned)p.C), kThreads, bytes, stream, p);
}

template <typename T, int D, int RT>
cudaError_t launch_b(const TreeParams &p, cudaStream_t s) {
    return p.b.lb == 3 ? launch_one<T, D, RT, 3>(p, s) : p.b.lb == 4 ? launch_one<T, D, RT, 4>(p, s) : launch_one<T, D, RT, 5>(p, s);
}

template <typename T, int D>
cudaError_t launch_rt(const TreeParams &p, cudaStream_t s) {
    return p.RC <= kTile ? launch_b<T, D, 1>(p, s) : launch_b<T, D, 2>(p, s);
}

}  // namespace

namespace pkv {

cudaError_t launch_tree_mma(int dtype, int D, const TreeParams &p, cudaStream_t s) {
    if (dtype == PKV_F16) return D == 128 ? launch_rt<__half, 128>(p, s) : launch_rt<__half, 64>(p, s);
    return D == 128 ? launch_rt<__nv_bfloat16, 128>(p, s) : launch_rt<__nv_bfloat16, 64>(p, s);
}

}  // namespace pkv

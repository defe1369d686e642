// Decode attention over a 4-bit cache (include/pkv_q4.h).
//
// With value(c) = s c + m for each group y of 32 elements,
//   <q, k_t>  = sum_y s_ty <q_y, c_ty> + sum_y m_ty (sum of q over y)
//   sum_t p_t v_t[d] = sum_t (p_t s_ty) c_td + sum_t p_t m_ty          (d in y)
// so codes meet the matrix instructions as they are and the parameters enter
// per token and group, not per element.
//
// Codes as operands. A 4-bit code in an fp16 whose other bits are zero is a
// subnormal number, exactly: one AND makes two operands, with no bias to take
// off again and no conversion. mma.sync takes subnormals at full rate, but aligns
// products by their operands' exponent fields before it adds them: leading zeros
// of a subnormal are bits that the sum loses. All codes are brought to bits 4..7
// (c 2^-20), which keeps a sum of 16 to 2^-16.6 of the largest |q|, or weight
// times scale, for a code's unit (2^-12.6 with codes at bits 0..3, measured;
// normal numbers 2^-18); it takes 2 to 3 % of the time. (tcgen05 has no form that
// reads these rows: its 4-bit kinds want the contracted index along the row for
// both operands, and a V row holds one token.)
//
// Work. The batch's (sequence, kv head, up to 8 q heads) units, cut into
// subtiles of 32 tokens (two halves of 16, the m of the scores' product and the
// k of the other) and laid end to end, are split evenly over the CTAs and in
// each CTA over its warps. A warp runs alone (warp_decode.cuh): its own ring of
// two stages in shared memory filled by its own cp.async, its own softmax
// state; no barrier but the one before the CTA's pieces are joined. Pieces of a
// unit cut between warps are joined in shared memory, between CTAs through the
// workspace by the CTA that arrives last (nobody waits).
//
// What bounds it: HBM, D + D / 4 bytes a token and kv head for K and V, and the
// instructions beside it: 700 to 730 of a warp a subtile (D 128), 0.62 to 0.71 a
// cycle, the ANDs' pipe half busy. 256 sequences of 128 to 2048 tokens and 40
// heads (1.79 GB) take 305 to 312 us, 5.8 TB/s; 8 of 32768 to 131072 tokens and
// 8 kv heads of 8 q heads (0.84 GB) 150 to 171 us, 4.9 to 5.6: units of more
// than 4 heads have no free columns for the weights' low parts, and their
// instructions bound them. A step of 64 sequences of 512 to 4096 tokens and 8 kv
// heads (190 MB) takes 46 us: 30 in the loops (6.3 TB/s), the rest is the list
// (1.6 us), tables and first copies (2), the joins within the CTA and between
// CTAs (5), the launch. Single weights, and codes where they lie, took 46.5, 303
// and 152 us in the same process. Sixteen warps in a CTA against two CTAs of
// eight, with those: 52 and 54 us (the step), 359 and 383, 133 and 144.
//
// Softmax in base 2 with a reference exponent that moves only when a score
// passes it by more than the fp16 weights can hold, or a V scale grows past its
// group's bound: most subtiles need one vote instead of a reduction over lanes
// and a rescale of the accumulators. V scales are brought to at most 1 by a
// power of two for each group, so that neither a large scale pushes light tokens,
// other heads or other groups below fp16's range nor tiny scales lose bits.
// Weights, and weights times V scales, are pairs of fp16 (22 bits): codes are
// positive, so an error of the products would not cancel against the minimum's
// share.
//
// Sums over a long context. The matrix instruction cuts its sum towards zero:
// half a last place, 4e-8, a step, always the same way, and the codes' sum and
// the minima's cancel in the output (2000 tokens a warp: 2e-5 of either, where
// outputs are 5e-3). So codes are added up around zero: the second half of a
// subtile enters as 15 - c with its weights negated (an inverted mask and sign,
// no instruction more), and 15 times its weights times scales are added at the
// end. Minima, these and the denominator (rows of scales and of ones beside the
// minima) are small enough to be summed for each half alone and added in fp32,
// which rounds to nearest.
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
#include "warp_decode.cuh"

namespace {

using pkv::launch_chained;

constexpr int kSub = 32;             // tokens of a subtile: two halves of 16, the m and k of the mma
constexpr int kHeads = pkv::kWdHeads;
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSeqs = 1024;       // of one launch
// What a warp spends on a unit besides its subtiles (q to operands, the piece
// it leaves), in subtiles: 3.1 us against 2.07 us a subtile on the Llama-shaped
// batch. Counting units as 2 subtiles evened the warps' ends out (loops of 29.6
// and 29.8 us with one and two units, 31.7 and 35.3 us uncounted).
constexpr int kUnitCost = 2;
constexpr float kCodeUnit = 0x1p-20f;    // of a code as operand
// Sums of q over a group, 2^20 at most, as operands: in this unit they end below
// the largest fp16 number. (In the codes' own they would end near 1 and lose
// what lies below 2^-25, a part of the head's largest element that is more than
// another group's sum: a few large channels are the usual case.)
constexpr float kSumUnit = 0x1p-5f;
// Exponent that a reference gives the top score: up to 2^15 needs no new one, and
// what a pair of fp16 cannot hold of a light token is 2^-35 of the largest.
constexpr float kTop = 10.f;
constexpr uint32_t kMostUp = 0x78007800u;    // 2^15 twice
constexpr float kNone = pkv::kWdNone;

struct Q4Params {
    pkv::WdList list;
    pkv::WdOut o;
    const void *q;
    int act_f16;
    int Hk, NB;
    uint32_t code_bytes, par_bytes;  // of one (block, kv head) chunk, K or V
    float scale_log2;
    const uint8_t *kc, *vc;
    const __half *kp, *vp;
    float *ws_pieces;                // [C][warps][GC][D], or NULL: on chip
    int C;
};

template <int D>
struct Cfg {
    static constexpr int NG = D / 32;
    static constexpr int kCodes = kSub * D / 2;          // bytes of a subtile's K (or V) codes
    static constexpr int kPar = kSub * 4 * NG;           // bytes of its K (or V) parameters
    static constexpr int kStage = 2 * kCodes + 2 * kPar; // K codes, V codes, K parameters, V parameters
    static constexpr int kStages = 2;
    static constexpr int kRing = kStages * kStage;
};

using pkv::wd_ex2;

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma8_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%7,%7,%7,%7};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Two codes as operands, of bits 0..3 and of bits 4..7 of a word's halves: the
// former multiplied by 16, where a shift would wait for the pipe of the ANDs.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
    return as_u32(__hmul2(as_h2(w & 0x000f000fu), __float2half2_rn(16.f)));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return w & 0x00f000f0u; }

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t &a, uint32_t &b) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}

// cp.async of 16 bytes from src + FROM to dst + OFF.
template <int OFF, int FROM = 0>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(dst), "l"(src), "n"(OFF), "n"(FROM)
                 : "memory");
}

// The order of the 16-byte pieces of codes in a stage. Each 128-byte line has
// its eight pieces exclusive-ored by a number of the line (counted within a
// half of 16 tokens), so that the fragment loads of K and V meet 32 banks.
template <int D>
__device__ __forceinline__ int line_xor(int line) {
    return D == 128 ? (line & 6) : ((line & 1) << 2 | (line & 2));
}

// A lane's piece of the parameters: of which block of the subtile, where in the
// block's chunk (K and V alike), where in the stage. At D 128 every lane copies
// a piece of K and one of V; at D 64 lanes 0..15 copy K and 16..31 V.
template <int D, int LB>
struct ParPiece {
    using C = Cfg<D>;
    static constexpr int B = 1 << LB;
    static constexpr int kPieces = B * 4 * C::NG / 16;       // a block's, K or V
    __device__ __forceinline__ static int index(int lane) { return D == 128 ? lane : lane & 15; }
    __device__ __forceinline__ static int block(int lane) { return index(lane) / kPieces; }
    __device__ __forceinline__ static int source(int lane) { return index(lane) % kPieces * 16; }
    __device__ __forceinline__ static int dst_k(int lane) { return 2 * C::kCodes + index(lane) * 16; }
    // V: piece i of a block is tokens 8 (i % (B / 8)) .. of row i / (B / 8)
    __device__ __forceinline__ static int dst_v(int lane) {
        const int i = index(lane) % kPieces;
        return 2 * C::kCodes + C::kPar + i / (B / 8) * (2 * kSub) + block(lane) * (2 * B) + i % (B / 8) * 16;
    }
};

// A context's last subtile, or one with a block id outside the pool: what is
// not there becomes zeros.
template <int D, int LB>
__device__ __noinline__ void issue_ragged(const Q4Params &p, uint32_t stage, int32_t window, int at,
                                          int head, int left, int lane) {
    using C = Cfg<D>;
    using P = ParPiece<D, LB>;
    constexpr int B = 1 << LB;
#pragma unroll 1
    for (int j = 0; j < C::kCodes / 512; ++j) {
        const int c = lane + 32 * j, r = c / (D / 32), w = c % (D / 32);
        int id = __shfl_sync(~0u, window, at + (r >> LB));
        const bool ok = (unsigned)id < (unsigned)p.NB;
        if (!ok && r < left) atomicOr(p.list.err, PKV_DEVERR_BLOCK_ID);
        if (!ok) id = 0;
        const size_t src = (((size_t)id * p.Hk + head) * B + (r & (B - 1))) * (D / 2) + w * 16;
        constexpr int kHalfLines = 16 * D / 2 / 128;
        const int line = c >> 3;
        const uint32_t dst = stage + line * 128 + (((c & 7) ^ line_xor<D>(line & (kHalfLines - 1))) << 4);
        pkv::cp_async_16(dst, p.kc + src, ok && r < left);
        pkv::cp_async_16(dst + C::kCodes, p.vc + src, ok && r < left);
    }
    int id = __shfl_sync(~0u, window, at + P::block(lane));
    const bool ok = (unsigned)id < (unsigned)p.NB;
    if (!ok) id = 0;
    const size_t src = ((size_t)id * p.Hk + head) * p.par_bytes + P::source(lane);
    const int t0 = P::block(lane) * B;               // first token of the piece's block
    if (D == 128 || lane < 16) {
        constexpr int kTok = 16 / (4 * C::NG);       // tokens of a K piece: 1 or 2
        const int r = t0 + P::source(lane) / 16 * kTok;
        const int live = ok ? min(kTok, max(0, left - r)) : 0;
        pkv::cp_async_16_n(stage + P::dst_k(lane), reinterpret_cast<const uint8_t *>(p.kp) + src, live * 4 * C::NG);
    }
    if (D == 128 || lane >= 16) {
        const int r = t0 + P::source(lane) / 16 % (B / 8) * 8;
        const int live = ok ? min(8, max(0, left - r)) : 0;
        pkv::cp_async_16_n(stage + P::dst_v(lane), reinterpret_cast<const uint8_t *>(p.vp) + src, live * 2);
    }
}

// Copies one warp's subtiles into its stages, ahead of their use. The place of
// the next subtile is kept as the sequence and unit it belongs to, its first
// token and the tokens left from there.
template <int D, int LB>
struct Loader {
    using C = Cfg<D>;
    using P = ParPiece<D, LB>;
    static constexpr int kBlocks = kSub >> LB;       // of a subtile: 4, 2 or 1
    const Q4Params &p;
    const int *len;                  // shared memory: a sequence's length
    int lane, cost;                  // cost: places before a unit's first subtile
    int s, u, head, t0, left;
    int32_t window, next_window;     // table entries: lane holds entry `base + lane` of each
    int base;
    uint32_t dst0;                   // this lane's first piece of the codes in a stage
    uint32_t dst_v;                  // and of the V parameters
    // The warp's place for one unit's q rows [GC][D]. A unit whose turn comes
    // while the last rows there have been taken up gets its own copied with its
    // first subtile: 3.1 us a unit besides its subtiles, 3.7 where the rows are
    // read when they are wanted, behind the stream of K and V.
    uint32_t q_buf;
    int q_unit;                      // the unit whose rows lie there (s * U + u); -1: none

    __device__ __forceinline__ Loader(const Q4Params &p_, const int *len_, int lane_, int cost_, uint32_t q_buf_)
        : p(p_), len(len_), lane(lane_), cost(cost_), q_buf(q_buf_), q_unit(-1) {
        const int line = lane >> 3;
        dst0 = line * 128 + (((lane & 7) ^ line_xor<D>(line)) << 4);
        dst_v = P::dst_v(lane);
    }

    __device__ __forceinline__ int32_t entries(int from) const {
        const int e = from + lane;
        return e < p.list.M ? __ldg(p.list.tables + (int64_t)s * p.list.M + e) : -1;
    }
    __device__ __forceinline__ void windows() {
        base = (t0 >> LB) & ~31;
        window = entries(base);
        next_window = entries(base + 32);
    }
    __device__ __forceinline__ void fetch_q() {
        if (q_unit >= 0) return;
        q_unit = s * p.list.U + u;
        const int gca = p.o.heads(u);
        const uint8_t *src = static_cast<const uint8_t *>(p.q) + ((size_t)s * p.o.Hq + p.o.first_head(u)) * (D * 2);
        for (int i = lane * 16; i < gca * D * 2; i += 512) copy16<0>(q_buf + i, src + i);
    }
    __device__ __forceinline__ void start(int seq, int unit, int subtile) {
        s = seq;
        u = unit;
        head = unit / p.o.NC;
        t0 = subtile * kSub;
        left = len[s] - t0;
        windows();
        fetch_q();
    }
    // Next subtile; the table's row starts again with each unit. Returns the
    // places passed over.
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
        fetch_q();
        return cost;
    }
    // Piece J of the codes, K and V, FROM bytes past `src` in their pools.
    template <int J, int FROM>
    __device__ __forceinline__ void codes(uint32_t stage, uint64_t src) const {
        // at D 128 a half has eight lines, two pieces' worth (of the second one's
        // lines the number's bit 2 is set); at D 64 four
        constexpr int OFF = J * 512;
        const uint32_t dst = stage + (D == 128 && J % 2 ? dst0 ^ 64u : dst0);
        copy16<OFF, FROM>(dst, p.kc + src);
        copy16<OFF + C::kCodes, FROM>(dst, p.vc + src);
    }
    __device__ __forceinline__ void issue(uint32_t stage) {
        const int at = (t0 >> LB) - base;
        uint32_t chunk[kBlocks];
        bool ok = left >= kSub;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int id = __shfl_sync(~0u, window, at + k);
            ok &= (unsigned)id < (unsigned)p.NB;
            chunk[k] = id * p.Hk + head;
        }
        if (!ok) {
            issue_ragged<D, LB>(p, stage, window, at, head, left, lane);
            return;
        }
        // a chunk's codes lie in a row: lanes take neighbouring pieces (chunks are
        // 256 bytes or a multiple of 512, so lane offsets go into their low bits)
        const uint32_t piece = lane * 16;
        if constexpr (D == 128) {
            constexpr int PER = 1 << (LB - 3);           // 512-byte pieces of a chunk
            codes<0, 0>(stage, (uint64_t)chunk[0] * p.code_bytes | piece);
            codes<1, 1 % PER * 512>(stage, (uint64_t)chunk[1 / PER] * p.code_bytes | piece);
            codes<2, 2 % PER * 512>(stage, (uint64_t)chunk[2 / PER] * p.code_bytes | piece);
            codes<3, 3 % PER * 512>(stage, (uint64_t)chunk[3 / PER] * p.code_bytes | piece);
        } else if constexpr (LB == 3) {
            const bool up = lane >= 16;                  // 256-byte chunks: two in a piece
            const uint32_t half = (lane & 15) * 16;
            codes<0, 0>(stage, (uint64_t)(up ? chunk[1] : chunk[0]) * p.code_bytes | half);
            codes<1, 0>(stage, (uint64_t)(up ? chunk[3] : chunk[2]) * p.code_bytes | half);
        } else {
            constexpr int PER = 1 << (LB - 4);
            codes<0, 0>(stage, (uint64_t)chunk[0] * p.code_bytes | piece);
            codes<1, 1 % PER * 512>(stage, (uint64_t)chunk[1 / PER] * p.code_bytes | piece);
        }
        uint32_t c = chunk[0];
#pragma unroll
        for (int k = 1; k < kBlocks; ++k) c = P::block(lane) == k ? chunk[k] : c;
        const uint64_t src = (uint64_t)c * p.par_bytes | P::source(lane);
        if (D == 128 || lane < 16) copy16<2 * C::kCodes>(stage + P::index(lane) * 16, reinterpret_cast<const uint8_t *>(p.kp) + src);
        if (D == 128 || lane >= 16) copy16<0>(stage + dst_v, reinterpret_cast<const uint8_t *>(p.vp) + src);
    }
};

// WIDE: units of more than 4 heads. Narrower ones have half of the product's
// columns free: columns 4..7 carry the same heads' low parts.
template <int D, int LB, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) decode_q4_kernel(const __grid_constant__ Q4Params p) {
    using C = Cfg<D>;
    constexpr int NG = C::NG;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ pkv::WdListShared<kWarps, kMaxSeqs> list;
    __shared__ pkv::WdJoinShared<kWarps> join;
    uint8_t *ring_all = smem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // places of the pieces that end in a warp, [warp][GC][D]: behind the rings
    // where they fit, else this CTA's part of the workspace
    float *heads_o = p.ws_pieces ? p.ws_pieces + (size_t)blockIdx.x * kWarps * p.o.GC * D
                                 : reinterpret_cast<float *>(smem + kWarps * (C::kRing + p.o.GC * (D * 2)));
    pkv::grid_dependents_launch();
    pkv::wd_join_init(join);
    const pkv::WdShare share = pkv::wd_share<kWarps, kSub>(p.list, p.o, D, kUnitCost, list);
    if ((int)blockIdx.x >= share.CT) return;
    const int cost = share.cost, a = share.a, z = share.z;

    const uint32_t ring = pkv::smem_u32(ring_all) + warp * C::kRing;
    const int g = lane >> 2, t = lane & 3;
    const int hd = WIDE ? g : g & 3;         // head of the unit whose column this is

    if (a < z) {
        pkv::WdPlace at = pkv::wd_place(p.list, list, a, cost);
        Loader<D, LB> ld(p, list.len, lane, cost, pkv::smem_u32(smem) + kWarps * C::kRing + warp * p.o.GC * (D * 2));
        ld.start(at.s, at.u, at.i);
        int rem = z - (at.tu + at.i);             // places from the next subtile to copy on
#pragma unroll
        for (int st = 0; st < C::kStages; ++st) {
            if (rem > 0) {
                ld.issue(ring + st * C::kStage);
                if (--rem > 0) rem -= ld.advance();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        uint32_t sk = ring;                  // stage in use
        // this lane's places in a stage (see below)
        const int r0 = 4 * (g >> 1) + (g & 1);
        uint32_t k_at, v_at, m_at;
        if constexpr (NG == 4) {
            k_at = (r0 >> 1) * 128 + (((4 * (r0 & 1) + t) ^ line_xor<D>(r0 >> 1)) << 4);
            v_at = 2 * t * 128 + (((g >> 1) ^ (2 * t)) << 4) + 8 * (g & 1);
        } else {
            k_at = (r0 >> 2) * 128 + (((2 * (r0 & 3) + (t >> 1)) ^ line_xor<D>(r0 >> 2)) << 4) + 8 * (t & 1);
            v_at = t * 128 + (((g >> 2) ^ line_xor<D>(t)) << 4) + 4 * (g & 3);
        }
        m_at = 2 * NG + (NG == 4 ? 4 * (t & 1) : 0);                 // minima of two groups in a K row
        const uint32_t vs_at = (g & (NG - 1)) * (2 * kSub) + (g / NG & 1) * 32 + t * 8;      // scales of a group, V
        const uint32_t vm_at = ((g & (2 * NG - 1)) ^ NG) * (2 * kSub) + t * 8;       // minima, then scales of a group, V
        const uint32_t minima = g & NG ? 0u : ~0u;
        const uint32_t one = g == 0 ? 0x3c003c00u : 0u;

        while (true) {
            // ---- a unit, or the part of it that lies here: `count` subtiles
            const int n = at.nv - cost;
            const int count = min(n, z - at.tu) - at.i;
            if (count <= 0) break;
            const int gca = p.o.heads(at.u), h0 = p.o.first_head(at.u);
            int left = list.len[at.s] - at.i * kSub;     // tokens from the subtile in hand on
            uint32_t qb[NG][2][2];               // q as B operands
            uint32_t qsum;                       // sums of q over the groups, as a B operand
            float zs0, zs1;                      // scores to log2 units, heads 2t and 2t + 1
            {
                // lane (g, t) holds elements 32 y + 8 t .. + 7 of its head
                float x[NG][8], top = 0.f;
                const bool here = ld.q_unit == at.s * p.list.U + at.u;
                if (here) {
                    // copied with the unit's first subtile or before
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    __syncwarp();
                }
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    uint4 raw = make_uint4(0, 0, 0, 0);
                    if (hd < gca) {
                        if (here)
                            pkv::lds_u32x4(ld.q_buf + hd * (D * 2) + 64 * y + 16 * t, raw.x, raw.y, raw.z, raw.w);
                        else
                            raw = __ldg(reinterpret_cast<const uint4 *>(
                                static_cast<const uint16_t *>(p.q) +
                                ((size_t)at.s * p.o.Hq + h0 + hd) * D + 32 * y + 8 * t));
                    }
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
                if (here) {
                    __syncwarp();
                    ld.q_unit = -1;              // taken up
                }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                // a power of two that brings the head's largest element to
                // [2^14, 2^15): exact, and fp16 then holds q exactly down to
                // 2^-28 of it
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
                    sum[y] *= kSumUnit;              // at most 2^15
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        qb[y][k][0] = as_u32(__floats2half2_rn(x[y][2 * k], x[y][4 + 2 * k]));
                        qb[y][k][1] = as_u32(__floats2half2_rn(x[y][2 * k + 1], x[y][4 + 2 * k + 1]));
                    }
                }
                // sums as fp16 pairs: k = 0..NG-1 the high parts, then the low ones
                // (to 2^-22 of the sum, at least to 2^-34 of the head's largest
                // element: a head with a few large channels keeps the sums of its
                // other groups)
                const bool upper = NG == 4 && (t & 1);
                const float s0 = upper ? sum[NG - 2] : sum[0], s1 = upper ? sum[NG - 1] : sum[1];
                __half2 hi = __floats2half2_rn(s0, s1);
                if (NG == 4 ? t >= 2 : t == 1) {
                    const float2 f = __half22float2(hi);
                    hi = __floats2half2_rn(s0 - f.x, s1 - f.y);
                }
                qsum = NG == 2 && t >= 2 ? 0u : as_u32(hi);
                const float zq = p.scale_log2 / kCodeUnit * down;
                zs0 = __shfl_sync(~0u, zq, 8 * t);
                zs1 = __shfl_sync(~0u, zq, 8 * t + 4);
            }
            float mu0 = kNone, mu1 = kNone;      // reference exponents
            float room = -INFINITY;              // largest score above them that needs no new ones
            // V scales are multiplied, group by group, by a power of two that
            // brings the largest so far to [1/2, 1): of the groups in pairs, and
            // of the one that this lane watches
            uint32_t vm[NG / 2], vm_own = kMostUp;
#pragma unroll
            for (int i = 0; i < NG / 2; ++i) vm[i] = kMostUp;
            float acc[NG][2][4], accx[4];
#pragma unroll
            for (int y = 0; y < NG; ++y)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[y][k][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) accx[i] = 0.f;

          for (int it = 0; it < count; ++it) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const uint32_t sv = sk + C::kCodes, pk = sk + 2 * C::kCodes, pv = pk + C::kPar;
            constexpr int kHalfCodes = C::kCodes / 2, kHalfPar = C::kPar / 2;

            // ---- scores: rows g and g + 8 of the product are tokens r0 and r0 + 2 of a
            // half, so that after the transpose below lane t holds tokens 4t .. 4t + 3
            float sc[2][4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t k_row = sk + k_at + half * kHalfCodes;
                const uint32_t pk_row = pk + r0 * (4 * NG) + half * kHalfPar;
                uint32_t w[2][NG];
                if constexpr (NG == 4) {
                    pkv::lds_u32x4(k_row, w[0][0], w[0][1], w[0][2], w[0][3]);
                    pkv::lds_u32x4(k_row + 128, w[1][0], w[1][1], w[1][2], w[1][3]);
                } else {
                    lds64(k_row, w[0][0], w[0][1]);
                    lds64(k_row ^ 64u, w[1][0], w[1][1]);            // two rows on: piece + 4
                }
                float s0[NG], s1[NG];                // scales of tokens r0, r0 + 2
                uint32_t m0, m1;                     // minima of two groups
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t row = pk_row + h * (8 * NG);
                    uint32_t u[2];
                    if constexpr (NG == 4) lds64(row, u[0], u[1]);
                    else u[0] = pkv::lds_u32(row);
#pragma unroll
                    for (int y = 0; y < NG; y += 2) {
                        const float2 f = __half22float2(as_h2(u[y / 2]));
                        (h ? s1 : s0)[y] = f.x;
                        (h ? s1 : s0)[y + 1] = f.y;
                    }
                    uint32_t m = pkv::lds_u32(row + m_at);
                    if (NG == 2 && t >= 2) m = 0;
                    (h ? m1 : m0) = m;
                }
                float x[4];
                mma8_zero(x, m0, m1, qsum);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] *= kCodeUnit / kSumUnit;    // to the codes' unit
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    float d[4];
                    uint32_t wa = w[0][y], wb = w[1][y];
                    mma16_zero(d, low_codes(wa), low_codes(wb), high_codes(wa), high_codes(wb), qb[y][0][0], qb[y][0][1]);
                    wa >>= 8;
                    wb >>= 8;
                    mma16(d, low_codes(wa), low_codes(wb), high_codes(wa), high_codes(wb), qb[y][1][0], qb[y][1][1]);
                    x[0] = fmaf(d[0], s0[y], x[0]);
                    x[1] = fmaf(d[1], s0[y], x[1]);
                    x[2] = fmaf(d[2], s1[y], x[2]);
                    x[3] = fmaf(d[3], s1[y], x[3]);
                }
                // exponents of the weights, against the reference
                sc[half][0] = fmaf(x[0], zs0, -mu0);
                sc[half][1] = fmaf(x[1], zs1, -mu1);
                sc[half][2] = fmaf(x[2], zs0, -mu0);
                sc[half][3] = fmaf(x[3], zs1, -mu1);
            }
            if (left < kSub) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (r0 + 16 * half >= left) sc[half][0] = sc[half][1] = -INFINITY;
                    if (r0 + 16 * half + 2 >= left) sc[half][2] = sc[half][3] = -INFINITY;
                }
            }
            left -= kSub;

            // ---- V scales' bounds, and the reference exponent. Lane (g, t) looks at
            // four tokens' scales of one group
            uint32_t v0, v1;
            lds64(pv + vs_at, v0, v1);
            const __half2 big = __hmax2(as_h2(v0), as_h2(v1));
            const float over = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                                     fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
            if (__any_sync(~0u, over > room || !__hble2(__hmul2(big, as_h2(vm_own)), __float2half2_rn(1.f)))) {
                // the factors for this subtile's largest scales, the reference
                // to 10 below the top score
                float bs = fmaxf(__low2float(big), __high2float(big));
                float t0 = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2])) + mu0;
                float t1 = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3])) + mu1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    if (o < 4 || o >= 4 * NG) bs = fmaxf(bs, __shfl_xor_sync(~0u, bs, o));
                    if (o >= 4) {
                        t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, o));
                        t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, o));
                    }
                }
                // a largest scale of 2^(k - 1) to 2^k: 2^-k, 2^15 at most
                const float was = __low2float(as_h2(vm_own));
                const uint32_t top = __float_as_uint(fminf(fmaxf(bs, 0x1p-15f), 65504.f)) >> 23;
                const float now = fminf(was, __uint_as_float((253 - top) << 23));
                const float down = __uint_as_float(__float_as_uint(now) - __float_as_uint(was) + 0x3f800000u);
                vm_own = as_u32(__float2half2_rn(now));
                float u0 = mu0, u1 = mu1;
                const bool none0 = mu0 == kNone, none1 = mu1 == kNone;
                if (t0 > -INFINITY) u0 = none0 ? t0 - kTop : fmaxf(mu0, t0 - kTop);
                if (t1 > -INFINITY) u1 = none1 ? t1 - kTop : fmaxf(mu1, t1 - kTop);
                // (before the first score there is nothing to rescale)
                const float f0 = none0 ? 1.f : wd_ex2(mu0 - u0), f1 = none1 ? 1.f : wd_ex2(mu1 - u1);
                // a head that has had no score but -infinity keeps none, and
                // the next subtile asks again
                room = __any_sync(~0u, u0 == kNone || u1 == kNone) ? -INFINITY : 15.f;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    sc[half][0] = sc[half][0] + mu0 - u0;
                    sc[half][1] = sc[half][1] + mu1 - u1;
                    sc[half][2] = sc[half][2] + mu0 - u0;
                    sc[half][3] = sc[half][3] + mu1 - u1;
                }
                mu0 = u0;
                mu1 = u1;
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    const float d = __shfl_sync(~0u, down, 4 * y), g0 = f0 * d, g1 = f1 * d;
                    if (y % 2 == 0) vm[y / 2] = __byte_perm(__shfl_sync(~0u, vm_own, 4 * y), __shfl_sync(~0u, vm_own, 4 * y + 4), 0x5410);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        acc[y][k][0] *= g0;
                        acc[y][k][1] *= g1;
                        acc[y][k][2] *= g0;
                        acc[y][k][3] *= g1;
                    }
                }
                accx[0] *= f0;
                accx[1] *= f1;
                accx[2] *= f0;
                accx[3] *= f1;
            }

#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // ---- weights as pairs, transposed: lane (g, t) has its head, tokens 4t .. 4t + 3
                uint32_t ph[2], pl[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float w0 = wd_ex2(sc[half][2 * i]), w1 = wd_ex2(sc[half][2 * i + 1]);
                    const __half2 hi = __floats2half2_rn(w0, w1);
                    const float2 f = __half22float2(hi);
                    ph[i] = transpose8(as_u32(hi));
                    pl[i] = transpose8(as_u32(__floats2half2_rn(w0 - f.x, w1 - f.y)));
                }
                // narrow units: a column has the high parts or the low ones
                const uint32_t low = WIDE || g >= 4 ? ~0u : 0u;
                const uint32_t pc[2] = {WIDE || g < 4 ? ph[0] : pl[0], WIDE || g < 4 ? ph[1] : pl[1]};
                const uint32_t pm[2] = {ph[0] & low, ph[1] & low};
                pl[0] &= low, pl[1] &= low;
                // ---- V: rows of the product are d, its contracted index the tokens
                uint32_t v01[NG], v23[NG];
                {
                    // tokens 4t .. 4t + 3: two lines of two rows (D 64: one line of four)
                    const uint32_t v_row = sv + v_at + half * kHalfCodes;
                    uint32_t w[4][NG / 2];
                    if constexpr (NG == 4) {
                        lds64(v_row, w[0][0], w[0][1]);
                        lds64(v_row ^ 64u, w[1][0], w[1][1]);
                        lds64(v_row + 128, w[2][0], w[2][1]);
                        lds64((v_row ^ 64u) + 128, w[3][0], w[3][1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j][0] = pkv::lds_u32(v_row ^ (32u * j));
                    }
#pragma unroll
                    for (int y = 0; y < NG; ++y) {
                        const uint32_t sel = y & 1 ? 0x7632u : 0x5410u;
                        v01[y] = __byte_perm(w[0][y / 2], w[1][y / 2], sel);
                        v23[y] = __byte_perm(w[2][y / 2], w[3][y / 2], sel);
                    }
                }
                {
                    // minima as rows 0..NG-1, scales of the second half as rows
                    // NG..2NG-1 (rows up to 7 repeat them, unused), a row of ones
                    // as row 8
                    uint32_t m01, m23;
                    float sums[4];
                    lds64(pv + vm_at + half * 32, m01, m23);
                    if (half == 0) m01 &= minima, m23 &= minima;
                    mma16_zero(sums, m01, one, m23, one, pc[0], pc[1]);
                    if (WIDE) mma16(sums, m01, one, m23, one, pl[0], pl[1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) accx[i] += sums[i];
                }
#pragma unroll
                for (int y = 0; y < NG; ++y) {
                    uint32_t vs0, vs1;
                    lds64(pv + y * (2 * kSub) + half * 32 + t * 8, vs0, vs1);
                    __half2 m2 = y & 1 ? __high2half2(as_h2(vm[y / 2])) : __low2half2(as_h2(vm[y / 2]));
                    if (half) m2 = __hneg2(m2);
                    const __half2 s01 = __hmul2(as_h2(vs0), m2), s23 = __hmul2(as_h2(vs1), m2);
                    // high parts of the products, then what they leave (narrow units:
                    // in a column of high parts nothing is taken off or added)
                    const __half2 h01 = __hmul2(as_h2(pm[0]), s01), h23 = __hmul2(as_h2(pm[1]), s23);
                    const uint32_t l01 = as_u32(__hfma2(as_h2(pl[0]), s01, __hfma2(as_h2(ph[0]), s01, __hneg2(h01))));
                    const uint32_t l23 = as_u32(__hfma2(as_h2(pl[1]), s23, __hfma2(as_h2(ph[1]), s23, __hneg2(h23))));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t wa = v01[y] >> (8 * k), wb = v23[y] >> (8 * k);
                        if (half) wa = ~wa, wb = ~wb;
                        const uint32_t a0 = low_codes(wa), a1 = high_codes(wa), a2 = low_codes(wb), a3 = high_codes(wb);
                        if (WIDE) mma16(acc[y][k], a0, a1, a2, a3, as_u32(h01), as_u32(h23));
                        mma16(acc[y][k], a0, a1, a2, a3, l01, l23);
                    }
                }
            }

            // ---- the stage is used up: fill it with the subtile after next
            __syncwarp();
            if (rem > 0) {
                ld.issue(sk);
                if (--rem > 0) rem -= ld.advance();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            sk = 2 * ring + C::kStage - sk;
          }

            // ---- the unit's output, or a piece of it
            const bool whole = at.i == 0 && count == n;
            const int slot = at.i ? 0 : 1;       // i > 0: it began before this warp's part
            if (!WIDE) {                         // high and low parts
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    accx[i] += __shfl_xor_sync(~0u, accx[i], 2);
#pragma unroll
                    for (int y = 0; y < NG; ++y)
#pragma unroll
                        for (int k = 0; k < 2; ++k) acc[y][k][i] += __shfl_xor_sync(~0u, acc[y][k][i], 2);
                }
            }
            const float l0 = __shfl_sync(~0u, accx[2], t), l1 = __shfl_sync(~0u, accx[3], t);
            const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
            // a piece of a unit that goes on in the next warp lies in this
            // warp's ring, which is read to the end; the other has its own place
            float *po = slot ? reinterpret_cast<float *>(ring_all + warp * C::kRing)
                             : heads_o + (size_t)warp * p.o.GC * D;
            if (slot && !whole) __syncwarp();
#pragma unroll
            for (int y = 0; y < NG; ++y) {
                const float x0 = fmaf(__shfl_sync(~0u, accx[0], 4 * (NG + y) + t), 15.f, __shfl_sync(~0u, accx[0], 4 * y + t));
                const float x1 = fmaf(__shfl_sync(~0u, accx[1], 4 * (NG + y) + t), 15.f, __shfl_sync(~0u, accx[1], 4 * y + t));
                // one over the group's power of two, in the codes' unit
                const float m2 = y & 1 ? __high2float(as_h2(vm[y / 2])) : __low2float(as_h2(vm[y / 2]));
                const float up = __uint_as_float(0x7f000000u - __float_as_uint(m2)) / kCodeUnit;
#pragma unroll
                for (int e = 0; e < 2; ++e) {            // head 2t + e
                    const int h = 2 * t + e;
                    if (h >= gca) continue;
                    const float m = e ? x1 : x0, inv = e ? inv1 : inv0;
                    const int d = 32 * y + 4 * g;
                    float o4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o4[i] = fmaf(acc[y][i / 2][2 * (i & 1) + e], up, m) * inv;
                    if (whole) {
                        pkv::wd_store_row<4>(p.o, ((size_t)at.s * p.o.Hq + h0 + h) * D + d, o4);
                    } else {
                        pkv::wd_store_f32(po + h * D + d, o4);
                    }
                }
            }
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = 2 * t + e;
                    if (h >= gca) continue;
                    const float lse = (e ? mu1 : mu0) + log2f(e ? l1 : l0);
                    if (!whole) join.lse[warp][slot][h] = lse;
                    else if (p.o.lse_out) p.o.lse_out[(size_t)at.s * p.o.Hq + h0 + h] = lse;
                }
            }
            if (!whole && lane == 0) join.piece[warp][slot] = {at.tu, n, at.s, at.u};
            if (!pkv::wd_next_unit(p.list, list, at, z)) break;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    pkv::wd_join<kWarps, D>(p.o, share, join, heads_o, reinterpret_cast<const float *>(ring_all), C::kRing / 4);
}

// Whether the warps' pieces fit behind the rings (they do but for more than 4
// heads at D 128, which take them to the workspace).
constexpr bool pieces_on_chip(int GC, int D) { return D == 64 || GC <= 4; }

template <int D>
size_t smem_bytes(int GC) {
    return (size_t)kWarps * (Cfg<D>::kRing + GC * D * 2 + (pieces_on_chip(GC, D) ? GC * D * sizeof(float) : 0));
}

template <int D, int LB, bool WIDE>
cudaError_t launch_width(const Q4Params &p, cudaStream_t stream) {
    // the attribute is per device and idempotent; set once for each
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(decode_q4_kernel<D, LB, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<D>(WIDE ? kHeads : 4));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(decode_q4_kernel<D, LB, WIDE>, dim3((unsigned)p.C), kThreads, smem_bytes<D>(p.o.GC), stream, p);
}

template <int D, int LB>
cudaError_t launch(const Q4Params &p, cudaStream_t stream) {
    return p.o.GC > 4 ? launch_width<D, LB, true>(p, stream) : launch_width<D, LB, false>(p, stream);
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// workspace: [PKV_MAX_DECODE_CTAS] arrival counters (a fixed region, whatever
// the launch), then [C][2][GC][D] outputs, then the warps' pieces where they
// do not fit on chip, then [C][2][GC] log2 denominators
constexpr size_t kCounterBytes = PKV_MAX_DECODE_CTAS * sizeof(unsigned);
size_t workspace_for(int C, int GC, int D) {
    return kCounterBytes + (size_t)C * GC * (2 * (D + 1) + (pieces_on_chip(GC, D) ? 0 : kWarps * D)) * sizeof(float);
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
    // the list's places fit 32 bits; products with the CTAs are taken in 64
    const int64_t tokens = (int64_t)M * cache->block_size;
    const int64_t seqs = num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs;
    if (tokens > INT32_MAX / 2 ||
        seqs * Hk * NC * ((tokens + kSub - 1) / kSub + kUnitCost) >= (int64_t)INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
    if ((int64_t)cache->num_blocks * Hk > INT32_MAX)     // 2^31 chunks are over 500 GB
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is 2^31 or more");
    if (C == 0 && (st = pkv::device_sm_count(&C)) != PKV_OK) return st;
    const size_t need = workspace_for(C, GC, D);
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    Q4Params p = {};
    if ((st = pkv::device_error_word(&p.list.err)) != PKV_OK) return st;
    p.list.M = M;
    p.list.lb = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
    p.list.U = Hk * NC;
    p.list.tables_ready = o && o->tables_ready;
    p.o.out_dtype = out_dtype;
    p.o.Hq = num_q_heads;
    p.o.G = G;
    p.o.NC = NC;
    p.o.GC = GC;
    p.o.cnt = static_cast<unsigned *>(workspace);
    p.o.ws_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    float *after = p.o.ws_o + (size_t)C * 2 * GC * D;
    if (!pieces_on_chip(GC, D)) {
        p.ws_pieces = after;
        after += (size_t)C * kWarps * GC * D;
    }
    p.o.ws_lse = after;
    p.act_f16 = cache->act_dtype == PKV_F16;
    p.Hk = Hk;
    p.NB = cache->num_blocks;
    p.code_bytes = (uint32_t)(cache->block_size * D / 2);
    p.par_bytes = (uint32_t)(cache->block_size * D / 32 * 4);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.kc = static_cast<const uint8_t *>(pools->k_codes);
    p.vc = static_cast<const uint8_t *>(pools->v_codes);
    p.kp = static_cast<const __half *>(pools->k_params);
    p.vp = static_cast<const __half *>(pools->v_params);
    p.C = C;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int s0 = 0; s0 < num_seqs; s0 += kMaxSeqs) {
        p.list.S = num_seqs - s0 < kMaxSeqs ? num_seqs - s0 : kMaxSeqs;
        p.list.tables = block_tables + (size_t)s0 * M;
        p.list.lens = context_lens + s0;
        p.q = static_cast<const uint16_t *>(q) + (size_t)s0 * num_q_heads * D;
        p.o.out = static_cast<uint8_t *>(out) + (size_t)s0 * num_q_heads * D * oes;
        p.o.lse_out = o && o->lse_out ? static_cast<float *>(o->lse_out) + (size_t)s0 * num_q_heads : nullptr;
        cudaError_t e;
        if (s0 == 0 && o && o->timing_events[0] &&
            (e = pkv::record_event(static_cast<cudaEvent_t>(o->timing_events[0]), s)) != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "cudaEventRecord: %s", cudaGetErrorString(e));
        auto *go = D == 128 ? (p.list.lb == 3 ? &launch<128, 3> : p.list.lb == 4 ? &launch<128, 4> : &launch<128, 5>)
                            : (p.list.lb == 3 ? &launch<64, 3> : p.list.lb == 4 ? &launch<64, 4> : &launch<64, 5>);
        e = go(p, s);
        if (e != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "decode_q4 launch: %s", cudaGetErrorString(e));
        if (s0 == 0 && o && o->timing_events[1] &&
            (e = pkv::record_event(static_cast<cudaEvent_t>(o->timing_events[1]), s)) != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "cudaEventRecord: %s", cudaGetErrorString(e));
    }
    return PKV_OK;
}

}  // extern "C"

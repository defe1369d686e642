// Storing rows in the 4-bit cache and reading them back (include/pkv_q4.h).
//
// One lane holds 32 elements of a row: the 16 bytes of codes that lie together,
// which are 8 neighbouring elements of each group of 32 (D 64: 16 of each), so a
// row is D / 32 lanes and four 16-byte loads a lane. The lanes of a row find the
// groups' minima and maxima together, each lane ends up with one group's, makes
// its scale and minimum and hands them round. The 8 codes of a K row are exactly
// one of its 32-bit words, those of a V row two of its half-words. A warp takes
// K or V rows of neighbouring tokens of one kv head.
//
// A code is the quotient (x - m) / s rounded to the nearest whole number. The
// product with 1 / s is taken into a sum whose last 16 bits are the quotient's
// fraction and whose next 4 are the code: no conversion, and one comparison for
// two elements tells whether the fraction is too near a half to be sure. The
// sum is off by at most 0.75 of its last place (0.5 its own rounding, 16 * 2^-23
// the reciprocal's, 16 * 2^-24 the quotient's by definition); quotients within
// two places of a half are divided, one in 16000.
//
// What bounds it: HBM, and close to it the instructions. A row of 128 elements
// is 256 bytes read and 80 written: 103 instructions of a warp for a K and a V
// row (232 with 8 elements a lane, each lane its group's scale), 67 to read them
// back. 16383 tokens of 8 heads of 128 appended and read back take 36.0 us, 4.9
// TB/s of what the two calls must read and write (60.6 us with 8 elements a lane;
// CTAs of 256 and of 64 threads 1.1 and 2.6 more; rows read after their slots
// 1.5 more).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "q4_internal.h"

namespace {

using pkv::launch_chained;

constexpr int kThreads = 128;
constexpr float kMaxHalf = 65504.f;

struct StoreParams {
    const void *k, *v;           // append: new rows
    void *k_out, *v_out;         // gather: values
    const int64_t *slots;
    int T, Hk, NB, lb;           // tokens, kv heads, blocks, block size 1 << lb
    pkv_q4cache_pools pools;
    unsigned *err;
};

// Lane's place: which row of the warp's, which 32 elements of it.
template <int D>
struct Place {
    static constexpr int kLanes = D / 32;             // lanes a row, groups a row
    static constexpr int kRows = 32 / kLanes;         // rows of a warp
    __device__ Place() {
        row = (threadIdx.x & 31) / kLanes;
        l = threadIdx.x % kLanes;
    }
    // group of word j of a lane's four, and the word's first element in the row
    static __device__ constexpr int group(int j) { return j % kLanes; }
    __device__ __forceinline__ int element(int j) const {
        return 32 * group(j) + 8 * (l * (4 / kLanes) + j / kLanes);
    }
    int row, l;
};

// What a warp takes: K or V rows of a run of tokens, of the CTA's kv head (kv
// heads first, so that the rows of a token, which lie side by side, are read
// together).
template <int D>
struct Run {
    static constexpr int kTokens = kThreads / 64 * Place<D>::kRows;      // of a CTA
    __device__ __forceinline__ Run(const StoreParams &p, const Place<D> &at) {
        const int tile = blockIdx.x / p.Hk, warp = threadIdx.x >> 5;
        g = blockIdx.x - tile * p.Hk;
        is_v = warp & 1;
        tok = tile * kTokens + (warp >> 1) * Place<D>::kRows + at.row;
    }
    int g, tok;
    bool is_v;
};

// A slot as row of the pools ((block * Hk + head) * B + offset); -1: none.
__device__ __forceinline__ int64_t locate(const StoreParams &p, int64_t slot, int g, bool report) {
    if (slot < 0) return -1;
    const int64_t blk = slot >> p.lb;
    if (blk >= p.NB) {
        if (report) atomicOr(p.err, PKV_DEVERR_SLOT);
        return -1;
    }
    return ((blk * p.Hk + g) << p.lb) + (slot & ((1 << p.lb) - 1));
}

// The larger (smaller) of each of two pairs of T; a NaN wins over anything.
template <typename T>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A lane's words as a V row has them, by half-words with the groups side by
// side, and back.
template <int D>
__device__ __forceinline__ uint4 v_order(const uint32_t (&w)[4]) {
    if constexpr (D == 128)
        return make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                          __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
    return make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                      __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632));
}
template <int D>
__device__ __forceinline__ uint4 words_of(uint4 v) {
    if constexpr (D == 128)
        return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                          __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                      __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
}

// Eight codes by division, for the few where the product leaves one open.
template <typename T>
__device__ __noinline__ uint32_t exact_word(uint4 raw, float mf, float sf) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float2 f = pkv::Elem<T>::unpack2(w[e / 2]);
        word |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(f.x - mf, sf)), 0.f), 15.f) << (4 * e);
        word |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(f.y - mf, sf)), 0.f), 15.f) << (4 * e + 4);
    }
    return word;
}

// 192 and a half, and two last places: a sum with a quotient in [-0.5, 15.5) has
// the code in its bits 16..19 and the fraction's distance from a half, plus two,
// below.
constexpr float kCodeBase = 192.5f + 0x1p-15f;

// The codes of eight elements; `unsure`: all by division.
template <typename T>
__device__ __forceinline__ uint32_t code_word(uint4 raw, float mf, float sf, float inv, bool unsure) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    const pkv::Pair minus = pkv::pair_of(-mf, -mf), inv2 = pkv::pair_of(inv, inv);
    const pkv::Pair base = pkv::pair_of(kCodeBase, kCodeBase);
    uint32_t c[8], near = ~0u;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float2 f = pkv::Elem<T>::unpack2(w[e / 2]);
        float x, y;
        pkv::unpair(pkv::fma2(pkv::add2(pkv::pair_of(f.x, f.y), minus), inv2, base), x, y);
        c[e] = __float_as_uint(x);
        c[e + 1] = __float_as_uint(y);
        const uint32_t fractions = __byte_perm(c[e], c[e + 1], 0x5410);
        asm("min.u16x2 %0, %0, %1;" : "+r"(near) : "r"(fractions));
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) word = word * 16 + __byte_perm(c[i], c[i + 4], 0x7632);
    word -= 0x43404340u * 0x1111u;                   // what the sums' other bits come to
    if ((near & 0xffffu) < 4 || near < 4u << 16 || unsure) word = exact_word<T>(raw, mf, sf);
    return word;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    constexpr int NG = D / 32;
    const Place<D> at;
    const Run<D> run(p, at);
    int64_t slot = -1;
    uint4 raw[4] = {};
    if (run.tok < p.T) {                 // (a row without a slot is read too: nothing waits for the slot)
        slot = __ldg(p.slots + run.tok);
        const T *from = static_cast<const T *>(run.is_v ? p.v : p.k) + ((int64_t)run.tok * p.Hk + run.g) * D;
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = __ldg(reinterpret_cast<const uint4 *>(from + at.element(j)));
    }
    const int64_t r = locate(p, slot, run.g, at.l == 0 && !run.is_v && run.g == 0);
    // of each group, among this lane's elements: (largest, smallest)
    uint32_t ends[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        uint32_t hi = pair_max<T>(pair_max<T>(raw[i].x, raw[i].y), pair_max<T>(raw[i].z, raw[i].w));
        uint32_t lo = pair_min<T>(pair_min<T>(raw[i].x, raw[i].y), pair_min<T>(raw[i].z, raw[i].w));
        if constexpr (NG == 2) {
            const uint4 b = raw[i + 2];
            hi = pair_max<T>(hi, pair_max<T>(pair_max<T>(b.x, b.y), pair_max<T>(b.z, b.w)));
            lo = pair_min<T>(lo, pair_min<T>(pair_min<T>(b.x, b.y), pair_min<T>(b.z, b.w)));
        }
        // (the smallest negated: one maximum for both from here on)
        lo ^= 0x80008000u;
        ends[i] = pair_max<T>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    }
    // lane l keeps group l: half the groups are handed on at each step
#pragma unroll
    for (int o = NG / 2; o > 0; o >>= 1) {
        const bool upper = at.l & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const uint32_t give = upper ? ends[i] : ends[i + o];
            ends[i] = pair_max<T>(upper ? ends[i + o] : ends[i], __shfl_xor_sync(~0u, give, o));
        }
    }
    const float2 end = pkv::Elem<T>::unpack2(ends[0]);
    const float hi = end.x, lo = -end.y;
    __half m = __float2half_rn(fminf(fmaxf(lo, -kMaxHalf), kMaxHalf));
    __half s = __float2half_rn(fminf((hi - lo) * (1.f / 15.f), kMaxHalf));
    // a NaN is the largest of all; an infinity is one of the ends
    if (!(fabsf(hi) <= 3.402823466e38f) || !(fabsf(lo) <= 3.402823466e38f)) m = s = __ushort_as_half(0x7fff);
    // Quotients lie within 0.3 of [0, 15] and need no clamp where the minimum is
    // the group's own but for its rounding (2^-11 of it), that is small beside
    // the scale, and the scale's rounding is relative (no subnormal, not the
    // largest)
    const float own_m = fabsf(__half2float(m)), own_s = __half2float(s);
    const unsigned unsure = __ballot_sync(~0u, !(fabsf(lo) <= kMaxHalf) || !(own_m * 0x1p-9f < own_s) ||
                                                   own_s < 0x1p-13f || own_s >= kMaxHalf) >>
                            (threadIdx.x & 31 & ~(NG - 1));
    const uint32_t own = __half_as_ushort(s) | (uint32_t)__half_as_ushort(m) << 16;
    uint32_t word[4];
    float sf[NG], mf[NG], inv[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const uint32_t v = __shfl_sync(~0u, own, i, NG);
        sf[i] = __half2float(__ushort_as_half((unsigned short)v));
        mf[i] = __half2float(__ushort_as_half((unsigned short)(v >> 16)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv[i]) : "f"(sf[i]));
    }
    if (r < 0) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = Place<D>::group(j);
        word[j] = 0;
        // (a scale of 0 or NaN: codes 0)
        if (sf[i] > 0.f) word[j] = code_word<T>(raw[j], mf[i], sf[i], inv[i], unsure >> i & 1);
    }
    if (!run.is_v) {
        static_cast<uint4 *>(p.pools.k_codes)[r * (D / 32) + at.l] = make_uint4(word[0], word[1], word[2], word[3]);
        __half *par = static_cast<__half *>(p.pools.k_params) + r * 2 * NG + at.l;
        par[0] = s;
        par[NG] = m;
    } else {
        static_cast<uint4 *>(p.pools.v_codes)[r * (D / 32) + at.l] = v_order<D>(word);
        const int off = (int)r & ((1 << p.lb) - 1);
        __half *par = static_cast<__half *>(p.pools.v_params) + (r - off) * 2 * NG + off;
        par[at.l << p.lb] = s;
        par[(NG + at.l) << p.lb] = m;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        float a, b;
        uint4 v;
        v.x = pkv::Elem<T>::pack2(x[0], x[1], a, b);
        v.y = pkv::Elem<T>::pack2(x[2], x[3], a, b);
        v.z = pkv::Elem<T>::pack2(x[4], x[5], a, b);
        v.w = pkv::Elem<T>::pack2(x[6], x[7], a, b);
        *reinterpret_cast<uint4 *>(dst) = v;
    }
}

// Codes stay where they are in the word: the bits of 2^23 with code e's four
// bits in place are 2^23 + 16^e c, and the scale of the product has 16^-e.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const __grid_constant__ StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    constexpr int NG = D / 32;
    const Place<D> at;
    const Run<D> run(p, at);
    const int64_t slot = run.tok < p.T ? __ldg(p.slots + run.tok) : -1;
    const int64_t r = locate(p, slot, run.g, at.l == 0 && !run.is_v && run.g == 0);
    uint4 codes = make_uint4(0, 0, 0, 0);
    uint32_t own = 0;                    // group l's scale and minimum
    if (r >= 0) {
        const __half *par;
        int to_min;
        if (!run.is_v) {
            codes = __ldg(static_cast<const uint4 *>(p.pools.k_codes) + r * (D / 32) + at.l);
            par = static_cast<const __half *>(p.pools.k_params) + r * 2 * NG + at.l;
            to_min = NG;
        } else {
            codes = words_of<D>(__ldg(static_cast<const uint4 *>(p.pools.v_codes) + r * (D / 32) + at.l));
            const int off = (int)r & ((1 << p.lb) - 1);
            par = static_cast<const __half *>(p.pools.v_params) + (r - off) * 2 * NG + off + (at.l << p.lb);
            to_min = NG << p.lb;
        }
        own = __half_as_ushort(__ldg(par)) | (uint32_t)__half_as_ushort(__ldg(par + to_min)) << 16;
    }
    uint32_t params[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) params[i] = __shfl_sync(~0u, own, i, NG);
    if (run.tok >= p.T) return;
    T *to = static_cast<T *>(run.is_v ? p.v_out : p.k_out) + ((int64_t)run.tok * p.Hk + run.g) * D;
    const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
    const pkv::Pair back = pkv::pair_of(-8388608.f, -8388608.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = Place<D>::group(j);
        const float sf = __half2float(__ushort_as_half((unsigned short)params[i]));
        const float mf = __half2float(__ushort_as_half((unsigned short)(params[i] >> 16)));
        const pkv::Pair minimum = pkv::pair_of(mf, mf);
        const pkv::Pair scale[2] = {pkv::pair_of(sf, sf * 0x1p-4f), pkv::pair_of(sf * 0x1p-8f, sf * 0x1p-12f)};
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t w = e < 4 ? word[j] : word[j] >> 16;
            const pkv::Pair c = pkv::pair_of(__uint_as_float((w & (15u << (4 * (e & 3)))) | 0x4b000000u),
                                             __uint_as_float((w & (15u << (4 * (e & 3) + 4))) | 0x4b000000u));
            pkv::unpair(pkv::fma2(pkv::add2(c, back), scale[(e & 3) / 2], minimum), x[e], x[e + 1]);
        }
        store8(to + at.element(j), x);
    }
}

bool misaligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

template <int D>
dim3 grid_for(const StoreParams &p) {
    constexpr int per_cta = Run<D>::kTokens;
    return dim3((unsigned)((int64_t)(p.T + per_cta - 1) / per_cta * p.Hk));
}

template <int D, typename T>
cudaError_t launch_append(const StoreParams &p, cudaStream_t stream) {
    return launch_chained(append_q4_kernel<D, T>, grid_for<D>(p), kThreads, 0, stream, p);
}

template <int D, typename T>
cudaError_t launch_gather(const StoreParams &p, cudaStream_t stream) {
    return launch_chained(gather_q4_kernel<D, T>, grid_for<D>(p), kThreads, 0, stream, p);
}

pkv_status launch_failed(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return PKV_OK;
    return pkv::set_last_error(PKV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

namespace pkv {

pkv_status check_q4cache(const pkv_q4cache_desc *c) {
    if (!c) return set_last_error(PKV_ERR_INVALID_ARG, "cache descriptor is NULL");
    if (c->act_dtype != PKV_F16 && c->act_dtype != PKV_BF16)
        return set_last_error(PKV_ERR_UNSUPPORTED, "act_dtype %d (supported: PKV_F16, PKV_BF16)",
                              c->act_dtype);
    if (c->block_size != 8 && c->block_size != 16 && c->block_size != 32)
        return set_last_error(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)",
                              c->block_size);
    if (c->head_dim != 64 && c->head_dim != 128)
        return set_last_error(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", c->head_dim);
    if (c->num_kv_heads < 1)
        return set_last_error(PKV_ERR_INVALID_ARG, "num_kv_heads %d", c->num_kv_heads);
    if (c->num_blocks < 1) return set_last_error(PKV_ERR_INVALID_ARG, "num_blocks %d", c->num_blocks);
    return PKV_OK;
}

pkv_status check_q4pools(const pkv_q4cache_pools *pools) {
    if (!pools || !pools->k_codes || !pools->v_codes || !pools->k_params || !pools->v_params)
        return set_last_error(PKV_ERR_INVALID_ARG, "a pool pointer is NULL");
    if (misaligned(pools->k_codes) || misaligned(pools->v_codes) || misaligned(pools->k_params) ||
        misaligned(pools->v_params))
        return set_last_error(PKV_ERR_INVALID_ARG, "pools must be 16-byte aligned");
    return PKV_OK;
}

}  // namespace pkv

namespace {

pkv_status prepare(const pkv_q4cache_desc *cache, const pkv_q4cache_pools *pools, const void *k,
                   const void *v, const int64_t *slots, int32_t T, StoreParams *p) {
    pkv_status st = pkv::check_q4pools(pools);
    if (st != PKV_OK) return st;
    if (!k || !v || !slots) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (misaligned(k) || misaligned(v) || reinterpret_cast<uintptr_t>(slots) % 8)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "rows must be 16-byte aligned (slot_mapping 8)");
    if ((int64_t)T * cache->num_kv_heads > INT32_MAX / 2)      // (their rows are over 100 GB)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_tokens * num_kv_heads too large for one launch");
    p->slots = slots;
    p->T = T;
    p->Hk = cache->num_kv_heads;
    p->NB = cache->num_blocks;
    p->lb = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
    p->pools = *pools;
    return pkv::device_error_word(&p->err);
}

}  // namespace

extern "C" {

pkv_status pkv_append_q4(const pkv_q4cache_desc *cache, const void *k_new, const void *v_new,
                         const int64_t *slot_mapping, int32_t num_tokens,
                         const pkv_q4cache_pools *pools, void *stream) {
    pkv_status st = pkv::check_q4cache(cache);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", num_tokens);
    if (num_tokens == 0) return PKV_OK;
    StoreParams p = {};
    if ((st = prepare(cache, pools, k_new, v_new, slot_mapping, num_tokens, &p)) != PKV_OK) return st;
    p.k = k_new;
    p.v = v_new;
    const bool d64 = cache->head_dim == 64, h = cache->act_dtype == PKV_F16;
    auto *go = d64 ? (h ? &launch_append<64, __half> : &launch_append<64, __nv_bfloat16>)
                   : (h ? &launch_append<128, __half> : &launch_append<128, __nv_bfloat16>);
    return launch_failed(go(p, static_cast<cudaStream_t>(stream)), "append_q4");
}

pkv_status pkv_gather_q4(const pkv_q4cache_desc *cache, const pkv_q4cache_pools *pools,
                         const int64_t *slot_mapping, int32_t num_tokens, void *k_out,
                         void *v_out, int32_t out_dtype, void *stream) {
    pkv_status st = pkv::check_q4cache(cache);
    if (st != PKV_OK) return st;
    if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
    if (num_tokens < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", num_tokens);
    if (num_tokens == 0) return PKV_OK;
    StoreParams p = {};
    if ((st = prepare(cache, pools, k_out, v_out, slot_mapping, num_tokens, &p)) != PKV_OK) return st;
    p.k_out = k_out;
    p.v_out = v_out;
    const bool d64 = cache->head_dim == 64;
    auto *go = out_dtype == PKV_F32   ? (d64 ? &launch_gather<64, float> : &launch_gather<128, float>)
               : out_dtype == PKV_F16 ? (d64 ? &launch_gather<64, __half> : &launch_gather<128, __half>)
                                      : (d64 ? &launch_gather<64, __nv_bfloat16>
                                             : &launch_gather<128, __nv_bfloat16>);
    return launch_failed(go(p, static_cast<cudaStream_t>(stream)), "gather_q4");
}

pkv_status pkv_block_copy_q4(const pkv_q4cache_desc *cache, const int64_t *src_dst_pairs,
                             int32_t num_pairs, const pkv_q4cache_pools *pools, void *stream) {
    pkv_status st = pkv::check_q4cache(cache);
    if (st != PKV_OK) return st;
    if (num_pairs == 0) return PKV_OK;
    if ((st = pkv::check_q4pools(pools)) != PKV_OK) return st;
    const size_t rows = (size_t)cache->num_kv_heads * cache->block_size;
    // the pairs are checked by the first call; the second cannot fail on them
    if ((st = pkv::copy_block_pairs(cache->num_blocks, src_dst_pairs, num_pairs, pools->k_codes,
                                    pools->v_codes, rows * cache->head_dim / 2,
                                    static_cast<cudaStream_t>(stream))) != PKV_OK)
        return st;
    return pkv::copy_block_pairs(cache->num_blocks, src_dst_pairs, num_pairs, pools->k_params,
                                 pools->v_params, rows * cache->head_dim / 32 * 4,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"

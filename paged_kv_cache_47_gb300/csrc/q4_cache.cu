// Storing rows in the 4-bit cache and reading them back (include/pkv_q4.h).
//
// One thread holds 8 neighbouring elements (one 16-byte load), four threads a
// group of 32, so a group's minimum and maximum are two shuffles. The 8 codes
// of a K row are exactly one of its 32-bit words, those of a V row two of its
// half-words. Half the lanes of a warp hold K rows and half the V rows of the
// same (token, kv head), so both go in one pass. A CTA takes one kv head of a
// run of tokens, each warp every eighth of them, several at a time when there
// are many, so that their loads are under way together.
//
// A code is the quotient (x - m) / s rounded to the nearest whole number. The
// product with 1 / s, off by 2^-22 of it, decides all but quotients within
// 1e-4 of a half (16 times 2^-22 is 4e-6); only those are divided. Minima and
// maxima are taken on pairs in the rows' own type, the code out of the low bits
// of a sum: conversions to integers run at an eighth of the rate.
//
// What bounds it: HBM. A row of 128 elements is 256 bytes read and 80 written.
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

constexpr int kThreads = 256;
constexpr float kMaxHalf = 65504.f;

struct StoreParams {
    const void *k, *v;           // append: new rows
    void *k_out, *v_out;         // gather: values
    const int64_t *slots;
    int T, Hk, NB, lb;           // tokens, kv heads, blocks, block size 1 << lb
    pkv_q4cache_pools pools;
    unsigned *err;
};

// Lane's place: K or V, which row of the warp's, which 8 elements. A warp holds
// 128 / D rows of K and of V at a time, of as many tokens.
template <int D>
struct Place {
    static constexpr int kLanes = D / 8;              // lanes a row
    static constexpr int kRows = 16 / kLanes;
    __device__ Place() {
        const int lane = threadIdx.x & 31;
        is_v = lane >= 16;
        row = (lane & 15) / kLanes;
        l = lane % kLanes;
        group = l / 4;
        t = l % 4;
    }
    bool is_v;
    int row, l, group, t;
};

// The run of tokens and the kv head of a CTA: kv heads first, so that the rows
// of a token, which lie side by side, are read together.
template <int D, int ITER>
struct Run {
    static constexpr int kTokens = kThreads / 32 * Place<D>::kRows * ITER;
    __device__ __forceinline__ Run(const StoreParams &p) {
        const int tile = blockIdx.x / p.Hk;
        g = blockIdx.x - tile * p.Hk;
        first = tile * kTokens;
    }
    int g, first;
    // token of this lane's row in iteration i
    __device__ __forceinline__ int token(const Place<D> &at, int i) const {
        return first + (i * (kThreads / 32) + (threadIdx.x >> 5)) * at.kRows + at.row;
    }
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

constexpr uint32_t kSigns = 0x80008000u;

// The larger of each of two pairs of T; a NaN is larger than anything.
template <typename T>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const __nv_bfloat162 r =
            __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
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

template <int D, typename T, int ITER>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const Place<D> at;
    const Run<D, ITER> run(p);
    constexpr int NG = D / 32;
    const T *from = static_cast<const T *>(at.is_v ? p.v : p.k) + 8 * at.l;
    int64_t row[ITER];
    uint4 raw[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int tok = run.token(at, i);
        const int64_t slot = tok < p.T ? __ldg(p.slots + tok) : -1;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (slot >= 0) raw[i] = __ldg(reinterpret_cast<const uint4 *>(from + ((int64_t)tok * p.Hk + run.g) * D));
        row[i] = locate(p, slot, run.g, at.l == 0 && !at.is_v && run.g == 0);
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        // largest element and largest negated element of the group, as a pair
        uint32_t ends = pair_max<T>(pair_max<T>(w[0], w[1]), pair_max<T>(w[2], w[3]));
        uint32_t down = pair_max<T>(pair_max<T>(w[0] ^ kSigns, w[1] ^ kSigns),
                                    pair_max<T>(w[2] ^ kSigns, w[3] ^ kSigns));
        ends = pair_max<T>(__byte_perm(ends, down, 0x5410), __byte_perm(ends, down, 0x7632));
        ends = pair_max<T>(ends, __shfl_xor_sync(~0u, ends, 1));
        ends = pair_max<T>(ends, __shfl_xor_sync(~0u, ends, 2));
        const float2 end = pkv::Elem<T>::unpack2(ends);
        const float hi = end.x, lo = -end.y;
        __half m = __float2half_rn(fminf(fmaxf(lo, -kMaxHalf), kMaxHalf));
        __half s = __float2half_rn(fminf((hi - lo) * (1.f / 15.f), kMaxHalf));
        // a NaN is the largest of all; an infinity is one of the ends
        if (!(fabsf(hi) <= 3.402823466e38f) || !(fabsf(lo) <= 3.402823466e38f)) m = s = __ushort_as_half(0x7fff);
        const float mf = __half2float(m), sf = __half2float(s);
        uint32_t word = 0;
        if (sf > 0.f) {                   // not 0, not NaN
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sf));
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 f = pkv::Elem<T>::unpack2(w[e / 2]);
                q[e] = (f.x - mf) * inv;
                q[e + 1] = (f.y - mf) * inv;
            }
            // Quotients lie within 0.3 of [0, 15] and need no clamp where the
            // minimum's rounding (2^-11 of it) is small beside the scale and
            // the scale's own is relative (no subnormal, not the largest)
            bool close = !(fabsf(mf) * 0x1p-9f < sf) || sf < 0x1p-13f || sf >= kMaxHalf;
            // rounded by adding 1.5 * 2^23, whose low bits are then the code
            uint32_t code[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = q[e] + 12582912.f;
                close |= fabsf(q[e] - (c - 12582912.f)) > 0.4999f;
                code[e] = __float_as_uint(c);
            }
#pragma unroll
            for (int e = 7; e >= 0; --e) word = word * 16 + code[e];
            word -= 0x4b400000u * 0x11111111u;       // what all the codes' high bits come to
            if (close) word = exact_word<T>(raw[i], mf, sf);
        }
        const int64_t r = row[i];
        if (r < 0) continue;
        if (!at.is_v) {
            static_cast<uint32_t *>(p.pools.k_codes)[r * (D / 8) + at.t * NG + at.group] = word;
            if (at.t == 0) {
                __half *par = static_cast<__half *>(p.pools.k_params) + r * 2 * NG + at.group;
                par[0] = s;
                par[NG] = m;
            }
        } else {
            uint16_t *codes = static_cast<uint16_t *>(p.pools.v_codes) + r * (D / 4) + 2 * at.t * NG + at.group;
            codes[0] = (uint16_t)word;
            codes[NG] = (uint16_t)(word >> 16);
            if (at.t == 0) {
                const int off = (int)r & ((1 << p.lb) - 1);
                __half *par = static_cast<__half *>(p.pools.v_params) + (r - off) * 2 * NG + off;
                par[at.group << p.lb] = s;
                par[(NG + at.group) << p.lb] = m;
            }
        }
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

template <int D, typename T, int ITER>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const __grid_constant__ StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const Place<D> at;
    const Run<D, ITER> run(p);
    constexpr int NG = D / 32;
    uint32_t word[ITER];
    __half s[ITER], m[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int tok = run.token(at, i);
        const int64_t slot = tok < p.T ? __ldg(p.slots + tok) : -1;
        const int64_t r = locate(p, slot, run.g, at.l == 0 && !at.is_v && run.g == 0);
        word[i] = 0;
        s[i] = m[i] = __ushort_as_half(0);
        if (r < 0) continue;
        if (!at.is_v) {
            word[i] = __ldg(static_cast<const uint32_t *>(p.pools.k_codes) + r * (D / 8) + at.t * NG + at.group);
            const __half *par = static_cast<const __half *>(p.pools.k_params) + r * 2 * NG + at.group;
            s[i] = __ldg(par);
            m[i] = __ldg(par + NG);
        } else {
            const uint16_t *codes =
                static_cast<const uint16_t *>(p.pools.v_codes) + r * (D / 4) + 2 * at.t * NG + at.group;
            word[i] = __ldg(codes) | (uint32_t)__ldg(codes + NG) << 16;
            const int off = (int)r & ((1 << p.lb) - 1);
            const __half *par = static_cast<const __half *>(p.pools.v_params) + (r - off) * 2 * NG + off;
            s[i] = __ldg(par + (at.group << p.lb));
            m[i] = __ldg(par + ((NG + at.group) << p.lb));
        }
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int tok = run.token(at, i);
        if (tok >= p.T) continue;
        const float sf = __half2float(s[i]), mf = __half2float(m[i]);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf((float)((word[i] >> (4 * e)) & 15u), sf, mf);
        store8(static_cast<T *>(at.is_v ? p.v_out : p.k_out) + ((int64_t)tok * p.Hk + run.g) * D + at.l * 8, x);
    }
}

bool misaligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

// One row of a warp's at a time while that fills the GPU (152 SMs of 64 warps),
// four from then on.
constexpr int64_t kManyRows = 4 * 152 * 64;

template <int D, int ITER>
dim3 grid_for(const StoreParams &p) {
    constexpr int per_cta = Run<D, ITER>::kTokens;
    return dim3((unsigned)((int64_t)(p.T + per_cta - 1) / per_cta * p.Hk));
}

template <int D, typename T>
cudaError_t launch_append(const StoreParams &p, cudaStream_t stream) {
    return (int64_t)p.T * p.Hk >= kManyRows
               ? launch_chained(append_q4_kernel<D, T, 4>, grid_for<D, 4>(p), kThreads, 0, stream, p)
               : launch_chained(append_q4_kernel<D, T, 1>, grid_for<D, 1>(p), kThreads, 0, stream, p);
}

template <int D, typename T>
cudaError_t launch_gather(const StoreParams &p, cudaStream_t stream) {
    return (int64_t)p.T * p.Hk >= kManyRows
               ? launch_chained(gather_q4_kernel<D, T, 4>, grid_for<D, 4>(p), kThreads, 0, stream, p)
               : launch_chained(gather_q4_kernel<D, T, 1>, grid_for<D, 1>(p), kThreads, 0, stream, p);
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

// Storing rows in the 4-bit cache and reading them back (include/pkv_q4.h).
//
// One thread holds 8 neighbouring elements (one 16-byte load), four threads a
// group of 32, so a group's minimum and maximum are two shuffles. The 8 codes
// of a K row are exactly one of its 32-bit words, those of a V row two of its
// half-words. Half the lanes of a warp hold K rows and half the V rows of the
// same (token, kv head), so both go in one pass.
//
// What bounds it: HBM. A row of 128 elements is 256 bytes read and 80 written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "q4_internal.h"

namespace {

using pkv::launch_chained;

constexpr int kThreads = 256;
constexpr float kMaxHalf = 65504.f;

struct StoreParams {
    const void *k, *v;           // append: new rows; gather: outputs (non-const)
    void *k_out, *v_out;
    const int64_t *slots;
    int64_t rows;                // tokens * Hk
    int Hk, NB, B;
    pkv_q4cache_pools pools;
    unsigned *err;
};

// Lane's place: which of K and V, which row of the warp's, which 8 elements.
// A warp holds 512 / (2 D) rows (2 at D 64, 1 at D 128) of K and of V.
template <int D>
struct Place {
    static constexpr int kLanes = D / 8;              // lanes a row
    static constexpr int kRows = 16 / kLanes;         // (token, kv head) rows a warp
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

// Slot of a row, as chunk (block * Hk + head) and offset; chunk -1: none.
__device__ __forceinline__ void locate(const StoreParams &p, int64_t r, int64_t &chunk, int &off,
                                       bool report) {
    const int64_t tok = r / p.Hk;
    const int g = (int)(r - tok * p.Hk);
    const int64_t slot = p.slots[tok];
    chunk = -1;
    off = 0;
    if (slot < 0) return;
    const int64_t blk = slot / p.B;
    if (blk >= p.NB) {
        if (report && g == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
        return;
    }
    chunk = blk * p.Hk + g;
    off = (int)(slot - blk * p.B);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const Place<D> at;
    constexpr int NG = D / 32;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * at.kRows;
    int64_t r = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * at.kRows + at.row;
    const int64_t last = r - at.row;     // uniform over the warp
    for (int64_t base = last; base < p.rows; base += step, r += step) {
        int64_t chunk = -1;
        int off = 0;
        if (r < p.rows) locate(p, r, chunk, off, at.l == 0 && !at.is_v);
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (chunk >= 0)
            raw = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(at.is_v ? p.v : p.k) +
                                                        r * D) + at.l);
        const T *e = reinterpret_cast<const T *>(&raw);
        float x[8], lo = INFINITY, hi = -INFINITY;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = pkv::Elem<T>::to_f32(e[i]);
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
            bad |= !(fabsf(x[i]) <= 3.402823466e38f);
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
            bad |= __shfl_xor_sync(~0u, (int)bad, o) != 0;
        }
        __half m = __float2half_rn(fminf(fmaxf(lo, -kMaxHalf), kMaxHalf));
        __half s = __float2half_rn(fminf(__fdiv_rn(hi - lo, 15.f), kMaxHalf));
        if (bad) m = s = __ushort_as_half(0x7fff);
        const float mf = __half2float(m), sf = __half2float(s);
        uint32_t word = 0;
        if (sf > 0.f) {                   // not 0, not NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = rintf(__fdiv_rn(x[i] - mf, sf));
                word |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
            }
        }
        if (chunk < 0) continue;
        const int64_t tr = chunk * p.B + off;
        if (!at.is_v) {
            uint32_t *row = reinterpret_cast<uint32_t *>(p.pools.k_codes) + tr * (D / 8);
            row[at.t * NG + at.group] = word;
            if (at.t == 0) {
                __half *par = static_cast<__half *>(p.pools.k_params) + tr * 2 * NG;
                par[at.group] = s;
                par[NG + at.group] = m;
            }
        } else {
            uint16_t *row = reinterpret_cast<uint16_t *>(p.pools.v_codes) + tr * (D / 4);
            row[2 * at.t * NG + at.group] = (uint16_t)word;
            row[(2 * at.t + 1) * NG + at.group] = (uint16_t)(word >> 16);
            if (at.t == 0) {
                __half *par = static_cast<__half *>(p.pools.v_params) + chunk * 2 * NG * p.B + off;
                par[at.group * p.B] = s;
                par[(NG + at.group) * p.B] = m;
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

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const StoreParams p) {
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const Place<D> at;
    constexpr int NG = D / 32;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * at.kRows;
    for (int64_t r = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * at.kRows + at.row;
         r < p.rows; r += step) {
        int64_t chunk;
        int off;
        locate(p, r, chunk, off, at.l == 0 && !at.is_v);
        float x[8] = {};
        if (chunk >= 0) {
            const int64_t tr = chunk * p.B + off;
            uint32_t word;
            __half s, m;
            if (!at.is_v) {
                word = (static_cast<const uint32_t *>(p.pools.k_codes) + tr * (D / 8))[at.t * NG + at.group];
                const __half *par = static_cast<const __half *>(p.pools.k_params) + tr * 2 * NG;
                s = par[at.group];
                m = par[NG + at.group];
            } else {
                const uint16_t *row = static_cast<const uint16_t *>(p.pools.v_codes) + tr * (D / 4);
                word = row[2 * at.t * NG + at.group] |
                       (uint32_t)row[(2 * at.t + 1) * NG + at.group] << 16;
                const __half *par =
                    static_cast<const __half *>(p.pools.v_params) + chunk * 2 * NG * p.B + off;
                s = par[at.group * p.B];
                m = par[(NG + at.group) * p.B];
            }
            const float sf = __half2float(s), mf = __half2float(m);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((word >> (4 * i)) & 15u), sf, mf);
        }
        store8(static_cast<T *>(at.is_v ? p.v_out : p.k_out) + r * D + at.l * 8, x);
    }
}

bool misaligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

dim3 grid_for(int64_t rows, int D) {
    const int64_t per_cta = (kThreads / 32) * (D == 64 ? 2 : 1);
    int64_t g = (rows + per_cta - 1) / per_cta;
    return dim3((unsigned)(g > 16384 ? 16384 : g));
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
    p->slots = slots;
    p->rows = (int64_t)T * cache->num_kv_heads;
    p->Hk = cache->num_kv_heads;
    p->NB = cache->num_blocks;
    p->B = cache->block_size;
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
    auto *kernel = d64 ? (h ? &append_q4_kernel<64, __half> : &append_q4_kernel<64, __nv_bfloat16>)
                       : (h ? &append_q4_kernel<128, __half> : &append_q4_kernel<128, __nv_bfloat16>);
    return launch_failed(launch_chained(kernel, grid_for(p.rows, cache->head_dim), kThreads, 0,
                                        static_cast<cudaStream_t>(stream), p), "append_q4");
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
    auto *kernel = out_dtype == PKV_F32
                       ? (d64 ? &gather_q4_kernel<64, float> : &gather_q4_kernel<128, float>)
                   : out_dtype == PKV_F16
                       ? (d64 ? &gather_q4_kernel<64, __half> : &gather_q4_kernel<128, __half>)
                       : (d64 ? &gather_q4_kernel<64, __nv_bfloat16>
                              : &gather_q4_kernel<128, __nv_bfloat16>);
    return launch_failed(launch_chained(kernel, grid_for(p.rows, cache->head_dim), kThreads, 0,
                                        static_cast<cudaStream_t>(stream), p), "gather_q4");
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

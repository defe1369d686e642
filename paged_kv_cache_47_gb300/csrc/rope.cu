// Rotary positions, alone or with the append (include/pkv_rope.h).
//
// A CTA takes one token (or one part of its heads, when tokens are few): its
// first threads compute the token's cosines and sines once, into shared
// memory, and all threads then turn heads. The angle is exact: the plan's
// fraction of a turn (64-bit fixed point) times the position modulo 2^64, so
// one integer multiply replaces the range reduction and far positions cost
// and lose nothing. It becomes fp32 in units of pi, for sincospif.
//
// Work item: 32 bytes of one head, read as two 16-byte vectors and written as
// two. PKV_ROPE_HALF: the vectors of the pairs' two members; INTERLEAVED and
// the part past rotary_dim: neighbours. A thread reads both before it writes
// either, so outputs may be the inputs. Rotary sizes that do not fill vectors
// take a form with two elements an item.
//
// What bounds it: HBM. Every element is read once and written once: 8191 tokens
// of 40 q and 40 kv heads of 128 with the append (fp16, 503 MB in all) take
// 74.5 us, 6.75 TB/s. A step of 64 tokens is a launch and two dependent loads:
// 4.3 us, the host's call, and 2.5 replayed as a graph.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/pkv_rope.h"
#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"

namespace {

using pkv::launch_chained;

constexpr int kThreads = 256;

struct RopeParams {
    const int32_t *pos;
    const int64_t *slots;        // with the append; else NULL
    const void *q, *k, *v;       // v: with the append only
    void *q_out, *k_out, *v_out; // k_out, v_out: the pools with the append
    int64_t q_st, k_st, v_st, qo_st, ko_st;   // strides, elements
    int T, Hq, Hk, D;
    int NB, B;
    int parts;                   // CTAs a token
    unsigned *err;
    pkv_rope_plan plan;
};

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T>
union Vec {
    uint4 raw;
    T e[16 / sizeof(T)];
};

// One pair turned; the fused multiply-adds keep each output at two roundings.
template <typename T>
__device__ __forceinline__ void turn(T &a, T &b, float2 cs) {
    const float x = pkv::Elem<T>::to_f32(a), y = pkv::Elem<T>::to_f32(b);
    a = from_f32<T>(fmaf(x, cs.x, -y * cs.y));
    b = from_f32<T>(fmaf(y, cs.x, x * cs.y));
}

// Two vectors of one head: item j of head row src, to dst.
template <typename T>
__device__ __forceinline__ void do_vectors(const T *src, T *dst, int j, bool rotate, int rd,
                                           bool half, const float2 *cs) {
    constexpr int V = 16 / sizeof(T);
    int a = 2 * j * V, b = a + V;             // neighbours
    const bool in = rotate && a < rd;
    if (in && half) {
        a = j * V;
        b = a + rd / 2;
    }
    Vec<T> x, y;
    x.raw = *reinterpret_cast<const uint4 *>(src + a);
    y.raw = *reinterpret_cast<const uint4 *>(src + b);
    if (in) {
        if (half) {
#pragma unroll
            for (int i = 0; i < V; ++i) turn(x.e[i], y.e[i], cs[a + i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) turn(x.e[i], x.e[i + 1], cs[(a + i) / 2]);
            if (b < rd) {
#pragma unroll
                for (int i = 0; i < V; i += 2) turn(y.e[i], y.e[i + 1], cs[(b + i) / 2]);
            }
        }
    }
    *reinterpret_cast<uint4 *>(dst + a) = x.raw;
    *reinterpret_cast<uint4 *>(dst + b) = y.raw;
}

// Two elements of one head: pair j, or two neighbours past rotary_dim.
template <typename T>
__device__ __forceinline__ void do_pair(const T *src, T *dst, int j, bool rotate, int rd, bool half,
                                        const float2 *cs) {
    int a = 2 * j, b = a + 1;
    const bool in = rotate && a < rd;
    if (in && half) {
        a = j;
        b = j + rd / 2;
    }
    T x = src[a], y = src[b];
    if (in) turn(x, y, cs[j]);
    dst[a] = x;
    dst[b] = y;
}

template <typename T, bool VECTORS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[PKV_ROPE_MAX_PAIRS];
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    const int tok = blockIdx.x / p.parts, part = blockIdx.x - tok * p.parts;
    const int rd = p.plan.rotary_dim;
    if (threadIdx.x < rd / 2) {
        const unsigned long long u = (unsigned long long)(long long)p.pos[tok] *
                                     p.plan.turns[threadIdx.x];
        // signed: half a turn either way, in units of pi
        float s, c;
        sincospif(__ll2float_rn((long long)u) * 0x1p-63f, &s, &c);
        cs[threadIdx.x] = make_float2(c * p.plan.amplitude, s * p.plan.amplitude);
    }
    int64_t row = -1;                          // (block * Hk) * B + offset
    if (p.slots) {
        const int64_t slot = p.slots[tok];
        if (slot >= 0) {
            const int64_t blk = slot / p.B;
            if (blk < p.NB) row = blk * p.Hk * p.B + (slot - blk * p.B);
            else if (part == 0 && threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
        }
    }
    __syncthreads();
    const bool half = p.plan.layout == PKV_ROPE_HALF;
    const int per_head = VECTORS ? p.D * (int)sizeof(T) / 32 : p.D / 2;
    const int heads = p.Hq + p.Hk + (p.slots ? p.Hk : 0);
    const int items = heads * per_head;
    for (int i = part * kThreads + threadIdx.x; i < items; i += p.parts * kThreads) {
        int h = i / per_head;
        const int j = i - h * per_head;
        const T *src;
        T *dst;
        bool rotate = true;
        if (h < p.Hq) {
            src = static_cast<const T *>(p.q) + tok * p.q_st + (int64_t)h * p.D;
            dst = static_cast<T *>(p.q_out) + tok * p.qo_st + (int64_t)h * p.D;
        } else {
            h -= p.Hq;
            rotate = h < p.Hk;
            if (!rotate) h -= p.Hk;
            src = rotate ? static_cast<const T *>(p.k) + tok * p.k_st
                         : static_cast<const T *>(p.v) + tok * p.v_st;
            src += (int64_t)h * p.D;
            dst = static_cast<T *>(rotate ? p.k_out : p.v_out);
            if (p.slots) {
                if (row < 0) continue;
                dst += (row + (int64_t)h * p.B) * p.D;
            } else {
                dst += tok * p.ko_st + (int64_t)h * p.D;
            }
        }
        if (VECTORS) do_vectors<T>(src, dst, j, rotate, rd, half, cs);
        else do_pair<T>(src, dst, j, rotate, rd, half, cs);
    }
}

bool misaligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

template <typename T>
cudaError_t launch(RopeParams &p, int sms, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int rd = p.plan.rotary_dim;
    const bool vectors = rd % (2 * V) == 0 || (p.plan.layout == PKV_ROPE_INTERLEAVED && rd % V == 0);
    const int heads = p.Hq + p.Hk + (p.slots ? p.Hk : 0);
    const int items = heads * (vectors ? p.D * (int)sizeof(T) / 32 : p.D / 2);
    // few tokens: several CTAs a token, one item a thread
    int parts = (items + kThreads - 1) / kThreads;
    const int wanted = 2 * sms / (p.T < 2 * sms ? p.T : 2 * sms);
    if (parts > wanted) parts = wanted;
    p.parts = parts;
    const dim3 grid((unsigned)(p.T * parts));
    return vectors ? launch_chained(rope_kernel<T, true>, grid, kThreads, 0, stream, p)
                   : launch_chained(rope_kernel<T, false>, grid, kThreads, 0, stream, p);
}

pkv_status run(int dtype, RopeParams &p, void *stream) {
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    const pkv_status st = pkv::device_sm_count(&sms);
    if (st != PKV_OK) return st;
    const cudaError_t e = dtype == PKV_F32   ? launch<float>(p, sms, s)
                          : dtype == PKV_F16 ? launch<__half>(p, sms, s)
                                             : launch<__nv_bfloat16>(p, sms, s);
    if (e != cudaSuccess)
        return pkv::set_last_error(PKV_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

pkv_status check_plan(const pkv_rope_plan *plan, int D) {
    if (!plan) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "the plan is NULL");
    if (plan->rotary_dim < 2 || plan->rotary_dim > 2 * PKV_ROPE_MAX_PAIRS || plan->rotary_dim % 2 ||
        (plan->layout != PKV_ROPE_HALF && plan->layout != PKV_ROPE_INTERLEAVED))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "not a plan of pkv_rope_plan_init");
    if (plan->rotary_dim > D)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "rotary_dim %d above head_dim %d",
                                   plan->rotary_dim, D);
    return PKV_OK;
}

// One strided tensor of `heads` heads a token.
pkv_status check_rows(const char *name, const void *ptr, int64_t stride, int heads, int D, int es) {
    if (!ptr) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "%s is NULL", name);
    if (misaligned(ptr) || stride * es % 16)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "%s: pointer and stride must be multiples of 16 bytes", name);
    if (stride < (int64_t)heads * D)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "%s: stride %lld below %d heads of %d", name,
                                   (long long)stride, heads, D);
    return PKV_OK;
}

pkv_status check_heads(int T, int Hq, int Hk) {
    if (T < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", T);
    if (T > INT32_MAX / 512)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_tokens %d too large for one launch", T);
    if (Hq < 0 || Hk < 0 || Hq > 65536 || Hk > 65536)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "head counts %d, %d", Hq, Hk);
    return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_plan_init(const pkv_rope_desc *d, pkv_rope_plan *plan) {
    if (!d || !plan) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    const int rd = d->rotary_dim;
    if (rd < 2 || rd > 2 * PKV_ROPE_MAX_PAIRS || rd % 2)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "rotary_dim %d (even, 2..%d)", rd,
                                   2 * PKV_ROPE_MAX_PAIRS);
    if (d->layout != PKV_ROPE_HALF && d->layout != PKV_ROPE_INTERLEAVED)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "layout %d", d->layout);
    if (d->scaling < PKV_ROPE_NONE || d->scaling > PKV_ROPE_YARN)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "scaling %d", d->scaling);
    if (!(d->base > 1) || !isfinite(d->base))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "base must be above 1");
    const int sc = d->scaling;
    const double f = sc == PKV_ROPE_NONE ? 1.0 : d->factor;
    if (!(f > 0) || !isfinite(f)) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "factor must be above 0");
    if ((sc == PKV_ROPE_BANDS || sc == PKV_ROPE_YARN) && d->original_len < 1)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "original_len %d", d->original_len);
    if (sc == PKV_ROPE_BASE && rd < 4)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "base scaling needs rotary_dim of 4 or more");
    if (sc == PKV_ROPE_BANDS && (!(d->low_freq_factor > 0) || !(d->high_freq_factor > d->low_freq_factor) ||
                                 !isfinite(d->high_freq_factor)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "band factors must satisfy 0 < low < high");
    if (sc == PKV_ROPE_YARN && (!(d->beta_slow > 0) || !(d->beta_fast >= d->beta_slow) ||
                                !isfinite(d->beta_fast) || !isfinite(d->attention_factor)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "betas must satisfy beta_fast >= beta_slow > 0");

    const double kTwoPi = 6.283185307179586476925286766559;
    const double base = sc == PKV_ROPE_BASE ? d->base * pow(f, (double)rd / (rd - 2)) : d->base;
    if (!(base > 1) || !isfinite(base))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "the scaled base must be finite and above 1");
    double lo = 0, hi = 0;
    if (sc == PKV_ROPE_YARN) {
        const double n = d->original_len;
        lo = floor(rd * log(n / (kTwoPi * d->beta_fast)) / (2 * log(base)));
        hi = ceil(rd * log(n / (kTwoPi * d->beta_slow)) / (2 * log(base)));
        lo = lo < 0 ? 0 : lo;
        hi = hi > rd - 1 ? rd - 1 : hi;
    }
    memset(plan, 0, sizeof(*plan));
    plan->rotary_dim = rd;
    plan->layout = d->layout;
    plan->amplitude = 1.f;
    if (sc == PKV_ROPE_YARN)
        plan->amplitude = (float)(d->attention_factor != 0 ? d->attention_factor : f > 1 ? 0.1 * log(f) + 1 : 1);
    for (int i = 0; i < rd / 2; ++i) {
        double w = pow(base, -2.0 * i / rd), t;
        switch (sc) {
            case PKV_ROPE_LINEAR: w /= f; break;
            case PKV_ROPE_BANDS:
                t = (d->original_len * w / kTwoPi - d->low_freq_factor) /
                    (d->high_freq_factor - d->low_freq_factor);
                t = t < 0 ? 0 : t > 1 ? 1 : t;
                w = t * w + (1 - t) * w / f;
                break;
            case PKV_ROPE_YARN:
                t = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
                t = t < 0 ? 0 : t > 1 ? 1 : t;
                w = (1 - t) * w + t * w / f;
                break;
            default: break;
        }
        // a fraction of a turn; whole turns (factors below 1) drop out
        double turns = w / kTwoPi;
        turns -= floor(turns);
        plan->turns[i] = (uint64_t)rint(ldexp(turns, 64));      // (turns < 1: below 2^64)
    }
    return PKV_OK;
}

pkv_status pkv_rope(int32_t dtype, int32_t head_dim, const pkv_rope_plan *plan,
                    const int32_t *positions, int32_t num_tokens, const void *q, int64_t q_stride,
                    int32_t num_q_heads, void *q_out, int64_t q_out_stride, const void *k,
                    int64_t k_stride, int32_t num_kv_heads, void *k_out, int64_t k_out_stride,
                    void *stream) {
    if (dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "dtype %d", dtype);
    if (head_dim != 64 && head_dim != 128)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
    pkv_status st = check_plan(plan, head_dim);
    if (st != PKV_OK) return st;
    if ((st = check_heads(num_tokens, num_q_heads, num_kv_heads)) != PKV_OK) return st;
    if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PKV_OK;
    const int es = dtype == PKV_F32 ? 4 : 2;
    if (!positions) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(positions) % 4)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    if (num_q_heads) {
        if ((st = check_rows("q", q, q_stride, num_q_heads, head_dim, es)) != PKV_OK) return st;
        if ((st = check_rows("q_out", q_out, q_out_stride, num_q_heads, head_dim, es)) != PKV_OK)
            return st;
    }
    if (num_kv_heads) {
        if ((st = check_rows("k", k, k_stride, num_kv_heads, head_dim, es)) != PKV_OK) return st;
        if ((st = check_rows("k_out", k_out, k_out_stride, num_kv_heads, head_dim, es)) != PKV_OK)
            return st;
    }
    if ((num_q_heads && q == q_out && q_stride != q_out_stride) ||
        (num_kv_heads && k == k_out && k_stride != k_out_stride))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "in place needs equal strides");
    RopeParams p = {};
    p.pos = positions;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_st = q_stride;
    p.k_st = k_stride;
    p.qo_st = q_out_stride;
    p.ko_st = k_out_stride;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hk = num_kv_heads;
    p.D = head_dim;
    p.plan = *plan;
    return run(dtype, p, stream);
}

pkv_status pkv_rope_append(const pkv_cache_desc *cache, const pkv_rope_plan *plan,
                           const int32_t *positions, const int64_t *slot_mapping,
                           int32_t num_tokens, const void *q, int64_t q_stride,
                           int32_t num_q_heads, void *q_out, int64_t q_out_stride,
                           const void *k_new, int64_t k_stride, const void *v_new,
                           int64_t v_stride, void *k_pool, void *v_pool, void *stream) {
    pkv_status st = pkv::check_cache_desc(cache);
    if (st != PKV_OK) return st;
    if ((st = check_plan(plan, cache->head_dim)) != PKV_OK) return st;
    const int D = cache->head_dim, Hk = cache->num_kv_heads, es = cache->dtype == PKV_F32 ? 4 : 2;
    if ((st = check_heads(num_tokens, num_q_heads, Hk)) != PKV_OK) return st;
    if (num_tokens == 0) return PKV_OK;
    if (!positions || !slot_mapping || !k_pool || !v_pool)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    if (reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(slot_mapping) % 8 ||
        misaligned(k_pool) || misaligned(v_pool))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "pools must be 16-byte aligned (slot_mapping 8, positions 4)");
    if (num_q_heads) {
        if ((st = check_rows("q", q, q_stride, num_q_heads, D, es)) != PKV_OK) return st;
        if ((st = check_rows("q_out", q_out, q_out_stride, num_q_heads, D, es)) != PKV_OK) return st;
        if (q == q_out && q_stride != q_out_stride)
            return pkv::set_last_error(PKV_ERR_INVALID_ARG, "in place needs equal strides");
    }
    if ((st = check_rows("k_new", k_new, k_stride, Hk, D, es)) != PKV_OK) return st;
    if ((st = check_rows("v_new", v_new, v_stride, Hk, D, es)) != PKV_OK) return st;
    RopeParams p = {};
    if ((st = pkv::device_error_word(&p.err)) != PKV_OK) return st;
    p.pos = positions;
    p.slots = slot_mapping;
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.q_out = q_out;
    p.k_out = k_pool;
    p.v_out = v_pool;
    p.q_st = q_stride;
    p.k_st = k_stride;
    p.v_st = v_stride;
    p.qo_st = q_out_stride;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hk = Hk;
    p.D = D;
    p.NB = cache->num_blocks;
    p.B = cache->block_size;
    p.plan = *plan;
    return run(cache->dtype, p, stream);
}

}  // extern "C"

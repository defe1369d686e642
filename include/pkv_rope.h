/*
 * pkv_rope.h — rotary positions, alone or with the append.
 *
 * A head x of head_dim elements at position p has its first rotary_dim
 * elements turned in pairs (x_a, x_b), i < rotary_dim / 2:
 *   y_a = x_a cos(p w_i) - x_b sin(p w_i)
 *   y_b = x_b cos(p w_i) + x_a sin(p w_i)
 * with (a, b) = (i, i + rotary_dim / 2) for PKV_ROPE_HALF and (2i, 2i + 1) for
 * PKV_ROPE_INTERLEAVED; the elements from rotary_dim on are copied. Cosine and
 * sine are multiplied by the plan's amplitude. Arithmetic in fp32, one
 * rounding to the output type.
 *
 * Frequencies, w_i = base^(-2 i / rotary_dim) before scaling, f = factor,
 * n = original_len:
 *   PKV_ROPE_NONE    w_i
 *   PKV_ROPE_LINEAR  w_i / f (positions divided by f)
 *   PKV_ROPE_BASE    base replaced by base * f^(rotary_dim / (rotary_dim - 2))
 *   PKV_ROPE_BANDS   by wavelength: with r_i = n w_i / (2 pi) turns over the
 *                    original length and t = clamp((r_i - low) / (high - low), 0, 1)
 *                    for low, high = low_freq_factor, high_freq_factor:
 *                    t w_i + (1 - t) w_i / f
 *   PKV_ROPE_YARN    by dimension: d(r) = rotary_dim ln(n / (2 pi r)) / (2 ln base),
 *                    lo = max(floor d(beta_fast), 0), hi = min(ceil d(beta_slow),
 *                    rotary_dim - 1), u = clamp((i - lo) / max(hi - lo, 0.001), 0, 1):
 *                    (1 - u) w_i + u w_i / f; amplitude attention_factor, or
 *                    0.1 ln(f) + 1 where that is 0 (1 for f <= 1)
 *
 * The angle of a far position would lose its low bits in fp32, so the plan
 * holds each w_i as a fraction of a turn in 64-bit fixed point: position times
 * fraction modulo 2^64 is the angle modulo one turn, without rounding. The
 * fraction itself is off by a few roundings of 2^-53 of its value (it is
 * computed in double) and 2^-65, below 2^-30 turns at position 2^21.
 */
#ifndef PKV_ROPE_H
#define PKV_ROPE_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PKV_ROPE_HALF = 0, PKV_ROPE_INTERLEAVED = 1 } pkv_rope_layout;
typedef enum {
    PKV_ROPE_NONE = 0,
    PKV_ROPE_LINEAR = 1,
    PKV_ROPE_BASE = 2,
    PKV_ROPE_BANDS = 3,
    PKV_ROPE_YARN = 4
} pkv_rope_scaling;

typedef struct {
    int32_t rotary_dim;       /* even, 2..128 (BASE: at least 4)                  */
    int32_t layout;           /* pkv_rope_layout                                  */
    int32_t scaling;          /* pkv_rope_scaling                                 */
    int32_t original_len;     /* BANDS, YARN: >= 1                                */
    double base;              /* > 1                                              */
    double factor;            /* > 0; not read by NONE                            */
    double low_freq_factor;   /* BANDS: 0 < low < high                            */
    double high_freq_factor;
    double beta_fast;         /* YARN: beta_fast >= beta_slow > 0                 */
    double beta_slow;
    double attention_factor;  /* YARN: 0 = from factor                            */
} pkv_rope_desc;

#define PKV_ROPE_MAX_PAIRS 64

/* What the kernels read, made once on the host by pkv_rope_plan_init and passed
 * by pointer to host memory; calls copy it into the launch. */
typedef struct {
    int32_t rotary_dim;
    int32_t layout;
    float amplitude;
    int32_t reserved;
    uint64_t turns[PKV_ROPE_MAX_PAIRS];  /* round(w_i / (2 pi) * 2^64) */
} pkv_rope_plan;

/* Fill *plan from *desc (host only; no device is needed). */
pkv_status pkv_rope_plan_init(const pkv_rope_desc *desc, pkv_rope_plan *plan);

/*
 * pkv_rope — rotate q and k.
 *
 * Token t's heads start at q + t * q_stride (strides in elements, so that q
 * and k may be parts of one projection's output), head h at h * head_dim from
 * there; k, q_out and k_out alike. q_out may be q and k_out may be k (same
 * stride); otherwise outputs do not overlap inputs. positions: device int32
 * [num_tokens], any value. num_q_heads or num_kv_heads 0: that side is left
 * out (its pointers are not read). dtype: of all four. Pointers 16-byte
 * aligned, strides multiples of 16 bytes, at least heads * head_dim.
 * head_dim 64 or 128.
 */
pkv_status pkv_rope(int32_t dtype, int32_t head_dim, const pkv_rope_plan *plan,
                    const int32_t *positions, int32_t num_tokens, const void *q, int64_t q_stride,
                    int32_t num_q_heads, void *q_out, int64_t q_out_stride, const void *k,
                    int64_t k_stride, int32_t num_kv_heads, void *k_out, int64_t k_out_stride,
                    void *stream);

/*
 * pkv_rope_append — pkv_rope and pkv_append in one launch: q turned into q_out
 * ([num_tokens][num_q_heads][head_dim], stride q_out_stride), k turned and v
 * copied to their slots. The pool bytes equal pkv_rope followed by pkv_append.
 * Tokens with a negative slot get q_out and write no cache row; a slot past
 * the pool sets PKV_DEVERR_SLOT and is skipped. Slots are unique per call.
 * Checks and types as pkv_rope and pkv_append.
 */
pkv_status pkv_rope_append(const pkv_cache_desc *cache, const pkv_rope_plan *plan,
                           const int32_t *positions, const int64_t *slot_mapping,
                           int32_t num_tokens, const void *q, int64_t q_stride,
                           int32_t num_q_heads, void *q_out, int64_t q_out_stride,
                           const void *k_new, int64_t k_stride, const void *v_new,
                           int64_t v_stride, void *k_pool, void *v_pool, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_ROPE_H */

/*
 * pkv_q4.h — a KV cache held in 4 bits.
 *
 * Passage: fewer bits per cached element are the lever that cuts the bytes
 * each decode step reads ("Contiguous vs Paged KV Cache on RDNA4", section
 * "The order of the memory levers"). The pages fix no format; this library's
 * 4-bit one is 5 bits an element in all:
 *
 * Each row of head_dim activations is cut into NG = head_dim / 32 groups of 32
 * neighbouring elements. A group has a scale s >= 0 and a minimum m, both
 * fp16, and element d of group y = d / 32 has a code c in 0..15:
 *   value = s * c + m
 *   m = fp16(min), s = fp16((max - min) * r), c = round((x - m) / s)
 * with r the fp32 number nearest 1 / 15 (differences, products, quotients and
 * the rounding to the nearest code in fp32, ties to even, clamped to 0..15;
 * s = 0 gives code 0). min and (max - min) * r are clamped to +-65504 before
 * they are rounded. A group that holds an infinity
 * or a NaN gets s = m = NaN and zero codes, so that it is not hidden.
 *
 *   k_codes   [num_blocks][num_kv_heads][block_size][head_dim / 2] uint8
 *             a row's 32-bit word w = (d % 32 / 8) * NG + y holds element d in
 *             bits 4 (d % 8) .. + 3
 *   v_codes   same shape; a row's 16-bit half-word h = (d % 32 / 4) * NG + y
 *             holds element d in bits 4 (d % 4) .. + 3
 *   k_params  [num_blocks][num_kv_heads][block_size][2 NG] fp16: s of each
 *             group, then m of each group
 *   v_params  [num_blocks][num_kv_heads][2 NG][block_size] fp16: the same,
 *             transposed within the block
 *
 * The word orders put what one thread feeds to the matrix instructions side by
 * side. q, k_new and v_new are PKV_F16 or PKV_BF16.
 */
#ifndef PKV_Q4_H
#define PKV_Q4_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t num_blocks;    /* >= 1                                             */
    int32_t block_size;    /* 8, 16 or 32                                      */
    int32_t num_kv_heads;  /* >= 1                                             */
    int32_t head_dim;      /* 64 or 128                                        */
    int32_t act_dtype;     /* PKV_F16 or PKV_BF16: q, k_new, v_new             */
} pkv_q4cache_desc;

/* The four pools, device memory, each 16-byte aligned. */
typedef struct {
    void *k_codes, *v_codes;
    void *k_params, *v_params;
} pkv_q4cache_pools;

/*
 * pkv_append_q4 — pkv_append for a 4-bit cache: quantizes row i of k_new and
 * v_new ([num_tokens][num_kv_heads][head_dim], 16-byte aligned) to
 * slot_mapping[i]. Negative slots are skipped, a slot past the pool sets
 * PKV_DEVERR_SLOT and is skipped, slots are unique per call. Codes and
 * parameters equal the rule above bit for bit.
 */
pkv_status pkv_append_q4(const pkv_q4cache_desc *cache, const void *k_new, const void *v_new,
                         const int64_t *slot_mapping, int32_t num_tokens,
                         const pkv_q4cache_pools *pools, void *stream);

/*
 * pkv_gather_q4 — cached rows as values: row i of k_out and v_out
 * ([num_tokens][num_kv_heads][head_dim], 16-byte aligned, out_dtype PKV_F32,
 * PKV_F16 or PKV_BF16) is the cached row at slot_mapping[i], s * c + m in fp32
 * rounded once. A negative slot gives zeros, a slot past the pool zeros and
 * PKV_DEVERR_SLOT. The same slot may be named more than once.
 */
pkv_status pkv_gather_q4(const pkv_q4cache_desc *cache, const pkv_q4cache_pools *pools,
                         const int64_t *slot_mapping, int32_t num_tokens, void *k_out,
                         void *v_out, int32_t out_dtype, void *stream);

/* Workspace bytes for pkv_decode_attention_q4 with num_ctas CTAs (0 = the
 * default launch); 0 on invalid arguments. Independent of the batch. */
size_t pkv_decode_q4_workspace_bytes(const pkv_q4cache_desc *cache, int32_t num_q_heads,
                                     int32_t num_ctas);

/*
 * pkv_decode_attention_q4 — pkv_decode_attention_ex over a 4-bit cache:
 * out[s][h] = softmax(scale * q K^T) V with K and V the cached values. q:
 * [num_seqs][num_q_heads][head_dim] in act_dtype. Tables, lengths, out
 * (aligned to four of its elements), the workspace (zero-filled before first
 * use, not shared by calls that may overlap) and errors as there. A
 * row that holds NaN parameters gives NaN where it is attended to; rows past a
 * context's length are not used, whatever they hold. options: num_ctas,
 * tables_ready (not with tables that pkv_tables_append wrote on the stream),
 * lse_out and timing_events apply; pending_tail is accepted and every other read
 * waits for the preceding kernel; consumer 1 (CUDA-core math) is
 * PKV_ERR_UNSUPPORTED.
 *
 * Sums are in fp32. Operands of fewer bits: weights, weights times V scales and
 * the sums of q that meet the minima are pairs of fp16 (22 bits); q times a power
 * of two is one fp16, exact for elements down to 2^-28 of the head's largest.
 */
pkv_status pkv_decode_attention_q4(const pkv_q4cache_desc *cache, const void *q, int32_t num_seqs,
                                   int32_t num_q_heads, const pkv_q4cache_pools *pools,
                                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                                   const int32_t *context_lens, float scale, void *out,
                                   int32_t out_dtype, void *workspace, size_t workspace_bytes,
                                   void *stream, const pkv_decode_options *options);

/* pkv_block_copy for a 4-bit cache: codes and parameters of whole blocks. */
pkv_status pkv_block_copy_q4(const pkv_q4cache_desc *cache, const int64_t *src_dst_pairs,
                             int32_t num_pairs, const pkv_q4cache_pools *pools, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_Q4_H */

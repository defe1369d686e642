/*
 * pkv_tree.h — a decode step that verifies drafted tokens.
 *
 * Several tokens a sequence are drafted by some cheaper means and put through
 * the model together; the model's answers confirm one branch of them. They
 * form a tree: each drafted token has a parent before it among its sequence's
 * tokens, or -1 (the token that is already decided, or the first of several
 * candidates). One attention over the cache then serves all of them, which
 * reads each K/V byte once for many queries: on long contexts the decode's
 * time is those bytes ("Contiguous vs Paged KV Cache on RDNA4", section "The
 * order of the memory levers").
 *
 * The batch's drafted tokens lie one sequence after another, sequence s at
 * rows token_offsets[s] .. token_offsets[s + 1] - 1 (what pkv_tables_append
 * writes for new_tokens[s] of them). In the cache they are the last n of the
 * sequence's L = context_lens[s] tokens, at places P .. L - 1, P = L - n: they
 * are appended first, and context_lens counts them. The tree is:
 *   parents  int32 [num_tokens]  -1, or the place among the sequence's drafted
 *                                tokens of one before it
 *   masks    [num_tokens][mask_words] 64-bit words; bit j of a token's words
 *            (word j / 64) tells that it sees the sequence's j-th drafted
 *            token. pkv_tree_plan makes each token see itself and those above
 *            it; any other masks are allowed.
 *
 * A step: pkv_tables_append (n tokens a sequence), pkv_tree_plan, then for
 * each layer the rotary append and pkv_decode_attention_tree, then
 * pkv_tree_accept, for each layer pkv_tree_commit, and pkv_tables_truncate
 * (pkv_tables.h) for the blocks behind the accepted tokens.
 *
 * Device values are checked by the kernels, which set bits of the device
 * error word (pkv_get_error):
 *   PKV_DEVERR_CONTEXT  a length < 0 or past the table's row
 *   PKV_DEVERR_TOKENS   offsets that descend or leave [0, num_tokens], more
 *                       tokens than max_tree (64 * mask_words) or than the
 *                       sequence holds
 *   PKV_DEVERR_TREE     a parent that is not before its token, a path that
 *                       does not ascend
 * A sequence with a bad length or offset is left out: what the calls would
 * write for it stays as it was, unless a call says otherwise. Rows from
 * token_offsets[num_seqs] on are left as they were.
 */
#ifndef PKV_TREE_H
#define PKV_TREE_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_TREE_MAX_TOKENS 256   /* drafted tokens of a sequence, at most */
#define PKV_TREE_MAX_AXES 4

/*
 * pkv_tree_plan — masks and positions of drafted tokens.
 *
 * For drafted token i of sequence s, with depth_i the number of tokens above it:
 *   masks[o_s + i]                     = bits of i and of the tokens above it
 *   positions[a * num_tokens + o_s + i] = P + position_deltas[s] + depth_i
 * for each axis a < num_axes (1: what pkv_rope_append takes; several: what
 * pkv_rope_axes_append takes; text has one position on all axes).
 * position_deltas: NULL, or int32 [num_seqs], how far a sequence's positions
 * run ahead of its places (after a picture they do not advance token by
 * token). parents: NULL for chains (the parent of i is i - 1). masks: NULL, or
 * [num_tokens][mask_words], mask_words 1..4; it bounds n by 64 * mask_words
 * with masks NULL too. positions: NULL, or int32 [num_axes][num_tokens]. A bad
 * parent counts as -1.
 */
pkv_status pkv_tree_plan(int32_t num_seqs, int32_t num_tokens, const int32_t *parents,
                         const int32_t *token_offsets, const int32_t *context_lens,
                         const int32_t *position_deltas, uint64_t *masks, int32_t mask_words,
                         int32_t *positions, int32_t num_axes, void *stream);

typedef struct {
    int32_t num_ctas;   /* CTAs of the attention kernel, 0..PKV_MAX_DECODE_CTAS; 0 = its default */
    int32_t reserved;
    float *lse_out;     /* optional device [num_tokens][num_q_heads] fp32: log2 of the softmax
                           denominator of each row (-inf for a row that sees nothing)          */
} pkv_tree_options;

/* Bytes of workspace pkv_decode_attention_tree needs on the current device; 0
 * on invalid arguments. It must be zero-filled before its first use: it begins
 * with counters of the pieces that are to be joined (a region of one size,
 * whatever the call), which every call leaves zero (but for one that sets
 * PKV_DEVERR_TIMEOUT: zero the workspace again after it). Calls that may overlap
 * need one each. */
size_t pkv_decode_tree_workspace_bytes(const pkv_cache_desc *cache, int32_t num_q_heads,
                                       int32_t max_tree, int32_t num_ctas);

/*
 * pkv_decode_attention_tree — attention of all drafted tokens over the cache.
 *
 * For drafted token i of sequence s and q head h (kv head g = h / G):
 *   z_t = scale * <q[o_s + i][h], K_t> for the t < P, and the t = P + j of the
 *         drafted tokens j < n that its mask shows,
 *         K_t = k_pool[tab[s][t / B]][g][t % B]
 *   out[o_s + i][h] = sum_t softmax(z)_t * V_t
 * in fp32 accumulation, written in out_dtype. A row that sees nothing is zeros.
 * What a row does not see never reaches it, whatever the pool holds there
 * (infinities and NaN included).
 * masks: NULL for chains (i sees j <= i). q, out: [num_tokens][num_q_heads]
 * [head_dim], q and the pools in the cache's dtype and 16-byte aligned, out
 * 32-byte aligned. max_tree: drafted tokens of a sequence at
 * most, 1..PKV_TREE_MAX_TOKENS (and 64 * mask_words with masks); it sizes the
 * work, so a bound near the truth is best (and so is a table's width: trees of more
 * than 128 rows a kv head are cut up by it). Block ids outside the pool set
 * PKV_DEVERR_BLOCK_ID and read as zeros. workspace: 32-byte aligned, at least
 * pkv_decode_tree_workspace_bytes. options: NULL for the defaults.
 */
pkv_status pkv_decode_attention_tree(const pkv_cache_desc *cache, const void *q,
                                     int32_t num_tokens, int32_t num_q_heads, const void *k_pool,
                                     const void *v_pool, const int32_t *block_tables,
                                     int32_t num_seqs, int32_t max_blocks_per_seq,
                                     const int32_t *context_lens, const int32_t *token_offsets,
                                     const uint64_t *masks, int32_t mask_words, int32_t max_tree,
                                     float scale, void *out, int32_t out_dtype, void *workspace,
                                     size_t workspace_bytes, void *stream,
                                     const pkv_tree_options *options);

/*
 * pkv_tree_accept — the branch that the model's answers confirm.
 *
 * tokens[o_s + i]: drafted token i; targets[o_s + i]: the token the model
 * answers after it. A token with parent -1 holds; another holds if its parent
 * does and tokens[i] == targets[parent]. The path leads to the deepest token
 * that holds, of several equally deep ones the first:
 *   path[o_s + k]       = place among the drafted tokens of the path's k-th,
 *                         k < counts[s]; -1 from there to n
 *   counts[s]           = tokens of the path (0 for n = 0)
 *   next_tokens[s]      = targets of its last token (-1 for n = 0)
 *   context_lens_out[s] = P + counts[s]
 * A token with a bad parent does not hold. A sequence left out gets count 0,
 * next token -1, and its length as it was. parents NULL: chains. max_tree:
 * 1..PKV_TREE_MAX_TOKENS. context_lens_out may be context_lens (then
 * pkv_tree_commit and pkv_tables_truncate need a copy of the lengths from
 * before); no other buffers overlap.
 */
pkv_status pkv_tree_accept(int32_t num_seqs, int32_t num_tokens, int32_t max_tree,
                           const int32_t *parents, const int32_t *tokens, const int32_t *targets,
                           const int32_t *token_offsets, const int32_t *context_lens,
                           int32_t *path, int32_t *counts, int32_t *next_tokens,
                           int32_t *context_lens_out, void *stream);

/*
 * pkv_tree_commit — move the accepted rows together.
 *
 * For each sequence and k < counts[s] with p = path[o_s + k], K and V of all kv
 * heads: the row at place P + p goes to place P + k, byte-exact, as if all rows
 * were read before any is written. context_lens counts all drafted tokens (the
 * lengths from before pkv_tree_accept). p has to ascend, k <= p < n: from the
 * first that does not, nothing more of the sequence is moved
 * (PKV_DEVERR_TREE); counts[s] outside 0..n sets PKV_DEVERR_TOKENS and moves
 * nothing. A block id outside the pool sets PKV_DEVERR_BLOCK_ID and its row is
 * not moved. Blocks are this sequence's alone.
 */
pkv_status pkv_tree_commit(const pkv_cache_desc *cache, int32_t num_seqs, int32_t num_tokens,
                           int32_t max_tree, const int32_t *path, const int32_t *counts,
                           const int32_t *token_offsets, const int32_t *context_lens,
                           const int32_t *block_tables, int32_t max_blocks_per_seq, void *k_pool,
                           void *v_pool, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_TREE_H */

/*
 * pkv_sparse.h — decode attention over the blocks that a score selects.
 *
 * Passage: on long contexts the decode's time is the bytes of K and V it
 * reads ("Contiguous vs Paged KV Cache on RDNA4", section "The order of the
 * memory levers"). Paging makes a block the natural piece to leave out: here
 * each (sequence, kv head) reads only the blocks whose mean key scores highest
 * for its queries, and always the first and last ones of the context.
 *
 *   k_means [num_blocks][num_kv_heads][head_dim], the cache's dtype: the mean
 *   of a full block's keys (pkv_block_means). Only full blocks' means are read.
 *   They are made from a pool of that dtype: a cache of codes that is to be read
 *   through a selection needs the keys of its last blocks in such a pool too.
 *
 * For sequence s of n = ceil(L / B) blocks and kv head g, blocks j < first and
 * j >= n - last are read always, and of the others the top ones by
 *   score_j = max over the q heads h of g of <q[s][h], k_means[tab[s][j]][g]>
 * ties going to the lower j, a NaN counting as +infinity. Scores are computed
 * in fp32 in one stated order, so that equal inputs select equal blocks:
 * products of eight neighbouring elements are added one after another, then
 * neighbouring sums in pairs, again and again. (16-bit types: product and
 * addition are one fused step, which is the same wherever a product is a normal
 * fp32 number; fp32: two steps.)
 *
 * The selection is written as a block table of its own: sel_tables[s][g]
 * lists, in ascending j, tab[s][j] * num_kv_heads + g, then -1 up to
 * W = top_blocks + first_blocks + last_blocks, and sel_lens[s][g] is the
 * number of tokens they hold (all but the context's last block are full).
 * Because one (block, kv head) chunk of a pool is contiguous, a pool
 * [NB][Hk][B][D] is also a pool [NB * Hk][1][B][D]: with that view, Hk
 * sequences per sequence and the selection as table and lengths, every decode
 * call of this library reads just the selected chunks.
 */
#ifndef PKV_SPARSE_H
#define PKV_SPARSE_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pkv_block_means — mean keys of the blocks that tokens have just filled.
 *
 * For every token i whose slot_mapping[i] is the last of its block, all kv
 * heads: k_means[block][g] = the mean of the block's B keys (added in order in
 * fp32, divided by B, rounded to the cache's dtype). Other slots, negative
 * ones among them, are passed over; a slot past the pool sets PKV_DEVERR_SLOT.
 * Called after the append that wrote the tokens. k_pool, k_means: 16-byte
 * aligned.
 */
pkv_status pkv_block_means(const pkv_cache_desc *cache, const int64_t *slot_mapping,
                           int32_t num_tokens, const void *k_pool, void *k_means, void *stream);

typedef struct {
    int32_t top_blocks;    /* >= 0: blocks taken by score                        */
    int32_t first_blocks;  /* >= 0: always read from the start of the context    */
    int32_t last_blocks;   /* >= 1: always read from its end                     */
} pkv_sparse_select;

/* Bytes of scores that a selection over num_seqs sequences and
 * max_blocks_per_seq table columns needs; 0 on invalid arguments. The memory
 * needs no zero-fill. */
size_t pkv_select_workspace_bytes(const pkv_cache_desc *cache, int32_t num_seqs,
                                  int32_t max_blocks_per_seq);

/*
 * pkv_select_blocks — score the blocks and write the selection.
 *
 * q: [num_seqs][num_q_heads][head_dim] in the cache's dtype. sel_tables: int32
 * [num_seqs][num_kv_heads][W]; sel_lens: int32 [num_seqs][num_kv_heads]. A
 * context length out of range is clamped and sets PKV_DEVERR_CONTEXT; a block
 * id out of range scores as a mean of zeros does, is listed as -1 if selected
 * and sets PKV_DEVERR_BLOCK_ID. num_blocks * num_kv_heads must stay below 2^31.
 */
pkv_status pkv_select_blocks(const pkv_cache_desc *cache, const void *q, int32_t num_seqs,
                             int32_t num_q_heads, const void *k_means,
                             const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *context_lens, const pkv_sparse_select *select,
                             int32_t *sel_tables, int32_t *sel_lens, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Workspace bytes of pkv_decode_attention_sparse; 0 on invalid arguments. */
size_t pkv_decode_sparse_workspace_bytes(const pkv_cache_desc *cache, int32_t num_seqs,
                                         int32_t num_q_heads, int32_t max_blocks_per_seq);

/*
 * pkv_decode_attention_sparse — pkv_select_blocks, then the decode attention
 * over the selection (pkv_decode_attention's contract for q, pools, out and
 * scale; out aligned to four of its elements). sel_tables and sel_lens are
 * outputs too. workspace: at least pkv_decode_sparse_workspace_bytes, 16-byte
 * aligned, zero-filled before its first use; not shared by calls that may
 * overlap.
 */
pkv_status pkv_decode_attention_sparse(const pkv_cache_desc *cache, const void *q,
                                       int32_t num_seqs, int32_t num_q_heads, const void *k_pool,
                                       const void *v_pool, const void *k_means,
                                       const int32_t *block_tables, int32_t max_blocks_per_seq,
                                       const int32_t *context_lens, float scale,
                                       const pkv_sparse_select *select, int32_t *sel_tables,
                                       int32_t *sel_lens, void *out, int32_t out_dtype,
                                       void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_SPARSE_H */

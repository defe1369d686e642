/*
 * pkv_tables.h — block tables and slot maps kept on the GPU.
 *
 * The block manager (pkv_block_manager.h) decides on the host which blocks a
 * step's new tokens take; its tables and slots are then copied to the device.
 * These calls take the same decisions on the device, from device memory, so
 * that a serving step needs no host work and can be captured into a CUDA graph
 * with everything that follows it (the rotary append, the decode).
 *
 * Passage: a sequence that needs slot B+1 gets a new block appended to its
 * table ("PagedAttention — Math + Memory Model", section "PagedAttention:
 * blocks and the block table"); a finished request's blocks go back to the
 * pool at once ("KV-Cache Optimization & PagedAttention for Long-Context
 * Agents", section "Key KV-Cache Optimization Principles", item 1).
 *
 * State, all in device memory and owned by the caller:
 *   block_tables  [num_seqs][max_blocks_per_seq] int32; row s holds the
 *                 ceil(L_s / B) blocks of request s, later entries anything
 *   context_lens  [num_seqs] int32, L_s tokens (0: an empty row)
 *   free_blocks   [num_blocks] int32, a stack: the first num_free[0] entries
 *                 are free, the last of them is taken next
 *   num_free      [1] int32
 * Blocks are taken request after request in row order, each request's in
 * table order: what pkv_bm_append_batch hands out for the same requests from
 * the same stack. Sharing (prefixes, forks) is the host manager's: here every
 * block has one owner.
 *
 * A call whose request cannot be met changes nothing (all or nothing) and sets
 * a bit of the device error word (pkv_get_error):
 *   PKV_DEVERR_NO_BLOCKS  more blocks needed than free, or (release,
 *                         truncate) more returned than the pool holds
 *   PKV_DEVERR_TOKENS     a negative token count, or more new tokens than
 *                         max_tokens
 *   PKV_DEVERR_CONTEXT    a length < 0 or past max_blocks_per_seq * B
 * A block id outside [0, num_blocks) among the entries used sets
 * PKV_DEVERR_BLOCK_ID: its tokens get slot -1 (append), or it is pushed as it
 * is (release, truncate).
 *
 * Calls on one state are ordered by the caller (one stream, or events).
 *
 * The tables, lengths and slots that these calls write are never "ready" in the
 * sense of pkv_decode_options.tables_ready or pkv_append_options.inputs_ready
 * for a call that follows on the stream, even with other calls in between: each
 * kernel lets the next one start before it has itself waited, so a chain of
 * them may run at once. A step made of them leaves both options 0.
 */
#ifndef PKV_TABLES_H
#define PKV_TABLES_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device memory each call needs: zero-filled once before its first use, zero
 * again after every call. Calls that may overlap need one each. */
#define PKV_TABLES_WORKSPACE_BYTES 64

/*
 * pkv_tables_append — blocks and slots for the new tokens of one step.
 *
 * Request s gets new_tokens[s] >= 0 tokens (device int32) at positions L_s ..
 * L_s + new_tokens[s] - 1. With o_s = sum of new_tokens below s, and i < new_tokens[s]:
 *   positions[o_s + i]    = L_s + i
 *   slot_mapping[o_s + i] = block_tables[s][(L_s + i) / B] * B + (L_s + i) % B
 *   token_offsets[s]      = o_s, token_offsets[num_seqs] = the number of tokens
 *   context_lens_out[s]   = L_s + new_tokens[s]
 *   num_free_out[0]       = num_free[0] - blocks taken
 * and the table entries of the blocks taken are written. Entries of
 * slot_mapping and positions past the last token, up to max_tokens, become -1
 * and 0, so that a captured append over max_tokens tokens skips them; a
 * refused call writes them so throughout, with all offsets 0.
 * slot_mapping: int64 [max_tokens]; positions: int32 [max_tokens];
 * token_offsets: int32 [num_seqs + 1]. context_lens_out may be context_lens,
 * num_free_out may be num_free; no other buffers overlap.
 */
pkv_status pkv_tables_append(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                             const int32_t *new_tokens, int32_t *block_tables,
                             int32_t max_blocks_per_seq, const int32_t *context_lens,
                             int32_t *context_lens_out, const int32_t *free_blocks,
                             const int32_t *num_free, int32_t *num_free_out,
                             int64_t *slot_mapping, int32_t *positions, int32_t max_tokens,
                             int32_t *token_offsets, void *workspace, void *stream);

/*
 * pkv_tables_release — give the blocks of finished requests back.
 *
 * For each s with released[s] != 0 (device bytes), in row order, its
 * ceil(L_s / B) blocks are pushed in table order and context_lens_out[s] = 0;
 * other lengths are copied. Table rows stay as they are. The aliases of
 * pkv_tables_append are allowed.
 */
pkv_status pkv_tables_release(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                              const uint8_t *released, const int32_t *block_tables,
                              int32_t max_blocks_per_seq, const int32_t *context_lens,
                              int32_t *context_lens_out, int32_t *free_blocks,
                              const int32_t *num_free, int32_t *num_free_out, void *workspace,
                              void *stream);

/*
 * pkv_tables_truncate — shorten requests and give the blocks behind them back.
 *
 * Request s keeps its first kept_lens[s] tokens, 0 <= kept_lens[s] <= L_s
 * (what pkv_tree_accept leaves of the drafted ones, say): blocks
 * ceil(kept / B) .. ceil(L_s / B) - 1 of its row are pushed in table order,
 * request after request, and context_lens_out[s] = kept_lens[s]. Table rows
 * stay as they are. A kept length outside its range refuses the call
 * (PKV_DEVERR_CONTEXT). The aliases of pkv_tables_append are allowed;
 * kept_lens overlaps no output.
 */
pkv_status pkv_tables_truncate(int32_t num_blocks, int32_t block_size, int32_t num_seqs,
                               const int32_t *kept_lens, const int32_t *block_tables,
                               int32_t max_blocks_per_seq, const int32_t *context_lens,
                               int32_t *context_lens_out, int32_t *free_blocks,
                               const int32_t *num_free, int32_t *num_free_out, void *workspace,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_TABLES_H */

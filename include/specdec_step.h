/*
 * specdec_step.h — the operators of a decode step around the verify call
 * (specdec.h), on the same GPU and without a host round trip:
 *
 *   kv_block_step        gives every request the blocks of a paged cache that
 *                        its next tokens need, from the accepted lengths that
 *                        spec_verify wrote, and lists the tokens' slots;
 *   kv_append            writes the new tokens' keys and values into the
 *                        cache, 8 bits a value, one scale a block and head;
 *   spec_attention       attention of the new tokens (one of a decode step,
 *                        n + 1 of a verify step, a prompt's) over that cache;
 *   spec_process_logits  penalties for repeated tokens, biases and grammar
 *                        masks on the rows that spec_verify reads.
 *
 * "Accelerating Sonar through speculation" (Perplexity Research, 2025) names
 * their places in the loop: §Inference with speculative decoding (KV pages
 * allocated per batch; "the number of accepted tokens determines the next
 * sequence length") and §MTP (sampling and logit processing shared by the
 * drafting methods).  It has no interface for any of them.
 *
 * Conventions are those of specdec.h: caller-owned device memory, argument
 * errors found on the host before anything is enqueued, bad values in device
 * arrays clamped and reported in an optional device error word (any 4-byte
 * word; a spec_verify workspace may be passed), every call asynchronous on
 * `stream` and safe to capture into a CUDA graph.
 *
 * The cache: k_cache and v_cache [num_blocks, H, block_size, D] of 8-bit
 * e4m3 codes, k_scale and v_scale float [num_blocks, H].  A value is its code
 * times the scale of its block and head.  A slot is block * block_size +
 * offset; a request's token p lives in block block_table[b][p / block_size]
 * at offset p % block_size.  D is 64 or 128, block_size 16, 32, 64 or 128,
 * and num_blocks * block_size below 2^31.
 */
#ifndef SPECDEC_STEP_H_
#define SPECDEC_STEP_H_

#include "specdec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the device error word, beside those of specdec.h. */
#define SPECDEC_DEV_ERR_BLOCKS 32u  /* kv_block_step: no block left, a table row
                                       too short, tokens beyond `capacity`, or
                                       lengths that the table cannot hold */
#define SPECDEC_DEV_ERR_PENALTY 64u /* spec_process_logits: a repetition penalty
                                       that is not a positive finite number
                                       (taken as 1), a presence or frequency
                                       penalty that is not finite (taken as 0),
                                       a length out of range (clamped), or a
                                       row's mask outside [-1, mask_count) (the
                                       row is not masked) */

/*
 * kv_block_step — block tables and slot maps from request lengths.
 *
 * Inputs (device int32 unless stated):
 *   kv_len        [B]: tokens in the cache before the last step's were added.
 *   accepted_len  [B] or NULL: the last step's accepted lengths; request b
 *                 keeps accepted_len[b] + 1 of the tokens it added then
 *                 (-1: none).  NULL: kv_len is what it keeps.
 *   new_tokens    [B]: tokens it adds in this step; 0 keeps the request
 *                 waiting; -1 ends it: it keeps nothing and all its blocks
 *                 go back.
 *   held          [B]: blocks that its table row names.
 *   free_ring     [num_blocks]: free block ids in a ring; ring_state [2] =
 *                 {head, count}.
 *   block_table   [B, max_blocks], read and written.
 * Per request, with kept tokens k and w = max(new, 0) new ones, blocks needed
 *   are ceil((k + w) / block_size).  Blocks past those go back to the ring's
 *   tail, missing ones come from its head, both in request order.  A request
 *   that needs more blocks than are left, or than max_blocks, is refused: it
 *   gets no new tokens in this step, keeps its blocks and sets
 *   SPECDEC_DEV_ERR_BLOCKS; so do all later requests that need new blocks
 *   (the ring serves in order), and others are served.
 * Outputs (device int32):
 *   kv_len_out [B] tokens kept (before the new ones); held_out [B];
 *   ring_state_out [2]; cu_tokens [B+1] prefix sums of the new tokens granted;
 *   cu_blocks [B+1] prefix sums of the blocks taken; slot_map [capacity] and
 *   positions [capacity]: slot and position of each new token, packed by
 *   request, -1 past the last.  Tokens past `capacity` are cut off
 *   (cu_tokens ends there) and set SPECDEC_DEV_ERR_BLOCKS.
 *   Table entries at and past held_out have no meaning.
 * kv_len_out, held_out and ring_state_out may be the inputs themselves.
 * Without requests (B = 0) the arrays that have an element a request are not
 * looked at and the other outputs are written all the same (no tokens, no
 * blocks, the ring as it was); nothing is where ring_state is not memory of a
 * device.
 */
specdec_status_t kv_block_step(int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                               const int32_t* kv_len, const int32_t* accepted_len, const int32_t* new_tokens,
                               const int32_t* held, int32_t* block_table, int32_t* free_ring,
                               const int32_t* ring_state, int32_t* kv_len_out, int32_t* held_out,
                               int32_t* ring_state_out, int32_t* cu_tokens, int32_t* cu_blocks,
                               int32_t* slot_map, int32_t* positions, int32_t capacity, uint32_t* error_word,
                               void* stream);

/*
 * kv_append — keys and values of new tokens into the cache.
 *
 *   k, v       [T, H, D] of dtype (F32 or BF16); token t's head h starts at
 *              t * token_stride + h * head_stride elements, its D values are
 *              contiguous.  16-byte aligned, strides multiples of 16 bytes.
 *   slot_map   [T] int32: token t's slot; a negative or too large one is
 *              skipped.
 * Neighbouring tokens in neighbouring slots of one block form a run; blocks
 * fill from their start, so the tokens before a run's first are the block's
 * older ones.  (No two runs of a call may share a block: tokens that are skipped
 * between others of a block make two runs of it, which write its scale both, and
 * what it holds then has no meaning.)  Per run and head
 * the scale is the least power of two that brings the largest magnitude
 * within 448, the type's largest number, and at least the block's scale where
 * it has older tokens, whose codes are then rescaled; 0 when all that is finite
 * is 0.  Codes are rounded to the nearest, ties to even; infinities become the
 * largest number and do not count for the scale, NaN stays NaN.
 */
specdec_status_t kv_append(const void* k, const void* v, specdec_dtype_t dtype, int32_t T, int32_t H, int32_t D,
                           int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                           int64_t v_head_stride, const int32_t* slot_map, int32_t num_blocks, int32_t block_size,
                           void* k_cache, void* v_cache, float* k_scale, float* v_scale, void* stream);

/*
 * spec_attention — attention of new tokens over the cache, causal among them.
 *
 *   q            [T, Hq, D] bf16; token t starts at t * q_token_stride
 *                elements (16-byte aligned, a multiple of 8), its heads are
 *                contiguous.  Hq is a multiple of H; query head h reads key
 *                and value head h / (Hq / H).
 *   cu_tokens    [B+1]: request b's tokens are cu_tokens[b] .. cu_tokens[b+1]-1.
 *                Values outside [0, T] are clamped and a decrease is a request
 *                without tokens; either sets SPECDEC_DEV_ERR_SEGMENT.  Where
 *                requests overlap so often that their tiles pass the count
 *                below, nothing is computed.
 *   kv_len       [B]: tokens in the cache before these; these tokens' own keys
 *                and values are in the cache (kv_append), so token i of
 *                request b attends to positions 0 .. kv_len[b] + i.
 *   out          [T, Hq, D] bf16, contiguous, 16-byte aligned.  Rows of
 *                tokens that belong to no request are left as they were; a
 *                request whose row of the table is too short for its tokens
 *                attends to what the row holds, and a token that thereby
 *                attends to nothing gets zeros.
 *   block ids outside [0, num_blocks) read as blocks of zeros.
 *   scale        factor of the scores, at most 2.3e38; 0 selects 1 / sqrt(D).
 *   workspace    SPECDEC_ATTENTION_WORKSPACE_BYTES, zero-filled once before
 *                its first use; every call leaves it ready for the next.  One
 *                workspace serves one call in flight at a time.  Its first
 *                word is the device error word (specdec_get_error reads it):
 *                after SPECDEC_DEV_ERR_TIMEOUT the call's outputs have no
 *                meaning and the workspace has to be zero-filled again.
 * Scores, their maxima and sums and the output's sums are held in 32 bits;
 * keys and values are taken as they are in the cache, queries to 2^-21 of a
 * row's largest.  Probabilities enter the second product in f16, times their
 * block's value scale over the largest that the request's tiles have had, and
 * 64 times their size over a reference (a score that later ones pass by 2^9 at
 * most): 11 significant bits down to 2^-20 of it, nothing below 2^-31.
 * SPECDEC_ERR_UNSUPPORTED also where the tiles of 128 positions, over heads
 * and groups of 64 rows, could pass some 400 million, or where
 * max_blocks * block_size + T passes 2^31 - 1.
 */
#define SPECDEC_ATTENTION_WORKSPACE_BYTES (64u << 20)
specdec_status_t spec_attention(const void* q, int64_t q_token_stride, int32_t T, int32_t Hq, int32_t H, int32_t D,
                                int32_t B, const int32_t* cu_tokens, const int32_t* kv_len,
                                const int32_t* block_table, int32_t max_blocks, int32_t num_blocks,
                                int32_t block_size, const void* k_cache, const void* v_cache,
                                const float* k_scale, const float* v_scale, float scale, void* out,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * spec_process_logits — penalties, biases and grammar masks.
 *
 *   logits, out   [B, n_max+1, V] of dtype, contiguous; out may be logits (with
 *                 long histories a call in place takes longer).
 *                 Rows j > draft_len[b] are neither read nor written.
 *   history       [B, history_stride] int32: a request's prompt, then the
 *                 tokens made so far; prompt_len [B] and history_len [B] say
 *                 how many.  Ids outside [0, V) are passed over.  NULL with
 *                 history_stride 0: no history.
 *   draft_tokens  [B, n_max], draft_len [B]: as for spec_verify; row j also
 *                 counts the drafts before it.  draft_len NULL: n_max.
 *   repetition, presence, frequency  [B] float, or NULL (1, 0, 0).
 *   bias_offsets  [B+1], bias_ids, bias_values: request b's biases are
 *                 entries bias_offsets[b] .. bias_offsets[b+1]-1; those of
 *                 one token add up.  NULL: none.  num_bias: entries in all.
 *   mask          [mask_count, ceil(V / 32)] words: bit v % 32 of word v / 32
 *                 allows token v.  mask_rows [B, n_max+1] names each row's
 *                 mask, -1 for none.  NULL: none.
 * history_stride stays below 2^29.
 * After SPECDEC_DEV_ERR_TIMEOUT in the error word (a device wait ran out; not
 * known without an error word) the rows that the call writes have no meaning;
 * nothing else is touched.
 * For token v of row j, with c = times it was made (drafts before j among
 * them), in 32 bits and rounded once:
 *   l = logit; made or in the prompt: l > 0 ? l / repetition : l * repetition;
 *   l -= frequency * c; c > 0: l -= presence; l += bias; masked: l = -inf.
 */
specdec_status_t spec_process_logits(const void* logits, void* out, specdec_dtype_t dtype, int32_t B,
                                     int32_t n_max, int32_t V, const int32_t* history, int32_t history_stride,
                                     const int32_t* prompt_len, const int32_t* history_len,
                                     const int32_t* draft_tokens, const int32_t* draft_len,
                                     const float* repetition, const float* presence, const float* frequency,
                                     const int32_t* bias_offsets, const int32_t* bias_ids,
                                     const float* bias_values, int32_t num_bias, const uint32_t* mask,
                                     int32_t mask_count, const int32_t* mask_rows, uint32_t* error_word,
                                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECDEC_STEP_H_ */

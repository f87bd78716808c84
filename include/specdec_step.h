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
 *                        masks on the rows that spec_verify reads;
 *   spec_sample          tokens drawn with temperature, top-k, top-p and min-p
 *                        from given random numbers, and the rows cut to what
 *                        may be drawn, as spec_verify reads them;
 *   spec_rotary          rotary positions of queries and keys;
 *   kv_fork, kv_compact  requests that go on from others' tokens, and the blocks
 *                        in use moved to the lowest ids: tables, holders, ring;
 *   kv_copy              the copies of blocks that both ask for.
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
#define SPECDEC_DEV_ERR_SAMPLE 128u /* spec_sample: a top-p below 0, a min-p outside
                                       [0, 1] or a random number outside [0, 1)
                                       (clamped; NaN as 1, 0 and 0), or a row
                                       without a number above -infinity */

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
 * kv_block_step_shared — the same where requests may share blocks (kv_fork).
 *
 *   shares   [num_blocks] int32 or NULL (none are shared): a block's holders beside
 *            the first.
 * A request that would write a block with other holders, or give one back, is
 * refused, as one for which no blocks are left: it gets no new tokens, keeps its
 * tokens and blocks, and sets SPECDEC_DEV_ERR_BLOCKS; others are served.  (kv_fork
 * ends such a request, or cuts it back, and gives it blocks of its own.)
 */
specdec_status_t kv_block_step_shared(int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                                      const int32_t* kv_len, const int32_t* accepted_len, const int32_t* new_tokens,
                                      const int32_t* held, int32_t* block_table, int32_t* free_ring,
                                      const int32_t* ring_state, const int32_t* shares, int32_t* kv_len_out,
                                      int32_t* held_out, int32_t* ring_state_out, int32_t* cu_tokens,
                                      int32_t* cu_blocks, int32_t* slot_map, int32_t* positions, int32_t capacity,
                                      uint32_t* error_word, void* stream);

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

/*
 * spec_sample — truncated sampling: the draft's tokens, and rows for spec_verify.
 *
 *   logits        [B, n_max+1, V] of dtype, contiguous.  NaN counts as -infinity.
 *   out           as logits, may be logits, or NULL: the rows with -infinity for
 *                 every id that is not kept.  (A verify step wants the draft's
 *                 rows and the target's cut alike.)
 *   draft_len     [B] or NULL (n_max): rows j > draft_len[b] are neither read nor
 *                 written, and their tokens are -1.
 *   temperature   [B] float or NULL (1): 0, or what spec_verify takes as 0 (above
 *                 3e38 too; SPECDEC_DEV_ERR_TEMPERATURE), keeps the largest logit
 *                 alone.
 *   top_k         [B] int32 or NULL: 0 and below, and V and above, keep all.
 *   top_p, min_p  [B] float or NULL (1 and above, 0: keep all).
 *   uniform       [B, n_max+1] float in [0, 1), and
 *   tokens        [B, n_max+1] int32: a token drawn of each row; both or neither.
 * But for out in logits' place, no output lies on an input or on another output
 * (refused).
 * Per row, with weights w = exp((logit - largest) / temperature) and the ids in
 * order of their logits, the largest first and equal ones by id: kept are the
 * first top_k; of those the shortest beginning whose weights sum to at least
 * top_p times that of all of them (one id at least); of those the ids with
 * w >= min_p.  The token is the first of the kept, in this order, up to which the
 * weights sum to more than uniform times that of all kept.  A row without a
 * number above -infinity gives -1 and keeps nothing; infinite logits are equal,
 * and the others count as -infinity beside them.
 * Weights are made to within 2^-40 of their value and rounded to whole numbers of 2^-44
 * of the largest, so that the smallest are 0 and a min_p means its value rounded up to
 * such a number; their sums are exact.  (bf16 logits within 1.01 * 2^-20 of 0 weigh as 0 does
 * where that changes the sum by less than 2^-40 of itself.)
 */
specdec_status_t spec_sample(const void* logits, void* out, specdec_dtype_t dtype, int32_t B, int32_t n_max, int32_t V,
                             const int32_t* draft_len, const float* temperature, const int32_t* top_k,
                             const float* top_p, const float* min_p, const float* uniform, int32_t* tokens,
                             uint32_t* error_word, void* stream);

/*
 * spec_rotary — rotary positions of the new tokens' queries and keys.
 *
 *   q, k          [T, Hq, D] and [T, H, D] of dtype; token t's head h starts at
 *                 t * token_stride + h * head_stride elements, its D values are
 *                 contiguous.  Hq or H may be 0 (their pointers are not looked at);
 *                 strides of one token or one head do not matter.
 *   q_out, k_out  the same, with strides of their own, rows apart from one another;
 *                 the inputs themselves with their strides, or memory that no input
 *                 shares.
 *   positions     [T] int32, as kv_block_step lists them; rows of tokens with
 *                 negative ones are left as they were.
 *   turns         [rotary_dim / 2]: what pair i turns by a position, in 2^-64 of a
 *                 whole turn (frequency / 2 pi * 2^64, rounded).
 *   rotary_dim    values of a head that are turned, its first ones; even.  The
 *                 others are as they were (copied to other outputs).
 *   interleaved   0: values i and i + rotary_dim / 2 are a pair; 1: 2 i and 2 i + 1.
 *   factor        of the turned values, positive.
 * A pair (a, b) becomes factor * (a cos - b sin, a sin + b cos) in 32 bits, rounded
 * once.  The angle is position * turns[i] in whole numbers: at any position its
 * sine and cosine are within 2^-21.  D is at most 1024.
 */
specdec_status_t spec_rotary(const void* q, const void* k, specdec_dtype_t dtype, int32_t T, int32_t Hq, int32_t H,
                             int32_t D, int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                             int64_t k_head_stride, const int32_t* positions, const uint64_t* turns,
                             int32_t rotary_dim, int32_t interleaved, float factor, void* q_out,
                             int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                             int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream);

/*
 * Holders of a block: shares [num_blocks] int32 says how many requests, or other
 * users of the cache, hold a block beside the first.  What kv_block_step hands out has
 * one holder and shares 0.  Without shares it gives back whatever it takes from a
 * request, and neither it nor kv_append looks whether a block that is written has other
 * holders: after kv_fork none has, and requests that hold shared blocks are ended, or
 * cut back into them, by kv_fork.  kv_block_step_shared looks, and refuses.
 *
 * The workspace of kv_fork and kv_compact: specdec_page_workspace_bytes(num_blocks)
 * bytes, zero-filled once before its first use; every call leaves it ready for the
 * next, which may be of another pool: one workspace, given whole, serves all numbers
 * of blocks that it has room for, one call in flight at a time.
 */
size_t specdec_page_workspace_bytes(int32_t num_blocks);

/*
 * kv_fork — requests that go on from the tokens of others: several continuations of
 * a prompt, beams that choose their parents anew, a step back, an end.
 *
 * Inputs (device int32):
 *   block_table [P, max_blocks], held [P], kv_len [P], accepted_len [P] or NULL: the
 *                 old requests, as kv_block_step leaves them; request p has
 *                 kv_len[p] + accepted_len[p] + 1 tokens (NULL: kv_len[p]).
 *   parent      [B]: the old request that new request b goes on from, -1 for none
 *                 (it has no tokens).  An old request without children ends.
 *   keep        [B] or NULL: tokens of the parent's that b keeps, at most (below 0: 0).
 *   shares, free_ring, ring_state  as above and as for kv_block_step.
 * New request b names its parent's first ceil(t / block_size) blocks for its t
 * tokens.  A request whose last block is part-filled will write it: where others
 * hold that block too, it takes a block of its own from the ring's head, in request
 * order, and asks for a copy; where all its holders are such requests the last one
 * keeps it.  Without blocks left, the request keeps its full blocks' tokens only and
 * SPECDEC_DEV_ERR_BLOCKS is set.  Blocks that no one holds any more go to the ring's
 * tail in order of their ids.
 * Outputs (device int32):
 *   table_out [B, max_blocks] (-1 past a request's blocks), held_out [B],
 *   kv_len_out [B]: tokens (a next kv_block_step has no accepted_len, or -1);
 *   shares_out [num_blocks], ring_state_out [2]; free_ring's tail in place;
 *   copies [B, 2] and count [1]: for kv_copy, from and to; those past count have no
 *                 meaning.
 * shares_out and ring_state_out may be the inputs; no other output lies on an input
 * or on another output (refused).  Out of range: a parent is none, a length is clamped to what is held, held to
 * the table's width, a block id (the ring's too) is left as it is; each sets
 * SPECDEC_DEV_ERR_BLOCKS.
 */
specdec_status_t kv_fork(int32_t P, int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                         const int32_t* block_table, const int32_t* kv_len, const int32_t* accepted_len,
                         const int32_t* held, const int32_t* parent, const int32_t* keep, const int32_t* shares,
                         int32_t* free_ring, const int32_t* ring_state, int32_t* table_out, int32_t* kv_len_out,
                         int32_t* held_out, int32_t* shares_out, int32_t* ring_state_out, int32_t* copies,
                         int32_t* count, void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream);

/*
 * kv_compact — blocks in use to the lowest ids, so that the cache's end is free.
 *
 * Blocks in use are those that the ring does not list; with n of them, the i-th in
 * use from id n on, in order, moves to the i-th free one before n.  The ring then
 * lists n .. num_blocks - 1 from its start.
 * Outputs (device int32); the first four may be the inputs of their name, and else no
 * output lies on an input or on another output (refused):
 *   table_out [B, max_blocks] (-1 past held), shares_out [num_blocks],
 *   ring_out [num_blocks] (what is behind its free ids is left), ring_state_out [2];
 *   renamed [num_blocks]: a block's new id, -1 for a free one, for other holders;
 *   copies [num_blocks / 2, 2] and count [1]: for kv_copy.
 * An entry that names no block, or a free one, becomes -1 and sets
 * SPECDEC_DEV_ERR_BLOCKS, as do ids of the ring out of range, which are passed over.
 */
specdec_status_t kv_compact(int32_t B, int32_t max_blocks, int32_t num_blocks, const int32_t* block_table,
                            const int32_t* held, const int32_t* shares, const int32_t* free_ring,
                            const int32_t* ring_state, int32_t* table_out, int32_t* shares_out, int32_t* ring_out,
                            int32_t* ring_state_out, int32_t* renamed, int32_t* copies, int32_t* count,
                            void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream);

/*
 * kv_copy — copies of blocks, codes and scales, in every layer's cache.
 *
 *   copies   [capacity, 2] int32: from and to; count [1] int32 on the device says how
 *            many of them hold (at most capacity).  No block is written twice, or
 *            both read and written.  Ids out of range, and a block onto itself, are
 *            passed over.
 *   caches   host array of 4 * layers device pointers, a layer's k_cache, v_cache
 *            (16-byte aligned), k_scale and v_scale in turn; it is read in the call.
 * A launch for every 64 layers.
 */
specdec_status_t kv_copy(const int32_t* copies, const int32_t* count, int32_t capacity, int32_t layers,
                         void* const* caches, int32_t num_blocks, int32_t block_size, int32_t H, int32_t D,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECDEC_STEP_H_ */

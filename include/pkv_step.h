/*
 * pkv_step.h -- C ABI of the serving-step operators that stand beside the calls of pkv.h: the
 * block tables and slots of a step built on the GPU, an FP8 cache with one scale per block and
 * kv head, and attention with score rules (capped scores, distance bias, sliding window,
 * documents, a prefix that stays visible) for one query token and for many.
 *
 * One step of a serving engine: pkv_kv_step_tables gives every request the blocks and slots of
 * its new tokens, pkv_kv_append (or pkv_kv_append_f8) writes their K and V rows there, and
 * pkv_paged_prefill_attention (prompt chunks, mixed batches) or one of the decode calls (one token
 * per request) attends.
 *
 * The conventions of pkv.h hold for every call here (device pointers, nothing allocated, kernels
 * enqueued on `stream` only, status codes, device errors through error_word, dense layouts).
 */
#ifndef PKV_STEP_H_
#define PKV_STEP_H_

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most new tokens of one pkv_kv_step_tables call. */
#define PKV_MAX_STEP_TOKENS 262144

/*
 * pkv_kv_step_tables -- the block tables, slots and lengths of one step, from the requests'
 * lengths ("KV Cache primer", cf-1.com/news/5988169, section 4.1: a request's blocks are taken
 * from a shared pool as its tokens arrive, one block per 16 tokens, and a block table maps them).
 * Sequence b holds c_b = context_lens[b] tokens in its first h_b = ceil(c_b / 16) table entries.
 * new_tokens[b] = n_b > 0 gives it n_b more tokens, 0 leaves it as it is, -1 ends it.  Free
 * blocks are a stack: free_blocks[0 : free_count].
 *   1. The blocks of ended sequences are pushed, in the order of (b, table entry).
 *   2. Sequence b takes d_b = ceil((c_b + n_b) / 16) - h_b blocks off the top, in the order of b:
 *      block_tables[b][h_b + j] = the stack's entry number (top - 1 - sum_{a<b} d_a - j).
 *   3. Token i of sequence b is row s_b + i of the step's packed batch, s_b = sum_{a<b} max(n_a, 0):
 *      positions = c_b + i, slot_mapping = block_tables[b][(c_b+i)/16] * 16 + (c_b+i) % 16.
 * Rows past the last token, up to max_new_tokens, get slot -1 (which the appends skip) and
 * position -1, so one captured graph serves steps of any size.
 *   block_tables     : [B, MB] int32, updated in place (entries of the blocks taken).
 *   context_lens     : [B] int32.    context_lens_out : [B] int32, c_b + n_b (0 for an ended one);
 *                      may be context_lens itself.
 *   new_tokens       : [B] int32, each >= -1.
 *   free_blocks      : [NB] int32, updated in place; entries past the new count are unspecified.
 *   free_count       : [1] int32.    free_count_out : [1] int32; may be free_count itself.
 *   query_starts     : [B + 1] int32, s_b and the total.
 *   slot_mapping     : [max_new_tokens] int64.    positions : [max_new_tokens] int32.
 *   max_new_tokens   : 0 .. PKV_MAX_STEP_TOKENS.
 *   dims             : uses batch (<= 4096), block_size, num_blocks, max_blocks_per_seq.
 *   error_word       : PKV_DEV_BAD_CONTEXT_LEN (a length, or a sequence's new length, outside its
 *                      table), PKV_DEV_BAD_QUERY_RANGE (n_b < -1, or more than max_new_tokens in
 *                      all), PKV_DEV_NO_BLOCKS (too few free blocks; a free count outside the stack
 *                      or one that the pushed blocks would take past it), PKV_DEV_BAD_BLOCK_ID (a
 *                      block outside the pool among those pushed, taken, or part filled and written on;
 *                      a sequence's other blocks are not looked at).
 * Arrays are aligned to their elements (slot_mapping to 8 bytes).
 * All or nothing: on an error the lengths and the count are passed through unchanged, the tables
 * and the stack's live entries stay as they were, every query_starts entry is 0 and every slot and
 * position -1.
 */
int pkv_kv_step_tables(int32_t* block_tables, int32_t* context_lens_out, int32_t* query_starts,
                       int64_t* slot_mapping, int32_t* positions, int32_t* free_count_out,
                       int32_t* free_blocks, const int32_t* free_count, const int32_t* context_lens,
                       const int32_t* new_tokens, int32_t max_new_tokens, const pkv_dims* dims,
                       int32_t* error_word, void* stream);

/*
 * FP8 KV cache: K and V as E4M3 numbers (4 exponent and 3 mantissa bits, largest 448), one fp32
 * scale per (block, kv head) and pool, value = code * scale ("KV Cache primer" section 4.2: 8-bit
 * storage halves the cache; section 5.2 names FP8 among vLLM's cache types).  Code pools are
 * [NB, Hkv, 16, d], one byte an element; scale pools are [NB, Hkv] fp32, finite and >= 0.
 *
 * pkv_kv_append_f8 -- pkv_kv_append into FP8 pools.  Per (block, kv head) that receives rows, for K
 * and for V on their own: the needed scale is the smallest power of two s with max|x| / s <= 448
 * over the call's rows of the block (exponent kept in [-120, 119]).  A block whose offset 0 is
 * written (not one whose row there is refused) starts anew with the needed scale; otherwise its scale
 * becomes the larger of the old and the needed one, and if it grew, the codes c of the rows that this
 * call does not write become rne(c * (old / new)) (exact but for results below the smallest normal
 * number).  Rows become rne(x / scale), saturated at 448.
 *   k_codes, v_codes   : [NB, Hkv, 16, d] E4M3, updated in place.
 *   k_scales, v_scales : [NB, Hkv] fp32, updated in place.
 *   k, v, slot_mapping, num_tokens, dims : as pkv_kv_append, and the tokens of one block are
 *                        adjacent in slot_mapping with ascending slots (the order of
 *                        pkv_kv_step_tables).  A token whose slot is in the block of the token
 *                        before it but not above that token's is reported (PKV_DEV_BAD_SLOT), and
 *                        neither it nor the tokens of that block that follow on it are written; those
 *                        before it are.  The same block in two places that are not adjacent is
 *                        invalid input.
 *   error_word         : PKV_DEV_BAD_SLOT; PKV_DEV_BAD_VALUE for a (token, kv head) whose K or V row
 *                        holds a non-finite value (it is left unwritten and does not count), or a
 *                        (block, kv head) whose old scale is negative or not finite (nothing of it
 *                        is written).
 * Code pools, k and v 16-byte aligned; scales 4-byte, slot_mapping 8-byte aligned.
 */
int pkv_kv_append_f8(void* k_codes, void* v_codes, float* k_scales, float* v_scales, const void* k,
                     const void* v, const int64_t* slot_mapping, int64_t num_tokens, const pkv_dims* dims,
                     int32_t* error_word, void* stream);

/*
 * Score rules of an attention call.  A query at position i of a sequence with L keys sees key t if
 *     lo <= t <= i   or   t < min(prefix_lens[b], L),
 *     lo = max(0, i - window + 1 if window > 0, doc_start of the query if given),
 * and its logit is
 *     x = scale * q . k;   x = softcap * tanh(x / softcap) if softcap > 0;   x -= slope_h * |i - t|.
 * So `window` slides, `doc_starts` keeps packed documents apart (the first position of the query's
 * document), and the prefix -- a shared prompt, or the bidirectional part of a prefix model -- stays
 * visible to every query of the sequence.  A row that sees no key is written as zeros.  Masked keys
 * contribute nothing, whatever their K and V hold.
 */
typedef struct pkv_score_rules {
  float softcap;               /* 0: scores are not capped; else 1e-30 .. 1e30 */
  int32_t window;              /* > 0: the last `window` positions; <= 0: all */
  const float* alibi_slopes;   /* [Hq] fp32 finite, or NULL */
  const int32_t* doc_starts;   /* decode: [B]; prefill: [total_tokens] (the packed rows); or NULL */
  const int32_t* prefix_lens;  /* [B] int32, or NULL; values are cut to [0, L] */
} pkv_score_rules;

/*
 * pkv_paged_decode_attention_rules -- pkv_paged_decode_attention with score rules (the query of
 * sequence b is at position L_b - 1).
 *   rules : required; its window replaces that call's argument.
 *   other arguments, supported sizes and errors : as pkv_paged_decode_attention (the same workspace).
 *           With PKV_DECODE_INPUTS_READY the rules' arrays are among the inputs declared final.
 */
int pkv_paged_decode_attention_rules(void* out, const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_tables, const int32_t* context_lens, float scale,
                                     const pkv_score_rules* rules, void* workspace, size_t workspace_bytes,
                                     const pkv_dims* dims, uint32_t flags, int32_t* error_word, void* stream);

/*
 * pkv_paged_decode_attention_f8 -- pkv_paged_decode_attention over FP8 pools (value = code * scale of
 * the key's block), with score rules.  Weights are fp32 numbers relative to the row's largest, and enter
 * the product with V times their block's scale as one fp16 term (11 bits).
 *   k_codes, v_codes   : [NB, Hkv, 16, d] E4M3, 16-byte aligned.
 *   k_scales, v_scales : [NB, Hkv] fp32, finite and >= 0.
 *   rules              : or NULL (plain softmax over all keys).
 *   other arguments    : as pkv_paged_decode_attention (the same workspace).  With
 *                        PKV_DECODE_INPUTS_READY the scales and the rules' arrays are among the inputs
 *                        declared final.
 */
int pkv_paged_decode_attention_f8(void* out, const void* q, const void* k_codes, const void* v_codes,
                                  const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                  const int32_t* context_lens, float scale, const pkv_score_rules* rules,
                                  void* workspace, size_t workspace_bytes, const pkv_dims* dims, uint32_t flags,
                                  int32_t* error_word, void* stream);

/*
 * pkv_prefill_workspace_bytes -- bytes of device workspace for pkv_paged_prefill_attention with these
 * dims and at most total_tokens packed query rows.  Its contents need no preparation and nothing is
 * kept in it between calls; calls that may overlap on the GPU (other streams, or captured graphs that
 * run at the same time) need one each.  Returns 0 if the arguments are invalid.
 */
size_t pkv_prefill_workspace_bytes(const pkv_dims* dims, int32_t total_tokens);

/*
 * pkv_paged_prefill_attention -- attention of many query tokens per sequence over the paged cache:
 * prompts, chunks of prompts and mixed steps, causal, with score rules (the prefill stage of "KV Cache
 * primer" section 2.1 over the blocks of section 4.1).  The K and V rows of the queries' own tokens
 * are in the cache already.  bf16 pools only: a prompt over an FP8 cache is not offered.  Weights enter
 * the product with V as two bf16 terms in sequences of at most 512 keys, as one (8 bits) in longer ones;
 * their sum is fp32.
 *   out, q        : [total_tokens, Hq, d] bf16.  Sequence b's queries are rows query_starts[b] ..
 *                   query_starts[b+1] - 1, n_b of them, at positions L_b - n_b + r.  Rows from
 *                   query_starts[B] on (a padded batch) are neither read nor written.
 *   query_starts  : [B + 1] int32, ascending, query_starts[0] >= 0, query_starts[B] <= total_tokens.
 *   context_lens  : [B] int32, L_b including the step's tokens, n_b <= L_b <= MB * 16.
 *   total_tokens  : rows of q and out.
 *   rules         : or NULL (causal).
 *   error_word    : PKV_DEV_BAD_BLOCK_ID, _BAD_CONTEXT_LEN, _WAIT_TIMEOUT; _BAD_QUERY_RANGE for a
 *                   sequence whose rows are not within the packed batch or which starts below a start
 *                   before its own.  Rows of a refused sequence are not written.
 * Arrays of int32 are 4-byte aligned, the others 16-byte.
 * Supported: d in {64, 128}; G = Hq / Hkv in 1..8; B <= 4096; MB * 16 < 2^30.
 */
int pkv_paged_prefill_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, const int32_t* context_lens,
                                const int32_t* query_starts, int32_t total_tokens, float scale,
                                const pkv_score_rules* rules, void* workspace, size_t workspace_bytes,
                                const pkv_dims* dims, int32_t* error_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_STEP_H_ */

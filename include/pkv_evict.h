/*
 * pkv_evict.h -- C ABI of eviction from the paged cache by accumulated attention weight: sequences
 * past a limit shrink to a budget in place, and the blocks behind it go back on the free stack of
 * pkv_kv_step_tables.
 *
 * ("How KV Sparsity Achieves 1.5x Acceleration for vLLM", blogs.novita.ai, "System model": keep sinks, the
 * recent window and the tokens of the highest score; "Key technique 1": the blocks so freed take other
 * requests.)  pkv_kv_select_topk and pkv_kv_compact take the kept rows to other pools; this call leaves
 * them where they are, but for those that fill the places of evicted ones.
 *
 * The conventions of pkv.h hold (device pointers, nothing allocated, kernels enqueued on `stream`
 * only, status codes, device errors through error_word, dense layouts).
 */
#ifndef PKV_EVICT_H_
#define PKV_EVICT_H_

#include "pkv_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most cached tokens of a sequence that an eviction takes. */
#define PKV_MAX_EVICT_TOKENS 262144

/* What an eviction keeps: n_sink + k_top + n_recent tokens (the budget) of a sequence of more than
 * max(trigger, budget). */
typedef struct pkv_evict_rules {
  int32_t n_sink;    /* >= 0: tokens of position < n_sink are kept */
  int32_t k_top;     /* >= 0 */
  int32_t n_recent;  /* >= 0: the last n_recent positions are kept */
  int32_t trigger;   /* sequences of up to this many cached tokens are left alone (any value; the budget is the least) */
} pkv_evict_rules;

/* The state of a layer that evictions read and bring forward.  An _out array may be its input itself, and
 * may not overlap it otherwise. */
typedef struct pkv_evict_state {
  const float* scores;       /* [B, Hkv, stride] fp32: accumulated attention weight of each slot */
  float* scores_out;
  const int32_t* slot_pos;   /* [B, Hkv, stride] int32: position of the token in each slot; < 0: the slots are in
                                order, position = slot + dropped[b].  -1 throughout for a sequence that has lost none */
  int32_t* slot_pos_out;
  const int32_t* dropped;    /* [B] int32 >= 0: tokens that the sequence has lost so far */
  int32_t* dropped_out;
  int32_t stride;            /* slots of a row of scores and slot_pos */
} pkv_evict_state;

/*
 * pkv_evict_workspace_bytes -- bytes of device workspace for an eviction of `dims` (batch, num_kv_heads) with
 * these rules.  Its contents need no preparation and nothing is kept in it between calls; calls that may
 * overlap on the GPU need one each.  Returns 0 if the arguments are invalid.
 */
size_t pkv_evict_workspace_bytes(const pkv_dims* dims, const pkv_evict_rules* rules);

/*
 * pkv_kv_evict -- evict tokens of every sequence b with L_b = context_lens[b] > max(trigger, budget), for
 * each kv head on its own:
 *   1. A token is protected if its position is below n_sink or at least L_b + dropped[b] - n_recent.  The budget
 *      goes to the protected tokens, then to the others by descending score; of equal scores (and -0.0 equals
 *      0.0), and of protected tokens where they alone are more, the lower slots.
 *   2. Slots below the budget whose token is evicted are filled: the j-th of them, ascending, with the j-th
 *      kept slot at or past the budget, ascending.  K and V rows, score and position move.
 *   3. scores_out and slot_pos_out: entries below the budget hold score and position (explicit, >= 0) of their
 *      token, those from the budget to L_b hold 0 and -1, so that tokens appended later start at no weight and
 *      in order; entries from L_b on are left as they were.  Of a sequence that is left alone, entries below
 *      L_b are copied.
 *   4. context_lens_out[b] = budget, dropped_out[b] = dropped[b] + L_b - budget (L_b and dropped[b] of a
 *      sequence that is left alone).
 *   5. Blocks ceil(budget / 16) .. ceil(L_b / 16) - 1 of the sequence are pushed on the free stack, in the order of
 *      (b, table entry).  block_tables itself is not changed.
 * The token that follows has position L_b + dropped[b] (pkv_kv_step_tables numbers slots: a model that wants a token's
 * position adds dropped[b] to its `positions`), and attention without position rules over the
 * shrunk cache is that over the kept tokens (slots are in no order, so a window or a distance bias over slots has
 * no meaning).  No block of a shrinking sequence may belong to another one too.
 *   k_cache, v_cache : [NB, Hkv, 16, d] bf16, changed in place.
 *   block_tables     : [B, MB] int32.
 *   context_lens     : [B] int32.    context_lens_out : [B] int32; may be context_lens itself.
 *   free_blocks      : [NB] int32 with free_count [1] int32 live entries, or NULL (with free_count and
 *                      free_count_out): nothing is pushed.  Layers that share one table pass it once, and
 *                      all but the last get context_lens_out other than context_lens.
 *   free_count_out   : [1] int32; may be free_count itself.
 *   dims             : uses batch (<= 4096), num_kv_heads, head_dim, block_size, num_blocks (< 2^27),
 *                      max_blocks_per_seq.
 *   error_word       : PKV_DEV_BAD_CONTEXT_LEN (a length outside its table, past `stride` or past
 *                      PKV_MAX_EVICT_TOKENS, dropped < 0 or a length with it past 32 bits: the sequence is left alone,
 *                      without copies), PKV_DEV_BAD_SCORE
 *                      (a NaN of an unprotected token of a sequence that shrinks; it counts as the lowest score), PKV_DEV_BAD_BLOCK_ID (a block outside the pool
 *                      among those a row moves from or to -- the row is not moved -- or that would be pushed -- it
 *                      is not), PKV_DEV_NO_BLOCKS (a free count outside the stack: nothing is pushed; or a full
 *                      stack: the blocks past it are not pushed).
 * Pools 16-byte aligned, the other arrays to their elements.
 */
int pkv_kv_evict(void* k_cache, void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
                 int32_t* context_lens_out, const pkv_evict_state* state, const pkv_evict_rules* rules,
                 int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out, void* workspace,
                 size_t workspace_bytes, const pkv_dims* dims, int32_t* error_word, void* stream);

/*
 * pkv_kv_evict_q8 -- pkv_kv_evict over INT8 pools ([NB, Hkv, 16, d] bytes with [NB, Hkv, 16] fp32 row
 * scales, 16-byte aligned): a row's codes move with its scale.
 */
int pkv_kv_evict_q8(void* k_codes, void* v_codes, float* k_scales, float* v_scales, const int32_t* block_tables,
                    const int32_t* context_lens, int32_t* context_lens_out, const pkv_evict_state* state,
                    const pkv_evict_rules* rules, int32_t* free_blocks, const int32_t* free_count,
                    int32_t* free_count_out, void* workspace, size_t workspace_bytes, const pkv_dims* dims,
                    int32_t* error_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_EVICT_H_ */

/*
 * pkv_diff.h -- C ABI of differential attention over the paged cache: a head's output is the difference
 * of two softmax maps with a learned factor, for one query token and for many.
 *
 * A layer of this kind keeps two keys and one value a token and kv head.  They stand in ordinary pools: a K row
 * of d elements holds the first map's key in its first half and the second's in its second half, a q row the two
 * queries likewise, a V row d elements.  So pkv_kv_step_tables, the bf16 appends and copies, and pkv_kv_evict
 * serve it as they are.
 *
 * With x_m,t the logit of pkv_score_rules for the m-th halves (scale * q_m . k_m,t, then cap and distance bias), and
 * a_m its softmax over the keys that the query sees (the formula of "Transformer模型中的KV Cache优化推理策略",
 * yutianautomatic.com, for each half),
 *     y   = sum_t (a_1,t - lambda a_2,t) V_t,
 *     out = y,  or  y / sqrt(mean(y^2) + norm_eps) * norm_weight  with a norm over the head's d elements.
 * A row that sees no key is zero, whatever lambda and norm_weight are.  The maps' outputs are made
 * apart, with unnormalised fp32 weights, and then subtracted: an infinity in V that a query sees, or finite V whose weighted sum
 * passes fp32 (|V| up to 2^80 never does), may give NaN.
 *
 * The conventions of pkv.h hold (device pointers, nothing allocated, kernels enqueued on `stream` only, status
 * codes, device errors through error_word, dense layouts).
 */
#ifndef PKV_DIFF_H_
#define PKV_DIFF_H_

#include "pkv_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a differential layer has learned. */
typedef struct pkv_diff_params {
  const float* lambdas;      /* fp32 factors of the second map: [Hq], or [rows of q, Hq] */
  int32_t lambda_rows;       /* 0: one row of lambdas serves every row of q; 1: each row has its own */
  float norm_eps;            /* finite and > 0 where norm_weight is given */
  const float* norm_weight;  /* [d] fp32 (a constant factor of the output belongs into it), or NULL: no norm */
} pkv_diff_params;

/*
 * pkv_diff_decode_workspace_bytes -- bytes of device workspace for the decode calls below; score_stride is
 * that of pkv_paged_diff_decode_attention_scores, 0 for pkv_paged_diff_decode_attention.  As of the other decode
 * calls: zero-filled before its first use, left ready by each call, one each for calls that may overlap on the
 * GPU.  Returns 0 if the arguments are invalid.
 */
size_t pkv_diff_decode_workspace_bytes(const pkv_dims* dims, int32_t score_stride);

/*
 * pkv_paged_diff_decode_attention -- one query token a sequence, at position L_b - 1.
 *   out, q        : [B, Hq, d] bf16.
 *   params        : lambdas [Hq] or [B, Hq].
 *   rules         : or NULL (plain softmax over all keys).  alibi_slopes serve both maps of a head.
 *   scale         : of the half heads' products (1 / sqrt(d / 2) for the usual one).
 *   other arguments, supported sizes and errors : as pkv_paged_decode_attention_rules.  With
 *                   PKV_DECODE_INPUTS_READY lambdas and norm_weight may still be written by the preceding work.
 */
int pkv_paged_diff_decode_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens, float scale,
                                    const pkv_diff_params* params, const pkv_score_rules* rules, void* workspace,
                                    size_t workspace_bytes, const pkv_dims* dims, uint32_t flags, int32_t* error_word,
                                    void* stream);

/*
 * pkv_paged_diff_decode_attention_scores -- the same, which also adds the weight that each key receives, summed
 * over the query heads of its kv head, into the layer's scores ("How KV Sparsity...", section "2. Attention
 * modification", with the differential weight in place of the probability):
 *     scores_out[b, g, t] = scores[b, g, t] + sum_h |a_1,t - lambda_h a_2,t|   for the t < L_b that the query sees,
 *                           scores[b, g, t]                                    for the other t < L_b.
 *   scores, scores_out : [B, Hkv, score_stride] fp32; may be the same array and may not overlap otherwise.  Entries
 *                        from L_b on are left as they were.  Keys from score_stride on get no score, and are reported
 *                        (PKV_DEV_BAD_CONTEXT_LEN).  A logit of NaN or +infinity makes a map's weights NaN, as the
 *                        formula does: those of every key that the query sees.  Keys of a block outside the
 *                        pool get no weight.
 */
int pkv_paged_diff_decode_attention_scores(void* out, const float* scores, float* scores_out, int32_t score_stride,
                                           const void* q, const void* k_cache, const void* v_cache,
                                           const int32_t* block_tables, const int32_t* context_lens, float scale,
                                           const pkv_diff_params* params, const pkv_score_rules* rules, void* workspace,
                                           size_t workspace_bytes, const pkv_dims* dims, uint32_t flags,
                                           int32_t* error_word, void* stream);

/*
 * pkv_diff_prefill_workspace_bytes -- bytes of device workspace for pkv_paged_diff_prefill_attention, as
 * pkv_prefill_workspace_bytes (no preparation).  Returns 0 if the arguments are invalid.
 */
size_t pkv_diff_prefill_workspace_bytes(const pkv_dims* dims, int32_t total_tokens);

/*
 * pkv_paged_diff_prefill_attention -- many query tokens a sequence, causal: prompts, chunks, mixed steps.
 *   params          : lambdas [Hq] or [total_tokens, Hq] (the packed rows).
 *   the weights     : two bf16 terms for rows over at most 512 keys.  Over more, one term (8 bits) but for the nearest
 *                     keys, those of one 64-key step in six, which take two.  Their sums are fp32.  The maps are
 *                     subtracted, so one term shows more here than in pkv_paged_prefill_attention: normal values over
 *                     16384 keys in no order are 0.0025 off in norm, where a bf16 output by itself is 0.0017.
 *   other arguments, supported sizes and errors : as pkv_paged_prefill_attention.
 */
int pkv_paged_diff_prefill_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_tables, const int32_t* context_lens,
                                     const int32_t* query_starts, int32_t total_tokens, float scale,
                                     const pkv_diff_params* params, const pkv_score_rules* rules, void* workspace,
                                     size_t workspace_bytes, const pkv_dims* dims, int32_t* error_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_DIFF_H_ */

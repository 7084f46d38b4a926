/*
 * pa_sample.h -- from logits to the next tokens (C ABI).
 *
 * What stands behind a decode step's attention and the model's output projection: the
 * filters of a request (temperature, top-k, top-p, min-p) applied to a row of logits, and
 * either a token drawn from what is left (pa_sample_tokens) or the distribution itself as a
 * row of probabilities (pa_sampling_probs), which pa_verify_tree (pa_draft.h) takes as
 * target_probs and draft_probs: a drafter's tokens drawn by pa_sample_tokens follow the rows
 * that pa_sampling_probs writes for the same logits and filters.
 *
 * The distribution of a row.  x are its logits (NaN counts as -inf), m the largest, and the
 * order is by falling x, equal logits by rising index:
 *   weight     w_v = exp((x_v - m) / temperature); 1 where x_v = m (so a row whose largest
 *              logits are +inf is uniform over them), 0 where x_v = -inf;
 *   top-k      the first top_k tokens of the order stay (top_k <= 0, or >= V: all);
 *   top-p      of those, a token stays if the weights before it in the order sum to less
 *              than top_p times the sum of all of them; the first always stays (top_p >= 1:
 *              all);
 *   min-p      of those, a token stays if w_v >= min_p (the largest weight is 1; min_p > 1
 *              counts as 1, min_p <= 0: all);
 *   temperature 0: the first token with x_v = m alone (the filters change nothing).
 * Probabilities are the weights left over their sum.
 *
 * Temperatures from 2^-60 to 2^80 are used as they are, lower ones above 0 and higher ones as
 * these.
 *
 * Weights are computed to about 2^-28 relative (2^-25 for the smallest) and held as whole
 * numbers of 2^-44 (2^-(62 - ceil(log2 V)) for V > 2^18).  Their sums are the same from call to
 * call, and off by at most about 2^-28 of the sum and half a unit a token (2^-27 of the largest
 * weight for V = 2^18, 2^-23 for 2^20; a row of all equal logits under a large one comes near
 * that, ordinary rows stay at 2^-32).  Borders and draws come out as they do in 64 bits unless
 * what they compare is closer than that.  (A weight below half of the unit is never drawn;
 * pa_sampling_probs still writes its probability.)
 *
 * Conventions (streams, device-side checks, err_flag) as in pa.h, but logits and
 * probabilities need only be aligned to their type: rows of any length and stride.
 */
#ifndef PA_SAMPLE_H
#define PA_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"
#include "pa_draft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_SAMPLE_MAX_VOCABULARY (1 << 20)

/*
 * Draw one token for each of R rows.
 *   tokens_out     [R] int32 (written): the first token, in index order, whose running sum of
 *                  the weights left exceeds uniforms[r] times their sum.
 *   probs_out      [R] fp32 (written), or NULL: the token's probability.
 *   logits         [R] rows of V, fp32 or bf16 (logit_dtype, PA_PROB_*), rows logit_stride
 *                  elements (>= V) apart.
 *   temperature, top_p, min_p  [R] fp32, top_k [R] int32, device; each may be NULL (1, and off).
 *   uniforms       [R] fp32 in [0, 1).
 * A row with a temperature that is negative or not finite, or a NaN among top_p and min_p,
 * gives token -1 and probability 0 (PA_FLAG_SAMPLING), as does a row without any logit above
 * -inf (PA_FLAG_PROBABILITY).  1 <= V <= PA_SAMPLE_MAX_VOCABULARY, R <= 2^20.
 */
pa_status pa_sample_tokens(int32_t *tokens_out, float *probs_out, const void *logits, int64_t logit_stride,
                           int logit_dtype, const float *temperature, const int32_t *top_k,
                           const float *top_p, const float *min_p, const float *uniforms, int R, int V,
                           int *err_flag, void *stream);

/*
 * The distributions of R rows.
 *   probs_out      [R] rows of V, fp32 or bf16 (prob_dtype), rows prob_stride elements (>= V)
 *                  apart (written; what lies between rows is not).  Must not overlap logits.
 * Other arguments as in pa_sample_tokens; a row that gives no token there is all zeros here.
 */
pa_status pa_sampling_probs(void *probs_out, int64_t prob_stride, int prob_dtype, const void *logits,
                            int64_t logit_stride, int logit_dtype, const float *temperature,
                            const int32_t *top_k, const float *top_p, const float *min_p, int R, int V,
                            int *err_flag, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_SAMPLE_H */

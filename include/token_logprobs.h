/*
 * token_logprobs.h -- C ABI of what is read off a matrix of logits on MI355X (gfx950): the
 * log-probability of one given token a row, the entropy, the top alternatives, and the
 * gradient with respect to the logits.
 *
 * Conventions and the order of validation are gemm_i8.h's. Rows may start at any address
 * aligned to the element. All arithmetic is FP32; logits of 16 bits are widened exactly.
 *
 * Per row of V logits x (M rows, leading dimension ld), with m = max x and
 * s = sum_j exp(x_j - m):
 *     lse     = m + log s
 *     logprob = x_t - lse                      for the row's token t
 *     entropy = log s - sum_j (x_j - m) exp(x_j - m) / s
 *     alternatives: the `top` largest logits in descending order, equal ones by ascending
 *     index, as x - lse and their indices
 *
 * Edges:
 *   - a token below 0 marks a row without one (padding): logprob 0, no gradient from it. A
 *     token >= V gives a NaN logprob, and NaN in that row's gradient.
 *   - a logit of -infinity has probability 0. A row of nothing else has lse and logprobs
 *     -infinity (0 without a token), entropy 0 and gradient 0.
 *   - a NaN or +infinity makes the row's lse, entropy, logprobs and gradient NaN. Among
 *     the alternatives a NaN comes after every number.
 *   - 0.0 and -0.0 are equal.
 */
#ifndef TOKEN_LOGPROBS_H
#define TOKEN_LOGPROBS_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm_dtype.h"
#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most alternatives token_logprobs returns for a row. */
#define TOKEN_LOGPROBS_MAX_TOP 64

/*
 * tokens: M indices of token_bytes (4 or 8) each. logprobs, entropy, lse: M floats each;
 * entropy and lse may be NULL. top: 0 to 64 and at most V (else SGEMM_EINVAL_ARG);
 * top_logprobs: M x top floats, top_tokens: M x top int64, packed, not NULL where top > 0.
 * V must be at least 1 where M is (else SGEMM_EINVAL_DIM).
 *
 * workspace: few rows are split over workgroups along V and joined by a second kernel.
 * Caller-owned device memory of token_logprobs_workspace_size bytes, 16-byte aligned;
 * SGEMM_EINVAL_ARG if smaller. NULL with 0 bytes runs without a split. No initialisation
 * needed; calls that share one must not overlap in time. Results do not depend on timing:
 * repeated calls with the same arguments give identical bits.
 */
int token_logprobs(int M, int V,
                   const void *logits, int dtype, int64_t ld,
                   const void *tokens, int token_bytes,
                   float *logprobs, float *entropy, float *lse,
                   int top, float *top_logprobs, int64_t *top_tokens,
                   void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * token_logprobs, and what rounding lse to FP32 leaves off it: lse + lse_low is m + log s with the
 * error of log s alone, however large m is. lse_low holds M floats, or is NULL; 0 where |lse| < 64,
 * whose rounding, 2^-19 at most, is within the exponential's own error.
 */
int token_logprobs_low(int M, int V,
                       const void *logits, int dtype, int64_t ld,
                       const void *tokens, int token_bytes,
                       float *logprobs, float *entropy, float *lse, float *lse_low,
                       int top, float *top_logprobs, int64_t *top_tokens,
                       void *workspace, size_t workspace_bytes,
                       void *stream);

/* Bytes of workspace token_logprobs uses for this shape on the current device (0: none,
 * also for arguments it would refuse and where no device answers). */
size_t token_logprobs_workspace_size(int M, int V, int dtype, int top);

/*
 * The gradient of sum_i g_logprob_i logprob_i + g_entropy_i entropy_i + g_lse_i lse_i with
 * respect to the logits, from the lse and entropy that token_logprobs returned:
 *     p_j  = exp(x_j - lse)
 *     dx_j = g_logprob ([j = t] - p_j) - g_entropy p_j (x_j - lse + entropy) + g_lse p_j
 * g_logprob, g_entropy and g_lse are M floats each; any may be NULL (zeros). entropy is
 * needed where g_entropy is given. grad has the logits' type and leading dimension ldg,
 * and may be the logits themselves (same pointer and leading dimension: in place); any
 * other overlap is SGEMM_EALIAS. The alternatives have no gradient.
 */
int token_logprobs_backward(int M, int V,
                            const void *logits, int dtype, int64_t ld,
                            const void *tokens, int token_bytes,
                            const float *lse, const float *entropy,
                            const float *g_logprob, const float *g_entropy,
                            const float *g_lse,
                            void *grad, int64_t ldg,
                            void *stream);

/*
 * The same with lse_low (M floats as token_logprobs_low wrote them, or NULL for zeros) taken off too:
 *     p_j  = exp(x_j - lse - lse_low)
 * For logits far from 0 an FP32 lse alone is too coarse: at 60000 its rounding moves every p_j by 0.2 %,
 * and a row of nothing but the type's lowest value (a mask that leaves nothing) would get p_j = 1
 * where 1 / V is meant.
 */
int token_logprobs_backward_low(int M, int V,
                                const void *logits, int dtype, int64_t ld,
                                const void *tokens, int token_bytes,
                                const float *lse, const float *lse_low, const float *entropy,
                                const float *g_logprob, const float *g_entropy,
                                const float *g_lse,
                                void *grad, int64_t ldg,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TOKEN_LOGPROBS_H */

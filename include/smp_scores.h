/*
 * smp_scores.h -- C ABI of libsmp, third part: log probabilities of tokens
 * under a block of logits, and what a draft model is trained on.
 *
 * smp_token_logprobs scores tokens that were given or drawn: their log
 * probabilities, the entropy of each row's distribution and its likeliest
 * tokens.  Kept for the target's rows, the likeliest tokens and their log
 * probabilities are the teacher's record from which smp_distill trains the
 * draft model, so that smp_spec_verify accepts more of its drafts;
 * smp_token_logprobs_grad is the gradient for a loss of log probabilities and
 * entropies.
 *
 * The conventions are those of smp.h: calls are asynchronous on the caller's
 * stream, allocate nothing, may be captured in a CUDA graph, and report what
 * the host can see as a return code before anything is launched.  Problems of
 * one row give that row NaN (ids: -1) and OR a flag into the optional device
 * status word, which the call clears first.  Results do not depend on the
 * launch shape beyond the last bits of a sum, and are the same from run to run.
 *
 * Rows.  `logits` is device memory, [rows, vocab] elements of `dtype`, rows
 * `stride` elements apart (stride >= vocab; what lies between rows is neither
 * read nor written), base aligned to the element size.  Row r's temperature T
 * is temperatures[r] (device, [rows] float), or `temperature` when
 * `temperatures` is NULL; it has to lie in [SMP_MIN_TEMPERATURE,
 * SMP_MAX_TEMPERATURE], else the host answers SMP_ERR_INVALID_ARG and the
 * device SMP_ROW_BAD_PARAMS.  With y = z / T, p = softmax(y).  A logit that is
 * -inf or NaN has probability 0, a row whose maximum is not finite is an error
 * row (SMP_ROW_NONFINITE): the sampler's readings.  Sums and statistics are
 * held in binary32 or wider, and gradients are rounded once to `dtype`.
 *   rows 0 .. 2^24; vocab 1 .. SMP_MAX_VOCAB; stride up to 2^40.
 */
#ifndef SMP_SCORES_H
#define SMP_SCORES_H

#include "smp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most ids, alternatives or teacher's tokens per row. */
#define SMP_MAX_ROW_IDS 128
/* Range of the temperatures. */
#define SMP_MIN_TEMPERATURE 0x1p-30f
#define SMP_MAX_TEMPERATURE 0x1p+30f

/* Flag OR-ed into the device status word, beside those of smp.h and smp_cache.h. */
#define SMP_ROW_BAD_TOKEN 128   /* a token id at or past the vocabulary's end */

/*
 * smp_token_logprobs -- log probabilities of given tokens, entropies and
 * likeliest tokens, in one pass.
 *
 *   ids          device, [rows, count] int32, or NULL with count 0.  A negative
 *                id is no token (padding): its log probability is 0.  An id >=
 *                vocab gets NaN and SMP_ROW_BAD_TOKEN.  Ids may repeat.
 *   count, top   0 .. SMP_MAX_ROW_IDS.
 *   out_logprobs device, [rows, count] float (NULL with count 0): ln p of each
 *                id; -inf where p = 0.
 *   out_entropy  device, [rows] float, or NULL: -sum p ln p, in nats.
 *   out_top_ids, out_top_logprobs  device, [rows, top] int32 and float (NULL
 *                with top 0): the tokens with the largest logits, in descending
 *                order, the lower id first among equal ones.  Tokens of
 *                probability 0 (-inf or NaN logits) are none: where fewer than
 *                `top` are left, the rest is id -1 with -inf.  Rows with hundreds
 *                of equal logits among these, as under a finite mask that leaves
 *                fewer than `top`, are read `top` times: mask with -inf.
 * Something has to be asked for (count, top or out_entropy).  A row whose ids
 * are all padding is not read when only log probabilities are asked for.
 */
smp_status smp_token_logprobs(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                              float temperature, const float* temperatures, const int32_t* ids, int32_t count,
                              int32_t top, float* out_logprobs, float* out_entropy, int32_t* out_top_ids,
                              float* out_top_logprobs, int32_t* status, void* stream);

/*
 * smp_token_logprobs_grad -- the gradient of a loss in the logits, given its
 * gradients g (in the log probabilities) and h (in the entropies), with H the
 * entropy and G = sum of the row's g:
 *   dz_j = (1/T) (sum of g_i with ids_i = j  -  p_j (G + h (ln p_j + H)))
 * It needs nothing of the forward call: the row is read once, kept on chip and
 * its statistics made again.
 *
 *   ids, count   as above, 0 .. SMP_MAX_ROW_IDS; padding has no gradient, and
 *                an id >= vocab makes an error row (SMP_ROW_BAD_TOKEN).
 *   grad_logprobs  device, [rows, count] float (NULL with count 0).
 *   grad_entropy   device, [rows] float, or NULL (none).
 *   out_grad     device, like logits with its own stride, written for every
 *                row; may be the logits themselves with the same stride (in
 *                place).  Rows that overlap the logits otherwise are refused; two
 *                blocks of columns of one tensor do not.  Rows that do not lie to
 *                16-byte boundaries as the logits' do are written element by
 *                element, which takes up to 1.4 times as long.
 * A row without a token and with h = 0 is not read: its gradient is 0.
 */
smp_status smp_token_logprobs_grad(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                                   float temperature, const float* temperatures, const int32_t* ids, int32_t count,
                                   const float* grad_logprobs, const float* grad_entropy, void* out_grad,
                                   int64_t grad_stride, int32_t* status, void* stream);

/*
 * smp_distill -- the divergence of a student's rows from a teacher of whom
 * each row's likeliest tokens are known, and its gradient in the same pass.
 * With the row's teacher ids i_1 .. i_k and values l_1 .. l_k, s = softmax(z/T)
 * the student's distribution and s_rest its mass outside the ids:
 *   tail 0:  t = softmax(l) over the row's ids, r = 0;
 *   tail 1:  t_n = exp(l_n), r = max(0, 1 - sum t): the teacher's mass outside
 *            the ids, compared with the student's as one more outcome;
 *   loss = sum_n t_n (ln t_n - ln s_{i_n}) + r (ln r - ln s_rest)
 *   dz_j = (w/T) (s_j (sum t + r) - sum of t_n with i_n = j
 *                 - [j not among the ids] r s_j / s_rest)
 * The values are log probabilities at the temperature T, as smp_token_logprobs
 * gives them with the teacher's logits (for tail 0 anything that differs from
 * them by a constant per row, logits divided by T for instance).  Terms with
 * t_n = 0 are 0; t_n > 0 where s is 0 makes the loss +inf (its gradient is
 * finite).  Where the student has no mass at all outside the ids, r counts as 0.
 *
 *   teacher_ids  device, [rows, count] int32; count 1 .. SMP_MAX_ROW_IDS.  A
 *                negative id is an unused place.  A row of unused places is no
 *                token: it is not read, its loss is 0 and its gradient 0.  An id
 *                >= vocab makes an error row (SMP_ROW_BAD_TOKEN).  An id that
 *                repeats counts with the sum of its t.
 *   teacher_logprobs  device, [rows, count] float; a NaN or +inf, no finite
 *                value (tail 0) or a sum of t above 1 + 2^-6 (tail 1) makes an
 *                error row (SMP_ROW_BAD_PARAMS).
 *   weights      device, [rows] float, the gradients w of the row losses, or
 *                NULL (1); not used without out_grad.
 *   out_loss     device, [rows] float: the row losses, not weighted.
 *   out_grad     NULL (the loss alone), or as for smp_token_logprobs_grad.
 */
smp_status smp_distill(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                       float temperature, const float* temperatures, const int32_t* teacher_ids,
                       const float* teacher_logprobs, int32_t count, int32_t tail, const float* weights,
                       float* out_loss, void* out_grad, int64_t grad_stride, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SMP_SCORES_H */

/*
 * vce_policy.h -- C ABI of the post-training losses on [T, V] logits with a large vocabulary
 * (libvce.so):
 *
 *   ce_logprobs_forward, _backward      log-probabilities of chosen tokens, entropies of the rows
 *   policy_loss_forward, _backward,     the clipped policy loss with a KL and an entropy term, its
 *   _forward_backward                   gradient, and both in one pass
 *   preference_loss_forward, _backward  the preference loss over pairs of packed sequences
 *
 * The conventions of vce.h hold: device pointers owned by the caller, nothing allocated, work
 * only enqueued on `s`, row-major matrices with a leading dimension, element alignment, fp32
 * arithmetic, VCE_OK or a negative host-detected error, device-detected errors in a status word.
 * No call keeps state on the device between calls or shares any between launches, so calls may
 * run at once on any streams and in captured graphs, provided that their outputs differ.
 *
 * Below, x_ij = z_ij / temperature, p_i = softmax(x_i), and t = ids[i] (actions[i], labels[i]) is
 * the row's token.  A row whose token is ignore_index is left out: its logits are not read, what
 * it returns is +0.0 and so is its gradient.  Any other token outside [0, V) makes *status
 * VCE_ERR_LABEL, what the row returns NaN, and its gradient +0.0.  Masked logits may be -inf or
 * any value far below the others, such as -1e10 or the type's lowest.  A logit whose product with
 * log2(e) / temperature passes fp32 counts as -inf; of a row of nothing but -inf everything is NaN, and
 * it has no gradient (+0.0).  A row of nothing but lesser masks is a row like any other (where that
 * product of its largest logit but the token is 2^31 or more in size, logits count as equal when their
 * products round to the same fp32 number).  A NaN or +inf among a row's logits (or one whose product passes
 * fp32 upwards) makes all that the row returns, and its whole gradient, NaN.
 */
#ifndef VCE_POLICY_H
#define VCE_POLICY_H

#include "vce.h"
#include "vce_logits.h"   /* VCE_ERR_OFFSETS */

#ifdef __cplusplus
extern "C" {
#endif

#define VCE_MAX_POLICY_V 2097152      /* most columns of every call of this header */
#define VCE_MAX_POLICY_T 8388608      /* most rows */
#define VCE_MAX_PAIRS 4194304         /* most pairs of preference_loss_* */

/*
 * ce_logprobs_forward -- per row
 *   logprobs[i] = log p_it,   entropy[i] = -sum_j p_ij log p_ij
 * The logarithm is -softplus(L' - x_t) with L' the log-sum-exp of the other columns, and the
 * entropy a sum of terms >= 0 that splits off the token's own probability, so a row that is sure of
 * its token keeps its digits (where it is sure of another column, the entropy of the rest among itself is
 * off by up to about 3e-7).  A token on a column of -inf has log-probability -inf.
 *   logits, dt, T, V, ld   as ce_forward; V <= VCE_MAX_POLICY_V
 *   ids, ignore_index      [T] int64
 *   temperature            finite, > 0, with a finite reciprocal
 *   logprobs [T] fp32, written;  entropy [T] fp32, written, or NULL (not worked out, and
 *                          row_stats then hold none for ce_logprobs_backward's grad_entropy)
 *   row_stats              [T * VCE_ROW_STATS] fp32, 16-byte aligned: for the backward
 *   status                 [1] int32: 0, VCE_ERR_LABEL, or 105 .. 109 when a bounded device-side
 *                          wait gave up (the rows that it may have touched are NaN then)
 */
VCE_API int ce_logprobs_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                const int64_t* ids, int64_t ignore_index, float temperature, float* logprobs,
                                float* entropy, float* row_stats, int32_t* status, vce_stream_t s);

/*
 * ce_logprobs_backward -- with a = grad_logprobs[i] and b = grad_entropy[i] (NULL: 0),
 *   grad_ij = (a ([j = t] - p_ij) - b p_ij (log p_ij + entropy_i)) / temperature
 *  row_stats, ids, temperature  as given to and written by the forward, which worked the entropy
 *                out if grad_entropy is given (else the gradient is NaN)
 *   grad_logprobs  [T] fp32 or NULL (0);  grad_logits  [T, ld_grad] of dtype grad_dt, written;
 *                VCE_ERR_ARG if it overlaps the logits.  Columns behind a device-side wait that
 *                gave up after 2 s hold NaN.
 */
VCE_API int ce_logprobs_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                 const int64_t* ids, float temperature, const float* row_stats,
                                  const float* grad_logprobs, const float* grad_entropy, void* grad_logits,
                                 vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s);

/* The constants of the policy loss (host memory, read during the call). */
typedef struct {
    float clip_low, clip_high; /* the ratio is clipped to [1 - clip_low, 1 + clip_high]; >= 0 */
    float dual_clip;           /* 0: none; else >= 1, the bound for negative advantages */
    float kl_coef;             /* >= 0 or < 0, finite; not 0 only with ref_logprobs */
    float entropy_coef;        /* finite; 0: no entropy term */
} vce_policy_params;

/*
 * policy_loss_forward -- with lp_i = log p_it, ratio r_i = exp(lp_i - old_logprobs[i]) (NULL: the
 * policy's own, r = 1), A_i = advantages[i], d_i = ref_logprobs[i] - lp_i, H_i the row's entropy:
 *   s_i = min(r_i A_i, clip(r_i, 1 - clip_low, 1 + clip_high) A_i)
 *         and, with dual_clip, at least dual_clip A_i where A_i < 0
 *   loss_rows[i] = weights[i] (-s_i + kl_coef (exp(d_i) - d_i - 1) - entropy_coef H_i)
 * loss_out is their sum (SUM) or that over the rows that are not left out (MEAN; NaN when none).
 *   actions, ignore_index  [T] int64, the rows' tokens
 *   old_logprobs, ref_logprobs, weights  [T] fp32 or NULL;  advantages  [T] fp32
 *   p                      host pointer
 *   loss_rows [T], logprobs [T] fp32, written;  entropy [T] fp32, written, or NULL
 *   loss_out               [1] fp32, written for SUM / MEAN
 *   row_stats, status      as ce_logprobs_forward (the row_stats here are policy_loss_backward's)
 * An advantage of 0 makes s_i 0 whatever the ratio.
 */
VCE_API int policy_loss_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                const int64_t* actions, int64_t ignore_index, float temperature,
                                const float* old_logprobs, const float* advantages, const float* ref_logprobs,
                                const float* weights, const vce_policy_params* p, vce_reduction red,
                                float* loss_rows, float* loss_out, float* logprobs, float* entropy,
                                float* row_stats, int32_t* status, vce_stream_t s);

/*
 * policy_loss_backward -- the gradient w.r.t. the logits from what policy_loss_forward saved (through
 * lp and H; old_logprobs, advantages, ref_logprobs and weights are constants).
 *   logits .. temperature, red: as given to the forward;  row_stats: from it
 *   grad_output   fp32 [1] (SUM, MEAN) or [T] (NONE);  grad_logits as ce_logprobs_backward
 */
VCE_API int policy_loss_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                 const int64_t* actions, float temperature, vce_reduction red,
                                 const float* row_stats, const float* grad_output, void* grad_logits,
                                 vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s);

/*
 * policy_loss_forward_backward -- both with one read of the logits, for callers that know grad_output
 * when the forward runs: each row is held in the shared memory of a thread-block cluster between
 * its statistics and its gradient (rows too long for that are read again).  The arguments and
 * results are the two calls' (where a wait gave up, NaN over the columns of the block that waited too, in all of
 * its rows); for MEAN *loss_out holds 1/N while the work runs, and row_stats is scratch.
 */
VCE_API int policy_loss_forward_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                         const int64_t* actions, int64_t ignore_index, float temperature,
                                         const float* old_logprobs, const float* advantages,
                                         const float* ref_logprobs, const float* weights,
                                         const vce_policy_params* p, vce_reduction red, const float* grad_output,
                                         float* loss_rows, float* loss_out, float* logprobs, float* entropy,
                                         float* row_stats, void* grad_logits, vce_dtype grad_dt, int64_t ld_grad,
                                         int32_t* status, vce_stream_t s);

typedef enum { VCE_PREF_SIGMOID = 0, VCE_PREF_HINGE = 1, VCE_PREF_IPO = 2 } vce_preference_kind;

/* The constants of the preference loss (host memory, read during the call). */
typedef struct {
    vce_preference_kind kind;
    float beta;            /* finite, > 0 */
    float label_smoothing; /* [0, 1/2]; SIGMOID alone, else 0 */
    float margin;          /* finite */
    int average;           /* 1: a sequence's sum is divided by the number of its tokens */
} vce_preference_params;

/*
 * preference_loss_forward -- the T rows hold 2 P sequences one after another, sequence q the rows
 * offsets[q] .. offsets[q + 1]; sequence 2 p is the preferred one of pair p, 2 p + 1 the other.
 * With l_i = log p_it - ref_logprobs[i] (NULL: no reference, 0):
 *   rewards[q] = beta sum of l_i over the sequence's rows (their mean with average; 0 of no rows)
 *   x_p = rewards[2 p] - rewards[2 p + 1] - margin, and pair_losses[p] by kind
 *     SIGMOID  -(1 - eps) log sigma(x) - eps log sigma(-x),  eps = label_smoothing
 *     HINGE    max(0, 1 - x)
 *     IPO      ((x - 1/2) / beta)^2
 * loss_out is their sum (SUM) or mean over the P pairs (MEAN; NaN when P = 0).  Rows whose label is
 * ignore_index, and rows in no sequence (padding before the first or behind the last), are left out.
 *   labels, ignore_index   [T] int64
 *   offsets                [2 P + 1] int64, ascending, in [0, T]; where they are not, every pair's
 *                          loss and rewards are NaN, no row has a gradient, and *status is
 *                          VCE_ERR_OFFSETS
 *   P                      0 .. VCE_MAX_PAIRS
 *   ref_logprobs           [T] fp32 or NULL
 *   p                      host pointer
 *   pair_losses [P], rewards [2 P], logprobs [T] fp32, written;  loss_out [1] fp32, written for SUM / MEAN
 *   row_stats, status      as ce_logprobs_forward.  A sequence with an error in one of its rows, or a row of
 *                          nothing but -inf, has a NaN reward, and its pair a NaN loss and no gradient.
 */
VCE_API int preference_loss_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                    const int64_t* labels, int64_t ignore_index, float temperature,
                                    const int64_t* offsets, int64_t P, const float* ref_logprobs,
                                    const vce_preference_params* p, vce_reduction red, float* pair_losses,
                                    float* loss_out, float* rewards, float* logprobs, float* row_stats,
                                    int32_t* status, vce_stream_t s);

/*
 * preference_loss_backward -- the gradient w.r.t. the logits from what preference_loss_forward saved.
 *   logits .. temperature, P, red: as given to the forward;  row_stats: from it
 *   grad_output   fp32 [1] (SUM, MEAN) or [P] (NONE);  grad_logits as ce_logprobs_backward
 */
VCE_API int preference_loss_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                     const int64_t* labels, float temperature, int64_t P, vce_reduction red,
                                     const float* row_stats, const float* grad_output, void* grad_logits,
                                     vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s);

/*
 * Test hooks for the paths of waits that give up, every wait bounded by wait_ns (1 ms .. 2 s), bf16
 * logits and gradients (ld = V), temperature 1, reduction SUM, no row left out.  The kernels return,
 * with their copies landed, and the context stays usable.
 *   vce_test_policy_stall      policy_loss_forward_backward (clipped at 0.2, nothing else) where the last
 *                              block of every cluster never gets its gradient's coefficients, after the
 *                              statistics have been exchanged
 *   vce_test_policy_bwd_stall  policy_loss_backward where a row's last block never gets its last stage
 */
VCE_API int vce_test_policy_stall(const void* logits, int64_t T, int64_t V, const int64_t* actions,
                                  const float* advantages, const float* grad_output, float* loss_rows,
                                  float* loss_out, float* logprobs, float* row_stats, void* grad_logits,
                                  uint64_t wait_ns, int32_t* status, vce_stream_t s);
VCE_API int vce_test_policy_bwd_stall(const void* logits, int64_t T, int64_t V, const int64_t* actions,
                                      const float* row_stats, const float* grad_output, void* grad_logits,
                                      uint64_t wait_ns, vce_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* VCE_POLICY_H */

/*
 * vce_logits.h -- C ABI of the operators around the cross-entropy on [T, V] logits with a large
 * vocabulary (libvce.so):
 *
 *   ce_topk                        a row's K largest logits and its log-sum-exps
 *   ce_distill_forward, _backward, the distillation loss against a teacher's top K logits, its
 *   _forward_backward              gradient, and both in one pass
 *   logits_process, _backward      penalties for repeated tokens, biases, temperature and masks on
 *                                  logits before sampling or a loss, and the gradient through them
 *
 * The conventions of vce.h hold: device pointers owned by the caller, nothing allocated, work
 * only enqueued on `s`, row-major matrices with a leading dimension, element alignment, fp32
 * arithmetic, VCE_OK or a negative host-detected error, device-detected errors in a status word.
 * No call keeps state on the device between calls or shares any between launches, so calls may
 * run at once on any streams and in captured graphs, provided that their outputs differ.
 */
#ifndef VCE_LOGITS_H
#define VCE_LOGITS_H

#include "vce.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VCE_MAX_TOPK 256            /* most entries per row of ce_topk and ce_distill_* */
#define VCE_MAX_TOPK_V 2097152      /* most columns of ce_topk and ce_distill_* */
#define VCE_MAX_TOPK_T 8388608      /* most rows of every call of this header */

enum {
    VCE_ERR_TEACHER = 2,  /* device-detected: a teacher id outside [0, V) other than -1, an id twice
                             in a row, or a row whose teacher has no finite mass */
    VCE_ERR_PARAM = 3,    /* device-detected: a temperature or repetition penalty not finite and > 0 */
    VCE_ERR_OFFSETS = 4   /* device-detected: row offsets descending or outside their list */
};

/*
 * ce_topk -- the K largest logits of each row, in order, and the log-sum-exp of the row.
 *   values[i][0..K)  the row's K largest logits, descending (fp32, the logits' exact values; -0
 *                    is returned as 0); equal logits in ascending column order
 *   ids[i][0..K)     their columns
 *   lse[i]           log sum_j exp(z_ij / temperature) over all columns
 *   tail_lse[i]      the same over the columns that are not among the K, summed without them (not
 *                    as a difference), so it stays accurate when the K carry nearly all the mass;
 *                    -inf when nothing is left
 * A logit of -inf (a masked column) is never among the K: where a row has fewer than K other
 * logits the remaining entries are (-inf, -1).  +inf and NaN logits: unspecified.
 *   logits, dt, T, V, ld  as ce_forward; V <= VCE_MAX_TOPK_V
 *   K                     1 .. min(V, VCE_MAX_TOPK)
 *   temperature           finite, > 0, with a finite reciprocal
 *   values [T, K] fp32, ids [T, K] int64, lse [T] fp32, tail_lse [T] fp32, written
 * A device-side wait that gives up after 2 s makes the outputs of the rows it may have touched NaN
 * (ids -1).
 */
VCE_API int ce_topk(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld, int K,
                    float temperature, float* values, int64_t* ids, float* lse, float* tail_lse,
                    vce_stream_t s);

/*
 * ce_distill_forward -- the distillation loss of a student's logits against a teacher's top K.
 * With tau the temperature, the outcomes of row i are its teacher entries (the columns ids[i][k],
 * their logits t_k) and "any other column" (the tail):
 *     q_k = exp(t_k / tau) / Z,  q_T = exp(R_i) / Z,  Z = sum_k exp(t_k / tau) + exp(R_i)
 *     p   = softmax(z_i / tau),  p_T = the sum of p over the other columns
 *     loss_rows[i] = tau^2 [ sum_k q_k log(q_k / p_k) + q_T log(q_T / p_T) ]
 * R_i = teacher_tail[i], the log-sum-exp of the teacher's other logits over tau (tail_lse of
 * ce_topk at the same temperature).  Without it (NULL, or R_i = -inf) the teacher is renormalised
 * over its entries (q_T = 0); with K = 1 that is the cross-entropy of ce_forward.  p_T is summed
 * without the entries' columns and the loss is a sum of terms >= 0, so neither a confident
 * student nor one that matches its teacher cancels to 0.
 *
 *   logits, dt, T, V, ld   the student's, as ce_forward; V <= VCE_MAX_TOPK_V
 *   teacher_ids            [T, K] int64.  -1: no entry (anywhere in a row).  A row whose first id
 *                          is -1 has no teacher and is ignored.
 *   teacher_values, tdt    [T, K] fp32 or bf16 logits (any shift; with a tail, the tail's)
 *   teacher_tail           [T] fp32, or NULL
 *   K                      1 .. min(V, VCE_MAX_TOPK)
 *   temperature            finite, > 0, with a finite reciprocal
 *   labels, ignore_index   [T] int64 or NULL: rows whose label is ignore_index are ignored too
 *                          (the label is not read otherwise)
 *   red                    NONE, SUM, or MEAN over the rows that are not ignored (NaN when none)
 *   loss_rows              [T] fp32; +0.0 for ignored rows
 *   loss_out               [1] fp32, written for SUM / MEAN
 *   row_stats              [T * VCE_ROW_STATS] fp32, 16-byte aligned; per row (log-sum-exp of the
 *                          other columns' z / tau, p_T - q_T, 0, weight), weight as ce_forward's
 *   top_grads              [T, K] fp32: tau (p_k - q_k), 0 where there is no entry
 *   status                 [1] int32: 0, VCE_ERR_TEACHER, or 105 .. 109 when a bounded device-side
 *                          wait gave up (the largest of the rows' codes).  A row with an error has a
 *                          NaN loss and no gradient (the one pass's of 105 .. 109: unspecified).
 * A student's logit whose product with log2(e) / temperature is -2^31 or less (a mask: -1e10, the type's
 * lowest value) counts as -inf.  A student row of nothing else has a NaN loss and no gradient; an entry with
 * q_k > 0 on a logit of -inf, and a teacher's tail on nothing but such, make the loss +inf.  A NaN or +inf among a
 * student's logits, or a logit but an entry's whose product is 2^31 or more, makes its loss and its whole gradient
 * NaN (not the status).
 */
VCE_API int ce_distill_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                               const int64_t* teacher_ids, const void* teacher_values, vce_dtype tdt,
                               const float* teacher_tail, int K, float temperature,
                               const int64_t* labels, int64_t ignore_index, vce_reduction red,
                               float* loss_rows, float* loss_out, float* row_stats, float* top_grads,
                               int32_t* status, vce_stream_t s);

/*
 * ce_distill_backward -- the gradient w.r.t. the student's logits from what ce_distill_forward saved:
 *     grad_ij = c_i tau (p_T - q_T) exp(z_ij / tau - L'_i)   (j not an entry; L' in row_stats)
 *     grad_ij = c_i top_grads[i][k]                          (j = teacher_ids[i][k])
 * with c_i as in ce_backward.  Ignored rows are written as +0.0 and their logits are not read.
 *   logits .. temperature: as given to the forward;  row_stats, top_grads: from it
 *   grad_output  fp32 [1] (SUM, MEAN) or [T] (NONE);  grad_logits [T, ld_grad] of dtype grad_dt,
 *                written; VCE_ERR_ARG if it overlaps the logits.  Columns behind a device-side wait
 *                that gave up after 2 s hold NaN.
 */
VCE_API int ce_distill_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                const int64_t* teacher_ids, int K, float temperature, vce_reduction red,
                                const float* row_stats, const float* top_grads, const float* grad_output,
                                void* grad_logits, vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s);

/*
 * ce_distill_forward_backward -- both in one pass over the logits, for callers that know
 * grad_output when the forward runs: each row is held in the shared memory of a thread-block
 * cluster between its statistics and its gradient (rows too long for that are read again).  The
 * arguments and results are the two calls'; for MEAN *loss_out holds 1/N while the work runs.
 */
VCE_API int ce_distill_forward_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                        const int64_t* teacher_ids, const void* teacher_values, vce_dtype tdt,
                                        const float* teacher_tail, int K, float temperature,
                                        const int64_t* labels, int64_t ignore_index, vce_reduction red,
                                        const float* grad_output, float* loss_rows, float* loss_out,
                                        float* row_stats, void* grad_logits, vce_dtype grad_dt,
                                        int64_t ld_grad, int32_t* status, vce_stream_t s);

/*
 * logits_process -- the logits that are sampled from (or trained through):
 *     y = z                                   and, for a token of the row's history,
 *     y = z > 0 ? z / r : z * r               (r the repetition penalty)
 *     y = y - f n - (n > 0 ? p : 0)           (n its count behind the prompt; f, p the frequency
 *                                              and presence penalties)
 *     y = (y + bias) / temperature
 *     out = y where the mask allows the column, -inf elsewhere
 * Each parameter may be NULL (none).  Masked logits have no effect, whatever they hold.
 *   logits, dt, T, V, ld         as ce_forward; V <= 2^28
 *   temperature, repetition, frequency, presence   [T] fp32
 *   history_ids, n_history       [n_history] int64: all rows' tokens, oldest first
 *   history_offsets              [T + 1] int64: row i's tokens are [offsets[i], offsets[i + 1])
 *   prompt_lens                  [T] int64: a row's first so many tokens are its prompt, seen by the
 *                                repetition penalty alone (NULL: 0)
 *   bias_ids, bias_values, n_bias, bias_offsets    [n_bias] int64 (ascending within a row, each
 *                                column once), [n_bias] fp32, [T + 1] int64
 *   mask, mask_ld                [T, mask_ld] 32-bit words, bit j % 32 of word j / 32 allows column j;
 *                                mask_ld >= ceil(V / 32) words
 *   out, out_dt, ld_out          [T, ld_out]; VCE_ERR_ARG if it overlaps the logits
 *   row_status                   [T] int32, written for every row: 0; VCE_ERR_LABEL (a history or
 *                                bias id outside [0, V), or bias ids not ascending);
 *                                VCE_ERR_PARAM (a temperature or repetition penalty that is not
 *                                finite and > 0, or a temperature without a finite reciprocal);
 *                                VCE_ERR_OFFSETS (also a history of 2^30 tokens or
 *                                more).  A row with an error is NaN in every column.
 */
VCE_API int logits_process(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                           const float* temperature, const float* repetition, const float* frequency,
                           const float* presence, const int64_t* history_ids, int64_t n_history,
                           const int64_t* history_offsets, const int64_t* prompt_lens,
                           const int64_t* bias_ids, const float* bias_values, int64_t n_bias,
                           const int64_t* bias_offsets, const int32_t* mask, int64_t mask_ld,
                           void* out, vce_dtype out_dt, int64_t ld_out, int32_t* row_status,
                           vce_stream_t s);

/*
 * logits_process_backward -- the gradient w.r.t. the logits of logits_process:
 *     grad_logits = grad_out / temperature * (history: z > 0 ? 1 / r : r; else 1), +0.0 where masked
 * The penalties n f, p and the biases do not enter.  A row with an error (row_status) is +0.0 in every
 * column.
 *   grad_out, gdt, ld_gout   [T, ld_gout];  logits, dt, ld: the unprocessed ones (read at the
 *                            columns of the history only; may be NULL without a history)
 *   grad_logits, grad_dt, ld_grad   [T, ld_grad]; VCE_ERR_ARG if it overlaps grad_out or the logits
 */
VCE_API int logits_process_backward(const void* grad_out, vce_dtype gdt, int64_t T, int64_t V, int64_t ld_gout,
                                    const void* logits, vce_dtype dt, int64_t ld,
                                    const float* temperature, const float* repetition,
                                    const int64_t* history_ids, int64_t n_history,
                                    const int64_t* history_offsets, const int32_t* mask, int64_t mask_ld,
                                    void* grad_logits, vce_dtype grad_dt, int64_t ld_grad,
                                    int32_t* row_status, vce_stream_t s);

/*
 * Test hooks for the paths of waits that give up, every wait bounded by wait_ns (1 ms .. 2 s), bf16
 * logits and gradients (ld = V), temperature 1, reduction SUM, no tail, no labels.  The kernels return,
 * with their copies landed, and the context stays usable.
 *   vce_test_topk_stall         ce_topk with the last stage of every slice never copied
 *   vce_test_distill_stall      ce_distill_forward_backward where the last block of every cluster never
 *                               gets what its gradient waits for (its coefficients; in rows longer than
 *                               shared memory the last stage), after the statistics have been exchanged
 *   vce_test_distill_bwd_stall  ce_distill_backward where a row's last block never gets its last stage
 */
VCE_API int vce_test_topk_stall(const void* logits, int64_t T, int64_t V, int K, float* values, int64_t* ids,
                                float* lse, float* tail_lse, uint64_t wait_ns, vce_stream_t s);
VCE_API int vce_test_distill_stall(const void* logits, int64_t T, int64_t V, const int64_t* teacher_ids,
                                   const float* teacher_values, int K, const float* grad_output, float* loss_rows,
                                   float* loss_out, float* row_stats, void* grad_logits, uint64_t wait_ns,
                                   int32_t* status, vce_stream_t s);
VCE_API int vce_test_distill_bwd_stall(const void* logits, int64_t T, int64_t V, const int64_t* teacher_ids, int K,
                                       const float* row_stats, const float* top_grads, const float* grad_output,
                                       void* grad_logits, uint64_t wait_ns, vce_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* VCE_LOGITS_H */

/*
 * ga_loss.h -- the losses whose gradients the workers aggregate, part of the
 * C ABI of libga.so (ga.h holds the conventions: ownership, pointers,
 * streams, errors; they apply here unchanged).
 *
 *   ga_top_logits      a teacher's K largest logits of every row, in order,
 *                      with the row's log-sum-exp
 *   ga_distill_loss    distillation from a teacher's top logits: the loss and
 *                      its gradient with respect to the student's logits
 *   ga_balance_loss    a router's balance loss, the tokens every expert got,
 *                      and the gradient with respect to the router's logits
 *
 * The batch is spread over P simulated data-parallel workers, worker i holding
 * tokens[i] rows. Like the extremes of THC's grid, what a loss is normalised
 * by -- the weights' sum, the experts' counts -- is taken over ALL workers'
 * rows, and each worker's gradient is then its part of the whole batch's
 * gradient: the workers' parameter gradients are to be SUMMED
 * (ga_ring_allreduce_sim, GA_SUM), whatever their shares of the batch.
 *
 * Rows: a matrix of worker i has tokens[i] rows; row r starts at element
 *   r * ld of its buffer (ld >= the row's length). Elements of a row past its
 *   length are neither read nor written. Rows need no alignment beyond their
 *   elements' own.
 * Overlap: a buffer reaches from its first row's start to its last row's end,
 *   padding between rows included. An output that overlaps another buffer is
 *   refused, except a gradient that replaces the logits.
 * tokens: host array of P row counts >= 0. Buffers of a worker without rows
 *   are not looked at (they may be null). All workers together hold fewer
 *   than 2^31 rows. No rows at all is a success: the loss is 0 / 0 -> 0.
 * Values: logits are finite or -inf (an entry that is masked out: it has
 *   probability 0, and gradient 0 but for what a teacher's slot on it adds). Rows that do not count (weight 0, mask 0)
 *   are not read and may hold anything; their gradient is written as zeros.
 *   A row that counts and holds NaN or +inf gives NaN, never an access out of
 *   bounds. (A router's sigmoid of +inf is 1, though, and gives numbers.)
 * Results do not depend on timing: no sum's order does (no floating-point
 *   atomics), so two calls on the same inputs give the same bits.
 * Workspaces belong to one call at a time: two calls that may overlap (two
 *   streams, two captured graphs replayed at once) need one each.
 */
#ifndef GA_LOSS_H
#define GA_LOSS_H

#include "ga.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most teacher slots (top logits) of a row, and the most experts. */
#define GA_TOP_MAX 1024
#define GA_MAX_EXPERTS 1024

typedef enum { GA_SCORE_SOFTMAX = 0, GA_SCORE_SIGMOID = 1 } ga_score;

/*
 * ga_top_logits -- for every row x of V logits: its K largest, in descending
 * order, equal values in the order of their columns (-0 equals +0), and
 *   lse = log sum_v exp(x_v / temp)     (binary32 sums; -inf for a row of -inf)
 *   logits    P device matrices of dt, tokens[i] x V, row stride ld
 *   K         1 .. min(V, GA_TOP_MAX)
 *   temp      > 0, finite, log2(e) / temp too (used by lse alone; an lse past
 *             binary32's ends is infinite)
 *   vals      P device matrices of dt, tokens[i] x K, dense: the values (a -0
 *             of the logits as +0)
 *   idx       P device matrices of int32, tokens[i] x K, dense: their columns
 *   lse       null, or P device vectors of tokens[i] binary32 values
 * Rows with NaN: some K columns, none twice, and lse = NaN.
 * Errors (nothing enqueued): GA_EINVAL for a bad size, dt, P, K, temp, null or
 * misaligned pointer, or an output that overlaps another buffer.
 */
ga_status ga_top_logits(const void* const* logits, const int64_t* tokens, int32_t P, int64_t V,
                        int64_t ld, ga_dtype dt, int32_t K, float temp, void* const* vals,
                        int32_t* const* idx, float* const* lse, void* stream);

/*
 * ga_distill_loss -- the forward divergence of a student from a teacher of
 * which a few logits per row are known. With p = softmax(z / temp) over the V
 * logits z of a row and the teacher's probabilities of its K slots
 *   q_k = exp(t_k / temp - L),  L = the teacher's own lse of the row (lse
 *   given: the slots hold what the teacher gives them, less than 1 together)
 *   or log sum_k exp(t_k / temp) (lse null: renormalised over the slots),
 *   row   l_r = temp^2 sum_k q_k (log q_k - log p[idx_k])
 *   loss  = scale * (sum_r w_r l_r) / (sum_r w_r)    over all workers' rows
 *   grad  dz_v = scale w_r / (sum w) temp (p_v sum_k q_k - sum_{idx_k = v} q_k)
 * in binary32 per row, binary64 over the rows; a gradient is rounded once to dt.
 *   logits    P device matrices of dt, tokens[i] x V, row stride ld
 *   idx       P device matrices of int32, tokens[i] x K, dense. A slot whose
 *             column lies outside [0, V) is empty (-1 by custom); a column
 *             may stand in several slots, whose q then add up
 *   vals      P device matrices of vals_dt, tokens[i] x K, dense: the
 *             teacher's logits t (finite, or -inf: q = 0)
 *   lse       null, or P device vectors of tokens[i] binary32 values, finite,
 *             or -inf where the slots are -inf too
 *   K         1 .. GA_TOP_MAX
 *   weight    null (every row 1), or P device vectors of tokens[i] binary32
 *             weights >= 0; a row whose weight is not above 0 does not count
 *   temp      > 0, finite, log2(e) / temp too;  scale  finite (1: none). The
 *             sum in l_r is binary32: its rounding, of about 2^-21, is
 *             multiplied by temp^2, which need not be a binary32 number itself
 *   grad      null (the loss alone), or P device matrices of dt, tokens[i] x
 *             V, row stride ldg. They may be the logits themselves (same
 *             addresses and stride): the gradient then replaces them
 *   row_loss  null, or P device vectors: l_r (0 for a row that does not count)
 *   d_loss    device, 3 binary32 values: sum_r w_r l_r, sum_r w_r, the loss
 *   d_ws      device workspace of ga_distill_loss_ws_bytes(total rows) bytes,
 *             8-byte aligned
 * A row with no slot left, or whose logits are all -inf, has l_r = 0 and a
 * gradient of zeros; its weight counts. Weights that sum to 0: loss and
 * gradients are 0. A slot with q > 0 on a column of -inf gives l_r = +inf.
 * Errors (nothing enqueued): GA_EINVAL as above.
 */
ga_status ga_distill_loss(const void* const* logits, const int64_t* tokens, int32_t P, int64_t V,
                          int64_t ld, ga_dtype dt, const int32_t* const* idx,
                          const void* const* vals, ga_dtype vals_dt, const float* const* lse,
                          int32_t K, const float* const* weight, float temp, float scale,
                          void* const* grad, int64_t ldg, float* const* row_loss, float* d_loss,
                          void* d_ws, size_t ws_bytes, void* stream);
size_t ga_distill_loss_ws_bytes(int64_t rows);

/*
 * ga_balance_loss -- the auxiliary loss that keeps a router's experts evenly
 * used. The rows are cut into groups: group_len = 0 makes one group of all
 * workers' rows; otherwise every worker's rows are cut into groups of
 * group_len consecutive rows (its last one shorter), the loss of every
 * sequence for itself. In a group of n rows that count,
 *   c_e = how many of their K slots name expert e,  f_e = E c_e / (K n),
 *   p_t = softmax(x_t) or sigmoid(x_t) / sum sigmoid(x_t),
 *   L   = 1/n sum_t s_t,  s_t = sum_e f_e p_te;
 *   loss = scale * (sum of L) / (number of groups with n > 0)
 *   grad = scale / (groups) / n * p_te (f_e - s_t)                  (softmax)
 *                               * p_te (1 - sigmoid(x_te)) (f_e - s_t)
 * (the counts are taken as constants: they have no gradient).
 *   logits    P device matrices of dt, tokens[i] x E, row stride ld
 *   E         1 .. GA_MAX_EXPERTS
 *   idx       P device matrices of int32, tokens[i] x K, dense: the experts
 *             that were chosen. A slot outside [0, E) is counted nowhere (-1
 *             by custom: dropped); one that repeats counts again
 *   K         1 .. GA_TOP_MAX
 *   mask      null, or P device vectors of tokens[i] bytes: rows with 0 do
 *             not count
 *   grad      null, or P device matrices of dt, tokens[i] x E, row stride
 *             ldg; may be the logits themselves (same addresses and stride)
 *   d_counts  device int32 [groups][E] with groups =
 *             ga_balance_groups(tokens, P, group_len), worker by worker (may
 *             be null where that is 0)
 *   d_loss    device, 3 binary32 values: sum of the groups' L, the number of
 *             groups that hold a row that counts, the loss
 *   d_ws      device workspace of ga_balance_loss_ws_bytes(tokens, P, E,
 *             group_len) bytes, 8-byte aligned
 * A row whose logits are all -inf (sigmoid: whose sigmoids are all 0) has
 * p = 0; a sigmoid below 2^-126, of a logit below -87.3, is taken as 0. All workers together hold fewer than 2^31 slots.
 * Errors (nothing enqueued): GA_EINVAL as above.
 */
ga_status ga_balance_loss(const void* const* logits, const int64_t* tokens, int32_t P, int32_t E,
                          int64_t ld, ga_dtype dt, const int32_t* const* idx, int32_t K,
                          const uint8_t* const* mask, ga_score score, int64_t group_len,
                          float scale, void* const* grad, int64_t ldg, int32_t* d_counts,
                          float* d_loss, void* d_ws, size_t ws_bytes, void* stream);
int64_t ga_balance_groups(const int64_t* tokens, int32_t P, int64_t group_len);
size_t ga_balance_loss_ws_bytes(const int64_t* tokens, int32_t P, int32_t E, int64_t group_len);

#ifdef __cplusplus
}
#endif

#endif /* GA_LOSS_H */

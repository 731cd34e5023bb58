/*
 * moe_router.h - the router's choice of experts, its balance loss with the
 * per-expert counts, and the gradient of both.
 *
 * A router gives each token t a row of logits l[t][0 .. E).  From them
 *   score    s[t] = softmax(l[t]), or s[t][e] = 1 / (1 + exp(-l[t][e]))
 *   choice   by score plus a bias per expert that only the choice sees:
 *            c[t][e] = s[t][e] + bias[e].  The experts form `groups` runs of
 *            E / groups; a group's value is the sum of its two largest c (of
 *            its one where it has one), and the top_groups groups of the
 *            largest values are kept.  ids[t] are the top_k experts of largest
 *            c within them, in descending order.
 *   weight   w[t][j] = scale * s[t][ids[t][j]], divided by
 *            sum_i s[t][ids[t][i]] + 1e-20 with normalise
 * The choice is that of scores, choices and groups' values in 64 bits: it does not
 * depend on how fp32 rounds them (close ones are computed again); without a bias and
 * with one group it is the order of the logits.  Equal values, those among them that
 * 64 bits do not tell apart (sigmoids of logits above 37 are 1), go to the lowest index.
 * Large top_k are slow: of 18 a tenth of the rows, of 24 nearly all take top_k maxima
 * over all experts in 64 bits.
 *
 * A logit of -inf masks its expert: it is never chosen, has the score 0 and the
 * gradient 0.  A bias of -inf or NaN keeps its expert from being chosen.  Where
 * fewer than top_k experts are left the last ids are -1 with weight 0 (moe_permute
 * skips and reports them).  A row that holds a NaN (under softmax also +inf) gets
 * ids -1, weights NaN and a gradient of NaN.
 *
 * Balance loss over sequences s of T_s rows each (rows seq_offsets[s] ..
 * seq_offsets[s + 1] - 1), with S the number of those that have rows:
 *   q[t]     = s[t] / sum_e s[t][e]   (softmax: s[t] itself; 0 where every logit is
 *              -inf), of the exact scores: rows whose sigmoids fp32 does not hold too
 *   count_se = entries of ids in the sequence's rows that are e
 *   loss     = coef / S * sum_s E / (top_k T_s^2) * sum_e count_se * sum_t q[t][e]
 * which is coef where every expert gets the same.  Counts are constants to the
 * gradient.  Rows of no sequence (padding behind the last) add nothing.
 *
 * Logits are fp32 or bf16, arithmetic is fp32, weights, bias and their gradients
 * fp32; in weights and their gradients a score below 2^-126 is 0.  All pointers
 * except the struct are device pointers; every call is asynchronous on `stream`,
 * allocates nothing, does not synchronise and can be captured.  Results do not depend
 * on the order in which the GPU runs the work.  n = 0 is MOE_OK.
 */
#ifndef MOE_ROUTER_H
#define MOE_ROUTER_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

#define MOE_LOGITS_F32 0
#define MOE_LOGITS_BF16 1

typedef struct {
    int32_t num_experts;    /* E, 1 to 1024 */
    int32_t top_k;          /* 1 to 32, at most top_groups * E / groups */
    int32_t score;          /* MOE_SCORE_* */
    int32_t logits_type;    /* MOE_LOGITS_* */
    int32_t groups;         /* 1 to 32, a divisor of E */
    int32_t top_groups;     /* 1 to groups */
    int32_t normalise;
    float scale;
} moe_router;

/* The choice and its weights.
 *   logits       [n] rows of E, logits_ld elements apart (>= E)
 *   bias         [E] fp32 or NULL
 *   topk_ids     [n, top_k] int32 out;  topk_weight  [n, top_k] fp32 out */
moe_status moe_route(const moe_router *r, int64_t n_tokens, const void *logits, int64_t logits_ld, const float *bias,
                     int32_t *topk_ids, float *topk_weight, cudaStream_t stream);

/* Bytes of workspace of moe_balance_loss; 0 for unsupported sizes. */
size_t moe_balance_workspace_size(const moe_router *r, int64_t n_tokens, int64_t num_sequences);

/* The balance loss and the counts.
 *   topk_ids     [n, top_k] int32; entries outside [0, E) are not counted
 *   seq_offsets  [num_sequences + 1] int32, ascending from >= 0 to <= n; NULL: one sequence of all rows
 *                (num_sequences = 1).  Anything else gives a loss of NaN, and counts that mean nothing.
 *   counts       [num_sequences, E] int32 out
 *   loss         [1] fp32 out
 *   workspace    moe_balance_workspace_size bytes, 256-byte aligned; calls that may run at the same time (two
 *                captured graphs, two streams) need one each
 * num_sequences 1 to 65536.  n = 0: counts and loss are set to 0. */
moe_status moe_balance_loss(const moe_router *r, int64_t n_tokens, const void *logits, int64_t logits_ld,
                            const int32_t *topk_ids, float coef, const int32_t *seq_offsets, int64_t num_sequences,
                            int32_t *counts, float *loss, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/* The gradient of the logits, of the weights' part, the loss's part or their sum:
 *   d_logits[t] = sum_j d_weight[t][j] dw[t][j]/dl[t]  +  d_loss dloss/dl[t]
 *   d_weight     [n, top_k] fp32, or NULL: no such part.  Entries of topk_ids outside [0, E) add nothing.
 *   counts       [num_sequences, E] as moe_balance_loss wrote them, or NULL: no such part
 *   coef, seq_offsets, num_sequences   as in moe_balance_loss; not used without counts
 *   d_loss       [1] fp32, NULL = 1
 *   d_logits     [n] rows of E in the logits' type, d_ld elements apart (>= E); may be logits itself (same stride), else
 *                nothing that logits' rows hold
 * Every row is written, one without a part with zeros. */
moe_status moe_route_backward(const moe_router *r, int64_t n_tokens, const void *logits, int64_t logits_ld,
                              const int32_t *topk_ids, const float *d_weight, float coef, const int32_t *counts,
                              const float *d_loss, const int32_t *seq_offsets, int64_t num_sequences, void *d_logits,
                              int64_t d_ld, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTER_H */

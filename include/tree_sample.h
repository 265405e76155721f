/*
 * tree_sample.h -- the next token of every rollout, drawn from its logits with
 * given random numbers (libtreeattn).
 *
 * Rollouts branch by sampling (TreePO, segment-level tree sampling).  The draw is
 * a function of the logits and of one uniform number per row, so it is
 * reproducible, and it returns the log-probability that tree_attn_traj_logprobs
 * (tree_loss.h) gives the token later: under the untempered softmax of the row.
 *
 * Row r with logits x, temperature T, and w_i = exp((x_i - max x) / T):
 *   order    tokens by x descending, equal x by index ascending
 *   top_k    keep the first k (k <= 0: all)
 *   top_p    of those, keep the shortest prefix whose weights reach p times their
 *            sum, at least one token (p >= 1: all)
 *   min_p    of those, keep the tokens with w_i >= min_p (<= 0: all; above 1 counts
 *            as 1)
 *   token    the first kept token whose cumulated weight exceeds u times the kept
 *            tokens' sum, u in [0, 1) (below 0 counts as 0, 1 and above picks the
 *            last kept token of positive weight)
 *   T = 0    the largest logit, lowest index
 *   logprob  x_token - ln sum_i exp(x_i)
 * Infinite temperatures, T < 0 and NaN parameters are errors of the row: token -1,
 * logprob NaN, and TREE_ATTN_ERR_INVALID_SAMPLING in the device status word.  A
 * row without a distribution (a NaN, +inf, or nothing but -inf) gets token -1 and
 * logprob NaN.  Tokens at -inf are never drawn.
 *
 * Weights are held in 64-bit fixed point (2^45 for the largest) and summed as
 * integers: the cuts and the draw are exact for those weights, whatever the order
 * of the sums, and the same on every run.  A weight below 2^-46 of the largest
 * counts as zero.
 */
#ifndef TREE_SAMPLE_H
#define TREE_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#include "tree_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status only: a row's parameters are invalid (above). */
#define TREE_ATTN_ERR_INVALID_SAMPLING -15

/* A parameter of every row: one value, or an array of one per row. */
typedef struct {
    const float* temperatures;  /* [n_rows] device, or NULL: `temperature` for all */
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    float temperature;
    int32_t top_k;
    float top_p;
    float min_p;
} tree_attn_sampling_t;

/* logits bf16, row r at element r * row_stride (>= vocab; any alignment of 2
 * bytes), 1 <= vocab <= 262144; u fp32 [n_rows]; tokens int32 [n_rows]; logprobs
 * fp32 [n_rows] or NULL.  Device pointers, asynchronous on `stream`; no workspace.
 * n_rows = 0 does nothing. */
int tree_attn_sample(const void* logits, int64_t row_stride, int64_t n_rows, int64_t vocab, const float* u,
                     const tree_attn_sampling_t* params, int32_t* tokens, float* logprobs, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TREE_SAMPLE_H */

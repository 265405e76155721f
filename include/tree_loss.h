/*
 * tree_loss.h -- the calls around the attention at the loss boundary of
 * packed-tree training (libtreeattn): per-trajectory views of a plan, token
 * weights folded into a gradient, per-trajectory next-token log-probs from
 * compact logits, and subtree (segment-level) advantages.
 *
 * Trajectories.  One per leaf of the tree or forest, in ascending leaf node
 * id; trajectory l is the compact tokens of the nodes on the root-to-leaf path,
 * in path order.  A compact token belongs to every trajectory through its node
 * (its multiplicity) and sits at the same position in each of them (its
 * position id, for rotary embeddings) -- the HARTS abstract's compact-token
 * view of trajectories that share histories.
 *
 * Conventions are those of tree_attn.h: status 0 = success, negative =
 * TREE_ATTN_ERR_*; host outputs are caller-allocated; device pointers belong to
 * the caller, are 16-byte aligned and are used asynchronously on `stream`.
 * The first device call with a plan on a device uploads its trajectory tables
 * (allocates and synchronises once).
 */
#ifndef TREE_LOSS_H
#define TREE_LOSS_H

#include <stddef.h>
#include <stdint.h>

#include "tree_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Trajectory counts: n_leaves, and n_expanded = sum of trajectory lengths
 * (the tokens training every trajectory on its own would process). */
int tree_attn_plan_trajectory_info(tree_attn_plan_t plan, int32_t* n_leaves, int64_t* n_expanded);

/* Host copies: leaf_ids [n_leaves] (ascending), traj_ptr [n_leaves+1] offsets
 * into traj_tokens [n_expanded] = compact (packed) token index of every
 * trajectory position.  Any pointer may be NULL. */
int tree_attn_plan_trajectories(tree_attn_plan_t plan, int32_t* leaf_ids, int64_t* traj_ptr, int32_t* traj_tokens);

/* Host copies, [n_tokens] each, packed order: multiplicity = trajectories
 * containing the token (leaves under its node); position id = its 0-based
 * position along those trajectories.  Either pointer may be NULL. */
int tree_attn_plan_token_info(tree_attn_plan_t plan, int32_t* multiplicity, int32_t* position_ids);

/* Token weights folded into a gradient (HARTS abstract: compact tokens stand
 * for several trajectory tokens; a loss weights each compact token by how
 * many trajectory tokens it stands for, or by any other per-token weight):
 *   y[t, e] = bf16(x[t, e] * w[t])   for t < n_rows, e < row_elems
 * x, y bf16 [n_rows, row_elems] (may be the same buffer), w fp32 [n_rows];
 * row_elems a multiple of 8.  Device pointers, asynchronous on `stream`. */
int tree_attn_scale_rows(const void* x, const float* w, void* y, int64_t n_rows, int64_t row_elems, void* stream);

/* Per-trajectory next-token log-probs from compact logits.  logits bf16
 * [n_tokens, vocab] in packed order (vocab a multiple of 8); tokens int32
 * [n_tokens] = the token id at each compact position.  Writes
 *   row_lse[t]  = ln sum_v exp(logits[t, v])                    [n_tokens]
 *   logprobs[k] = logits[r, tokens[s]] - row_lse[r]             [n_expanded - n_leaves]
 * where prediction k is the k-th (position p, p+1) pair of the trajectories in
 * order, r = the compact token at p and s = the one at p+1.  At the end of a
 * shared segment r is the same for every child trajectory and s differs: the
 * one compact row predicts each child's first token.  A token id outside
 * [0, vocab) gives NaN.  Device pointers, asynchronous on `stream`. */
int tree_attn_traj_logprobs(tree_attn_plan_t plan, const void* logits, int64_t vocab, const int32_t* tokens,
                            float* row_lse, float* logprobs, void* stream);

/* Subtree (segment-level) advantages.  Section: TreePO (Approach: advantages
 * estimated over sub-trees from collective descendant outcomes; tree-based
 * advantage estimation with trajectory subgroups that share predecessor nodes;
 * discussion: simple subgroup averaging vs size-weighted aggregation, root
 * group removable).  Reading of this library (the pages give no formula):
 *   group G(u) = the leaves under node u; mean_u, std_u their rewards' mean and
 *   population standard deviation;
 *   for leaf l, the subgroups are the nodes u on its root path (u = l included)
 *   with |G(u)| >= 2 (without roots if TREE_ADV_NO_ROOT);
 *   a_u(l) = R_l - mean_u, divided by (std_u + eps) with TREE_ADV_NORM_STD;
 *   A(l)   = sum_u w_u a_u(l) / sum_u w_u with w_u = 1, or |G(u)| with
 *            TREE_ADV_SIZE_WEIGHTED; 0 when l has no subgroup;
 *   node_coef[u] = sum of A(l) over G(u); token_coef[t] = node_coef of t's node
 *   (the policy-gradient weight of a compact token: the advantages of every
 *   trajectory through it).
 * leaf_reward / leaf_adv: fp32 [n_leaves], leaves in ascending node id;
 * node_coef fp32 [n_nodes] by node id; token_coef fp32 [n_tokens], packed
 * order.  Device pointers, asynchronous on `stream`; n_nodes <= 16384. */
#define TREE_ADV_NORM_STD      1
#define TREE_ADV_SIZE_WEIGHTED 2
#define TREE_ADV_NO_ROOT       4
int tree_attn_subtree_advantage(tree_attn_plan_t plan, const float* leaf_reward, int32_t flags, float eps,
                                float* leaf_adv, float* node_coef, float* token_coef, void* stream);

/* Clipped policy loss of the trajectories, and its gradient for the compact logits.  The pages
 * train policies on rollout trees (HARTS, AReaL-DTA: the compact tokens' results equal those of
 * training every trajectory on its own; TreePO: advantages of segments) and print no loss; this
 * is the clipped ratio with a penalty towards a reference policy that such training uses.
 *
 * Prediction k (as in tree_attn_traj_logprobs) is made by the compact row r of the logits x for
 * the token y at the next position.  With LSE_r = ln sum_v e^x_rv, p_rv = e^(x_rv - LSE_r),
 * lp = x_ry - LSE_r, rho = e^(lp - old_k), H_r = LSE_r - sum_v p_rv x_rv and A the advantage:
 *
 *   loss = sum_k w_k (-min(rho A, clip(rho, 1 - clip_low, 1 + clip_high) A)
 *                     + kl_coef (e^(ref_k - lp) - (ref_k - lp) - 1) - entropy_coef H_r)
 *   g_k  = w_k (dsurrogate + kl_coef (1 - e^(ref_k - lp)))
 *          dsurrogate = -rho A where the clip does not bind (its borders included), else 0
 *   dlogits_rv = grad_scale (sum_k g_k (1[v = y_k] - p_rv)
 *                            + entropy_coef sum_k w_k p_rv (x_rv - LSE_r + H_r))
 *
 * over the predictions with w_k != 0.  At the end of a shared segment one row predicts every
 * child's first token, and above it every trajectory's copy of a prediction counts on its own.
 * A = 0 gives a surrogate of 0 whatever the ratio.  -inf in the logits is probability 0; a row
 * with a NaN, a +inf or nothing but -inf, and a token id outside [0, vocab), give NaN.  Where
 * w_k = 0 the prediction is left out whatever its other inputs hold, and its log-prob is written
 * as 0; the logits of a row without any weight are not read, its entropy and gradient are 0. */
typedef struct {
    const float* old_logprobs;   /* [n_pred], n_pred = n_expanded - n_leaves; NULL: rho = 1, as if old = lp */
    const float* advantages;     /* [n_leaves] by leaf id ascending, or [n_pred] with per_token */
    const float* weights;        /* [n_pred]; NULL: 1 / n_pred each */
    const float* ref_logprobs;   /* [n_pred]; may be NULL when kl_coef is 0 */
    int32_t per_token;
    float clip_low;              /* in [0, 1] */
    float clip_high;             /* >= 0, infinity for no upper clip */
    float kl_coef;               /* finite, as the next two */
    float entropy_coef;
    float grad_scale;            /* of dlogits only */
} tree_attn_policy_t;

/* Device workspace that tree_attn_policy_loss needs. */
int tree_attn_policy_loss_workspace(tree_attn_plan_t plan, size_t* ws_bytes);

/* logits bf16, row t at element t * row_stride (>= vocab; any alignment of 2 bytes),
 * 1 <= vocab <= 262144; tokens int32 [n_tokens]; loss fp32 [1]; logprobs fp32 [n_pred] and entropy
 * fp32 [n_tokens], either may be NULL; dlogits bf16 [n_tokens] rows of d_stride elements, NULL for the
 * loss alone, or the logits themselves with the same stride (each row is read before it is
 * written); fast where each row's address agrees with the logits' row modulo 16 bytes.  The
 * struct is read during the call.  Log-probs, ratios and sums are fp32 or wider
 * (whether a ratio lies beyond the clip is decided in pairs of floats); dlogits is
 * rounded once.  Bitwise reproducible, and loss, log-probs and entropies are the same bits with and
 * without dlogits.  workspace: 256-byte aligned, contents ignored; calls that may
 * overlap need one each.  Asynchronous on `stream`; the plan's first call on a device uploads
 * its tables (allocates and synchronises once: make it outside stream capture). */
int tree_attn_policy_loss(tree_attn_plan_t plan, const void* logits, int64_t row_stride, int64_t vocab,
                          const int32_t* tokens, const tree_attn_policy_t* policy, float* loss, float* logprobs,
                          float* entropy, void* dlogits, int64_t d_stride, void* workspace, size_t ws_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TREE_LOSS_H */

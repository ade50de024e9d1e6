/*
 * i8h_scored — the choice of experts by scores: softmax or sigmoid over all
 * experts, a bias that balances the load, groups of experts, weights with or
 * without renormalisation. Part of libi8h.so; i8h.h's conventions hold
 * (device pointers, the caller's buffers, host-side validation before any
 * launch, T == 0 a no-op). The outputs are those of moe_route_permute, so the
 * grouped products take them as they are.
 */
#ifndef I8H_SCORED_H
#define I8H_SCORED_H

#include "i8h_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scores of the experts from the logits l of a token. */
enum { I8H_SCORE_SOFTMAX = 0, I8H_SCORE_SIGMOID = 1 };

#define I8H_MAX_GROUPS 64

/* For each token, with its E logits l:
 *
 *   s(e) = exp(l(e) - max l) / sum of them    (I8H_SCORE_SOFTMAX; a token with
 *                                              only -inf has scores 0)
 *        = 1 / (1 + exp(-l(e)))               (I8H_SCORE_SIGMOID)
 *   c(e) = s(e) + bias(e), or without a bias the order of l(e) itself, which
 *          is that of the scores
 *   The experts form `groups` runs of E / groups. A group's worth is its
 *   largest c (group_top 1), or the sum of its two largest c (group_top 2; of
 *   the two largest s without a bias). The topk_groups groups of most worth
 *   stay (groups == topk_groups: all of them).
 *   The topk experts of largest c in them are chosen, in that order.
 *   w(j) = s(chosen j), divided by their sum if `renormalize` (0 where that
 *          sum is 0), times `scale`
 *
 * Ties go to the lower index, of groups as of experts. A NaN (a NaN logit, or
 * bias; +inf under softmax makes the whole token's scores NaN) ranks after
 * every number, so every id is an expert. The order is that of c and of the
 * worths in float64. A -inf logit masks an expert: its score is 0, and only a
 * bias, or a lack of others, has it chosen.
 *
 * Weights are computed in float32 (in float64 where a score that counts leaves
 * its range), each within 40 units of 2^-24 of its own value, for
 * I8H_SCORE_SOFTMAX (40 + 2 d) units with d the distance of its logit from the
 * token's largest; a weight below 2^-126 may be 0.
 *
 * logits [T, E] (logits_type: I8H_F32 or I8H_BF16, aligned to the element);
 * bias [E] float32 or NULL; topk_ids, topk_w, expert_off, sorted_pairs and
 * pair_pos as for moe_route_permute. E % groups == 0, 1 <= topk_groups <=
 * groups, group_top 1 or 2 and with more than one group at most E / groups,
 * topk <= topk_groups * (E / groups) (else I8H_EINVAL); groups <=
 * I8H_MAX_GROUPS, E and topk as in i8h.h, T <= (2^22 - 1) * min(64, 512 / topk),
 * so that T * topk is below 2^31 (else I8H_EUNSUPPORTED).
 * workspace: at least moe_route_scored_workspace_size(T, E, topk) bytes,
 * 256-B aligned, contents on entry ignored (may be NULL when that size is 0).
 * Sizes never fall as T, E or topk grow: one for the largest batch serves
 * smaller ones. */
size_t moe_route_scored_workspace_size(int T, int E, int topk);
int moe_route_scored_permute(const void* logits, int logits_type, int T, int E, int topk, int score,
                             const float* bias, int groups, int topk_groups, int group_top, int renormalize,
                             float scale, int32_t* topk_ids, float* topk_w, int32_t* expert_off,
                             int32_t* sorted_pairs, int32_t* pair_pos, void* workspace, size_t workspace_bytes,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* I8H_SCORED_H */

/*
 * i8h_draft — verification of drafted tokens: which tokens of a speculative
 * step stay, and the token sampled after them. Part of libi8h.so; i8h.h's
 * conventions hold (device pointers, host-side validation before any launch).
 *
 * The drafter of the int8 card (model table, row "Speculator") proposes 15
 * tokens a step; the target model then gives a distribution at each of their
 * positions and one more (a verify batch). The rule is the published one of
 * speculative sampling: it leaves the target's distribution unchanged.
 */
#ifndef I8H_DRAFT_H
#define I8H_DRAFT_H

#include "i8h_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For each of B sequences with up to D drafted tokens and V vocabulary
 * entries (p = target, q = draft, len = draft_len[b] clamped to [0, D]):
 *
 *   token i stays while  u[b, i] * q[b, i, x_i] < p[b, i, x_i],  x_i = drafted[b, i]
 *   n = accepted[b] = how many stay in a row from the front (n <= len)
 *   rest(v) = max(p[b, n, v] - q[b, n, v], 0)  if n < len   (token n was refused)
 *             p[b, n, v]                       if n == len  (all stayed)
 *   next = the lowest v with  rest(0) + ... + rest(v) > u_next[b] * sum(rest)
 *   tokens[b] = x_0 .. x_{n-1}, next, then -1
 *
 * draft_probs NULL stands for drafts taken without sampling (q = 1 at x_i, 0
 * elsewhere): token i stays while u < p(x_i), and rest is p without x_n.
 * Products, differences and sums are float64 (products exact). Entries of
 * rest that are not positive and finite count as zero; if none is left, rest is
 * p itself, and if p has none either, next is V - 1. A drafted token outside
 * [0, V) is refused. u and u_next are uniform in [0, 1). Results are the same,
 * bit for bit, in every run.
 *
 * target_probs [B, D+1, V], draft_probs [B, D, V] or NULL (both of prob_type,
 * I8H_F32 or I8H_BF16, aligned to the element); drafted [B, D] int32;
 * draft_len [B] int32, or NULL for D everywhere; u [B, D], u_next [B] float32;
 * tokens [B, D+1], accepted [B] int32 out. B >= 0, 0 <= D <= 1023 and V >= 1;
 * B <= 65535 (else I8H_EUNSUPPORTED). With D == 0 draft_probs, drafted and u
 * may be NULL. workspace: at least draft_verify_workspace_size(B, V) bytes,
 * 256-B aligned, contents on entry ignored. */
size_t draft_verify_workspace_size(int B, int V);
int draft_verify(const void* target_probs, const void* draft_probs, int prob_type, const int32_t* drafted,
                 const int32_t* draft_len, const float* u, const float* u_next, int B, int D, int V,
                 int32_t* tokens, int32_t* accepted, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* I8H_DRAFT_H */

/*
 * Routing of tokens to experts, for mixture-of-experts layers: from a router's
 * logits to the rows, offsets and weights that the grouped products
 * (gemm_grouped.h, gemm_mx4.h, gemm_i8.h) and the sum over a token's experts
 * take, and the gradient of the logits.
 *
 * gemm_route       For every token t (row t of the logits, at logits + t*ld):
 *
 *                  score    softmax over the row, or with GEMM_ROUTE_SIGMOID
 *                           1 / (1 + exp(-x)) of each logit.
 *                  ranking  by logit; with a bias (one float an expert, for
 *                           balance) by score + bias.  Equal ones rank by
 *                           index, the lower first.
 *                  groups   experts / groups neighbouring experts form a
 *                           group.  A group's score is the sum of its two best
 *                           score + bias (of one, where it has only one); the
 *                           top_groups best groups stay open, equal ones by
 *                           index.  groups = 1: no restriction.
 *                  choices  the k first of the ranking, in its order.
 *                  weights  scale * score (without the bias); with
 *                           GEMM_ROUTE_RENORMALISE scale * score / the sum of
 *                           the chosen scores (sigmoid: + 1e-20).
 *
 *                  weights[t*k + i] and expert[t*k + i] hold choice i.  Sums
 *                  with a bias, and of groups, that FP32 cannot tell apart are
 *                  decided in 64 bits.  An expert whose logit (or bias) is
 *                  minus infinity is no choice (a finite bias, however low,
 *                  excludes nothing, and one far above the scores' range makes
 *                  every sum a close one): where fewer than k are left
 *                  the last choices are expert -1 with weight 0.  A row of
 *                  padding is a row of minus infinities.  A row that holds a
 *                  NaN (for softmax: or plus infinity), or meets a bias
 *                  that is NaN, has no choices, and NaN weights.
 *
 *                  order[0 .. tokens*k - 1] lists the rows t*k + i by expert
 *                  (rows of one expert in rising order, those of expert -1
 *                  first) and offsets[0 .. experts] are the experts' bounds
 *                  in it: expert e owns order[offsets[e]] ..
 *                  order[offsets[e+1] - 1].  Rows before offsets[0] belong to
 *                  no expert, as the grouped products read it.  offsets[experts]
 *                  is tokens * k.
 *
 * gemm_route_grad  dlogits from dweights (tokens x k) for the choices
 *                  `expert` of gemm_route: the derivative of the weights with
 *                  the choices held fixed.  Choices outside 0 .. experts - 1
 *                  have none; an expert that appears twice in a row counts as
 *                  often.  Softmax, renormalised: rows outside the choices are
 *                  zero.
 *
 * dtype is GEMM_F32 or GEMM_BF16, of the logits and of dlogits; arithmetic is
 * FP32.  weights, expert, order, dweights are contiguous.  Limits: experts <=
 * GEMM_ROUTE_MAX_EXPERTS, k <= GEMM_ROUTE_MAX_K and <= top_groups * experts /
 * groups, groups <= GEMM_ROUTE_MAX_GROUPS and a divisor of experts, tokens * k
 * <= 2^30.  tokens = 0 writes zero offsets.  Handles, streams, workspace
 * and errors are those of gemm_run; results are bit-identical from call to call.
 */
#ifndef DENSE_GEMM_SM100_GB300_GEMM_ROUTE_H
#define DENSE_GEMM_SM100_GB300_GEMM_ROUTE_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ROUTE_MAX_EXPERTS 1024
#define GEMM_ROUTE_MAX_K 31
#define GEMM_ROUTE_MAX_GROUPS 32

#define GEMM_ROUTE_SIGMOID 1
#define GEMM_ROUTE_RENORMALISE 2

int gemm_route(gemm_handle_t h, int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
               const float *bias, int64_t groups, int64_t top_groups, int flags, float scale, float *weights,
               int64_t *expert, int64_t *order, int64_t *offsets, cudaStream_t stream);

int gemm_route_grad(gemm_handle_t h, int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld,
                    int dtype, const int64_t *expert, const float *dweights, int flags, float scale, void *dlogits,
                    int64_t ldd, cudaStream_t stream);

/* Argument checks without touching the GPU, exactly as the calls make them. */
int gemm_route_validate(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
                        const float *bias, int64_t groups, int64_t top_groups, int flags, float scale,
                        const float *weights, const int64_t *expert, const int64_t *order, const int64_t *offsets);
int gemm_route_grad_validate(int64_t tokens, int64_t experts, int64_t k, const void *logits, int64_t ld, int dtype,
                             const int64_t *expert, const float *dweights, int flags, float scale,
                             const void *dlogits, int64_t ldd);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_SM100_GB300_GEMM_ROUTE_H */

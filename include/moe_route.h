/*
 * moe_route.h - C ABI of expert routing from scores (gfx950).
 *
 * moe_layer.h's router takes the k largest logits and the softmax over them.
 * Other routers score every expert (softmax over all experts, or a sigmoid of
 * each logit), choose by score plus a per-expert bias that balances the load
 * without entering the weights, restrict the choice to the best groups of
 * experts, and weight by the scores themselves.  This entry point computes
 * that, per token with logits l[E] and an optional bias b[E]:
 *
 *   s_e   = exp(l_e - m) / sum_j exp(l_j - m), m = max l      MOE_SCORE_SOFTMAX
 *         = 1 / (1 + exp(-l_e))                               MOE_SCORE_SIGMOID
 *   v_e   = s_e + b_e (s_e without a bias)
 *   key_e = v_e with a bias, l_e without one
 *   group g holds experts [g E/G, (g + 1) E/G); its score is the sum of its
 *     group_top largest v_e; the top_groups best groups stay (ties: the lower
 *     group), the experts of the others are out
 *   ids   = the first k experts that are not out by (-key, id)
 *   w_i   = scale * s_{ids_i} (/ sum_j s_{ids_j} with renormalize)
 *
 * An expert whose logit is -inf is masked: it has score 0, counts in no
 * group's score and comes after every other expert that is not out.  A NaN
 * key is ordered like a masked expert's, a NaN v_e counts in no group's
 * score; masked experts and NaN keys follow one another by id.  A row whose
 * mask leaves fewer than k experts still gets k distinct ids; the masked ones
 * have weight 0, and a row that it leaves empty has weights 0 only.  Where
 * every chosen score is 0, renormalize leaves the weights 0.  NaN scores give
 * NaN weights; under softmax a logit that is NaN or +inf makes the denominator
 * NaN, and so every score and weight of its row.
 *
 * Scores that order experts or groups (a bias, or more than one group) are
 * formed in double precision, so that the choice does not depend on single-
 * precision rounding; without either the logits themselves are compared.
 * Equal keys go to the lower id.
 *
 * Conventions as in moe_layer.h: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before anything is enqueued,
 * MOE_OK or a negative MOE_E* code with the reason in moe_last_error(),
 * deterministic results.  No workspace.
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

typedef struct moe_route_desc {
  int32_t n_experts;    /* E, 1 .. 1024                                         */
  int32_t top_k;        /* k, 1 .. min(64, top_groups E / n_groups)             */
  int32_t score;        /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID               */
  int32_t n_groups;     /* G, 1 .. 64, divides E (1: no groups)                 */
  int32_t top_groups;   /* groups that stay, 1 .. G                             */
  int32_t group_top;    /* experts whose scores make a group's score: 1 or 2    */
  int32_t renormalize;  /* 0 or 1                                               */
  int32_t logit_dtype;  /* MOE_F32 or MOE_BF16                                  */
  float scale;          /* factor on the weights (finite)                       */
} moe_route_desc;

/*
 * Routing of T tokens from their logits.
 *   logits     row t at logits + t * logits_stride elements (>= E), logit_dtype
 *   bias       [E] fp32, or NULL
 *   topk_ids   [T, k] int32, by descending key
 *   topk_w     [T, k] fp32
 * T = 0 enqueues nothing.  T <= 2^20.  Errors: MOE_EINVAL (descriptor, T,
 * stride, a NULL pointer or one not aligned to its element, an output that
 * overlaps an input or the other output), MOE_EHIP if the launch fails.
 */
int moe_route_forward(const moe_route_desc* r, int32_t T, const void* logits, int64_t logits_stride,
                      const float* bias, int32_t* topk_ids, float* topk_w, void* stream);

/*
 * The first half of a layer with this routing in place of moe_router_topk's:
 * logits R x by the kernels that moe_router_topk would run for this d and T
 * (kept as fp32 in the workspace), then the routing above.  topk_ids and
 * topk_w go to moe_experts_forward as they are.  r->n_experts and r->top_k
 * must equal d's, and r->logit_dtype must be MOE_F32.  Workspace and x,
 * router_w as in moe_router_topk; bias, topk_ids and topk_w as above.
 * MOE_EINVAL also where x, router_w, bias or an output overlaps the workspace,
 * or an output an input.
 */
int moe_router_route(const moe_desc* d, const moe_route_desc* r, int32_t T, const void* x, const void* router_w,
                     const float* bias, int32_t* topk_ids, float* topk_w, void* workspace, size_t ws_bytes,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_H */

/*
 * moe_scores.h -- C ABI of libmoe.so, part 6: routing to experts from given router logits, with softmax
 * or sigmoid scores, a balance bias that enters the choice only, expert groups, top-k and renormalised
 * weights, forward and backward, on one GB300 GPU.  Its topk_idx and weights are the topk_idx and gates
 * of moe_forward and moe_experts_backward (moe.h); moe_route is the softmax router whose bias also
 * enters the gates.
 *
 *   s[e]  = 1 / (1 + exp(-l[e]))  or  exp(l[e]) / sum_i exp(l[i])
 *   c[e]  = s[e] + bias[e]                                (the value experts are chosen by)
 *   group score = the sum of the group_top largest c of the group (group g
 *           holds experts [g E / groups, (g + 1) E / groups))
 *   the topk_groups groups of the largest scores are open; the k experts of the largest c in the open
 *           groups are chosen, in descending order of c
 *   weights[j] = scale s[e_j] / S,   S = sum of the chosen s (renormalize = 1) or 1
 * Ties go to the lower group and the lower expert.  The order is that of the values before rounding:
 * scores are computed in fp32, and where two of them lie within fp32's error of each other they are
 * compared in fp64.
 *
 *   backward, for dw = gradient of weights, the chosen set held fixed, the bias without gradient:
 *   ds_j  = scale (dw_j - [renormalize] sum_i dw_i s_i / S) / S
 *   sigmoid: dl[e_j] = ds_j s_j (1 - s_j)
 *   softmax: dl[e]   = s[e] ([e = e_j] ds_j - sum_i ds_i s_i); the sum is 0 when renormalize = 1
 *   and dl[e] = 0 for every other expert.
 *
 * Conventions are those of moe.h (MOE_OK / MOE_ERR_* codes, stream as void*, asynchronous, capturable,
 * the caller owns every buffer and the workspace), and:
 *   - logits [N, E] have a row stride ld (elements, >= E) and one of the MOE_TYPE_* types; dlogits is
 *     dense and of the same type.  bias and weights are fp32.
 *   - logits may be -inf (an expert that is masked for a token): its score is 0, it is chosen only when
 *     nothing else is left, with weight 0; a row of -inf alone has weights and gradients 0.  Scores
 *     below fp32's range still share out the renormalised weights; a sigmoid logit below -709, whose
 *     score is 0 in fp64 too, counts as -inf there.  A bias may be -inf.
 *     A NaN ranks below every number; the weights it reaches are NaN.
 *   - backward: an index outside [0, E) is reported as MOE_ERR_DEVICE_CHECK through the workspace status
 *     word (moe_check_status) and takes no part; the k indices of a row are distinct.
 *   - shapes: N >= 0; 1 <= E <= 1024; groups divides E, 1 <= groups <= 32; 1 <= topk_groups <= groups;
 *     1 <= k <= min(32, topk_groups E / groups).  Else MOE_ERR_UNSUPPORTED_SHAPE.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_SCORES_H_
#define TOP_SOFTMAX_ROUTER_MOE_SCORES_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };

typedef struct moe_scores_config {
  int32_t N, E, k;
  int32_t groups, topk_groups;
  int32_t group_top;     /* 1 or 2: how many of a group's values make its score */
  int32_t score;         /* MOE_SCORE_* */
  int32_t renormalize;   /* 0 or 1 */
  float scale;
} moe_scores_config;

/* Workspace bytes of both calls. */
int moe_scores_workspace_bytes(const moe_scores_config* cfg, size_t* bytes);

/* topk_idx [N, k] int32, weights [N, k] fp32, counts [E] int32 (or NULL; how many tokens chose each
 * expert): out, overwritten. */
int moe_scores_forward(const moe_scores_config* cfg, const void* logits, int64_t ld, int32_t type,
                       const float* bias, int32_t* topk_idx, float* weights, int32_t* counts, void* ws,
                       size_t ws_bytes, void* stream);

/* dlogits [N, E] out, overwritten. */
int moe_scores_backward(const moe_scores_config* cfg, const void* logits, int64_t ld, int32_t type,
                        const int32_t* topk_idx, const float* dweights, void* dlogits, void* ws, size_t ws_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_SCORES_H_ */

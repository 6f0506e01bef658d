/*
 * moe_types.h -- element types of the layer operators (moe_norm.h, moe_embed.h, moe_scores.h,
 * moe_distill.h), passed as int32_t beside an untyped pointer.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_TYPES_H_
#define TOP_SOFTMAX_ROUTER_MOE_TYPES_H_

enum { MOE_TYPE_F32 = 0, MOE_TYPE_BF16 = 1, MOE_TYPE_F16 = 2 };
/* index types */
enum { MOE_INDEX_I32 = 0, MOE_INDEX_I64 = 1 };

#endif /* TOP_SOFTMAX_ROUTER_MOE_TYPES_H_ */

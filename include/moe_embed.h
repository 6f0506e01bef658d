/*
 * moe_embed.h -- C ABI of libmoe.so, part 5: token embedding with scaling, and its gradient by sorted
 * tokens, on one GB300 GPU.
 *
 *   y[n]  = scale table[ids[n]]                          (fp32 product, rounded to the table's type)
 *   dW[v] = scale sum over the n with ids[n] = v of dy[n]   (fp32, summed in ascending n in pieces
 *           of 32 tokens, so the same inputs always give the same bits)
 *
 * Conventions are those of moe.h (MOE_OK / MOE_ERR_* codes, stream as void*, asynchronous, capturable,
 * the caller owns every buffer and the workspace), and:
 *   - table [V, H] and y [N, H] are dense and of one type (MOE_TYPE_*); dy [N, H] has a row stride lddy
 *     (elements, >= H) and any of the types; ids [N] are MOE_INDEX_I32 or MOE_INDEX_I64; the gradient
 *     is fp32.  Pointers need only their element's alignment.
 *   - an id outside [0, V) is reported as MOE_ERR_DEVICE_CHECK through the workspace status word
 *     (moe_check_status); its row of y is zero and it adds to no gradient.
 *   - rows whose id equals padding_idx (-1: none) are looked up like any other but add to no gradient.
 *   - shapes: 0 <= N <= 2^24, 1 <= V < 2^30, 1 <= H <= 2^20.  Else MOE_ERR_UNSUPPORTED_SHAPE.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_EMBED_H_
#define TOP_SOFTMAX_ROUTER_MOE_EMBED_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

/* N tokens, a table of V rows of H values. */
typedef struct moe_embed_config {
  int32_t N, V, H;
  int32_t padding_idx;
  float scale;
} moe_embed_config;

/* Workspace bytes (either pointer may be NULL): a function of the shape, not decreasing in N. */
int moe_embed_workspace_bytes(const moe_embed_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes);

int moe_embed_forward(const moe_embed_config* cfg, const void* ids, int32_t id_type, const void* table, void* y,
                      int32_t type, void* ws, size_t ws_bytes, void* stream);

/* dW [V, H] fp32.  accumulate = 0: overwritten, every row; 1: the gradient is added to what dW holds, and
 * rows of tokens that do not occur are neither read nor written. */
int moe_embed_backward(const moe_embed_config* cfg, const void* ids, int32_t id_type, const void* dy, int64_t lddy,
                       int32_t type, float* dW, int32_t accumulate, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_EMBED_H_ */

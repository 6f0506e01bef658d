/*
 * moe_norm.h -- C ABI of libmoe.so, part 4: layer normalisation, forward and backward with the
 * reduction of the parameter gradients, on one GB300 GPU.
 *
 *   mean[n] = sum_h x[n, h] / H,   rstd[n] = 1 / sqrt(sum_h (x[n, h] - mean[n])^2 / H + eps)
 *   xh      = (x - mean) rstd,     y = xh weight + bias
 *   t       = dy weight
 *   dx      = rstd (t - sum_h t / H - xh sum_h (t xh) / H)
 *   dweight = sum_n dy xh,         dbias = sum_n dy
 *
 * Conventions are those of moe.h (MOE_OK / MOE_ERR_* codes, stream as void*, asynchronous, capturable,
 * the caller owns every buffer), and:
 *   - x, y, dy and dx have one type (MOE_TYPE_* of moe_types.h); weight and bias have that type or
 *     fp32; mean, rstd, dweight and dbias are fp32.  Statistics and sums are fp32; the variance is
 *     summed around the mean, in a second pass over the row held in registers.
 *   - x and dy may have a row stride (ldx, lddy elements, >= H); y and dx are dense.  Pointers need
 *     only their element's alignment: rows that are 16-byte aligned take 16-byte loads.
 *   - shapes: N >= 0, 1 <= H <= 16384.  Else MOE_ERR_UNSUPPORTED_SHAPE.  eps >= 0 and finite.
 *   - repeated calls on the same inputs give the same bits (every sum has a fixed order).
 *   - a wait of the backward that runs out (moe_set_wait_limit_ns) is reported as MOE_ERR_TIMEOUT through
 *     the workspace status word (moe_check_status); the call's gradients are then of no use.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_NORM_H_
#define TOP_SOFTMAX_ROUTER_MOE_NORM_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LAYERNORM_MAX_H 16384

/* N rows of H values. */
typedef struct moe_layernorm_config {
  int32_t N, H;
  float eps;
} moe_layernorm_config;

/* Workspace bytes of moe_layernorm_backward (a function of the shape only, not decreasing in N: a
 * workspace for N rows serves fewer).  The forward needs none. */
int moe_layernorm_workspace_bytes(const moe_layernorm_config* cfg, size_t* bwd_bytes);

/* weight (NULL = ones) and bias (NULL = zeros) [H]; mean, rstd [N] out (either may be NULL). */
int moe_layernorm_forward(const moe_layernorm_config* cfg, const void* x, int64_t ldx, const void* weight,
                          const void* bias, void* y, float* mean, float* rstd, int32_t type, int32_t param_type,
                          void* stream);

/* mean, rstd [N] from the forward; dx [N, H] out (NULL: not wanted); dweight, dbias [H] fp32 out
 * (either may be NULL), overwritten. */
int moe_layernorm_backward(const moe_layernorm_config* cfg, const void* x, int64_t ldx, const void* weight,
                           const float* mean, const float* rstd, const void* dy, int64_t lddy, void* dx,
                           float* dweight, float* dbias, int32_t type, int32_t param_type, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_NORM_H_ */

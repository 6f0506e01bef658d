/*
 * moe_rmsnorm.h -- C ABI of libmoe.so, part 10: root-mean-square norm with the residual's addition, its output in the
 * inputs' type or in 8 bits with scales (moe_blocks8.h), forward and backward.
 *
 *   h[n]    = x[n] + residual[n], rounded to their type       (x itself without a residual)
 *   rstd[n] = 1 / sqrt(sum_h h[n, h]^2 / H + eps)
 *   y       = h rstd weight;   codes, scales: y (before any rounding) packed as by moe_blocks8_pack
 *
 *   t       = dy weight,       xh = h rstd
 *   dx      = rstd (t - xh sum_h (t xh) / H) + dh             (the gradient of x and of the residual alike)
 *   dweight = sum_n dy xh
 *
 * Conventions are those of moe_norm.h: x, residual, h, y, dy, dh and dx have one type (MOE_TYPE_*), weight has that
 * type or fp32, rstd and dweight are fp32; statistics and sums are fp32; x, residual, h (in the backward), dy and dh
 * may have row strides, what is written is dense; pointers need only their element's alignment, rows that lie on 16
 * bytes take 16-byte loads; repeated calls give the same bits.  Shapes: N >= 0, 1 <= H <= 16384.  eps >= 0 and finite.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_RMSNORM_H_
#define TOP_SOFTMAX_ROUTER_MOE_RMSNORM_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_RMSNORM_MAX_H 16384

/* N rows of H values. */
typedef struct moe_rmsnorm_config {
  int32_t N, H;
  float eps;
} moe_rmsnorm_config;

/* Workspace bytes of moe_rmsnorm_backward (a function of the shape only, not decreasing in N).  The forward needs none. */
int moe_rmsnorm_workspace_bytes(const moe_rmsnorm_config* cfg, size_t* bwd_bytes);

/* residual NULL: none; weight [H] NULL: ones.  Out, each NULL where it is not wanted: h [N][H] (only with a residual),
 * y [N][H], codes [N][H] with scales [N][ceil(H / 128)], rstd [N]. */
int moe_rmsnorm_forward(const moe_rmsnorm_config* cfg, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                        const void* weight, void* h, void* y, uint8_t* codes, uint8_t* scales, float* rstd,
                        int32_t type, int32_t param_type, void* stream);

/* h and rstd as the forward left them; dh NULL: 0.  dx [N][H] and dweight [H] out, each NULL where it is not wanted. */
int moe_rmsnorm_backward(const moe_rmsnorm_config* cfg, const void* h, int64_t ldh, const void* weight,
                         const float* rstd, const void* dy, int64_t lddy, const void* dh, int64_t lddh, void* dx,
                         float* dweight, int32_t type, int32_t param_type, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_RMSNORM_H_ */

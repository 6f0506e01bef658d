/*
 * moe_linear.h -- C ABI of libmoe.so, part 9: matrix products grouped by expert, with as many rows for each expert as
 * there are (none, one, or all), in bf16 or in 8 bits with a scale for each block of 128, forward and backward.
 *
 * Rows offsets[e] .. offsets[e + 1] - 1 of x belong to expert e, with the weights W[e] [O][K]:
 *
 *   y[n]  = x[n] W[e]^T                                      n a row of e
 *   dx[n] = dy[n] W[e]
 *   dW[e] = sum over e's rows of dy[n]^T x[n]                (0 where e has none)
 *
 * E = 1 with offsets = NULL is the dense layer: all N rows are the one expert's.  Rows before offsets[0] and from
 * offsets[E] on belong to nobody: their y and dx are 0, and what x and dy hold there is not used, be it NaN.
 *
 * In 8 bits x and W are e4m3 codes with their scales (moe_blocks8.h: [N][ceil(K / 128)] and
 * [E][ceil(O / 128)][ceil(K / 128)] bytes):
 *
 *   y[n, o] = sum over blocks b of 2^(sx[n, b] + sw[o / 128, b]) sum over k in b of cx[n, k] cw[o, k]
 *
 * dx takes dy packed as moe_blocks8_pack does, along O; dW takes dy as it is and
 * the values that x's codes stand for.  The backward also takes x in codes beside bf16 weights: an activation
 * checkpoint in 8 bits.
 *
 * Conventions are those of moe.h (codes, stream as void*, asynchronous, capturable, the caller owns every buffer), and:
 *   - x, dy, y and dx: bf16 (x: or codes); x may have a row stride (ldx elements, a multiple of 16 bytes).  dy, y, dx,
 *     W and the scales are dense.  Every matrix lies on 16 bytes, offsets on 4.
 *   - shapes: 0 <= N <= 2^31 - 4096, 1 <= E <= 1024, K and O multiples of 16 up to 2^20; with blocks8 N times the blocks of 128
 *     of K or O below 2^31.  Else MOE_ERR_UNSUPPORTED_SHAPE.
 *   - offsets [E + 1] int32 on the device: 0 <= offsets[0] <= .. <= offsets[E] <= N.  Others are reported as
 *     MOE_ERR_DEVICE_CHECK in the workspace status word (moe_check_status); nothing is then written.
 *   - sums are fp32, over accumulators of the tensor cores, which cut their additions off towards zero: 1024 products of
 *     bf16 or 4096 of codes go to each, whatever the length of the sum.
 *   - repeated calls on the same inputs give the same bits.  A row's y and dx may depend in their last bits on how
 *     many rows the call has (few rows are split along K).
 *   - a wait that runs out (moe_set_wait_limit_ns) is reported as MOE_ERR_TIMEOUT; outputs are then of no use, and the
 *     workspace's first fwd_bytes have to be cleared (to zeros, as at the start) before the next call.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_LINEAR_H_
#define TOP_SOFTMAX_ROUTER_MOE_LINEAR_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LINEAR_MAX_E 1024
#define MOE_LINEAR_MAX_N (2147483647 - 4095)

/* N rows (the call's), K columns of x, O of y, E experts.  blocks8: the workspace has room for the backward pass of
 * operands in 8 bits (dy's codes and x's values). */
typedef struct moe_linear_config {
  int32_t N, K, O, E;
  int32_t blocks8;
} moe_linear_config;

/* Functions of the shape only, not decreasing in N; a workspace starts zeroed and serves fewer rows, too. */
int moe_linear_workspace_bytes(const moe_linear_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes);

/* x_scales and w_scales: both NULL (bf16 x and w) or neither (e4m3 codes).  y [N][O] bf16 out. */
int moe_linear_forward(const moe_linear_config* cfg, const void* x, int64_t ldx, const uint8_t* x_scales, const void* w,
                       const uint8_t* w_scales, const int32_t* offsets, uint16_t* y, void* ws, size_t ws_bytes,
                       void* stream);

/* dx [N][K] bf16 and dw [E][O][K] (dw_type MOE_TYPE_F32 or MOE_TYPE_BF16) out; either may be NULL.  x is not read
 * without dw, w not without dx.  x_scales and w_scales: NULL where that operand is bf16, each on its own. */
int moe_linear_backward(const moe_linear_config* cfg, const void* x, int64_t ldx, const uint8_t* x_scales, const void* w,
                        const uint8_t* w_scales, const int32_t* offsets, const uint16_t* dy, uint16_t* dx, void* dw,
                        int32_t dw_type, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_LINEAR_H_ */

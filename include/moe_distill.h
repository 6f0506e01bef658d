/*
 * moe_distill.h -- C ABI of libmoe.so, part 7: distillation of a vocabulary head from a teacher's top
 * logits, without keeping the student's logits, on one GB300 GPU.  The head is that of moe_ce.h.
 *
 *   z[n, v]  = X[n] . W[v] / T                        (bf16 products, fp32 accumulation; T = temperature)
 *   lse[n]   = log sum_v exp(z[n, v])
 *   q[n, j]  = exp(t[n, j] / T) / sum_i exp(t[n, i] / T)     over the row's entries (class id[n, j],
 *              teacher logit t[n, j]), K at most; the student's softmax runs over all V classes
 *   loss[n]  = T^2 sum_j q[n, j] (log q[n, j] - z[n, id[n, j]] + lse[n])       (KL, scaled by T^2)
 *   and, for an upstream gradient g[n] of loss[n],
 *   d[n, v]  = g[n] T (exp(z[n, v] - lse[n]) - sum over j with id[n, j] = v of q[n, j])   (stored in bf16,
 *              relative to T times the first g whose size is 2^-30 to 2^30, or to T where there is none:
 *              where all rows have one gradient, or 0, that factor is not rounded)
 *   dX[n]    = sum_v d[n, v] W[v]    (fp32 accumulation, stored bf16)
 *   dW[v]    = sum_n d[n, v] X[n]    (fp32 accumulation, stored bf16 or fp32)
 *
 * Rows may have fewer than K entries: an id of -1, or a teacher logit of -inf, is no entry.  A row without
 * entries has loss 0 and gradient 0 (its X must still be finite).  A class may occur twice in a row.
 *
 * Schedule: that of moe_ce.h.  Forward: one tcgen05 GEMM whose epilogue folds each logit tile in tensor
 * memory into (max, sum) pairs and picks out the entries' logits.  Backward: for each of P vocabulary
 * strips (one where d of the whole vocabulary takes at most 8 MB) the logits are recomputed, d is written for that
 * strip only, dX accumulates d W_strip in fp32
 * and dW_strip = d^T X is written.
 *
 * Conventions are those of moe.h (MOE_OK / MOE_ERR_* codes, stream as void*, asynchronous, capturable,
 * the caller owns every buffer and the workspace; X, W, dX and dW 16-byte aligned), and:
 *   - shapes: N >= 0; H a multiple of 64; 1 <= V <= 2^20; 1 <= P <= V; 1 <= K <= 256;
 *     temperature > 0 and finite.  Else MOE_ERR_UNSUPPORTED_SHAPE (the temperature: MOE_ERR_INVALID_ARG).
 *   - an id below -1 or at or above V is reported as MOE_ERR_DEVICE_CHECK through the workspace status
 *     word (moe_check_status) and is no entry.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_DISTILL_H_
#define TOP_SOFTMAX_ROUTER_MOE_DISTILL_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

/* N tokens of hidden size H, V classes, K teacher entries a token, P vocabulary strips in the backward. */
typedef struct moe_distill_config {
  int32_t N, H, V, K, P;
  float temperature;
} moe_distill_config;

/* Workspace bytes (either pointer may be NULL): a function of the shape, not decreasing in N. */
int moe_distill_workspace_bytes(const moe_distill_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes);

/* X [N, H], W [V, H] bf16; ids [N, K] int32; teacher [N, K] fp32.
 * loss, lse [N] fp32 out; loss_mean [1] fp32 out or NULL: sum_n loss[n] / N, summed in a fixed order. */
int moe_distill_forward(const moe_distill_config* cfg, const uint16_t* X, const uint16_t* W, const int32_t* ids,
                        const float* teacher, float* loss, float* lse, float* loss_mean, void* ws, size_t ws_bytes,
                        void* stream);

/* lse [N] from the forward; dloss [N] fp32.  dX [N, H] bf16 out; dW [V, H] out, bf16 or fp32 (dw_type:
 * MOE_TYPE_BF16 or MOE_TYPE_F32; d's rounding to bf16 bounds what either says); both overwritten. */
int moe_distill_backward(const moe_distill_config* cfg, const uint16_t* X, const uint16_t* W, const int32_t* ids,
                         const float* teacher, const float* lse, const float* dloss, uint16_t* dX, void* dW,
                         int32_t dw_type, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_DISTILL_H_ */

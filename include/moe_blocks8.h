/*
 * moe_blocks8.h -- C ABI of libmoe.so, part 8: matrices in 8 bits with a scale for each block of 128, as activation
 * checkpoints and as operands of the products of moe_linear.h.
 *
 * A value is code x scale: the code is e4m3 (no infinities, largest 448), the scale a power of two held as its biased
 * exponent (e8m0: 2^(byte - 127)).  A row of activations has one scale for each 128 columns, a weight matrix one for
 * each 128 x 128 values; the last block of a row or column may be short.  With amax the largest finite magnitude of
 * a block,
 *
 *   scale = 2^e, e >= -127 the smallest with amax <= 448 x 2^e       (1 where amax is 0)
 *   code  = value / scale rounded to nearest even
 *
 * so that a value of ordinary size is off by at most 2^-4 of itself, one below 2^-6 x scale by at most 2^-10 x scale.
 * Because the scale is a power of two, the division is exact and code x scale is a bf16 number without rounding (where
 * it is not below bf16's range).  NaN and infinities become NaN codes and leave the others of their block alone.
 * Magnitudes above 240 x 2^120, of fp32 or bf16, become that (the next code would be an infinity), and so do those above
 * 240 x 2^8 of a block of fp16 rows whose scale is 2^8: what is packed in a type is finite when it is restored in it.
 *
 * Conventions are those of moe.h, and: x has type MOE_TYPE_* and rows `ldx` elements apart; codes and scales are dense
 * ([N][H] and [N][ceil(H / 128)] bytes).  Pointers need only their element's alignment; rows that lie on 16 bytes take
 * 16-byte loads.  Shapes: N >= 0, 1 <= H <= 2^20; weights E, O >= 0, 1 <= K <= 2^20.
 */
#ifndef TOP_SOFTMAX_ROUTER_MOE_BLOCKS8_H_
#define TOP_SOFTMAX_ROUTER_MOE_BLOCKS8_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_types.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_BLOCK8 128

/* codes [N][H], scales [N][ceil(H / 128)] out. */
int moe_blocks8_pack(const void* x, int64_t ldx, int32_t type, int64_t N, int32_t H, uint8_t* codes, uint8_t* scales,
                     void* stream);

/* y [N][H] out, in `type`: code x scale, rounded where the type needs it (bf16 and fp32 do not, above their
 * smallest numbers). */
int moe_blocks8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t N, int32_t H, void* y, int32_t type,
                       void* stream);

/* w [E][O][K] dense; codes [E][O][K], scales [E][ceil(O / 128)][ceil(K / 128)] out. */
int moe_blocks8_pack_weight(const void* w, int32_t type, int32_t E, int32_t O, int32_t K, uint8_t* codes,
                            uint8_t* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SOFTMAX_ROUTER_MOE_BLOCKS8_H_ */

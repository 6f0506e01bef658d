// 8-bit blocks: e4m3 codes with a power-of-two scale for each block of 128 (include/moe_blocks8.h), shared by the packing
// kernels, the RMS norm and the products.
#pragma once

#include "ops_common.cuh"

namespace moe {

// The scale's byte for a block whose largest finite magnitude is amax: 2^e with the smallest e that keeps amax within
// 448 = 1.75 x 2^8, from the exponent and the mantissa of amax alone (no rounding anywhere).
__device__ __forceinline__ int block_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return u == 0 ? 127 : max(b, 0);
}
// 1 / scale; the bytes that block_scale_byte makes (0 .. 247) keep it within the normal numbers.
__device__ __forceinline__ float block_scale_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
// The scale; byte 0 is 2^-127, below the normal numbers, 255 is NaN.
__device__ __forceinline__ float block_scale(int byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)byte << 23);
}
// Largest code: at byte 247 the code above 240, 256 x 2^120, would stand for an infinity.
__device__ __forceinline__ float block_code_limit(int byte) { return byte >= 247 ? 240.0f : 448.0f; }

__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;
}
// v / scale, ready for e4m3: what is not finite becomes NaN.
__device__ __forceinline__ float block_quotient(float v, float inverse, float limit) {
  const float q = v * inverse;
  return fabsf(v) < INFINITY ? fminf(fmaxf(q, -limit), limit) : __uint_as_float(0x7FFFFFFFu);
}
// Two values to two e4m3 codes (lo in the low byte), to nearest even.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes to two fp16 values, which hold every code.
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Eight values of a block by one lane, after amax is known: eight codes.
__device__ __forceinline__ uint2 block_codes(const float (&v)[8], int byte) {
  const float inv = block_scale_inverse(byte), lim = block_code_limit(byte);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = block_quotient(v[i], inv, lim);
  return make_uint2(e4m3_pair(q[0], q[1]) | e4m3_pair(q[2], q[3]) << 16, e4m3_pair(q[4], q[5]) | e4m3_pair(q[6], q[7]) << 16);
}
// The largest over the 16 lanes of a half warp.
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// A half warp's lane holds eight of the 128 values of a block: consecutive ones where the row lies on 16 bytes (VEC),
// else every sixteenth.  f(i, column in block).
template <bool VEC>
__device__ __forceinline__ int block_column(int lane16, int i) { return VEC ? lane16 * 8 + i : lane16 + 16 * i; }

// Loads a lane's eight of the block that starts at p, `valid` values long; zeros past them.
template <class T, bool VEC>
__device__ __forceinline__ void load_block8(const T* p, int lane16, int valid, float (&v)[8]) {
  if constexpr (VEC) {   // valid is a multiple of 8 here
    if (lane16 * 8 < valid) {
      const Pack<T, 8> a = load_pack<T, 8>(p + lane16 * 8);
      unpack<T, 8>(a, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lane16 + 16 * i < valid ? to_f32<T>(p[lane16 + 16 * i]) : 0.0f;
  }
}
template <class T, bool VEC>
__device__ __forceinline__ void store_block8(T* p, int lane16, int valid, const float (&v)[8]) {
  if constexpr (VEC) {
    if (lane16 * 8 < valid) store_pack<T, 8>(p + lane16 * 8, pack<T, 8>(v));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane16 + 16 * i < valid) p[lane16 + 16 * i] = from_f32<T>(v[i]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* p, int lane16, int valid, uint2 c) {
  if constexpr (VEC) {
    if (lane16 * 8 < valid) *reinterpret_cast<uint2*>(p + lane16 * 8) = c;
  } else {
    const uint64_t all = (uint64_t)c.y << 32 | c.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane16 + 16 * i < valid) p[lane16 + 16 * i] = (uint8_t)(all >> (8 * i));
  }
}

}  // namespace moe

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
// Scales from this byte on have codes above 240 that would stand for an infinity of the values' type: 256 x 2^120, of fp32 and
// bf16, and 256 x 2^8 of fp16.
template <class T>
constexpr int kTopByte = std::is_same<T, f16>::value ? 135 : 247;

__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;
}
// Two values to two e4m3 codes (lo in the low byte), to nearest even; NaN to NaN.
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

// A half warp's lane holds eight of the 128 values of a block, as four pairs: consecutive ones where the row lies on 16
// bytes (VEC), else every sixteenth.
template <bool VEC>
__device__ __forceinline__ int block_column(int lane16, int i) { return VEC ? lane16 * 8 + i : lane16 + 16 * i; }

// The lane's eight of the block that starts at p, `valid` values long (a multiple of eight with VEC); zeros past them.
template <class T, bool VEC>
__device__ __forceinline__ Pack<T, 8> load_block8(const T* p, int lane16, int valid) {
  Pack<T, 8> a = zero_pack<T, 8>();
  if constexpr (VEC) {
    if (lane16 * 8 < valid) a = load_pack<T, 8>(p + lane16 * 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane16 + 16 * i < valid) a.v[i] = p[lane16 + 16 * i];
  }
  return a;
}
template <class T, bool VEC>
__device__ __forceinline__ void store_block8(T* p, int lane16, int valid, const Pack<T, 8>& a) {
  if constexpr (VEC) {
    if (lane16 * 8 < valid) store_pack<T, 8>(p + lane16 * 8, a);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane16 + 16 * i < valid) p[lane16 + 16 * i] = a.v[i];
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

// The largest magnitude among a lane's eight (infinity where there is one, NaN passed over), and the largest finite one.
__device__ __forceinline__ float lane_max(const f32x2 (&f)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f[i].get(a, b);
    m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
  }
  return m;
}
__device__ __forceinline__ float lane_finite_max(const f32x2 (&f)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f[i].get(a, b);
    m = fmaxf(m, fmaxf(finite_magnitude(a), finite_magnitude(b)));
  }
  return m;
}
// The largest finite magnitude of each of PER blocks that a half warp holds; the whole warp calls it.  Infinities, which
// are rare, cost a second search; returns whether there was one among the warp's.
template <int PER>
__device__ __forceinline__ bool blocks_max(const f32x2 (&f)[PER][4], float (&m)[PER]) {
  auto among_lanes = [&] {   // the blocks' shuffles side by side
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < PER; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
  };
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    m[i] = lane_max(f[i]);
    most = fmaxf(most, m[i]);
  }
  among_lanes();
  if (!__any_sync(0xffffffffu, most == INFINITY)) return false;
#pragma unroll
  for (int i = 0; i < PER; ++i) m[i] = lane_finite_max(f[i]);
  among_lanes();
  return true;
}
// A lane's eight codes.  infinite: there may be infinities (else the quotients are within the codes, but for bytes from `top`
// on, whose codes end at 240).
__device__ __forceinline__ uint2 block_codes(const f32x2 (&f)[4], int byte, bool infinite, int top) {
  const float inv = block_scale_inverse(byte);
  const f32x2 inv2(inv);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    mul2(f[i], inv2).get(a, b);
    if (infinite || byte >= top) {
      const float lim = byte >= top ? 240.0f : 448.0f;
      a = fabsf(a) < INFINITY ? fminf(fmaxf(a, -lim), lim) : __uint_as_float(0x7FFFFFFFu);
      b = fabsf(b) < INFINITY ? fminf(fmaxf(b, -lim), lim) : __uint_as_float(0x7FFFFFFFu);
    }
    c[i] = e4m3_pair(a, b);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// n / d for n < 2^31, by a multiplication: m = floor(2^32 (2^s - d) / d) + 1 with 2^s >= d (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, m, s;
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

}  // namespace moe

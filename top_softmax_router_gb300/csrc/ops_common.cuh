// Element types, vector loads and reductions shared by the layer operators (norm.cu, embed.cu, scores.cu).
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/moe_types.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

using bf16 = __nv_bfloat16;
using f16 = __half;

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<bf16>(bf16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<f16>(f16 v) { return __half2float(v); }

// Rounds to nearest even.
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float v) { return __float2half_rn(v); }

// VEC consecutive elements as they lie in memory: VEC * sizeof(T) bytes, one aligned access up to 16 bytes.
template <class T, int VEC>
struct alignas(VEC * sizeof(T) >= 16 ? 16 : VEC * sizeof(T)) Pack {
  T v[VEC];
};
// Loads and stores a pack 16 bytes at a time (left to itself the compiler takes a pack of 32 bytes apart into its
// elements: 8-way bank conflicts and eight times the loads).
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* src) {
  Pack<T, VEC> p;
  if constexpr (sizeof(p) >= 16) {
    uint4* d = reinterpret_cast<uint4*>(&p);
#pragma unroll
    for (int i = 0; i < (int)sizeof(p) / 16; ++i) d[i] = reinterpret_cast<const uint4*>(src)[i];
  } else {
    p = *reinterpret_cast<const Pack<T, VEC>*>(src);
  }
  return p;
}
template <class T, int VEC>
__device__ __forceinline__ void store_pack(T* dst, const Pack<T, VEC>& p) {
  if constexpr (sizeof(p) >= 16) {
    const uint4* s = reinterpret_cast<const uint4*>(&p);
#pragma unroll
    for (int i = 0; i < (int)sizeof(p) / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = s[i];
  } else {
    *reinterpret_cast<Pack<T, VEC>*>(dst) = p;
  }
}

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> filled_pack(float v) {
  Pack<T, VEC> p;
#pragma unroll
  for (int i = 0; i < VEC; ++i) p.v[i] = from_f32<T>(v);
  return p;
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> zero_pack() { return filled_pack<T, VEC>(0.0f); }
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> one_pack() { return filled_pack<T, VEC>(1.0f); }

template <class T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&f)[VEC]) {
  if constexpr (std::is_same<T, bf16>::value && VEC % 2 == 0) {   // a bf16 is the upper half of its fp32
    const uint32_t* u = reinterpret_cast<const uint32_t*>(p.v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32<T>(p.v[i]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const float (&f)[VEC]) {
  Pack<T, VEC> p;
  if constexpr (std::is_same<T, bf16>::value && VEC % 2 == 0) {
    uint32_t* u = reinterpret_cast<uint32_t*>(p.v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  } else if constexpr (std::is_same<T, f16>::value && VEC % 2 == 0) {
    __half2* u = reinterpret_cast<__half2*>(p.v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) u[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p.v[i] = from_f32<T>(f[i]);
  }
  return p;
}

// Two fp32 values in a register pair: one instruction adds, multiplies or fuses both (sm_100 and later), each
// rounded as the scalar instruction would.
struct f32x2 {
  uint64_t r;
  __device__ __forceinline__ f32x2() {}
  __device__ __forceinline__ f32x2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit f32x2(float a) : f32x2(a, a) {}
  __device__ __forceinline__ float sum() const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
    return a + b;
  }
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
};
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.r) : "l"(a.r), "l"(b.r));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.r) : "l"(a.r), "l"(b.r));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.r) : "l"(a.r), "l"(b.r), "l"(c.r));
  return d;
}
// A pack as pairs; an odd one (VEC = 1) is a pair whose second value is `fill`.
template <int VEC>
constexpr int pairs_of = (VEC + 1) / 2;
template <class T, int VEC>
__device__ __forceinline__ void unpack2(const Pack<T, VEC>& p, f32x2 (&f)[pairs_of<VEC>], float fill = 0.0f) {
  float v[VEC];
  unpack<T, VEC>(p, v);
  if constexpr (VEC == 1) {
    f[0] = f32x2(v[0], fill);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = f32x2(v[2 * i], v[2 * i + 1]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack2(const f32x2 (&f)[pairs_of<VEC>]) {
  float v[2 * pairs_of<VEC>];
#pragma unroll
  for (int i = 0; i < pairs_of<VEC>; ++i) f[i].get(v[2 * i], v[2 * i + 1]);
  float o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = v[i];
  return pack<T, VEC>(o);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

inline int type_size(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }
inline bool known_type(int type) { return type == MOE_TYPE_F32 || type == MOE_TYPE_BF16 || type == MOE_TYPE_F16; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Calls f(T{}) for the element type.
template <class F>
auto with_type(int type, F&& f) {
  if (type == MOE_TYPE_BF16) return f(bf16{});
  if (type == MOE_TYPE_F16) return f(f16{});
  return f(float{});
}

}  // namespace moe

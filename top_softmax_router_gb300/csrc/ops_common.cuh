// Element types, vector loads and reductions shared by the layer operators (norm.cu, embed.cu, scores.cu).
#pragma once

#include <cuda_fp16.h>

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
template <class T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&f)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = to_f32<T>(p.v[i]);
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const float (&f)[VEC]) {
  Pack<T, VEC> p;
#pragma unroll
  for (int i = 0; i < VEC; ++i) p.v[i] = from_f32<T>(f[i]);
  return p;
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

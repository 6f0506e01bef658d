// Matrices in 8 bits with a scale for each block of 128 (include/moe_blocks8.h): packing of rows and of weights, unpacking.
//
// All three are one pass over memory: 2 + 1 + 1/128 bytes a bf16 value.  A half warp holds a row's block of 128, eight
// values a lane (16 bytes of bf16), and finds its largest magnitude by four shuffles; four blocks side by side keep enough
// loads in flight.  A block's row comes from a multiplication (divisions of 64 bits and the tests for infinities of every
// value held the pair of passes below at 443 us).  65536 x 4096 bf16, packed and restored: 257 us, 6.3 TB/s of the
// measured 6.8.  Weights wait longer for their 128 x 128 block: two blocks of threads a SM (92 to 106 registers), each with one
// round of loads before its maximum; 128 x 1536 x 4096 bf16 571 us, 4.2 TB/s.
#include <algorithm>

#include "../../include/moe_blocks8.h"
#include "blocks8.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // blocks a half warp has in flight

// VEC: rows of x and codes lie on 16 and 8 bytes and hold a multiple of eight values.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    pack_rows_kernel(const T* __restrict__ x, int64_t ldx, int blocks, FastDiv nb, int H, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane16 = threadIdx.x & 15;
  const int64_t first = ((int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kBatch;
  f32x2 f[kBatch][4];
  int64_t to[kBatch];
  int valid[kBatch];
  Pack<T, 8> raw[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int at = (int)min(first + j, (int64_t)blocks - 1);
    const int row = (int)nb(at), col = (at - row * (int)nb.d) * MOE_BLOCK8;
    valid[j] = first + j < blocks ? min(MOE_BLOCK8, H - col) : 0;
    to[j] = (int64_t)row * H + col;
    raw[j] = load_block8<T, VEC>(x + row * ldx + col, lane16, valid[j]);
  }
#pragma unroll
  for (int j = 0; j < kBatch; ++j) unpack2<T, 8>(raw[j], f[j]);
  float m[kBatch];
  const bool infinite = blocks_max<kBatch>(f, m);
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int byte = block_scale_byte(m[j]);
    if (valid[j]) {
      store_codes8<VEC>(codes + to[j], lane16, valid[j], block_codes(f[j], byte, infinite, kTopByte<T>));
      if (lane16 == 0) scales[first + j] = (uint8_t)byte;
    }
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    unpack_rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int blocks, FastDiv nb,
                       int H, T* __restrict__ y) {
  pdl_wait();
  pdl_trigger();
  const int lane16 = threadIdx.x & 15;
  const int64_t first = ((int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kBatch;
  uint64_t c[kBatch];
  int byte[kBatch], valid[kBatch];
  int64_t from[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int at = (int)min(first + j, (int64_t)blocks - 1);
    const int row = (int)nb(at), col = (at - row * (int)nb.d) * MOE_BLOCK8;
    valid[j] = first + j < blocks ? min(MOE_BLOCK8, H - col) : 0;
    from[j] = (int64_t)row * H + col;
    c[j] = 0;
    byte[j] = scales[at];
    if constexpr (VEC) {
      if (lane16 * 8 < valid[j]) c[j] = *reinterpret_cast<const uint64_t*>(codes + from[j] + lane16 * 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane16 + 16 * i < valid[j]) c[j] |= (uint64_t)codes[from[j] + lane16 + 16 * i] << (8 * i);
    }
  }
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const f32x2 s(block_scale(byte[j]));
    f32x2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = e4m3_values((uint32_t)(c[j] >> (16 * i)) & 0xFFFFu);
      v[i] = mul2(f32x2(p.x, p.y), s);
    }
    store_block8<T, VEC>(y + from[j], lane16, valid[j], pack2<T, 8>(v));
  }
}

// One block of threads for 128 x 128 values: a half warp takes every sixteenth row.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    pack_weight_kernel(const T* __restrict__ w, int O, int K, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  __shared__ float most[2][kThreads / 32];
  const int nk = (K + MOE_BLOCK8 - 1) / MOE_BLOCK8, no = (O + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  const int kb = blockIdx.x % nk;
  const int eo = blockIdx.x / nk;                   // (expert, block of rows)
  const int ob = eo % no;
  const int64_t e = eo / no;
  const int lane16 = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int valid = min(MOE_BLOCK8, K - kb * MOE_BLOCK8);
  const int64_t base = (e * O + ob * MOE_BLOCK8) * K + kb * MOE_BLOCK8;
  const int rows = min(MOE_BLOCK8, O - ob * MOE_BLOCK8);
  f32x2 f[8][4];
  Pack<T, 8> raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = sub + 16 * j;
    raw[j] = load_block8<T, VEC>(w + base + (r < rows ? (int64_t)r * K : 0), lane16, r < rows ? valid : 0);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) unpack2<T, 8>(raw[j], f[j]);
  auto among_threads = [&](float m, int turn) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((threadIdx.x & 31) == 0) most[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, most[turn][i]);
    return m;
  };
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, lane_max(f[j]));
  m = among_threads(m, 0);
  const bool infinite = m == INFINITY;              // of all threads alike
  if (infinite) {
    m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, lane_finite_max(f[j]));
    m = among_threads(m, 1);
  }
  const int byte = block_scale_byte(m);
  if (threadIdx.x == 0) scales[blockIdx.x] = (uint8_t)byte;   // [e][ob][kb]
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = sub + 16 * j;
    if (r < rows) store_codes8<VEC>(codes + base + (int64_t)r * K, lane16, valid, block_codes(f[j], byte, infinite, kTopByte<float>));
  }
}

constexpr int kMaxWidth = 1 << 20;
inline int64_t row_blocks(int64_t N, int nb) { return (N * nb + kThreads / 16 * kBatch - 1) / (kThreads / 16 * kBatch); }
// Blocks of 128 are counted in 31 bits (2.7e11 values).
inline bool too_many(int64_t N, int64_t nb) { return N > INT32_MAX / nb; }

}  // namespace

cudaError_t launch_pack_rows(const void* x, int64_t ldx, int type, int64_t N, int H, uint8_t* codes, uint8_t* scales,
                             cudaStream_t s) {
  const int nb = (H + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  const bool vec = aligned_to(x, 16) && H % 8 == 0 && (ldx * type_size(type)) % 16 == 0 && aligned_to(codes, 8);
  return with_type(type, [&](auto tv) {
    using T = decltype(tv);
    auto go = [&](auto kern) {
      return launch_pdl(kern, dim3((unsigned)row_blocks(N, nb)), dim3(kThreads), 0, s, static_cast<const T*>(x), ldx,
                        (int)(N * nb), FastDiv(nb), H, codes, scales);
    };
    return vec ? go(pack_rows_kernel<T, true>) : go(pack_rows_kernel<T, false>);
  });
}

cudaError_t launch_unpack_rows(const uint8_t* codes, const uint8_t* scales, int64_t N, int H, void* y, int type,
                               cudaStream_t s) {
  const int nb = (H + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  const bool vec = aligned_to(y, 16) && H % 8 == 0 && aligned_to(codes, 8);
  return with_type(type, [&](auto tv) {
    using T = decltype(tv);
    auto go = [&](auto kern) {
      return launch_pdl(kern, dim3((unsigned)row_blocks(N, nb)), dim3(kThreads), 0, s, codes, scales, (int)(N * nb),
                        FastDiv(nb), H, static_cast<T*>(y));
    };
    return vec ? go(unpack_rows_kernel<T, true>) : go(unpack_rows_kernel<T, false>);
  });
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_blocks8_pack(const void* x, int64_t ldx, int32_t type, int64_t N, int32_t H, uint8_t* codes, uint8_t* scales,
                     void* stream) {
  if (N < 0 || H < 1 || !known_type(type) || ldx < H) return MOE_ERR_INVALID_ARG;
  const int64_t nb = (H + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  if (H > kMaxWidth || too_many(N, nb)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned_to(x, type_size(type))) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed_launch(MOE_K_BLOCKS8, "pack in 8 bits", s,
                      [&] { return launch_pack_rows(x, ldx, type, N, H, codes, scales, s); });
}

int moe_blocks8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t N, int32_t H, void* y, int32_t type,
                       void* stream) {
  if (N < 0 || H < 1 || !known_type(type)) return MOE_ERR_INVALID_ARG;
  const int64_t nb = (H + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  if (H > kMaxWidth || too_many(N, nb)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return MOE_OK;
  if (!y || !codes || !scales || !aligned_to(y, type_size(type))) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed_launch(MOE_K_BLOCKS8, "unpack from 8 bits", s,
                      [&] { return launch_unpack_rows(codes, scales, N, H, y, type, s); });
}

int moe_blocks8_pack_weight(const void* w, int32_t type, int32_t E, int32_t O, int32_t K, uint8_t* codes,
                            uint8_t* scales, void* stream) {
  if (E < 0 || O < 0 || K < 1 || !known_type(type)) return MOE_ERR_INVALID_ARG;
  const int64_t nk = (K + MOE_BLOCK8 - 1) / MOE_BLOCK8, no = ((int64_t)O + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  if (K > kMaxWidth || O > kMaxWidth || E * no > INT32_MAX / nk) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (E == 0 || O == 0) return MOE_OK;
  if (!w || !codes || !scales || !aligned_to(w, type_size(type))) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = aligned_to(w, 16) && K % 8 == 0 && aligned_to(codes, 8);
  return timed_launch(MOE_K_BLOCKS8, "pack weights in 8 bits", s, [&] {
    return with_type(type, [&](auto tv) {
      using T = decltype(tv);
      auto go = [&](auto kern) {
        return launch_pdl(kern, dim3((unsigned)(E * no * nk)), dim3(kThreads), 0, s, static_cast<const T*>(w), O, K,
                          codes, scales);
      };
      return vec ? go(pack_weight_kernel<T, true>) : go(pack_weight_kernel<T, false>);
    });
  });
}

}  // extern "C"

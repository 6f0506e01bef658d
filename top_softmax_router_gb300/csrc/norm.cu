// Layer normalisation, forward and backward (include/moe_norm.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/moe.h"
#include "../../include/moe_norm.h"
#include "ops_common.cuh"

namespace moe {
namespace {

// A row is held in registers by `tpr` threads (32, or a multiple of 128), PER packs of VEC elements each:
// pack i of thread t holds columns VEC (t + i tpr) ..  A block of max(tpr, 128) threads holds
// block / tpr rows at a time.
struct RowShape {
  int tpr, block, rows;   // threads per row, threads per block, rows per block
};

// Sums of two values over the tpr threads of a row: one shuffle tree per warp, then the warps' sums in
// order.  `red`: 2 x 32 floats of shared memory, used alternately by the caller (`slot`).
__device__ __forceinline__ float2 row_sum2(float a, float b, int tpr, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (tpr == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = tpr >> 5;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const int w0 = warp / warps * warps;
  const float2 v = lane < warps ? red[w0 + lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// One pass: x is read once, kept in registers for the mean, the variance around it and the output.
template <class T, class P, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_fwd_kernel(const T* __restrict__ x, int64_t ldx,
                                                       const P* __restrict__ weight, const P* __restrict__ bias,
                                                       T* __restrict__ y, float* __restrict__ mean,
                                                       float* __restrict__ rstd, int N, int H, float eps, int tpr) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % tpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int packs = H / VEC;
  const bool row_ok = row < N;
  const T* xr = x + row * ldx;
  Pack<T, VEC> raw[PER];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = t + i * tpr;
    if (row_ok && c < packs) raw[i] = *reinterpret_cast<const Pack<T, VEC>*>(xr + (int64_t)c * VEC);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (row_ok && t + i * tpr < packs) {
      float f[VEC];
      unpack<T, VEC>(raw[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += f[j];
    }
  }
  const float inv_h = 1.0f / (float)H;
  const float mu = row_sum2(s, 0.0f, tpr, red[0]).x * inv_h;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (row_ok && t + i * tpr < packs) {
      float f[VEC];
      unpack<T, VEC>(raw[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) q = fmaf(f[j] - mu, f[j] - mu, q);
    }
  }
  const float rs = 1.0f / sqrtf(row_sum2(q, 0.0f, tpr, red[1]).x * inv_h + eps);
  if (!row_ok) return;
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = t + i * tpr;
    if (c < packs) {
      float f[VEC], o[VEC];
      unpack<T, VEC>(raw[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = (f[j] - mu) * rs;
      if (weight) {
        Pack<P, VEC> w = *reinterpret_cast<const Pack<P, VEC>*>(weight + c * VEC);
        unpack<P, VEC>(w, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] *= f[j];
      }
      if (bias) {
        Pack<P, VEC> b = *reinterpret_cast<const Pack<P, VEC>*>(bias + c * VEC);
        unpack<P, VEC>(b, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += f[j];
      }
      *reinterpret_cast<Pack<T, VEC>*>(y + row * H + (int64_t)c * VEC) = pack<T, VEC>(o);
    }
  }
}

// Persistent: block b takes row groups b, b + grid, ..  x and dy are read once; dx is written, and each
// thread keeps the sums of dy xh and dy of its columns in registers over all its rows.  The block's sums
// go to part[block][2][H]; norm_param_kernel adds the blocks in order, so the result has a fixed order.
template <class T, class P, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_bwd_kernel(const T* __restrict__ x, int64_t ldx,
                                                       const P* __restrict__ weight, const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, const T* __restrict__ dy,
                                                       int64_t lddy, T* __restrict__ dx, float* __restrict__ part,
                                                       int N, int H, int tpr) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 red[2][32];
  extern __shared__ float cols[];   // [2][H]: sums of the block's rows, when it holds several at a time
  const int t = threadIdx.x % tpr, rpb = blockDim.x / tpr, sub = threadIdx.x / tpr;
  const int packs = H / VEC;
  const float inv_h = 1.0f / (float)H;
  float gw[PER][VEC], gb[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) gw[i][j] = gb[i][j] = 0.0f;
  int it = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < N; base += (int64_t)gridDim.x * rpb, ++it) {
    const int64_t row = base + sub;
    const bool row_ok = row < N;
    Pack<T, VEC> rx[PER], rd[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * tpr;
      if (row_ok && c < packs) {
        rx[i] = *reinterpret_cast<const Pack<T, VEC>*>(x + row * ldx + (int64_t)c * VEC);
        rd[i] = *reinterpret_cast<const Pack<T, VEC>*>(dy + row * lddy + (int64_t)c * VEC);
      }
    }
    const float mu = row_ok ? mean[row] : 0.0f, rs = row_ok ? rstd[row] : 0.0f;
    float s = 0.0f, sx = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * tpr;
      if (row_ok && c < packs) {
        float fx[VEC], fd[VEC], fw[VEC];
        unpack<T, VEC>(rx[i], fx);
        unpack<T, VEC>(rd[i], fd);
        if (weight) {
          Pack<P, VEC> w = *reinterpret_cast<const Pack<P, VEC>*>(weight + c * VEC);
          unpack<P, VEC>(w, fw);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (fx[j] - mu) * rs;
          gw[i][j] = fmaf(fd[j], xh, gw[i][j]);
          gb[i][j] += fd[j];
          const float tj = weight ? fd[j] * fw[j] : fd[j];
          s += tj;
          sx = fmaf(tj, xh, sx);
        }
      }
    }
    if (dx) {
      const float2 sums = row_sum2(s, sx, tpr, red[it & 1]);
      const float a = sums.x * inv_h, b = sums.y * inv_h;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = t + i * tpr;
        if (row_ok && c < packs) {
          float fx[VEC], fd[VEC], fw[VEC], o[VEC];
          unpack<T, VEC>(rx[i], fx);
          unpack<T, VEC>(rd[i], fd);
          if (weight) {
            Pack<P, VEC> w = *reinterpret_cast<const Pack<P, VEC>*>(weight + c * VEC);
            unpack<P, VEC>(w, fw);
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float xh = (fx[j] - mu) * rs;
            const float tj = weight ? fd[j] * fw[j] : fd[j];
            o[j] = rs * (tj - a - xh * b);
          }
          *reinterpret_cast<Pack<T, VEC>*>(dx + row * H + (int64_t)c * VEC) = pack<T, VEC>(o);
        }
      }
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * 2 * H;
  // the rows of the block are added in turn: row group 0 first
  for (int r = 0; r < rpb; ++r) {
    if (sub == r) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = t + i * tpr;
        if (c < packs) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int h = c * VEC + j;
            float a = gw[i][j], b = gb[i][j];
            if (r > 0) a += cols[h], b += cols[H + h];
            if (r + 1 < rpb) cols[h] = a, cols[H + h] = b;
            else out[h] = a, out[H + h] = b;
          }
        }
      }
    }
    if (r + 1 < rpb) __syncthreads();
  }
}

// dweight[h], dbias[h]: the blocks' partial sums added in a fixed order.  A block owns 32 columns; its 8
// warps take the partials round robin and their sums are added in warp order.
__global__ void __launch_bounds__(256) norm_param_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                        float* __restrict__ dbias, int blocks, int H) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;   // column of the [2 H] row of partials
  const bool second = blockIdx.y == 1;
  float* out = second ? dbias : dweight;
  if (!out) return;
  float a = 0.0f;
  if (c < H) {
    const float* p = part + (second ? H : 0) + c;
    for (int b = warp; b < blocks; b += 8) a += p[(int64_t)b * 2 * H];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int w = 1; w < 8; ++w) a += s[w][lane];
    out[c] = a;
  }
}

int norm_validate(const moe_layernorm_config* c) {
  if (!c || c->N < 0 || c->H <= 0 || !(c->eps >= 0.0f) || !std::isfinite(c->eps)) return MOE_ERR_INVALID_ARG;
  if (c->H > MOE_LAYERNORM_MAX_H) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

constexpr int kMaxBwdBlocks = 152 * 4;

// Threads for `packs` packs a row, at most `per` packs a thread.
RowShape row_shape(int packs, int per) {
  RowShape s;
  s.tpr = packs <= 32 * per ? 32 : (packs + per - 1) / per;
  if (s.tpr > 32) s.tpr = s.tpr <= 128 ? 128 : (s.tpr + 127) / 128 * 128;
  s.block = std::max(s.tpr, 128);
  s.rows = s.block / s.tpr;
  return s;
}

int bwd_blocks(int N) { return std::min(N, kMaxBwdBlocks); }

template <class T, class P, int VEC, int PER, int THREADS>
cudaError_t fwd_launch(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight,
                       const void* bias, void* y, float* mean, float* rstd, cudaStream_t s) {
  const RowShape r = row_shape(c.H / VEC, PER);
  return launch_pdl(norm_fwd_kernel<T, P, VEC, PER, THREADS>,
                    dim3((unsigned)((c.N + (int64_t)r.rows - 1) / r.rows)), dim3(r.block), 0, s,
                    static_cast<const T*>(x), ldx, static_cast<const P*>(weight), static_cast<const P*>(bias),
                    static_cast<T*>(y), mean, rstd, c.N, c.H, c.eps, r.tpr);
}

template <class T, class P, int VEC, int PER, int THREADS>
cudaError_t bwd_launch(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight,
                       const float* mean, const float* rstd, const void* dy, int64_t lddy, void* dx, float* part,
                       int* blocks, cudaStream_t s) {
  const RowShape r = row_shape(c.H / VEC, PER);
  auto kern = norm_bwd_kernel<T, P, VEC, PER, THREADS>;
  const size_t smem = r.rows > 1 ? 32 * PER * VEC * 8 : 0;   // [2][H], H <= 32 PER VEC; at most 16 KB
  static std::atomic<int> cached[33];                        // resident blocks an SM by block size
  int per_sm = cached[r.block / 32].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, r.block, smem);
    if (e != cudaSuccess) return e;
    cached[r.block / 32].store(per_sm = std::max(1, per_sm), std::memory_order_relaxed);
  }
  const int64_t groups = ((int64_t)c.N + r.rows - 1) / r.rows;
  *blocks = (int)std::min<int64_t>(groups, std::min(bwd_blocks(c.N), per_sm * device_sm_count()));
  return launch_pdl(kern, dim3(*blocks), dim3(r.block), smem, s, static_cast<const T*>(x), ldx,
                    static_cast<const P*>(weight), mean, rstd, static_cast<const T*>(dy), lddy, static_cast<T*>(dx),
                    part, c.N, c.H, r.tpr);
}

// Calls f(T, P, VEC, PER, THREADS) with compile-time values.  vec: rows and parameters take 16-byte packs.
// Up to 128 packs a row a warp holds it; above, a block with two packs a thread (four where that would
// pass 1024 threads).
template <class F>
cudaError_t with_shape(int type, int param_type, bool vec, int H, F&& f) {
  return with_type(type, [&](auto tv) {
    using T = decltype(tv);
    auto by_param = [&](auto pv) {
      constexpr int V = 16 / sizeof(T);
      auto go = [&](auto v, auto per, auto threads) { return f(tv, pv, v, per, threads); };
#define MOE_INT(n) std::integral_constant<int, n>{}
      if (vec) {
        const int packs = H / V;
        if (packs <= 32) return go(MOE_INT(V), MOE_INT(1), MOE_INT(128));
        if (packs <= 64) return go(MOE_INT(V), MOE_INT(2), MOE_INT(128));
        if (packs <= 128) return go(MOE_INT(V), MOE_INT(4), MOE_INT(128));
        if (packs <= 1024) return go(MOE_INT(V), MOE_INT(2), MOE_INT(512));
        return go(MOE_INT(V), MOE_INT(4), MOE_INT(1024));
      }
      if (H <= 128) return go(MOE_INT(1), MOE_INT(4), MOE_INT(128));
      if (H <= 4096) return go(MOE_INT(1), MOE_INT(8), MOE_INT(512));
      return go(MOE_INT(1), MOE_INT(16), MOE_INT(1024));
#undef MOE_INT
    };
    if (param_type == MOE_TYPE_F32) return by_param(float{});
    return by_param(tv);
  });
}

bool vec_rows(const void* p, int64_t ld, int H, int type) {
  const int v = 16 / type_size(type);
  return aligned_to(p, 16) && H % v == 0 && ld % v == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_layernorm_workspace_bytes(const moe_layernorm_config* cfg, size_t* bwd_bytes) {
  const int v = norm_validate(cfg);
  if (v != MOE_OK) return v;
  if (bwd_bytes) *bwd_bytes = align256((size_t)bwd_blocks(cfg->N) * 2 * cfg->H * 4);
  return MOE_OK;
}

int moe_layernorm_forward(const moe_layernorm_config* cfg, const void* x, int64_t ldx, const void* weight,
                          const void* bias, void* y, float* mean, float* rstd, int32_t type, int32_t param_type,
                          void* stream) {
  const int v = norm_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_layernorm_config& c = *cfg;
  if (!known_type(type) || !(param_type == type || param_type == MOE_TYPE_F32) || ldx < c.H)
    return MOE_ERR_INVALID_ARG;
  const size_t ts = type_size(type), ps = type_size(param_type);
  if (!aligned_to(weight, ps) || !aligned_to(bias, ps) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (c.N == 0) return MOE_OK;
  if (!x || !y || !aligned_to(x, ts) || !aligned_to(y, ts)) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = vec_rows(x, ldx, c.H, type) && aligned_to(y, 16) && aligned_to(weight, 16) && aligned_to(bias, 16);
  return timed_launch(MOE_K_NORM_FWD, "layer norm", s, [&] {
    return with_shape(type, param_type, vec, c.H, [&](auto tv, auto pv, auto vv, auto per, auto threads) {
      return fwd_launch<decltype(tv), decltype(pv), decltype(vv)::value, decltype(per)::value,
                        decltype(threads)::value>(
          c, x, ldx, weight, bias, y, mean, rstd, s);
    });
  });
}

int moe_layernorm_backward(const moe_layernorm_config* cfg, const void* x, int64_t ldx, const void* weight,
                           const float* mean, const float* rstd, const void* dy, int64_t lddy, void* dx,
                           float* dweight, float* dbias, int32_t type, int32_t param_type, void* ws, size_t ws_bytes,
                           void* stream) {
  int v = norm_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_layernorm_config& c = *cfg;
  if (!known_type(type) || !(param_type == type || param_type == MOE_TYPE_F32) || ldx < c.H || lddy < c.H)
    return MOE_ERR_INVALID_ARG;
  if (!aligned_to(weight, type_size(param_type)) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return MOE_ERR_INVALID_ARG;
  const bool params = dweight || dbias;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N == 0) {
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)c.H * 4, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)c.H * 4, s);
    return e == cudaSuccess ? MOE_OK : record_cuda_error(e, "clear the norm's gradients");
  }
  const size_t ts = type_size(type);
  if (!x || !dy || !mean || !rstd || !aligned_to(x, ts) || !aligned_to(dy, ts) || !aligned_to(dx, ts) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (params) {
    if (!ws || !aligned_to(ws, 16)) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_layernorm_workspace_bytes(cfg, &need);
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (!dx && !params) return MOE_OK;
  const bool vec = vec_rows(x, ldx, c.H, type) && vec_rows(dy, lddy, c.H, type) && aligned_to(dx, 16) &&
                   aligned_to(weight, 16);
  float* part = params ? static_cast<float*>(ws) : nullptr;
  int blocks = 0;
  v = timed_launch(MOE_K_NORM_BWD, "layer norm backward", s, [&] {
    return with_shape(type, param_type, vec, c.H, [&](auto tv, auto pv, auto vv, auto per, auto threads) {
      return bwd_launch<decltype(tv), decltype(pv), decltype(vv)::value, decltype(per)::value,
                        decltype(threads)::value>(
          c, x, ldx, weight, mean, rstd, dy, lddy, dx, part, &blocks, s);
    });
  });
  if (v != MOE_OK || !params) return v;
  return timed_launch(MOE_K_NORM_BWD, "layer norm parameter gradients", s, [&] {
    return launch_pdl(norm_param_kernel, dim3((c.H + 31) / 32, 2), dim3(256), 0, s, static_cast<const float*>(part),
                      dweight, dbias, blocks, c.H);
  });
}

}  // extern "C"

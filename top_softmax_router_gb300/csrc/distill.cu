// Distillation of a vocabulary head from a teacher's top logits (include/moe_distill.h).
//
// The entries (row, class, probability q) are put into buckets of 32 rows x 256 classes first, so that the GEMM
// epilogues find those of their tile: the forward reads their logits out of tensor memory, the backward subtracts q
// at their places.  Everything else of d is one exponential.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe.h"
#include "../../include/moe_distill.h"
#include "head_gemm.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

constexpr int kMaxK = 256;
constexpr int kGroup = 32;        // rows of a bucket
// Row tiles of a band: the 76 clusters at work then hold 16 x ~5 tiles, 43 MB of operands at H = 4096 (a training step of
// 8192 x 4096 x 65536 with 4: 11.99 ms, 8: 11.62, 16: 11.58, 32: 12.21).
constexpr int kHeadBand = 16;
constexpr int kClusters = 76;     // CTA pairs of the GPU
// A d of the whole vocabulary of at most this is one strip whatever P: three launches instead of 3 P (53 x 640 x 60341,
// P = 3: 168 us of backward instead of 220).
constexpr int64_t kOneStrip = 8 << 20;

// One block a group of 32 rows, a row a warp: q of each entry, equal classes of a row joined at the first of
// them (class[j] = -1 for every other), the row's sum of q log q, and the group's entries by class tile.  Latency:
// 2048 rows of 32 entries 10 us.
__global__ void __launch_bounds__(1024) distill_prep_kernel(const int32_t* __restrict__ ids,
                                                           const float* __restrict__ teacher,
                                                           const float* __restrict__ dloss, float* __restrict__ q_out,
                                                           int32_t* __restrict__ class_out, float* __restrict__ qlogq,
                                                           float* __restrict__ coef, float* __restrict__ out_scale,
                                                           int* __restrict__ bucket,
                                                           uint32_t* __restrict__ entry, int N, int V, int K, int tiles,
                                                           float T, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int count[];            // [tiles + 1], then each warp's classes and q [K]
  __shared__ int scratch[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x, r0 = group * kGroup, row = r0 + warp;
  int* s_class = count + tiles + 1 + warp * 2 * K;
  float* s_q = reinterpret_cast<float*>(s_class + K);
  for (int i = threadIdx.x; i <= tiles; i += 1024) count[i] = 0;
  float c0 = 1.0f;
  if (coef) {
    // d is stored relative to the first gradient of an ordinary size (a masked row's is 0), which the products'
    // epilogues put back in fp32: with one gradient for all rows (a mean) its rounding would otherwise be the same in
    // every d and not average out
    for (int base = 0; base < N; base += 1024) {
      const int i = base + threadIdx.x;
      const float g = i < N ? fabsf(dloss[i]) : 0.0f;
      const uint32_t found = __ballot_sync(0xffffffffu, g >= 0x1p-30f && g <= 0x1p30f);
      if (lane == 0) scratch[warp] = found ? base + warp * 32 + __ffs(found) - 1 : N;
      if (__syncthreads_or(found != 0)) break;
    }
    const int first = __reduce_min_sync(0xffffffffu, scratch[lane]);
    if (first < N) c0 = dloss[first];
    if (group == 0 && threadIdx.x == 0) *out_scale = c0 * T;
  }
  __syncthreads();
  if (row < N) {                            // the same for the whole warp
    const int64_t base = (int64_t)row * K;
    float m = -INFINITY;
    for (int j = lane; j < K; j += 32) {
      const int c = ids[base + j];
      if (c < -1 || c >= V) report(status, MOE_ERR_DEVICE_CHECK, 711);
      const float t = teacher[base + j];
      const bool there = c >= 0 && c < V && t != -INFINITY;
      s_class[j] = there ? c : -1;
      s_q[j] = t;
      if (there) m = fmaxf(m, t);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float sum = 0.0f, dot = 0.0f;
    for (int j = lane; j < K; j += 32) {
      const bool there = s_class[j] >= 0;
      const float x = there ? (s_q[j] - m) / T : 0.0f;
      const float e = there ? expf(x) : 0.0f;
      s_q[j] = e;
      sum += e;
      if (e != 0.0f) dot = fmaf(e, x, dot);   // a finite logit's distance from m, over T, may pass fp32: x is -inf
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    const bool some = sum != 0.0f;          // the largest entry's e is 1
    if (lane == 0) {
      qlogq[row] = some ? dot / sum - logf(sum) : 0.0f;
      if (coef) coef[row] = some ? dloss[row] / c0 : 0.0f;
    }
    __syncwarp();
    for (int j = lane; j < K; j += 32) {
      int c = s_class[j];
      float q = 0.0f;
      if (c >= 0) {
        bool first = true;
        for (int i = 0; i < j; ++i) first &= s_class[i] != c;
        if (first)
          for (int i = j; i < K; ++i) q += s_class[i] == c ? s_q[i] : 0.0f;
        else
          c = -1;
      }
      q_out[base + j] = some ? q / sum : 0.0f;
      class_out[base + j] = c;
      if (c >= 0) atomicAdd(count + (c >> 8), 1);
    }
    __syncwarp();
  }
  __syncthreads();
  // exclusive scan of the counts; thread t owns a run of tiles
  const int per = (tiles + 1023) / 1024, t0 = threadIdx.x * per, t1 = min(tiles, t0 + per);
  int own = 0;
  for (int t = t0; t < t1; ++t) own += count[t];
  int x = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int at = x - own;
  for (int w = 0; w < warp; ++w) at += scratch[w];
  at += group * kGroup * K;
  int* b = bucket + (int64_t)group * (tiles + 1);
  for (int t = t0; t < t1; ++t) {
    const int c = count[t];
    b[t] = at;
    count[t] = at;
    at += c;
  }
  if (t0 < tiles && t1 == tiles) b[tiles] = at;
  __syncthreads();
  // an entry's place within its bucket does not change any result
  if (row < N) {
    for (int j = lane; j < K; j += 32) {
      const int c = class_out[(int64_t)row * K + j];   // this lane's own
      if (c >= 0) entry[atomicAdd(count + (c >> 8), 1)] = (uint32_t)warp | (uint32_t)(c & 255) << 5 | (uint32_t)j << 13;
    }
  }
}

// Folds (m2, z2) into (m, z): z counts in units of 2^m.
__device__ __forceinline__ void fold2(float& m, float& z, float m2, float z2) {
  const float mn = fmaxf(m, m2);
  if (mn == -INFINITY) return;
  z = z * exp2f(m - mn) + z2 * exp2f(m2 - mn);
  m = mn;
}

// 32 rows a block: lse from the half tiles' pairs (warp w takes half tiles w, w + 32, .. in order, four loads at a time;
// then the warps are folded in order), and the loss from the entries' logits, a row a warp.  2048 x 32000: 8 us.
__global__ void __launch_bounds__(1024) distill_loss_kernel(const float* __restrict__ part_m,
                                                            const float* __restrict__ part_z,
                                                            const float* __restrict__ entry_logit,
                                                            const float* __restrict__ q,
                                                            const int32_t* __restrict__ cls,
                                                            const float* __restrict__ qlogq, float* __restrict__ loss,
                                                            float* __restrict__ lse, float* __restrict__ mean, int N,
                                                            int K, int parts, float T) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[32][33], sz[32][33], s_loss[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * 32;
  {
    const int row = r0 + lane;
    float m = -INFINITY, z = 0.0f;
    if (row < N)
      for (int i = warp; i < parts; i += 128) {
        float pm[4], pz[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = i + 32 * k < parts;
          pm[k] = in ? part_m[(int64_t)(i + 32 * k) * N + row] : -INFINITY;
          pz[k] = in ? part_z[(int64_t)(i + 32 * k) * N + row] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) fold2(m, z, pm[k], pz[k]);
      }
    sm[lane][warp] = m;
    sz[lane][warp] = z;
  }
  __syncthreads();
  // warp w: row r0 + w; the fold of its 32 pairs is a fixed tree
  const int row = r0 + warp;
  float value = 0.0f;
  if (row < N) {
    float m = sm[warp][lane], z = sz[warp][lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off), z2 = __shfl_xor_sync(0xffffffffu, z, off);
      fold2(m, z, m2, z2);
    }
    const float l = m * 0.6931471805599453f + logf(z);
    const float inv_t = 1.0f / T;
    const int64_t base = (int64_t)row * K;
    float a = 0.0f;
    bool some = false;
    for (int j = lane; j < K; j += 32)
      if (cls[base + j] >= 0) {
        a = fmaf(q[base + j], l - entry_logit[base + j] * inv_t, a);
        some = true;
      }
    a = warp_sum(a);
    some = __any_sync(0xffffffffu, some);
    value = some ? T * T * (qlogq[row] + a) : 0.0f;
    if (lane == 0) {
      lse[row] = l;
      loss[row] = value;
    }
  }
  if (!mean) return;
  // the only block also takes the mean, as distill_mean_kernel would
  if (lane == 0) s_loss[warp] = value;
  __syncthreads();
  if (warp == 0) {
    value = warp_sum(s_loss[lane]);
    if (lane == 0) *mean = value / (float)N;
  }
}

// sum_n loss[n] / N in a fixed order: strided sums of the threads, then a tree over the block.
__global__ void __launch_bounds__(1024) distill_mean_kernel(const float* __restrict__ loss, float* out, int N) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32];
  float a = 0.0f;
  for (int i = threadIdx.x; i < N; i += 1024) a += loss[i];
  a = warp_sum(a);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    a = warp_sum(s[threadIdx.x]);
    if (threadIdx.x == 0) *out = N > 0 ? a / (float)N : 0.0f;
  }
}

// dX = the sum of its shares, in order (2 shares of 2048 x 1024: 6 us).
__global__ void __launch_bounds__(256) distill_join_kernel(const float* __restrict__ acc, uint16_t* __restrict__ dX,
                                                          int64_t n, int shares) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
    float a[8];
    unpack<float, 8>(load_pack<float, 8>(acc + i), a);
    for (int s = 1; s < shares; ++s) {
      float b[8];
      unpack<float, 8>(load_pack<float, 8>(acc + (int64_t)s * n + i), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
    }
    store_pack<bf16, 8>(reinterpret_cast<bf16*>(dX) + i, pack<bf16, 8>(a));
  }
}

struct DistillLayout {
  int groups, tiles;     // groups of 32 rows; class tiles of 256
  int Vs, S;             // classes a strip (a multiple of 256), strips
  int splits;            // shares of a strip's classes in the dX GEMM
  size_t q, cls, qlogq, coef, out_scale, bucket, entry;
  size_t part_m, part_z, entry_logit, fwd_total;
  size_t d, acc, bwd_total;
};

DistillLayout distill_layout(const moe_distill_config& c) {
  DistillLayout L = {};
  const int64_t N = c.N, V = c.V, K = c.K;
  L.groups = (int)((N + kGroup - 1) / kGroup);
  L.tiles = (int)((V + 255) / 256);
  const int64_t whole = (int64_t)L.tiles * 256, strip = ((V + c.P - 1) / c.P + 255) / 256 * 256;
  L.Vs = (int)(N * whole * 2 <= kOneStrip ? whole : strip);
  L.S = (int)((V + L.Vs - 1) / L.Vs);
  // dX has N x H tiles of 256 x 256 and a long K: where its tiles fill less than half of the 76 clusters, each strip's
  // K is split among them, at least 8 blocks of 64 classes to a share.  (2048 x 1024 from 8192 classes a strip, 32
  // tiles: 58 us a strip unsplit.)
  const int64_t tiles_n = (c.H + 255) / 256, dx_tiles = ((N + 255) / 256) * tiles_n;
  L.splits = (int)std::max<int64_t>(1, std::min<int64_t>(L.Vs / 512, dx_tiles > 0 ? kClusters / dx_tiles : 1));
  size_t o = align256(sizeof(WsHeader));
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  L.q = take((size_t)N * K * 4);
  L.cls = take((size_t)N * K * 4);
  L.qlogq = take((size_t)N * 4);
  L.coef = take((size_t)N * 4);
  L.out_scale = take(4);
  L.bucket = take((size_t)L.groups * (L.tiles + 1) * 4);
  L.entry = take((size_t)L.groups * kGroup * K * 4);
  const size_t common = o;
  L.part_m = take((size_t)N * 2 * L.tiles * 4);
  L.part_z = take((size_t)N * 2 * L.tiles * 4);
  L.entry_logit = take((size_t)N * K * 4);
  L.fwd_total = o;
  o = common;
  // (a workspace serves fewer tokens too, whose one strip may be larger)
  L.d = take((size_t)std::max(N * L.Vs * 2, std::min(N, kOneStrip / (whole * 2)) * whole * 2));
  // rows of fp32: N, or shares x N of any smaller N (a workspace serves fewer tokens too)
  const int64_t most = std::min<int64_t>(whole / 512, kClusters / tiles_n);   // shares of a single row tile
  const int64_t rows = std::max<int64_t>(L.S > 1 ? N : 0, most > 1 ? std::min<int64_t>(N * most, 256 * kClusters / tiles_n) : 0);
  L.acc = take((size_t)rows * c.H * 4);
  L.bwd_total = o;
  return L;
}

int distill_validate(const moe_distill_config* c) {
  if (!c || c->N < 0 || c->H < 0 || c->V < 0 || c->K < 0 || c->P < 0 || !(c->temperature > 0.0f) ||
      !std::isfinite(c->temperature) || !std::isfinite(1.0f / c->temperature))
    return MOE_ERR_INVALID_ARG;
  if (c->H < 64 || c->H % 64 != 0 || c->V < 1 || c->V > (1 << 20) || c->P < 1 || c->P > c->V || c->K < 1 ||
      c->K > kMaxK)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)c->N * c->K > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

bool ok16(const void* p) { return p != nullptr && aligned_to(p, 16); }
bool ok4(const void* p) { return p != nullptr && aligned_to(p, 4); }

int prepare(const moe_distill_config& c, const DistillLayout& L, const int32_t* ids, const float* teacher,
            const float* dloss, uint8_t* w, cudaStream_t s) {
  return timed_launch(MOE_K_DISTILL_PREP, "distill entries", s, [&] {
    const size_t smem = (size_t)(L.tiles + 1 + kGroup * 2 * c.K) * 4;   // at most 16 + 64 KB
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(distill_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(distill_prep_kernel, dim3(L.groups), dim3(1024), smem, s, ids, teacher, dloss,
                      reinterpret_cast<float*>(w + L.q), reinterpret_cast<int32_t*>(w + L.cls),
                      reinterpret_cast<float*>(w + L.qlogq),
                      dloss ? reinterpret_cast<float*>(w + L.coef) : static_cast<float*>(nullptr),
                      reinterpret_cast<float*>(w + L.out_scale),
                      reinterpret_cast<int*>(w + L.bucket), reinterpret_cast<uint32_t*>(w + L.entry), c.N, c.V, c.K,
                      L.tiles, c.temperature, reinterpret_cast<int*>(w));
  });
}

HeadGemm head_params(const moe_distill_config& c, const DistillLayout& L, uint8_t* w) {
  HeadGemm p = {};
  p.band = kHeadBand;
  p.status = reinterpret_cast<int*>(w);
  p.limit_ns = wait_limit_ns();
  p.to_log2 = (float)(1.4426950408889634 / (double)c.temperature);
  p.tiles_all = L.tiles;
  p.K = c.K;
  p.bucket = reinterpret_cast<const int*>(w + L.bucket);
  p.entry = reinterpret_cast<const uint32_t*>(w + L.entry);
  p.q = reinterpret_cast<const float*>(w + L.q);
  p.out_scale = reinterpret_cast<const float*>(w + L.out_scale);
  return p;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_distill_workspace_bytes(const moe_distill_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes) {
  const int v = distill_validate(cfg);
  if (v != MOE_OK) return v;
  const DistillLayout L = distill_layout(*cfg);
  if (fwd_bytes) *fwd_bytes = L.fwd_total;
  if (bwd_bytes) *bwd_bytes = L.bwd_total;
  return MOE_OK;
}

int moe_distill_forward(const moe_distill_config* cfg, const uint16_t* X, const uint16_t* W, const int32_t* ids,
                        const float* teacher, float* loss, float* lse, float* loss_mean, void* ws, size_t ws_bytes,
                        void* stream) {
  int v = distill_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_distill_config& c = *cfg;
  const DistillLayout L = distill_layout(c);
  if (!ok16(ws) || !ok16(W) || !aligned_to(loss_mean, 4)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.fwd_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (c.N > 0 && (!ok16(X) || !ok4(ids) || !ok4(teacher) || !ok4(loss) || !ok4(lse))) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (c.N > 0) {
    CUtensorMap a, b;
    if (!make_map_2d(&a, X, c.H, c.N, 64, 128) || !make_map_2d(&b, W, c.H, c.V, 64, 128))
      return record_cuda_error(cudaErrorInvalidValue, "distill tensor maps");
    if ((v = prepare(c, L, ids, teacher, nullptr, w, s)) != MOE_OK) return v;
    HeadGemm p = head_params(c, L, w);
    p.M = c.N;
    p.N = c.V;
    p.nk = c.H / GEMM_BK;
    p.share = kLseShare;
    p.part_m = reinterpret_cast<float*>(w + L.part_m);
    p.part_z = reinterpret_cast<float*>(w + L.part_z);
    p.entry_logit = reinterpret_cast<float*>(w + L.entry_logit);
    if ((v = timed_launch(MOE_K_DISTILL_LOGITS, "distill logits", s, [&] {
           return launch_head_gemm<HEAD_LSE, false, false>(a, b, p, device_sm_count(), s);
         })) != MOE_OK)
      return v;
    if ((v = timed_launch(MOE_K_DISTILL_LOSS, "distill loss", s, [&] {
           return launch_pdl(distill_loss_kernel, dim3(L.groups), dim3(1024), 0, s, static_cast<const float*>(p.part_m),
                             static_cast<const float*>(p.part_z), static_cast<const float*>(p.entry_logit), p.q,
                             reinterpret_cast<const int32_t*>(w + L.cls),
                             reinterpret_cast<const float*>(w + L.qlogq), loss, lse,
                             L.groups == 1 ? loss_mean : static_cast<float*>(nullptr), c.N, c.K, 2 * L.tiles,
                             c.temperature);
         })) != MOE_OK)
      return v;
  }
  if (!loss_mean || L.groups == 1) return MOE_OK;
  return timed_launch(MOE_K_DISTILL_LOSS, "distill mean", s, [&] {
    return launch_pdl(distill_mean_kernel, dim3(1), dim3(1024), 0, s, static_cast<const float*>(loss), loss_mean, c.N);
  });
}

int moe_distill_backward(const moe_distill_config* cfg, const uint16_t* X, const uint16_t* W, const int32_t* ids,
                         const float* teacher, const float* lse, const float* dloss, uint16_t* dX, void* dW,
                         int32_t dw_type, void* ws, size_t ws_bytes, void* stream) {
  int v = distill_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_distill_config& c = *cfg;
  const DistillLayout L = distill_layout(c);
  if (!ok16(ws) || !ok16(W) || !ok16(dW) || (dw_type != MOE_TYPE_BF16 && dw_type != MOE_TYPE_F32))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.bwd_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N == 0) {
    const cudaError_t e = cudaMemsetAsync(dW, 0, (size_t)c.V * c.H * type_size(dw_type), s);
    return e == cudaSuccess ? MOE_OK : record_cuda_error(e, "clear dW");
  }
  if (!ok16(X) || !ok4(ids) || !ok4(teacher) || !ok4(lse) || !ok4(dloss) || !ok16(dX)) return MOE_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int sms = device_sm_count();
  uint16_t* d = reinterpret_cast<uint16_t*>(w + L.d);
  float* acc = reinterpret_cast<float*>(w + L.acc);
  CUtensorMap xk, xm;   // X with K along the row (logits) and across the rows (dW)
  if (!make_map_2d(&xk, X, c.H, c.N, 64, 128) || !make_map_2d(&xm, X, c.H, c.N, 64, 64))
    return record_cuda_error(cudaErrorInvalidValue, "distill tensor maps");
  if ((v = prepare(c, L, ids, teacher, dloss, w, s)) != MOE_OK) return v;
  for (int st = 0; st < L.S; ++st) {
    const int v0 = st * L.Vs, width = std::min(L.Vs, c.V - v0);
    const uint16_t* Ws = W + (size_t)v0 * c.H;
    CUtensorMap wk, wm, dk, dm;
    if (!make_map_2d(&wk, Ws, c.H, width, 64, 128) || !make_map_2d(&wm, Ws, c.H, width, 64, 64) ||
        !make_map_2d_strided(&dk, d, width, c.N, L.Vs, 64, 128) || !make_map_2d_strided(&dm, d, width, c.N, L.Vs, 64, 64))
      return record_cuda_error(cudaErrorInvalidValue, "distill tensor maps");
    HeadGemm p = head_params(c, L, w);   // d of the strip
    p.M = c.N;
    p.N = width;
    p.nk = c.H / GEMM_BK;
    p.tile0 = v0 / 256;
    p.lse = lse;
    p.coef = reinterpret_cast<const float*>(w + L.coef);
    p.d = d;
    p.ldd = L.Vs;
    if ((v = timed_launch(MOE_K_DISTILL_D, "distill d", s, [&] {
           return launch_head_gemm<HEAD_D, false, false>(xk, wk, p, sms, s);
         })) != MOE_OK)
      return v;
    HeadGemm x = head_params(c, L, w);   // dX (+)= d W_strip, in bf16 after the last strip
    x.M = c.N;
    x.N = c.H;
    x.nk = (width + GEMM_BK - 1) / GEMM_BK;
    x.splits = L.splits;
    x.add = st > 0 ? acc : nullptr;
    if (st + 1 < L.S || L.splits > 1) x.out32 = acc;
    else x.out16 = dX;
    x.ldo = c.H;
    if ((v = timed_launch(MOE_K_DISTILL_DX, "distill dX", s, [&] {
           return launch_head_gemm<HEAD_OUT, false, true>(dk, wm, x, sms, s);
         })) != MOE_OK)
      return v;
    HeadGemm g = head_params(c, L, w);   // dW_strip = d^T X
    g.M = width;
    g.N = c.H;
    g.nk = (int)(((int64_t)c.N + GEMM_BK - 1) / GEMM_BK);
    if (dw_type == MOE_TYPE_BF16) g.out16 = static_cast<uint16_t*>(dW) + (size_t)v0 * c.H;
    else g.out32 = static_cast<float*>(dW) + (size_t)v0 * c.H;
    g.ldo = c.H;
    if ((v = timed_launch(MOE_K_DISTILL_DW, "distill dW", s, [&] {
           return launch_head_gemm<HEAD_OUT, true, true>(dm, xm, g, sms, s);
         })) != MOE_OK)
      return v;
  }
  if (L.splits == 1) return MOE_OK;
  return timed_launch(MOE_K_DISTILL_DX, "distill dX shares", s, [&] {
    const int64_t n = (int64_t)c.N * c.H;
    return launch_pdl(distill_join_kernel, dim3((unsigned)std::min<int64_t>((n / 8 + 255) / 256, sms * 8)), dim3(256), 0, s,
                      static_cast<const float*>(acc), dX, n, L.splits);
  });
}

}  // extern "C"

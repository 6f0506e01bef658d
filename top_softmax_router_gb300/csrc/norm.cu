// Layer normalisation, forward and backward (include/moe_norm.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe.h"
#include "../../include/moe_norm.h"
#include "ops_common.cuh"

namespace moe {
namespace {

// A row is held in registers by TPR threads (a multiple of 32), PER packs of VEC elements each: pack i of
// thread t holds columns VEC (t + i TPR) ..  A block of THREADS holds THREADS / TPR rows at a time: four rows of a
// warp each, or one.
//
// Sums of two values over the tpr threads of a row: a shuffle tree in each warp, then one over the warps' sums.
// `red`: the caller uses two of them in turn.
__device__ __forceinline__ float2 row_sum2(float a, float b, int tpr, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (tpr == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < tpr >> 5 ? red[lane] : make_float2(0.0f, 0.0f);   // one row a block
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// Bound by memory: 32768 x 7168 bf16 with fp32 parameters 160 us, 5.9 TB/s of its 0.94 GB, with bf16 ones 149; 4099 x
// 1001 fp32, where a row starts on no 16 bytes, 10 us.  With 16-bit parameters eight packs of eight spill 96 to 116
// bytes.
// One pass: x is read once, kept in registers for the mean, the variance around it and the output.  TPR threads a row
// at compile time, so that the packs' addresses are constants from the thread's first; places past the row hold zeros
// and are masked by data, not by branches (with both at run time the arithmetic of 32768 x 7168 held it at 195 us).
template <class T, class P, int VEC, int PER, int TPR, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    norm_fwd_kernel(const T* __restrict__ x, int64_t ldx, const P* __restrict__ weight, const P* __restrict__ bias,
                    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int N, int H, float eps) {
  pdl_wait();
  pdl_trigger();
  constexpr int PAIRS = pairs_of<VEC>;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
  if (row >= N) return;   // only where a row is a warp's own
  const int left = H / VEC - t;   // pack i of the thread is in the row where i TPR < left
  const T* xr = x + row * ldx + t * VEC;
  Pack<T, VEC> raw[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    raw[i] = zero_pack<T, VEC>();
    if (i * TPR < left) raw[i] = load_pack<T, VEC>(xr + i * TPR * VEC);
  }
  f32x2 s2(0.0f);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    f32x2 f[PAIRS];
    unpack2<T, VEC>(raw[i], f);
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) s2 = add2(s2, f[j]);
  }
  const float inv_h = 1.0f / (float)H;
  const float mu = row_sum2(s2.sum(), 0.0f, TPR, red[0]).x * inv_h;
  f32x2 q2(0.0f);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const f32x2 minus_mu(i * TPR < left ? -mu : 0.0f, VEC > 1 && i * TPR < left ? -mu : 0.0f);
    f32x2 f[PAIRS];
    unpack2<T, VEC>(raw[i], f);
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const f32x2 d = add2(f[j], minus_mu);
      q2 = fma2(d, d, q2);
    }
  }
  const float rs = 1.0f / sqrtf(row_sum2(q2.sum(), 0.0f, TPR, red[1]).x * inv_h + eps);
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
  const f32x2 rs2(rs), minus_mu(-mu);
  T* yr = y + row * H + t * VEC;
  const P* wt = weight + t * VEC;
  const P* bt = bias + t * VEC;
  const bool has_w = weight != nullptr, has_b = bias != nullptr;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool in = i * TPR < left;
    f32x2 f[PAIRS], w[PAIRS], b[PAIRS];
    Pack<P, VEC> pw = one_pack<P, VEC>(), pb = zero_pack<P, VEC>();
    if (in && has_w) pw = load_pack<P, VEC>(wt + i * TPR * VEC);
    if (in && has_b) pb = load_pack<P, VEC>(bt + i * TPR * VEC);
    unpack2<T, VEC>(raw[i], f);
    unpack2<P, VEC>(pw, w);
    unpack2<P, VEC>(pb, b);
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) f[j] = fma2(mul2(add2(f[j], minus_mu), rs2), w[j], b[j]);
    if (in) store_pack<T, VEC>(yr + i * TPR * VEC, pack2<T, VEC>(f));
  }
}

// Persistent: block b takes row groups b, b + grid, ..  x and dy are read once; dx is written, and each
// thread keeps the sums of dy xh and dy of its columns in registers over all its rows.  The block's sums
// go to part[block][2][H]; norm_param_kernel adds the blocks in order, so the result has a fixed order.
// Places past the row (and rows past the last) hold dy = 0, which adds nothing.  4099 x 1001 fp32: 15 us, 3.3 TB/s.
template <class T, class P, int VEC, int PER, int TPR, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    norm_bwd_kernel(const T* __restrict__ x, int64_t ldx, const P* __restrict__ weight, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const T* __restrict__ dy, int64_t lddy, T* __restrict__ dx,
                    float* __restrict__ part, int N, int H) {
  pdl_wait();
  pdl_trigger();
  constexpr int PAIRS = pairs_of<VEC>, ROWS = THREADS / TPR;
  __shared__ float2 red[2][32];
  __shared__ float cols[ROWS > 1 ? 2 * 32 * PER * VEC : 1];   // the block's sums, when it holds several rows at a time
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int left = H / VEC - t;   // pack i of the thread is in the row where i TPR < left
  const float inv_h = 1.0f / (float)H;
  f32x2 gw[PER][PAIRS], gb[PER][PAIRS];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) gw[i][j] = gb[i][j] = f32x2(0.0f);
  int it = 0;
  Pack<T, VEC> nx[PER], nd[PER];   // the next row, loaded while this one is worked on
  float mu_next = 0.0f, rs_next = 0.0f;
  auto load = [&](int64_t row) {
    const bool ok = row < N;
    const T* xr = x + row * ldx + t * VEC;
    const T* dr = dy + row * lddy + t * VEC;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      nx[i] = nd[i] = zero_pack<T, VEC>();
      if (ok && i * TPR < left) {
        nx[i] = load_pack<T, VEC>(xr + i * TPR * VEC);
        nd[i] = load_pack<T, VEC>(dr + i * TPR * VEC);
      }
    }
    mu_next = ok ? mean[row] : 0.0f;
    rs_next = ok ? rstd[row] : 0.0f;
  };
  const P* wt = weight + t * VEC;
  const bool has_w = weight != nullptr;
  load((int64_t)blockIdx.x * ROWS + sub);
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < N; base += (int64_t)gridDim.x * ROWS, ++it) {
    const int64_t row = base + sub;
    Pack<T, VEC> rx[PER], rd[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) rx[i] = nx[i], rd[i] = nd[i];
    const f32x2 minus_mu(-mu_next), rs2(rs_next);
    const float rs = rs_next;
    load(row + (int64_t)gridDim.x * ROWS);
    f32x2 s2(0.0f), sx2(0.0f);
    auto weight_of = [&](int i, f32x2 (&w)[PAIRS]) {
      Pack<P, VEC> pw = one_pack<P, VEC>();
      if (has_w && i * TPR < left) pw = load_pack<P, VEC>(wt + i * TPR * VEC);
      unpack2<P, VEC>(pw, w);
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      f32x2 xh[PAIRS], d[PAIRS], w[PAIRS];
      unpack2<T, VEC>(rx[i], xh);
      unpack2<T, VEC>(rd[i], d);
      weight_of(i, w);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        xh[j] = mul2(add2(xh[j], minus_mu), rs2);
        gw[i][j] = fma2(d[j], xh[j], gw[i][j]);
        gb[i][j] = add2(gb[i][j], d[j]);
        const f32x2 tw = mul2(d[j], w[j]);
        s2 = add2(s2, tw);
        sx2 = fma2(tw, xh[j], sx2);
      }
    }
    if (dx) {
      const float2 sums = row_sum2(s2.sum(), sx2.sum(), TPR, red[it & 1]);
      const f32x2 by_x(-rs * rs * (sums.y * inv_h)), by_1(-rs * (sums.x * inv_h));
      T* out = dx + row * H + t * VEC;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        f32x2 xv[PAIRS], d[PAIRS], w[PAIRS];
        unpack2<T, VEC>(rx[i], xv);
        unpack2<T, VEC>(rd[i], d);
        weight_of(i, w);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
          xv[j] = fma2(mul2(d[j], w[j]), rs2, fma2(add2(xv[j], minus_mu), by_x, by_1));
        if (row < N && i * TPR < left) store_pack<T, VEC>(out + i * TPR * VEC, pack2<T, VEC>(xv));
      }
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * 2 * H;
  // the rows of the block are added in turn: row group 0 first
  for (int r = 0; r < ROWS; ++r) {
    if (sub == r) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (i * TPR < left) {
          Pack<float, VEC> a = pack2<float, VEC>(gw[i]), b = pack2<float, VEC>(gb[i]);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int h = (t + i * TPR) * VEC + j;
            if (r > 0) a.v[j] += cols[h], b.v[j] += cols[H + h];
            if (r + 1 < ROWS) cols[h] = a.v[j], cols[H + h] = b.v[j];
            else out[h] = a.v[j], out[H + h] = b.v[j];
          }
        }
      }
    }
    if (r + 1 < ROWS) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Wide rows: a ring of rows in shared memory
// ---------------------------------------------------------------------------
// The last warp of a block streams the block's rows of x and dy into `stages` places of shared memory with bulk
// copies; the other threads (`workers`) hold up to four packs of columns each and meet once a row for its
// sums.  The copies run ahead of the reductions, so the memory stays busy, and the blocks that share an SM work while
// the others meet.  The weight lies in shared memory in fp32.  A thread whose last packs are past the row reads
// the row's last pack in their place and adds nothing, so that the arithmetic has no branches.  Bound by memory: 32768 x
// 7168 bf16 233 us, 6.0 TB/s of 1.41 GB; the register form, whose loads wait for each row's sums, took 462.
constexpr int kRingMost = 8;
constexpr int kRingSm = 228 * 1024;            // shared memory of an SM, of which a block costs 1 KB and its own variables
constexpr int kRingFixed = 2 * kRingMost * 8;  // full[kRingMost], empty[kRingMost]

// One contiguous copy of global memory into shared memory, completing on `bar` (16-byte multiples).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

struct Ring {
  uint32_t base, bars;
  int stages, stage_bytes;
  volatile int* abort_flag;
  int64_t limit_ns;
  int* status;
  __device__ __forceinline__ uint32_t full(int s) const { return bars + 8 * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8 * (kRingMost + s); }
  // Rows blockIdx.x, + gridDim.x, ..: one thread.
  __device__ __forceinline__ void stream(const void* a, int64_t lda, const void* b, int64_t ldb, int row_bytes, int N) const {
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
      if (!wait_bounded(empty(stage), phase ^ 1u, abort_flag, limit_ns, status, 801)) break;
      const uint32_t dst = base + stage * stage_bytes;
      mbar_expect_tx(full(stage), stage_bytes);
      bulk_load(dst, static_cast<const uint8_t*>(a) + row * lda, row_bytes, full(stage));
      if (b) bulk_load(dst + row_bytes, static_cast<const uint8_t*>(b) + row * ldb, row_bytes, full(stage));
      ++issued;
      if (++stage == stages) stage = 0, phase ^= 1u;
    }
    // every copy has landed before the block leaves, also after a wait that ran out
    for (int q = 1; q <= min(issued, stages); ++q) {
      int s = stage - q;
      uint32_t ph = phase;
      if (s < 0) s += stages, ph ^= 1u;
      volatile int no_abort = 0;
      wait_bounded(full(s), ph, &no_abort, max(limit_ns, kSettleNs), nullptr, 0);
    }
  }
};

// Sums of two values over the worker threads, in warp order (`red`: used alternately by the caller).
__device__ __forceinline__ float2 workers_sum2(float a, float b, int workers, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  asm volatile("bar.sync 1, %0;" ::"r"(workers) : "memory");
  a = b = 0.0f;
  for (int k = 0; k < workers / 32; ++k) a += red[k].x, b += red[k].y;
  return make_float2(a, b);
}

// Where column h of the weight lies in shared memory: the first four columns of 32 consecutive packs, then their other
// four, so that a warp reads 512 consecutive bytes at a time.
template <int VEC>
__device__ __forceinline__ int weight_at(int h) {
  if constexpr (VEC == 4) return h;
  const int c = h / VEC, half = (h >> 2) & 1;
  return ((c >> 5) * 64 + half * 32 + (c & 31)) * 4 + (h & 3);
}
__host__ __device__ constexpr int weight_floats(int H) { return (H + 255) / 256 * 256; }

// The weight in fp32 (ones where there is none): the whole block.
template <int VEC>
__device__ __forceinline__ void weight_to_smem(float* dst, const void* src, int type, int H) {
  for (int h = threadIdx.x; h < H; h += blockDim.x) {
    float v = 1.0f;
    if (src) {
      if (type == MOE_TYPE_F32) v = static_cast<const float*>(src)[h];
      else if (type == MOE_TYPE_BF16) v = to_f32<bf16>(static_cast<const bf16*>(src)[h]);
      else v = to_f32<f16>(static_cast<const f16*>(src)[h]);
    }
    dst[weight_at<VEC>(h)] = v;
  }
}
template <int VEC>
__device__ __forceinline__ void load_weight(const float* v, int pack, f32x2 (&f)[VEC / 2]) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    const float4 w = *reinterpret_cast<const float4*>(v + weight_at<VEC>(pack * VEC + 4 * i));
    f[2 * i] = f32x2(w.x, w.y);
    f[2 * i + 1] = f32x2(w.z, w.w);
  }
}

template <class T, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    norm_bwd_ring_kernel(const T* __restrict__ x, int64_t ldx, const void* __restrict__ weight, int param_type,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const T* __restrict__ dy,
                         int64_t lddy, T* __restrict__ dx, float* __restrict__ part, int N, int H, int stages,
                         int* status, int64_t limit_ns) {
  constexpr int VEC = 16 / sizeof(T), PER = 4, PAIRS = VEC / 2;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float2 red[2][16];
  __shared__ int abort_word;
  const int row_bytes = H * (int)sizeof(T);
  float* w_s = reinterpret_cast<float*>(ring_mem);
  uint8_t* places = reinterpret_cast<uint8_t*>(w_s + weight_floats(H));
  const Ring ring = {smem_u32(places), smem_u32(places) + stages * 2 * row_bytes, stages, 2 * row_bytes, &abort_word, limit_ns, status};
  const int workers = blockDim.x - 32, warps = workers >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(ring.full(i), 1);
      mbar_init(ring.empty(i), warps);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  weight_to_smem<VEC>(w_s, weight, param_type, H);
  __syncthreads();
  const int lane = threadIdx.x & 31, t = threadIdx.x;
  if (t >= workers) {
    if (lane == 0) ring.stream(x, ldx * (int64_t)sizeof(T), dy, lddy * (int64_t)sizeof(T), row_bytes, N);
    return;
  }
  const int packs = H / VEC;
  const float inv_h = 1.0f / (float)H;
  f32x2 gw[PER][PAIRS], gb[PER][PAIRS];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) gw[i][j] = gb[i][j] = f32x2(0.0f);
  int stage = 0, it = 0;
  uint32_t phase = 0;
  bool good = true;   // lane 0: no wait has run out
  float mu = 0.0f, rs = 0.0f;
  if ((int)blockIdx.x < N) mu = mean[blockIdx.x], rs = rstd[blockIdx.x];
  for (int64_t row = blockIdx.x; row < N; row += gridDim.x, ++it) {
    const int64_t next = row + gridDim.x;
    float mu_next = 0.0f, rs_next = 0.0f;
    if (next < N) mu_next = mean[next], rs_next = rstd[next];
    // After a wait that ran out the sums are of no use (the status says so), and no place is given back: its copies may
    // still be on their way.  Every warp still meets the others below.
    if (lane == 0) good &= wait_bounded(ring.full(stage), phase, ring.abort_flag, limit_ns, status, 803);
    __syncwarp();
    const T* at = reinterpret_cast<const T*>(places + (size_t)stage * 2 * row_bytes);
    f32x2 s2(0.0f), sx2(0.0f);
    const f32x2 minus_mu(-mu), rs2(rs);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * workers, k = min(c, packs - 1);
      Pack<T, VEC> rd = load_pack<T, VEC>(at + H + k * VEC);
      if (c >= packs) rd = zero_pack<T, VEC>();   // dy = 0 adds nothing
      f32x2 xh[PAIRS], d[PAIRS], w[PAIRS];
      unpack2<T, VEC>(load_pack<T, VEC>(at + k * VEC), xh);
      unpack2<T, VEC>(rd, d);
      load_weight<VEC>(w_s, k, w);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        xh[j] = mul2(add2(xh[j], minus_mu), rs2);
        gw[i][j] = fma2(d[j], xh[j], gw[i][j]);
        gb[i][j] = add2(gb[i][j], d[j]);
        const f32x2 tw = mul2(d[j], w[j]);
        s2 = add2(s2, tw);
        sx2 = fma2(tw, xh[j], sx2);
      }
    }
    if (dx) {
      const float2 sums = workers_sum2(s2.sum(), sx2.sum(), workers, red[it & 1]);
      // dx = rs t - rs a - (x - mu) rs^2 b, with a = s / H and b = sx / H; the packs are read from the ring again (kept
      // in registers beside the sums they spilled)
      const f32x2 by_x(-rs * rs * (sums.y * inv_h)), by_1(-rs * (sums.x * inv_h));
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = t + i * workers, k = min(c, packs - 1);
        f32x2 xv[PAIRS], d[PAIRS], w[PAIRS];
        unpack2<T, VEC>(load_pack<T, VEC>(at + k * VEC), xv);
        unpack2<T, VEC>(load_pack<T, VEC>(at + H + k * VEC), d);
        load_weight<VEC>(w_s, k, w);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
          xv[j] = fma2(mul2(d[j], w[j]), rs2, fma2(add2(xv[j], minus_mu), by_x, by_1));
        if (c < packs) store_pack<T, VEC>(dx + row * H + (int64_t)c * VEC, pack2<T, VEC>(xv));
      }
    }
    __syncwarp();
    if (lane == 0 && good) mbar_arrive(ring.empty(stage));
    if (++stage == stages) stage = 0, phase ^= 1u;
    mu = mu_next;
    rs = rs_next;
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = t + i * workers;
    if (c < packs) {
      store_pack<float, VEC>(out + c * VEC, pack2<float, VEC>(gw[i]));
      store_pack<float, VEC>(out + H + c * VEC, pack2<float, VEC>(gb[i]));
    }
  }
}

// dweight[h], dbias[h]: the blocks' partial sums added in a fixed order.  A block owns 32 columns; its 32
// warps take the partials round robin, and their sums are added in a fixed tree.  304 blocks of 7168 columns: 9 us.
__global__ void __launch_bounds__(1024) norm_param_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                         float* __restrict__ dbias, int blocks, int H) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const bool second = blockIdx.y == 1;
  float* out = second ? dbias : dweight;
  if (!out) return;
  float a = 0.0f;
  if (c < H) {
    const float* p = part + (second ? H : 0) + c;
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) a += p[(int64_t)b * 2 * H];
  }
  s[lane][warp] = a;
  __syncthreads();
  // warp w adds the 32 partial sums of column w in a fixed tree
  a = warp_sum(s[warp][lane]);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < H) out[col] = a;
}

int norm_validate(const moe_layernorm_config* c) {
  if (!c || c->N < 0 || c->H <= 0 || !(c->eps >= 0.0f) || !std::isfinite(c->eps)) return MOE_ERR_INVALID_ARG;
  if (c->H > MOE_LAYERNORM_MAX_H) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

constexpr int kMaxBwdBlocks = 152 * 4;   // rows of partial sums in the workspace

int bwd_blocks(int N) { return std::min(N, kMaxBwdBlocks); }

template <class T, class P, int VEC, int PER, int TPR, int BLOCKS>
cudaError_t fwd_launch(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight,
                       const void* bias, void* y, float* mean, float* rstd, cudaStream_t s) {
  constexpr int THREADS = TPR == 32 ? 128 : TPR, ROWS = THREADS / TPR;
  return launch_pdl(norm_fwd_kernel<T, P, VEC, PER, TPR, THREADS, BLOCKS>,
                    dim3((unsigned)((c.N + (int64_t)ROWS - 1) / ROWS)), dim3(THREADS), 0, s, static_cast<const T*>(x),
                    ldx, static_cast<const P*>(weight), static_cast<const P*>(bias), static_cast<T*>(y), mean, rstd, c.N,
                    c.H, c.eps);
}

// Up to 256 packs a row stays in one warp, so that no warps have to meet; then in 128, 256 or 1024 threads of up to
// 16 packs each.  1024 threads an SM (64 registers each): fewer keep too little memory in flight (32768 x 7168 with
// 768: 189 us, 1024: 164, 1536: 216 as the packs spill).
template <class T, class P, int VEC>
cudaError_t fwd_shape(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight, const void* bias,
                      void* y, float* mean, float* rstd, cudaStream_t s) {
  const int packs = c.H / VEC;
  if (packs <= 64) return fwd_launch<T, P, VEC, 2, 32, 8>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if (packs <= 128) return fwd_launch<T, P, VEC, 4, 32, 8>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if (packs <= 256) return fwd_launch<T, P, VEC, 8, 32, 8>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if (packs <= 512) return fwd_launch<T, P, VEC, 4, 128, 8>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if (packs <= 1024) return fwd_launch<T, P, VEC, 8, 128, 8>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if (packs <= 2048) return fwd_launch<T, P, VEC, 8, 256, 4>(c, x, ldx, weight, bias, y, mean, rstd, s);
  if constexpr (MOE_LAYERNORM_MAX_H / VEC > 2048) {
    if (packs <= 4096) return fwd_launch<T, P, VEC, 16, 256, 2>(c, x, ldx, weight, bias, y, mean, rstd, s);
  }
  if constexpr (VEC == 1) return fwd_launch<T, P, VEC, 16, 1024, 1>(c, x, ldx, weight, bias, y, mean, rstd, s);
  return cudaErrorInvalidValue;   // no row is wider
}

template <class T, class P, int VEC, int PER, int TPR, int BLOCKS>
cudaError_t bwd_launch(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight,
                       const float* mean, const float* rstd, const void* dy, int64_t lddy, void* dx, float* part,
                       int* blocks, cudaStream_t s) {
  constexpr int THREADS = TPR == 32 ? 128 : TPR, ROWS = THREADS / TPR;
  const int64_t groups = ((int64_t)c.N + ROWS - 1) / ROWS;
  *blocks = (int)std::min<int64_t>(groups, std::min(bwd_blocks(c.N), BLOCKS * device_sm_count()));
  return launch_pdl(norm_bwd_kernel<T, P, VEC, PER, TPR, THREADS, BLOCKS>, dim3(*blocks), dim3(THREADS), 0, s,
                    static_cast<const T*>(x), ldx, static_cast<const P*>(weight), mean, rstd,
                    static_cast<const T*>(dy), lddy, static_cast<T*>(dx), part, c.N, c.H);
}

struct RingShape {
  int threads, per_sm, stages;
  size_t smem;
};
// Blocks an SM: as many as its registers (128 a thread) and its shared memory hold with three rows in each ring, up to
// 4.  fixed: bytes beside the ring; row: bytes of a place.
RingShape ring_shape(int packs, size_t fixed, size_t row) {
  RingShape r;
  r.threads = ((packs + 3) / 4 + 31) / 32 * 32 + 32;
  r.per_sm = std::max(1, std::min(4, 512 / r.threads));
  auto fits = [&](int per_sm) { return (int)((kRingSm / per_sm - 1024 - 512 - (int)fixed - kRingFixed) / (int64_t)row); };
  while (r.per_sm > 1 && fits(r.per_sm) < 3) --r.per_sm;
  r.stages = std::min(kRingMost, fits(r.per_sm));
  r.smem = fixed + r.stages * row + kRingFixed;
  return r;
}

template <class T, int THREADS, int BLOCKS>
cudaError_t bwd_ring_launch(const moe_layernorm_config& c, const RingShape& r, const void* x, int64_t ldx,
                            const void* weight, int param_type, const float* mean, const float* rstd, const void* dy,
                            int64_t lddy, void* dx, float* part, int* blocks, int* status, cudaStream_t s) {
  auto kern = norm_bwd_ring_kernel<T, THREADS, BLOCKS>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)r.smem);
  if (e != cudaSuccess) return e;
  *blocks = std::min(bwd_blocks(c.N), r.per_sm * device_sm_count());
  return launch_pdl(kern, dim3(*blocks), dim3(r.threads), r.smem, s, static_cast<const T*>(x), ldx, weight, param_type,
                    mean, rstd, static_cast<const T*>(dy), lddy, static_cast<T*>(dx), part, c.N, c.H, r.stages, status,
                    wait_limit_ns());
}

// A warp holds rows of up to 128 packs (one pack a thread, or four: the register form of 32768 x 7168 took 462 us, the
// ring 233, but the ring's threads would stand idle below): 262144 x 256 bf16 95 us, 4.2 TB/s; 262144 x 512, four
// packs a thread and two blocks an SM, 414 us, 1.9 TB/s.  Wider rows of 16-byte packs go through the ring of shared
// memory where a block has threads for them and three places (H up to 14336 in 16 bits, 7680 in fp32); the others stay
// in a block's registers.  Those of 1024 threads have 64 each, spill 672 to 1574 bytes and are far from memory's rate:
// 16384 x 8192 fp32 1070 us, where 7680 columns take 254 through the ring; 16384 x 16384 bf16 4276; 32768 x 7169 bf16,
// by single elements, 4726.
template <class T, class P, int VEC>
cudaError_t bwd_shape(const moe_layernorm_config& c, const void* x, int64_t ldx, const void* weight, const float* mean,
                      const float* rstd, const void* dy, int64_t lddy, void* dx, float* part, int* blocks, int* status,
                      cudaStream_t s) {
  const int packs = c.H / VEC;
  if constexpr (VEC > 1) {
#define MOE_BWD(PER, TPR, BLOCKS) \
  return bwd_launch<T, P, VEC, PER, TPR, BLOCKS>(c, x, ldx, weight, mean, rstd, dy, lddy, dx, part, blocks, s)
    if (packs <= 32) MOE_BWD(1, 32, 4);
    if (packs <= 128) MOE_BWD(4, 32, 2);
    const RingShape r = ring_shape(packs, (size_t)weight_floats(c.H) * 4, 2 * c.H * sizeof(T));
    const int pt = std::is_same<P, float>::value ? MOE_TYPE_F32 : std::is_same<T, bf16>::value ? MOE_TYPE_BF16 : MOE_TYPE_F16;
    if (r.threads <= 256 && r.stages >= 3)
      return bwd_ring_launch<T, 256, 2>(c, r, x, ldx, weight, pt, mean, rstd, dy, lddy, dx, part, blocks, status, s);
    if (r.threads <= 512 && r.stages >= 3)
      return bwd_ring_launch<T, 512, 1>(c, r, x, ldx, weight, pt, mean, rstd, dy, lddy, dx, part, blocks, status, s);
    MOE_BWD(4, 1024, 1);
  } else {
    if (packs <= 128) MOE_BWD(4, 32, 4);
    if (packs <= 1024) MOE_BWD(8, 128, 4);
    if (packs <= 4096) MOE_BWD(8, 512, 1);
    MOE_BWD(16, 1024, 1);
  }
#undef MOE_BWD
}

// Calls f(T, P, VEC) with compile-time values.  vec: rows and parameters take 16-byte packs.  BY_PARAM: a pack is 16
// bytes of the wider of T and P: fp32 parameters of a 16-bit row are then read 512 consecutive bytes a warp (as packs
// of eight, two loads with gaps of 16 bytes, they held the forward of 32768 x 7168 at 198 us).
template <bool BY_PARAM, class F>
cudaError_t with_pack(int type, int param_type, bool vec, F&& f) {
  return with_type(type, [&](auto tv) {
    using T = decltype(tv);
    auto by_param = [&](auto pv) {
      constexpr int wide = BY_PARAM && sizeof(pv) > sizeof(T) ? sizeof(pv) : sizeof(T);
      if (vec) return f(tv, pv, std::integral_constant<int, 16 / wide>{});
      return f(tv, pv, std::integral_constant<int, 1>{});
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
  if (bwd_bytes) *bwd_bytes = sizeof(WsHeader) + align256((size_t)bwd_blocks(cfg->N) * 2 * cfg->H * 4);
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
    return with_pack<true>(type, param_type, vec, [&](auto tv, auto pv, auto vv) {
      return fwd_shape<decltype(tv), decltype(pv), decltype(vv)::value>(
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
  if (!ws || !aligned_to(ws, 16)) return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  moe_layernorm_workspace_bytes(cfg, &need);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!dx && !params) return MOE_OK;
  const bool vec = vec_rows(x, ldx, c.H, type) && vec_rows(dy, lddy, c.H, type) && aligned_to(dx, 16) &&
                   aligned_to(weight, 16);
  int* status = static_cast<int*>(ws);
  float* part = params ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader)) : nullptr;
  int blocks = 0;
  v = timed_launch(MOE_K_NORM_BWD, "layer norm backward", s, [&] {
    return with_pack<false>(type, param_type, vec, [&](auto tv, auto pv, auto vv) {
      return bwd_shape<decltype(tv), decltype(pv), decltype(vv)::value>(
          c, x, ldx, weight, mean, rstd, dy, lddy, dx, part, &blocks, status, s);
    });
  });
  if (v != MOE_OK || !params) return v;
  return timed_launch(MOE_K_NORM_BWD, "layer norm parameter gradients", s, [&] {
    return launch_pdl(norm_param_kernel, dim3((c.H + 31) / 32, 2), dim3(1024), 0, s, static_cast<const float*>(part),
                      dweight, dbias, blocks, c.H);
  });
}

}  // extern "C"

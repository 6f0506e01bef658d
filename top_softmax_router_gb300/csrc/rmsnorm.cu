// Root-mean-square norm with the residual's addition and an output in 8 bits (include/moe_rmsnorm.h).
//
// A half warp holds blocks of 128 columns of a row, eight values a lane, so that a block's largest magnitude is four
// shuffles away: PER blocks a half warp, TPR threads a row (whole warps), several rows a block of threads where rows are
// short.  Rows stay in registers between the statistics and the output: x, the residual and the outputs pass memory once.
// A block of the forward takes one row a row group and leaves; the backward is persistent, and loads its next row while it
// works on this one where the registers allow it.
#include <algorithm>

#include "../../include/moe_blocks8.h"
#include "../../include/moe_rmsnorm.h"
#include "blocks8.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Most threads of a block.  Up to 7168 columns the forward has four blocks of 224 threads a SM (72 registers; with 78, and
// three blocks, 32768 x 7168 took 424 us for 365), the backward two blocks of 128 columns a half warp.
constexpr int kFwdThreads = 224, kFwdWide = 512;
constexpr int bwd_threads(int per) { return per <= 2 ? 448 : 512; }
constexpr int kMaxRows = 8;

// A row's warps leave their sums here; places without a warp hold 0.  The backward's rows take two of them in turn, so that
// one barrier a row suffices.
template <int TURNS>
struct RowSums {
  float4 v[TURNS][kMaxRows][4];
};
template <int TURNS>
__device__ __forceinline__ void clear(RowSums<TURNS>& r) {
  float4* p = &r.v[0][0][0];
  for (int i = threadIdx.x; i < TURNS * kMaxRows * 4; i += blockDim.x) p[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
}
// The sum over a row's threads (tpr of them, whole warps of row group `group`), in a fixed order, in every thread.
__device__ __forceinline__ float row_sum(float v, int tpr, int group, int t, float4 (&r)[kMaxRows][4]) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  if ((t & 31) == 0) reinterpret_cast<float*>(r[group])[t >> 5] = v;
  __syncthreads();
  const float4 a = r[group][0], b = r[group][1], c = r[group][2], d = r[group][3];
  return (((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w))) + (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}

// A thread's place in its row: block i of its half warp starts at column(i) and has valid(i) columns.
struct RowPlace {
  int group, rows, t, lane16, hw, hws, H;
  __device__ __forceinline__ RowPlace(int tpr, int H_) : H(H_) {
    rows = blockDim.x / tpr;
    group = threadIdx.x / tpr;
    t = threadIdx.x - group * tpr;
    lane16 = t & 15;
    hw = t >> 4;
    hws = tpr >> 4;
  }
  __device__ __forceinline__ int block(int i) const { return hw + i * hws; }
  __device__ __forceinline__ int column(int i) const { return block(i) * MOE_BLOCK8; }
  __device__ __forceinline__ int step() const { return hws * MOE_BLOCK8; }
  __device__ __forceinline__ int valid(int i) const { return max(0, min(MOE_BLOCK8, H - column(i))); }
  // What a thread asks of block i before it touches it, worked out once: with VEC whether its eight are in the row, else
  // how many of the block's columns are.  Pointers start at first(): the thread's eight, or the block.
  template <bool VEC>
  __device__ __forceinline__ int in(int i) const { return VEC ? lane16 * 8 < valid(i) : valid(i); }
  template <bool VEC>
  __device__ __forceinline__ int first() const { return column(0) + (VEC ? lane16 * 8 : 0); }
};
template <class T, bool VEC>
__device__ __forceinline__ Pack<T, 8> get8(const T* p, int lane16, int in) {
  if constexpr (VEC) {
    Pack<T, 8> a = zero_pack<T, 8>();
    if (in) a = load_pack<T, 8>(p);
    return a;
  } else {
    return load_block8<T, false>(p, lane16, in);
  }
}
template <class T, bool VEC>
__device__ __forceinline__ void put8(T* p, int lane16, int in, const Pack<T, 8>& a) {
  if constexpr (VEC) {
    if (in) store_pack<T, 8>(p, a);
  } else {
    store_block8<T, false>(p, lane16, in, a);
  }
}

template <class T, class P, bool VEC, int PER, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kFwdWide : kFwdThreads, WIDE ? 1 : 4)
    rms_fwd_kernel(const T* __restrict__ x, int64_t ldx, const T* __restrict__ res, int64_t ldr,
                   const P* __restrict__ weight, T* __restrict__ h, T* __restrict__ y, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales, float* __restrict__ rstd, int N, int H, int nb, int tpr, float eps) {
  pdl_wait();
  pdl_trigger();
  __shared__ RowSums<1> sums;
  const RowPlace at(tpr, H);
  const int64_t row = (int64_t)blockIdx.x * at.rows + at.group;
  const bool there = row < N;        // of a row group, so of whole warps
  int in[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) in[i] = at.template in<VEC>(i);
  const int first = at.template first<VEC>(), step = at.step();
  Pack<T, 8> v[PER];
  const T* xr = x + (there ? row * ldx : 0) + first;
  const T* rr = res + (there ? row * ldr : 0) + first;
  f32x2 sq(0.0f);
  {
    Pack<T, 8> r[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = get8<T, VEC>(xr + i * step, at.lane16, there ? in[i] : 0);
      if (res) r[i] = get8<T, VEC>(rr + i * step, at.lane16, there ? in[i] : 0);
    }
    if (tpr > 32) clear(sums);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      f32x2 f[4];
      unpack2<T, 8>(v[i], f);
      if (res) {
        f32x2 g[4];
        unpack2<T, 8>(r[i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = add2(f[j], g[j]);
        v[i] = pack2<T, 8>(f);
        unpack2<T, 8>(v[i], f);      // what is kept
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sq = fma2(f[j], f[j], sq);
    }
  }
  const float rs = 1.0f / sqrtf(row_sum(sq.sum(), tpr, at.group, at.t, sums.v[0]) * (1.0f / (float)H) + eps);
  if (!there) return;
  if (rstd && at.t == 0) rstd[row] = rs;
  const int64_t to = row * H + first;
  const f32x2 rs2(rs);
  f32x2 f[PER][4];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (h) put8<T, VEC>(h + to + i * step, at.lane16, in[i], v[i]);
    unpack2<T, 8>(v[i], f[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i][j] = mul2(f[i][j], rs2);
    if (weight) {
      f32x2 g[4];
      unpack2<P, 8>(get8<P, VEC>(weight + first + i * step, at.lane16, in[i]), g);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[i][j] = mul2(f[i][j], g[j]);
    }
    if (y) put8<T, VEC>(y + to + i * step, at.lane16, in[i], pack2<T, 8>(f[i]));
  }
  if (!codes) return;
  float m[PER];
  const bool infinite = blocks_max<PER>(f, m);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int byte = block_scale_byte(m[i]);
    const uint2 c = block_codes(f[i], byte, infinite, kTopByte<float>);
    if constexpr (VEC) {
      if (in[i]) *reinterpret_cast<uint2*>(codes + to + i * step) = c;
    } else {
      store_codes8<false>(codes + to + i * step, at.lane16, in[i], c);
    }
    if (in[i] && at.lane16 == 0) scales[row * nb + at.block(i)] = (uint8_t)byte;
  }
}

// Each thread keeps the sums of dy xh of its columns in registers over all its rows.  The row groups of a block add
// theirs up in order, into part[block][H]; rms_param_kernel adds the blocks in order.
template <class T, class P, bool VEC, int PER>
__global__ void __launch_bounds__(bwd_threads(PER), 1)
    rms_bwd_kernel(const T* __restrict__ h, int64_t ldh, const P* __restrict__ weight, const float* __restrict__ rstd,
                   const T* __restrict__ dy, int64_t lddy, const T* __restrict__ dh, int64_t lddh, T* __restrict__ dx,
                   float* __restrict__ part, int N, int H, int tpr) {
  pdl_wait();
  pdl_trigger();
  constexpr bool AHEAD = VEC && PER * (int)sizeof(T) <= 4;
  constexpr bool LATE = PER * (int)sizeof(T) > 8;   // dh is loaded when it is needed
  __shared__ RowSums<2> sums;
  extern __shared__ float cols[];    // [H] where a block holds several rows
  if (tpr > 32) clear(sums);
  const RowPlace at(tpr, H);
  const float inv_h = 1.0f / (float)H;
  f32x2 gw[PER][4];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) gw[i][j] = f32x2(0.0f);
  int in[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) in[i] = at.template in<VEC>(i);
  const int first = at.template first<VEC>(), step = at.step();
  const int64_t row0 = (int64_t)blockIdx.x * at.rows + at.group, jump = (int64_t)gridDim.x * at.rows;
  const T* hp = h + row0 * ldh + first;       // of the row that is loaded next
  const T* gp = dy + row0 * lddy + first;
  const T* dp = dh + row0 * lddh + first;     // only read where there is a dh
  const bool with_dh = dx && dh;
  Pack<T, 8> nh[PER], ng[PER], nd[PER];
  float rs_next = 0.0f;
  auto load = [&](int64_t row) {
    const bool there = row < N;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      nh[i] = get8<T, VEC>(hp + i * step, at.lane16, there ? in[i] : 0);
      ng[i] = get8<T, VEC>(gp + i * step, at.lane16, there ? in[i] : 0);
      if (!LATE) nd[i] = get8<T, VEC>(dp + i * step, at.lane16, there && with_dh ? in[i] : 0);
    }
    rs_next = there ? rstd[row] : 0.0f;
    hp += jump * ldh;
    gp += jump * lddy;
    if (!LATE) dp += jump * lddh;
  };
  // Read again for each use, from L1: held, the weights of a row would take the registers of the next row.
  auto weights = [&](int i, f32x2 (&f)[4]) {
    const P* p = weight;
    asm volatile("" : "+l"(p));
    if (p) {
      unpack2<P, 8>(get8<P, VEC>(p + first + i * step, at.lane16, in[i]), f);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = f32x2(1.0f);
    }
  };
  T* op = dx + row0 * H + first;
  if (AHEAD) load(row0);
  int it = 0;
  for (int64_t base = (int64_t)blockIdx.x * at.rows; base < N; base += jump, ++it, op += jump * H) {
    const int64_t row = base + at.group;
    if (!AHEAD) load(row);
    Pack<T, 8> v[PER], g[PER], d[PER];
    const float rs = rs_next;
    const f32x2 rs2(rs);
    f32x2 sum(0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = nh[i];
      g[i] = ng[i];
      d[i] = nd[i];
    }
    if (AHEAD) load(row + jump);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      f32x2 a[4], b[4], w[4];
      unpack2<T, 8>(v[i], a);
      unpack2<T, 8>(g[i], b);
      weights(i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 xh = mul2(a[j], rs2);
        gw[i][j] = fma2(b[j], xh, gw[i][j]);
        sum = fma2(mul2(b[j], w[j]), xh, sum);
      }
    }
    if (!dx) continue;               // all threads alike
    const float c = row_sum(sum.sum(), tpr, at.group, at.t, sums.v[it & 1]) * inv_h;
    if (row < N) {
      const f32x2 by_h(-rs * rs * c);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (LATE) d[i] = get8<T, VEC>(dp + i * step, at.lane16, with_dh ? in[i] : 0);
        f32x2 a[4], b[4], w[4], e[4];
        unpack2<T, 8>(v[i], a);
        unpack2<T, 8>(g[i], b);
        unpack2<T, 8>(d[i], e);
        weights(i, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = add2(fma2(mul2(b[j], w[j]), rs2, mul2(a[j], by_h)), e[j]);
        put8<T, VEC>(op + i * step, at.lane16, in[i], pack2<T, 8>(e));
      }
    }
    if (LATE) dp += jump * lddh;
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * H;
  for (int r = 0; r < at.rows; ++r) {
    if (r > 0) __syncthreads();
    if (at.group != r) continue;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float mine[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) gw[i][j].get(mine[2 * j], mine[2 * j + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = block_column<VEC>(at.lane16, j);
        if (c < at.valid(i)) {
          const float s = mine[j] + (r > 0 ? cols[at.column(i) + c] : 0.0f);
          if (r + 1 < at.rows) cols[at.column(i) + c] = s;
          else out[at.column(i) + c] = s;
        }
      }
    }
  }
}

// dweight[c] = the sum of part[0 .. groups - 1][c], 32 columns a block: each of 32 warps adds every 32nd, then the 32
// sums are added in order.
__global__ void __launch_bounds__(1024) rms_param_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                         int groups, int H) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 10
    for (int g = warp; g < groups; g += 32) s += part[(int64_t)g * H + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H) {
    for (int g = 1; g < 32; ++g) s += sums[g][lane];
    dweight[c] = s;
  }
}

int rms_validate(const moe_rmsnorm_config* c) {
  if (!c || c->N < 0 || c->H < 1 || !(c->eps >= 0.0f) || c->eps > 3.0e38f) return MOE_ERR_INVALID_ARG;
  return c->H > MOE_RMSNORM_MAX_H ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

// Threads of a row and rows of a block, by the row's blocks of 128 columns.  A half warp has one block up to 256 columns, two
// up to 512 in the forward and 7168 in the backward, else four; a row has whole warps of them, one up to 512 columns (1024 in
// the forward).  Threads with fewer values need fewer registers, and more blocks of them run on a SM.
struct RmsShape {
  int nb, per, tpr, rows;
};
RmsShape rms_shape(int H, bool forward) {
  RmsShape s;
  s.nb = (H + MOE_BLOCK8 - 1) / MOE_BLOCK8;
  s.per = s.nb <= 2 ? 1 : s.nb <= (forward ? 4 : 56) ? 2 : 4;
  s.tpr = ((s.nb + s.per - 1) / s.per * 16 + 31) / 32 * 32;
  s.rows = std::max(1, (forward ? kFwdThreads : 256) / s.tpr);
  return s;
}
// The backward's blocks of threads.
int rms_blocks(int N, const RmsShape& s) {
  return (int)std::min<int64_t>(304 * (4 / s.per), ((int64_t)N + s.rows - 1) / s.rows);
}

// f(T, P, VEC, PER) with compile-time values.
template <class F>
cudaError_t with_rms(int type, int param_type, bool vec, int per, F&& f) {
  return with_type(type, [&](auto tv) {
    auto by_param = [&](auto pv) {
      auto by_per = [&](auto vv) {
        if (per == 1) return f(tv, pv, vv, std::integral_constant<int, 1>{});
        if (per == 2) return f(tv, pv, vv, std::integral_constant<int, 2>{});
        return f(tv, pv, vv, std::integral_constant<int, 4>{});
      };
      return vec ? by_per(std::true_type{}) : by_per(std::false_type{});
    };
    if (param_type == MOE_TYPE_F32) return by_param(float{});
    return by_param(tv);
  });
}

bool vec_rows(const void* p, int64_t ld, int type) {
  return !p || (aligned_to(p, 16) && ld * type_size(type) % 16 == 0);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_rmsnorm_workspace_bytes(const moe_rmsnorm_config* cfg, size_t* bwd_bytes) {
  const int v = rms_validate(cfg);
  if (v != MOE_OK) return v;
  if (bwd_bytes) *bwd_bytes = sizeof(WsHeader) + align256((size_t)rms_blocks(cfg->N, rms_shape(cfg->H, false)) * cfg->H * 4);
  return MOE_OK;
}

int moe_rmsnorm_forward(const moe_rmsnorm_config* cfg, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                        const void* weight, void* h, void* y, uint8_t* codes, uint8_t* scales, float* rstd,
                        int32_t type, int32_t param_type, void* stream) {
  const int v = rms_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_rmsnorm_config& c = *cfg;
  if (!known_type(type) || !(param_type == type || param_type == MOE_TYPE_F32) || ldx < c.H || (residual && ldr < c.H))
    return MOE_ERR_INVALID_ARG;
  const size_t ts = type_size(type);
  if (!aligned_to(weight, type_size(param_type)) || !aligned_to(rstd, 4) || !aligned_to(residual, ts) ||
      !aligned_to(h, ts) || !aligned_to(y, ts) || (codes != nullptr) != (scales != nullptr) || (h && !residual))
    return MOE_ERR_INVALID_ARG;
  if (c.N == 0) return MOE_OK;
  if (!x || !aligned_to(x, ts)) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RmsShape r = rms_shape(c.H, true);
  const bool vec = c.H % 8 == 0 && vec_rows(x, ldx, type) && vec_rows(residual, ldr, type) && vec_rows(h, c.H, type) &&
                   vec_rows(y, c.H, type) && aligned_to(weight, 16) && aligned_to(codes, 8);
  return timed_launch(MOE_K_RMS_FWD, "rms norm", s, [&] {
    return with_rms(type, param_type, vec, r.per, [&](auto tv, auto pv, auto vv, auto n) {
      using T = decltype(tv);
      using P = decltype(pv);
      constexpr int PER = decltype(n)::value;
      // rows of more threads than kFwdThreads hold four blocks of 128 columns a half warp
      auto kern = PER == 4 && r.tpr > kFwdThreads ? rms_fwd_kernel<T, P, decltype(vv)::value, PER, PER == 4>
                                                  : rms_fwd_kernel<T, P, decltype(vv)::value, PER, false>;
      return launch_pdl(kern, dim3((unsigned)(((int64_t)c.N + r.rows - 1) / r.rows)),
                        dim3(r.tpr * r.rows), 0, s, static_cast<const T*>(x), ldx, static_cast<const T*>(residual), ldr,
                        static_cast<const P*>(weight), static_cast<T*>(h), static_cast<T*>(y), codes, scales, rstd, c.N,
                        c.H, r.nb, r.tpr, c.eps);
    });
  });
}

int moe_rmsnorm_backward(const moe_rmsnorm_config* cfg, const void* h, int64_t ldh, const void* weight,
                         const float* rstd, const void* dy, int64_t lddy, const void* dh, int64_t lddh, void* dx,
                         float* dweight, int32_t type, int32_t param_type, void* ws, size_t ws_bytes, void* stream) {
  int v = rms_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_rmsnorm_config& c = *cfg;
  if (!known_type(type) || !(param_type == type || param_type == MOE_TYPE_F32) || ldh < c.H || lddy < c.H ||
      (dh && lddh < c.H))
    return MOE_ERR_INVALID_ARG;
  const size_t ts = type_size(type);
  if (!aligned_to(weight, type_size(param_type)) || !aligned_to(dweight, 4) || !aligned_to(dh, ts) || !aligned_to(dx, ts))
    return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N == 0) {
    if (!dweight) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)c.H * 4, s);
    return e == cudaSuccess ? MOE_OK : record_cuda_error(e, "clear the norm's gradient");
  }
  if (!h || !dy || !rstd || !aligned_to(h, ts) || !aligned_to(dy, ts) || !aligned_to(rstd, 4) || !ws || !aligned_to(ws, 16))
    return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  moe_rmsnorm_workspace_bytes(cfg, &need);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!dx && !dweight) return MOE_OK;
  const RmsShape r = rms_shape(c.H, false);
  const bool vec = c.H % 8 == 0 && vec_rows(h, ldh, type) && vec_rows(dy, lddy, type) && vec_rows(dh, lddh, type) &&
                   vec_rows(dx, c.H, type) && aligned_to(weight, 16);
  float* part = dweight ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader)) : nullptr;
  const int blocks = rms_blocks(c.N, r);
  v = timed_launch(MOE_K_RMS_BWD, "rms norm backward", s, [&] {
    return with_rms(type, param_type, vec, r.per, [&](auto tv, auto pv, auto vv, auto n) {
      using T = decltype(tv);
      using P = decltype(pv);
      return launch_pdl(rms_bwd_kernel<T, P, decltype(vv)::value, decltype(n)::value>, dim3(blocks),
                        dim3(r.tpr * r.rows), r.rows > 1 ? c.H * 4 : 0, s, static_cast<const T*>(h), ldh,
                        static_cast<const P*>(weight), rstd, static_cast<const T*>(dy), lddy, static_cast<const T*>(dh),
                        lddh, static_cast<T*>(dx), part, c.N, c.H, r.tpr);
    });
  });
  if (v != MOE_OK || !dweight) return v;
  return timed_launch(MOE_K_RMS_BWD, "rms norm weight gradient", s, [&] {
    return launch_pdl(rms_param_kernel, dim3((c.H + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(part), dweight,
                      blocks, c.H);
  });
}

}  // extern "C"

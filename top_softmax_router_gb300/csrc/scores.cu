// Routing to experts from given logits: scores, balance bias, groups, top-k, weights, and the gradient
// (include/moe_scores.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe.h"
#include "../../include/moe_scores.h"
#include "ops_common.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;   // rows a block holds at a time

// Keys order floats as unsigned integers: 0 = not a candidate, 1 = NaN, then -inf upwards.  -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The same in three instructions for a value that is not -0; a NaN comes out beyond an infinity, and nan_last() puts it
// in its place.
__device__ __forceinline__ uint32_t quick_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t nan_last(uint32_t k) { return k > 0xff800000u || k < 0x007fffffu ? 1u : k; }
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct Params {
  const float* bias;
  int N, E, k, groups, topk_groups, group_top, group_size;
  uint32_t group_inv;   // ceil(2^20 / group_size): e / group_size = (e group_inv) >> 20 for e < 1024
  bool sigmoid, renormalize;
  float scale;
};

__device__ __forceinline__ float exp2_approx(float x) {   // PTX ex2.approx: relative error at most 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {    // PTX rcp.approx: relative error at most 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Below -64 the sigmoid is exp(l) to fp32, and exp(-l) would overflow.
__device__ __forceinline__ float sigmoid_of(float l) { return l < -64.0f ? expf(l) : 1.0f / (1.0f + expf(-l)); }

// What a row's scores are computed from: l -> s.
struct RowScore {
  float m, sum, inv;   // softmax: maximum, sum of exp(l - m), 1 / sum
  bool sigmoid;
  __device__ __forceinline__ float of(float l) const {
    if (sigmoid) return sigmoid_of(l);
    if (m == -INFINITY) return l == l ? 0.0f : l;
    return expf(l - m) / sum;
  }
  // For the choice: two instructions of the special function unit.  off() bounds how far it is from s.
  __device__ __forceinline__ float quick_sigmoid(float l) const { return rcp_approx(1.0f + exp2_approx(-kLog2e * l)); }
  __device__ __forceinline__ float quick_softmax(float l) const {
    const float s = exp2_approx((l - m) * kLog2e) * inv;
    return l == -INFINITY ? 0.0f : s;   // also where every logit is
  }
  // sigmoid: the exponent's rounding moves e by 2 x 2^-24 |l| of itself and s by s (1 - s) of that, s (1 - s) |l| <=
  // 0.23; ex2, the addition and rcp add 2^-22 + 2^-24 + 2^-23 of s: below 2^-21 together.
  // softmax: the exponent's roundings 3 x 2^-24 x exp(-x) <= 1.2 x 2^-24 of the row's largest score; ex2, the sum of up to
  // 32 + 5 steps, its reciprocal and the product: 50 x 2^-24 of it: below 2^-18.
  __device__ __forceinline__ float off() const { return sigmoid ? 0x1p-21f : 0x1p-18f * inv; }
};

// exp(l - m) of a chosen expert, relative to itself within a few 2^-24 however far l is from m: what the
// subtraction rounds off comes back as a factor.
__device__ __forceinline__ float chosen_exp(float l, float m) {
  if (l == -INFINITY) return 0.0f;
  const float d = l - m, b = d - l, off = (l - (d - b)) - (m + b);
  return expf(d) * (1.0f + off);
}
// A chosen expert's part of the sum that weights are renormalised by, up to a factor that all lanes share (l is -inf in
// a lane without one).  A sigmoid of 0 or more is at least 1/2, and the scores are summed as they are; where every one
// is smaller they are taken relative to the largest, as for the softmax, since fp32 holds none below exp(-104).
__device__ __forceinline__ float chosen_part(float l, bool sigmoid) {
  if (sigmoid && __any_sync(kFull, l >= 0.0f)) return sigmoid_of(l);
  if (sigmoid && l < -709.0f) l = -INFINITY;   // 0 in fp64 too: a mask
  const float e = chosen_exp(l, key_value(__reduce_max_sync(kFull, order_key(l))));
  return sigmoid ? e / (1.0f + expf(l)) : e;
}

// fp64 scores of a row, for values that fp32 cannot order.
struct ExactScore {
  double m, sum;
  bool sigmoid;
  __device__ __forceinline__ double of(float l) const {
    if (sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    if (isinf(m) && m < 0) return l == l ? 0.0 : (double)l;
    return exp((double)l - m) / sum;
  }
};

// (Reads the row again: taking the logits by reference would keep them in local memory for every row.)
template <class T>
__device__ __noinline__ ExactScore exact_score(const T* lr, float m, bool sigmoid, int E) {
  ExactScore x = {(double)m, 0.0, sigmoid};
  if (sigmoid) return x;
  double s = 0.0;
  for (int e = threadIdx.x & 31; e < E; e += 32) s += exp((double)to_f32<T>(lr[e]) - x.m);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
  x.sum = s;
  return x;
}

// The value an expert is chosen by, in fp64.
template <class T>
__device__ __noinline__ double exact_value(const ExactScore x, const T* lr, const float* bias, int e) {
  return x.of(to_f32<T>(lr[e])) + (bias ? (double)bias[e] : 0.0);
}

// The group's score from the values c[0 .. size) of its experts, spread over `width` lanes (a power of two):
// the sum of its `top` largest, and *mass the sum of their absolute values.  NaN values are passed over.
template <class F>
__device__ __forceinline__ F group_score(const F* c, int size, int sub, int width, int top, F* mass) {
  F m1 = (F)-INFINITY, m2 = (F)-INFINITY;
  for (int i = sub; i < size; i += width) {
    const F v = c[i];
    if (v > m1) m2 = m1, m1 = v;
    else if (v > m2) m2 = v;
  }
  for (int off = 1; off < width; off <<= 1) {
    const F o1 = __shfl_xor_sync(kFull, m1, off), o2 = __shfl_xor_sync(kFull, m2, off);
    const F hi = m1 > o1 ? m1 : o1, lo = m1 > o1 ? o1 : m1;
    const F second = m1 > o1 ? m2 : o2;
    m1 = hi;
    m2 = lo > second ? lo : second;
  }
  const bool two = top == 2 && size > 1;
  const F s = two ? m1 + m2 : m1;
  *mass = fabs(m1) + (two ? fabs(m2) : (F)0);
  return s == s ? s : (F)-INFINITY;
}

// The score of the lane's group in fp64, from each lane's `per` experts from `first` on.
template <class T>
__device__ __noinline__ double group_score_run(const ExactScore x, const T* lr, const float* bias, int first, int per,
                                               int width, int top, int size) {
  double m1 = -INFINITY, m2 = -INFINITY;
  for (int i = 0; i < per; ++i) {
    const double v = exact_value<T>(x, lr, bias, first + i);
    if (v > m1) m2 = m1, m1 = v;
    else if (v > m2) m2 = v;
  }
  for (int off = 1; off < width; off <<= 1) {
    const double o1 = __shfl_xor_sync(kFull, m1, off), o2 = __shfl_xor_sync(kFull, m2, off);
    const double lo = m1 > o1 ? o1 : m1, second = m1 > o1 ? m2 : o2;
    m1 = m1 > o1 ? m1 : o1;
    m2 = lo > second ? lo : second;
  }
  const double s = top == 2 && size > 1 ? m1 + m2 : m1;
  return s == s ? s : -INFINITY;
}

// One warp a row, its experts' values as integer keys in the lanes' registers.  The k best are ranked among the few candidates
// that can be among them (k rounds of a warp maximum over all of them took 148 us for 32768 x 384, k = 8).  Two fp32
// values can be in the wrong order only if they lie within `window` of each other; where that happens among the
// candidates they are compared in fp64 (unless their logit and bias are equal, when the tie rule decides).

// Bound by its arithmetic: 32768 x 384 with 8 groups, k = 8 takes 1102 instructions a row, 75 of them loads and stores
// of spilled registers, 55 us (the logits alone are 7.4 us of memory); 16384 x 64 483 a row, 13 us, of which their
// issue is 6 and the rest latency: a warp has three or four rows.
// Blocks an SM (four leave 64 registers a thread, and the forms of up to 12 experts a lane spill 48 to 276 bytes).
constexpr int fwd_blocks(int per) { return per <= 12 ? 4 : per <= 16 ? 2 : 1; }

// RUN: lane t holds the PER = E / 32 consecutive experts from t PER on, so that a lane's experts are of one group and the
// groups are scored in registers.  Else lane t holds experts t, t + 32, .. and the groups are scored from shared memory.
template <class T, int PER, bool RUN>
__global__ void __launch_bounds__(32 * kWarps, fwd_blocks(PER))
    scores_fwd_kernel(const T* __restrict__ logits, int64_t ld, Params p, int32_t* __restrict__ topk_idx,
                      float* __restrict__ weights, int32_t* __restrict__ counts) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ double sm[];
  __shared__ uint2 cands[kWarps][32];   // (key, expert)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  int* hist = reinterpret_cast<int*>(sm);                                       // [E] choices of this block
  double* vals = sm + (E + 1) / 2 + (int64_t)warp * (!RUN && p.groups > 1 ? E : 0);   // [E] values of the row's groups
  auto expert = [&](int q) { return RUN ? lane * PER + q : q * 32 + lane; };
  auto held = [&](int q) { return RUN || q * 32 + lane < E; };
  if (counts) {
    for (int e = threadIdx.x; e < E; e += 32 * kWarps) hist[e] = 0;
    __syncthreads();
  }
  const bool biased = p.bias != nullptr;
  constexpr bool KEEP_BIAS = PER <= 16;   // in registers over the warp's rows
  float bias[KEEP_BIAS ? PER : 1];
  if constexpr (KEEP_BIAS) {
#pragma unroll
    for (int q = 0; q < PER; ++q) bias[q] = biased && held(q) ? __ldg(p.bias + expert(q)) : 0.0f;
  }
  int width = 32;                 // lanes a group: 32 / (groups rounded up to a power of two)
  while (width > 1 && width * p.groups > 32) width >>= 1;
  // the scores enter the choice, or the weights as they are
  const bool by_score = !biased && p.groups > 1 && p.group_top == 2;
  const bool need_scores = biased || by_score || !p.renormalize;
  for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < p.N; row += (int64_t)gridDim.x * kWarps) {
    const T* lr = logits + row * ld;
    float l[PER];
    uint32_t key[PER];
    if constexpr (RUN) {
      constexpr int CH = PER % 4 == 0 ? 4 : PER;
#pragma unroll
      for (int q = 0; q < PER; q += CH) {
        float f[CH];
        unpack<T, CH>(load_pack<T, CH>(lr + lane * PER + q), f);
#pragma unroll
        for (int j = 0; j < CH; ++j) l[q + j] = f[j];
      }
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q) l[q] = held(q) ? to_f32<T>(lr[expert(q)]) : -INFINITY;
    }
    float m = -INFINITY;
    RowScore score = {m, 1.0f, 1.0f, p.sigmoid};
    if (!p.sigmoid && need_scores) {
#pragma unroll
      for (int q = 0; q < PER; ++q) m = fmaxf(m, l[q]);
      m = score.m = key_value(__reduce_max_sync(kFull, order_key(m)));
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (held(q)) s += expf(l[q] - m);
      s = warp_sum(s);
      score.sum = m == -INFINITY ? 1.0f : s;   // every logit masked: all scores are 0
      score.inv = rcp_approx(score.sum);
    }
    // Without a bias c grows with l, so the logits themselves order the experts exactly.  Else two values whose fp32
    // forms are further apart than 2 (off + 2^-24 |c|) are in the right order; the windows below are twice that.
    const float window0 = biased ? 4.0f * score.off() : 0.0f;
    // (The uniform cases stand outside the loops: a branch in each step would run the steps one after the other.)
    float s_q[PER];
    if (biased || by_score) {
      if (p.sigmoid) {
#pragma unroll
        for (int q = 0; q < PER; ++q) s_q[q] = score.quick_sigmoid(l[q]);
      } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) s_q[q] = score.quick_softmax(l[q]);
      }
    }
    bool odd = false;   // a NaN, which the quick keys put at an end
    auto set_key = [&](int q, float c) {
      key[q] = held(q) ? quick_key(c) : 0u;
      odd |= c != c;
    };
    if (biased) {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        set_key(q, s_q[q] + (KEEP_BIAS ? bias[KEEP_BIAS ? q : 0] : held(q) ? __ldg(p.bias + expert(q)) : 0.0f));
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q) set_key(q, l[q] + 0.0f);
    }
    odd = __any_sync(kFull, odd);
    if (odd) {
#pragma unroll
      for (int q = 0; q < PER; ++q) key[q] = held(q) ? nan_last(key[q]) : 0u;
    }
    if (p.groups > 1) {
      // values the groups are scored by: c, or s where there is no bias (the logit itself when only the
      // largest counts)
      const float wide = biased || by_score ? 8.0f * score.off() : 0.0f;
      const int g = lane / width, sub = lane % width;
      const bool mine = g < p.groups;
      float gs, mass;   // mass: what the two values' roundings are relative to, also where the values cancel
      if constexpr (RUN) {
        uint32_t k1 = 1u, k2 = 1u;   // the two largest keys
        if (by_score) {
#pragma unroll
          for (int q = 0; q < PER; ++q) {
            const uint32_t k = nan_last(quick_key(s_q[q]));
            k2 = max(k2, min(k1, k));
            k1 = max(k1, k);
          }
        } else {
#pragma unroll
          for (int q = 0; q < PER; ++q) {
            k2 = max(k2, min(k1, key[q]));
            k1 = max(k1, key[q]);
          }
        }
        for (int off = 1; off < width; off <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(kFull, k1, off), o2 = __shfl_xor_sync(kFull, k2, off);
          k2 = max(min(k1, o1), max(k2, o2));
          k1 = max(k1, o1);
        }
        const float v1 = k1 > 1u ? key_value(k1) : -INFINITY, v2 = k2 > 1u ? key_value(k2) : -INFINITY;
        const bool two = p.group_top == 2 && p.group_size > 1;
        gs = two ? v1 + v2 : v1;
        mass = fabsf(v1) + (two ? fabsf(v2) : 0.0f);
        if (gs != gs) gs = -INFINITY;
      } else {
        float* v32 = reinterpret_cast<float*>(vals);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (held(q)) v32[expert(q)] = by_score ? s_q[q] : key[q] > 1u ? key_value(key[q]) : NAN;
        __syncwarp();
        gs = group_score<float>(v32 + (mine ? g : 0) * p.group_size, p.group_size, sub, width, p.group_top, &mass);
      }
      const float w = wide + mass * (wide > 0.0f ? 0x1p-21f : 0.0f);
      // rank of the group: how many are surely before it, and how many may be
      int before = 0, sure = 0, maybe = 0;
#pragma unroll 4
      for (int h = 0; h < p.groups; ++h) {
        const float o = __shfl_sync(kFull, gs, h * width);
        before += o > gs || (o == gs && h < g);
        sure += o > gs + w;
        maybe += h != g && o >= gs - w;
      }
      bool open = mine && before < p.topk_groups;
      const bool unsure = mine && wide > 0.0f && sure < p.topk_groups && maybe >= p.topk_groups;
      if (__any_sync(kFull, unsure)) {
        const ExactScore exact = exact_score<T>(lr, m, p.sigmoid, E);
        double gd;
        if constexpr (RUN) {
          gd = group_score_run<T>(exact, lr, p.bias, lane * PER, PER, width, p.group_top, p.group_size);
        } else {
          __syncwarp();
          for (int e = lane; e < E; e += 32) vals[e] = exact_value<T>(exact, lr, p.bias, e);
          __syncwarp();
          double md;
          gd = group_score<double>(vals + (mine ? g : 0) * p.group_size, p.group_size, sub, width, p.group_top, &md);
        }
        before = 0;
        for (int h = 0; h < p.groups; ++h) {
          const double o = __shfl_sync(kFull, gd, h * width);
          before += o > gd || (o == gd && h < g);
        }
        open = mine && before < p.topk_groups;
      }
      if constexpr (RUN) {
#pragma unroll
        for (int q = 0; q < PER; ++q) key[q] = open ? key[q] : 0u;
      } else {
        const uint32_t open_lanes = __ballot_sync(kFull, open);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const uint32_t eg = ((uint32_t)(q * 32 + lane) * p.group_inv) >> 20;
          if (!((open_lanes >> (eg * width & 31)) & 1u)) key[q] = 0u;
        }
      }
    }
    // The choice.  Every one of the k best is at least the k-th largest of the lanes' largest keys; what lies that high
    // (window included), usually little more than k, is gathered, one candidate a lane, and ranked.
    int my_e = 0;
    uint32_t best = 0u;
#pragma unroll
    for (int q = 0; q < PER; ++q) best = max(best, key[q]);
    uint32_t floor_key = 1u;
    {
      uint32_t left = best;
      for (int j = 0; j < p.k; ++j) {
        floor_key = __reduce_max_sync(kFull, left);
        if (left == floor_key) left = 0u;
      }
    }
    if (biased && floor_key > 1u) {
      const float v = key_value(floor_key);
      floor_key = order_key(v - (window0 + fabsf(v) * 0x1p-22f));
    }
    floor_key = max(floor_key, 1u);
    uint32_t mine = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) mine |= (key[q] >= floor_key ? 1u : 0u) << q;
    int at = __popc(mine), many = at;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFull, at, off);
      if (lane >= off) at += v;
    }
    const int cand = __shfl_sync(kFull, at, 31);
    at -= many;
    if (cand <= 32) {
      uint2* list = cands[warp];
      __syncwarp();
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if ((mine >> q) & 1u) list[at++] = make_uint2(key[q], (uint32_t)expert(q));
      __syncwarp();
      const bool is = lane < cand;
      const uint2 own = is ? list[lane] : make_uint2(0u, 0u);
      const int own_e = (int)own.y;
      // rank, and whether another candidate is too near to be told from this one in fp32
      const float v = key_value(own.x);
      const uint32_t low = biased && own.x > 1u ? order_key(v - (window0 + fabsf(v) * 0x1p-22f)) : own.x;
      int rank = 0, close = 0;
#pragma unroll 4
      for (int j = 0; j < cand; ++j) {
        const uint2 o = list[j];
        const bool above = o.x > own.x || (o.x == own.x && o.y < own.y);
        rank += above;
        close += !above && o.x >= low;    // itself among them
      }
      if (biased) {
        const bool near = is && own.x > 1u && close > 1;
        if (__any_sync(kFull, near)) {
          // equal logits and biases are no question: the tie rule has decided
          const float lo = is ? to_f32<T>(lr[own_e]) : 0.0f, bo = is ? p.bias[own_e] : 0.0f;
          bool other = false;
          for (int j = 0; j < cand; ++j) {
            const uint2 o = list[j];
            const float lj = __shfl_sync(kFull, lo, j), bj = __shfl_sync(kFull, bo, j);
            other |= near && o.x <= own.x && o.x >= low && (lj != lo || bj != bo);
          }
          if (__any_sync(kFull, other)) {
            const ExactScore exact = exact_score<T>(lr, m, p.sigmoid, E);
            const double c = is ? exact_value<T>(exact, lr, p.bias, own_e) : 0.0;
            const bool number = own.x > 1u;
            rank = 0;
            for (int j = 0; j < cand; ++j) {
              const double cj = __shfl_sync(kFull, c, j);
              const uint2 o = list[j];
              const bool nj = o.x > 1u;
              rank += nj != number ? nj : number && cj != c ? cj > c : o.y < own.y;
            }
          }
        }
      }
      __syncwarp();
      if (is && rank < p.k) list[rank].y = (uint32_t)own_e;   // every lane has its own candidate in registers
      __syncwarp();
      if (lane < p.k) my_e = (int)list[lane].y;
    } else {
      // many equal values, or k far above the usual: k rounds of a warp maximum
      for (int j = 0; j < p.k; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        int q_first = 0;
#pragma unroll
        for (int q = PER - 1; q >= 0; --q)
          if (key[q] == top) q_first = q;
        int e = __reduce_min_sync(kFull, best == top ? expert(q_first) : 0x7fffffff);
        if (biased && top > 1u) {
          const float tv = key_value(top);
          const uint32_t near_key = order_key(tv - (window0 + fabsf(tv) * 0x1p-22f));
          bool near = false;
#pragma unroll
          for (int q = 0; q < PER; ++q) near |= key[q] >= near_key && expert(q) != e;
          if (__any_sync(kFull, near)) {
            const float le = to_f32<T>(lr[e]), be = p.bias[e];
            bool other = false;
#pragma unroll
            for (int q = 0; q < PER; ++q)
              if (key[q] >= near_key) other |= l[q] != le || p.bias[expert(q)] != be;
            if (__any_sync(kFull, other)) {
              const ExactScore exact = exact_score<T>(lr, m, p.sigmoid, E);
              uint32_t mine = 0;
#pragma unroll
              for (int q = 0; q < PER; ++q) mine |= (key[q] >= near_key ? 1u : 0u) << q;
              double bv = -INFINITY;
              int bq = 0x7fffffff;
              for (; mine; mine &= mine - 1) {
                const int i = expert(__ffs(mine) - 1);
                const double v = exact_value<T>(exact, lr, p.bias, i);
                if (bq == 0x7fffffff || v > bv) bv = v, bq = i;
              }
              __syncwarp();
#pragma unroll
              for (int off = 16; off > 0; off >>= 1) {
                const double ov = __shfl_xor_sync(kFull, bv, off);
                const int oq = __shfl_xor_sync(kFull, bq, off);
                if (oq != 0x7fffffff && (bq == 0x7fffffff || ov > bv || (ov == bv && oq < bq))) bv = ov, bq = oq;
              }
              e = bq;
            }
          }
        }
        if (lane == j) my_e = e;
        if ((RUN ? e / PER : e & 31) == lane) {
          best = 0u;
#pragma unroll
          for (int q = 0; q < PER; ++q) {
            if (expert(q) == e) key[q] = 0u;
            best = max(best, key[q]);
          }
        }
      }
    }
    // weights; a lane without a slot adds 0
    const float ls = lane < p.k ? to_f32<T>(lr[my_e]) : -INFINITY;
    float s = 0.0f, total = 1.0f;
    if (p.renormalize) {
      s = chosen_part(ls, p.sigmoid);
      total = warp_sum(s);
    } else if (lane < p.k) {
      s = score.of(ls);
    }
    if (lane < p.k) {
      topk_idx[row * p.k + lane] = my_e;
      weights[row * p.k + lane] = total == 0.0f ? 0.0f : p.scale * (s / total);
      if (counts) atomicAdd(hist + my_e, 1);
    }
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 32 * kWarps) {
      if (gridDim.x == 1) counts[e] = hist[e];
      else if (hist[e]) atomicAdd(counts + e, hist[e]);   // integer adds: the order does not change the result
    }
  }
}

// 32768 x 384 fp32: 19 us for the 50 MB it writes (half of them still in L2 when it ends), 312 instructions a row.
// One warp a row: the chosen experts' gradients (and, for a softmax that is not renormalised, everyone's) are
// put together in shared memory and the row is stored whole.
template <class T, int VEC>
__global__ void __launch_bounds__(32 * kWarps) scores_bwd_kernel(const T* __restrict__ logits, int64_t ld, Params p,
                                                                const int32_t* __restrict__ topk_idx,
                                                                const float* __restrict__ dweights,
                                                                T* __restrict__ dlogits, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float rows[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  float* out = rows + warp * ((E + 3) / 4 * 4);
  const bool dense = !p.sigmoid && !p.renormalize;
  for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < p.N; row += (int64_t)gridDim.x * kWarps) {
    const T* lr = logits + row * ld;
    const bool slot = lane < p.k;
    const int e = slot ? topk_idx[row * p.k + lane] : 0;
    const bool ok = slot && e >= 0 && e < E;
    if (slot && !ok) report(status, MOE_ERR_DEVICE_CHECK, 601);
    const float dw = ok ? dweights[row * p.k + lane] : 0.0f;
    const float l = ok ? to_f32<T>(lr[e]) : -INFINITY;
    float dl;   // of the chosen expert
    if (dense) {
      float m = -INFINITY, s = 0.0f;
      for (int i = lane; i < E; i += 32) {
        const float v = to_f32<T>(lr[i]);
        out[i] = v;
        m = fmaxf(m, v);
      }
      m = key_value(__reduce_max_sync(kFull, order_key(m)));
      for (int i = lane; i < E; i += 32) {
        const float v = m == -INFINITY ? (out[i] == out[i] ? 0.0f : out[i]) : expf(out[i] - m);
        out[i] = v;
        s += v;
      }
      s = warp_sum(s);
      const float inv = s == 0.0f ? 0.0f : 1.0f / s;
      __syncwarp();
      const float se = ok ? out[e] * inv : 0.0f;
      const float all = warp_sum(ok ? p.scale * dw * se : 0.0f);
      dl = se * (p.scale * dw - all);
      __syncwarp();
      for (int i = lane; i < E; i += 32) out[i] = -out[i] * inv * all;
    } else {
      for (int i = lane; i < E; i += 32) out[i] = 0.0f;
      // the derivative's factor beside the share of the renormalised sum (or the score)
      const float rest = !p.sigmoid ? 1.0f : ok ? 1.0f / (1.0f + expf(l)) : 0.0f;
      float s;
      if (p.renormalize) {
        s = chosen_part(l, p.sigmoid);   // l is -inf where there is no expert
        const float total = warp_sum(s);
        s = total == 0.0f ? 0.0f : s / total;
        dl = p.scale * s * (dw - warp_sum(dw * s)) * rest;
      } else {   // a sigmoid
        s = ok ? sigmoid_of(l) : 0.0f;
        dl = p.scale * s * dw * rest;
      }
    }
    __syncwarp();
    if (ok) out[e] = dl;
    __syncwarp();
    T* dst = dlogits + row * E;
    for (int i = lane * VEC; i < E; i += 32 * VEC) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = out[i + j];
      store_pack<T, VEC>(dst + i, pack<T, VEC>(f));
    }
    __syncwarp();
  }
}

int scores_validate(const moe_scores_config* c) {
  if (!c || c->N < 0 || c->E <= 0 || c->k <= 0 || c->groups <= 0 || c->topk_groups <= 0 ||
      (c->group_top != 1 && c->group_top != 2) || (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) ||
      (c->renormalize != 0 && c->renormalize != 1) || !std::isfinite(c->scale))
    return MOE_ERR_INVALID_ARG;
  if (c->E > 1024 || c->groups > 32 || c->E % c->groups != 0 || c->topk_groups > c->groups || c->k > 32 ||
      c->k > c->topk_groups * (c->E / c->groups))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

Params params(const moe_scores_config& c, const float* bias) {
  Params p = {};
  p.bias = bias;
  p.N = c.N;
  p.E = c.E;
  p.k = c.k;
  p.groups = c.topk_groups == c.groups ? 1 : c.groups;   // all open: no group is closed
  p.topk_groups = c.topk_groups;
  p.group_top = c.group_top;
  p.group_size = c.E / c.groups;
  p.group_inv = (uint32_t)(((1 << 20) + p.group_size - 1) / p.group_size);
  p.sigmoid = c.score == MOE_SCORE_SIGMOID;
  p.renormalize = c.renormalize != 0;
  p.scale = c.scale;
  return p;
}

unsigned row_blocks(int N, int per_sm) {
  const int64_t need = ((int64_t)N + kWarps - 1) / kWarps;
  return (unsigned)std::min<int64_t>(need, (int64_t)device_sm_count() * per_sm);
}

template <class F>
cudaError_t with_per(int E, F&& f) {
  const int per = (E + 31) / 32;
  if (per <= 1) return f(std::integral_constant<int, 1>{});
  if (per <= 2) return f(std::integral_constant<int, 2>{});
  if (per <= 4) return f(std::integral_constant<int, 4>{});
  if (per <= 8) return f(std::integral_constant<int, 8>{});
  if (per <= 12) return f(std::integral_constant<int, 12>{});
  if (per <= 16) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_scores_workspace_bytes(const moe_scores_config* cfg, size_t* bytes) {
  const int v = scores_validate(cfg);
  if (v != MOE_OK) return v;
  if (bytes) *bytes = sizeof(WsHeader);
  return MOE_OK;
}

int moe_scores_forward(const moe_scores_config* cfg, const void* logits, int64_t ld, int32_t type,
                       const float* bias, int32_t* topk_idx, float* weights, int32_t* counts, void* ws,
                       size_t ws_bytes, void* stream) {
  const int v = scores_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_scores_config& c = *cfg;
  if (!known_type(type) || ld < c.E || !ws || !aligned_to(ws, 16) || !aligned_to(bias, 4) || !aligned_to(counts, 4))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N > 0 && (!logits || !topk_idx || !weights || !aligned_to(logits, type_size(type)) ||
                  !aligned_to(topk_idx, 4) || !aligned_to(weights, 4)))
    return MOE_ERR_INVALID_ARG;
  if (counts && (c.N == 0 || c.N > kWarps)) {   // a single block stores them
    const cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)c.E * 4, s);
    if (e != cudaSuccess) return record_cuda_error(e, "clear counts");
  }
  if (c.N == 0) return MOE_OK;
  const Params p = params(c, bias);
  return timed_launch(MOE_K_SCORES_FWD, "expert scores", s, [&] {
    return with_type(type, [&](auto tv) {
      using T = decltype(tv);
      return with_per(c.E, [&](auto per) {
        constexpr int PER = decltype(per)::value, CH = PER % 4 == 0 ? 4 : PER;
        auto go = [&](auto kern, bool grouped_in_smem) {
          // [E] counters, then [E] values a warp where groups are scored there: at most 4 KB + 64 KB
          const size_t smem = ((size_t)(c.E + 1) / 2 + (grouped_in_smem ? (size_t)kWarps * c.E : 0)) * 8;
          if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
          }
          return launch_pdl(kern, dim3(row_blocks(c.N, fwd_blocks(PER))), dim3(32 * kWarps), smem, s,
                            static_cast<const T*>(logits), ld, p, topk_idx, weights, counts);
        };
        // runs of E / 32 experts a lane: whole lanes make a group, and rows can be read in packs of CH
        if (c.E == 32 * PER && 32 % p.groups == 0 && ld % CH == 0 && aligned_to(logits, CH * sizeof(T)))
          return go(scores_fwd_kernel<T, PER, true>, false);
        return go(scores_fwd_kernel<T, PER, false>, p.groups > 1);
      });
    });
  });
}

int moe_scores_backward(const moe_scores_config* cfg, const void* logits, int64_t ld, int32_t type,
                        const int32_t* topk_idx, const float* dweights, void* dlogits, void* ws, size_t ws_bytes,
                        void* stream) {
  const int v = scores_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_scores_config& c = *cfg;
  if (!known_type(type) || ld < c.E || !ws || !aligned_to(ws, 16)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (c.N == 0) return MOE_OK;
  const size_t ts = type_size(type);
  if (!logits || !topk_idx || !dweights || !dlogits || !aligned_to(logits, ts) || !aligned_to(dlogits, ts) ||
      !aligned_to(topk_idx, 4) || !aligned_to(dweights, 4))
    return MOE_ERR_INVALID_ARG;
  const Params p = params(c, nullptr);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  return timed_launch(MOE_K_SCORES_BWD, "expert scores backward", s, [&] {
    return with_type(type, [&](auto tv) {
      using T = decltype(tv);
      auto go = [&](auto vv) {
        const size_t smem = (size_t)kWarps * ((c.E + 3) / 4 * 4) * 4;   // at most 32 KB
        return launch_pdl(scores_bwd_kernel<T, decltype(vv)::value>, dim3(row_blocks(c.N, 8)), dim3(32 * kWarps), smem, s,
                          static_cast<const T*>(logits), ld, p, topk_idx, dweights, static_cast<T*>(dlogits), status);
      };
      if (c.E % 4 == 0 && aligned_to(dlogits, 4 * ts)) return go(std::integral_constant<int, 4>{});
      return go(std::integral_constant<int, 1>{});
    });
  });
}

}  // extern "C"

// Token embedding with scaling, and its gradient by sorted tokens (include/moe_embed.h).
//
// Backward: the token positions are sorted by id (stable radix sort, so equal ids keep ascending
// positions); then each table row's gradient is the sum over one run of the sorted list.  A run longer
// than kPiece positions is summed in pieces aligned to multiples of kPiece (embed_piece_kernel, one block
// a piece), which the row's block adds in order.  Every sum thus has a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/moe.h"
#include "../../include/moe_embed.h"
#include "ops_common.cuh"

namespace moe {
namespace {

constexpr int kPiece = 32;           // positions of a piece of a long run (64: 16384 x 2048 added 162 us a pass, 32: 157, 16: 170)
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTile = 8192;          // most positions sorted by one block
constexpr int kCluster = 8;          // blocks that sort together through distributed shared memory
constexpr int kMaxBits = 9;          // bits of a digit: kSortWarps x 512 counters are 64 KB

// ---------------------------------------------------------------------------
// Forward: a warp copies a piece of up to 32 x PER packs of a row, so that a short batch still spreads over the SMs: four
// packs of 16 bytes a lane, or 16 single elements where rows do not start on 16 bytes.  32768 x 4096 bf16: 59 us for
// 0.54 GB (hot rows come from L2).
// ---------------------------------------------------------------------------
template <int VEC>
constexpr int kFwdPer = VEC == 1 ? 16 : 4;
template <class T, class I, int VEC>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const I* __restrict__ ids, const T* __restrict__ table,
                                                       T* __restrict__ y, int N, int V, int H, int pieces,
                                                       float scale, int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t n = unit / pieces;
  constexpr int PER = kFwdPer<VEC>;
  const int c0 = (int)(unit - n * pieces) * (32 * PER * VEC);
  if (n >= N) return;
  const int64_t id = ids[n];
  const bool ok = id >= 0 && id < V;
  if (!ok && c0 == 0 && lane == 0) report(status, MOE_ERR_DEVICE_CHECK, 501);
  const T* src = table + (ok ? id : 0) * H;
  T* dst = y + n * H;
  Pack<T, VEC> p[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = c0 + (i * 32 + lane) * VEC;
    if (c < H) p[i] = load_pack<T, VEC>(src + c);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = c0 + (i * 32 + lane) * VEC;
    if (c >= H) continue;
    if (!ok || scale != 1.0f) {
      float f[VEC];
      unpack<T, VEC>(p[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = ok ? f[j] * scale : 0.0f;
      p[i] = pack<T, VEC>(f);
    }
    store_pack<T, VEC>(dst + c, p[i]);
  }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (id, position)
// ---------------------------------------------------------------------------
// A block sorts its positions by one digit: warp w owns the w-th consecutive `own` positions (a multiple of 32, at most
// kTile / kSortWarps), 32 at a time; lanes with the same digit rank themselves by lane, so equal digits keep their
// order.  cnt[w][d] counts them.
constexpr int kSteps = kTile / kSortWarps / 32;

// The key of a position: its id, or V (which sorts last) for one that adds to no gradient.
template <class I>
__device__ __forceinline__ uint32_t token_key(const I* ids, int64_t n, int V, int padding, int* status) {
  const int64_t id = ids[n];
  if (id < 0 || id >= V) {
    report(status, MOE_ERR_DEVICE_CHECK, 502);
    return (uint32_t)V;
  }
  return id == padding ? (uint32_t)V : (uint32_t)id;
}

// Counts the digits d[k] (of the warp's k-th 32 positions; 0xFFFFFFFF: no position) into the warp's counters, and
// turns each d[k] into digit | rank << 16: how many of the warp's positions before it have the digit.
__device__ __forceinline__ void rank_digits(int* cnt, uint32_t (&d)[kSteps]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const uint32_t peers = __match_any_sync(0xffffffffu, d[k]);
    const bool in = d[k] != 0xFFFFFFFFu;
    int before = 0;
    if (in) before = cnt[d[k]] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == __ffs(peers) - 1) cnt[d[k]] += __popc(peers);
    __syncwarp();
    if (in) d[k] |= (uint32_t)before << 16;   // at most 256 of 512 digits: 9 + 9 bits
  }
}

// Exclusive prefix sum over the block's threads.
__device__ __forceinline__ int exclusive_scan(int v, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int w = lane < warp ? scratch[lane] : 0;   // 32 warps
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
  return w + x - v;
}

// cnt[w][d] becomes the first place of warp w's digit d, where the block's digit d starts at `start` (of thread d).
__device__ __forceinline__ void warp_places(int* cnt, int bins, int start) {
  const int d = threadIdx.x;
  if (d < bins) {
    int at = start;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * bins + d];
      cnt[w * bins + d] = at;
      at += c;
    }
  }
}
__device__ __forceinline__ int digit_total(const int* cnt, int bins) {
  int s = 0;
  const int d = threadIdx.x;
  if (d < bins)
    for (int w = 0; w < kSortWarps; ++w) s += cnt[w * bins + d];
  return s;
}

__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int load_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// N <= kCluster x kTile: one launch of one cluster.  Block c holds places [c cap, (c + 1) cap) as (key, position) pairs
// in shared memory; a pass counts its digits, reads the other blocks' counts, and stores each pair into the block of
// its new place.  The cluster's barrier separates the passes.  Bound by latency: 32768 tokens of 200000 25 us, 16384 of
// 32000 18 us.  (As two launches a pass over global memory the same
// sort of 32768 tokens took 75 us.)
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_sort_cluster_kernel(const I* __restrict__ ids, uint32_t* __restrict__ keys, int* __restrict__ order, int N,
                              int V, int padding, int cap, int passes, int bits, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint32_t sm[];
  const int bins = 1 << bits;
  uint2* buf[2] = {reinterpret_cast<uint2*>(sm), reinterpret_cast<uint2*>(sm) + cap};
  int* cnt = reinterpret_cast<int*>(sm + 4 * cap);      // [kSortWarps][bins]
  int* total = cnt + kSortWarps * bins;                 // [bins], read by the other blocks
  __shared__ int scratch[32];
  const int rank = (int)cluster_ctarank(), blocks = (int)cluster_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = max(0, min(cap, N - rank * cap));    // places this block holds
  const int own = (cap / kSortWarps + 31) / 32 * 32, first = warp * own;
  const uint32_t total_addr = smem_u32(total);
  for (int p = 0; p < passes; ++p) {
    uint2* in = buf[p & 1];
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    uint2 pair[kSteps];
    uint32_t d[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = first + k * 32 + lane;
      d[k] = 0xFFFFFFFFu;
      if (k * 32 < own && i < mine) {
        pair[k] = p == 0 ? make_uint2(token_key(ids, rank * cap + i, V, padding, status), (uint32_t)(rank * cap + i)) : in[i];
        d[k] = (pair[k].x >> (p * bits)) & (bins - 1u);
      }
    }
    rank_digits(cnt + warp * bins, d);
    __syncthreads();
    const int sum = digit_total(cnt, bins);
    if ((int)threadIdx.x < bins) total[threadIdx.x] = sum;
    __syncwarp();
    cluster_sync();
    int all = 0, ahead = 0;
    if ((int)threadIdx.x < bins) {
      int v[kCluster];   // all on their way before the first is waited for
#pragma unroll
      for (int c = 0; c < kCluster; ++c) v[c] = c < blocks ? load_cluster(mapa_shared(total_addr + 4 * threadIdx.x, c)) : 0;
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        all += v[c];
        if (c < rank) ahead += v[c];
      }
    }
    const int before = exclusive_scan(all, scratch);
    warp_places(cnt, bins, before + ahead);
    __syncthreads();
    const bool last = p + 1 == passes;
    const uint32_t out = smem_u32(buf[(p & 1) ^ 1]);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (d[k] == 0xFFFFFFFFu) continue;
      const int at = cnt[warp * bins + (d[k] & 0xFFFFu)] + (int)(d[k] >> 16);
      if (last) {
        keys[at] = pair[k].x;
        order[at] = (int)pair[k].y;
      } else {
        const int c = at / cap;
        store_cluster(mapa_shared(out + 8 * (at - c * cap), c), pair[k].x, pair[k].y);
      }
    }
    __syncwarp();
    cluster_sync();   // every pair is in place, and nobody still reads this pass's totals
  }
}

// The first pass reads the ids themselves; later ones the pairs of the pass before.
template <class I>
struct SortIn {
  const I* ids;             // first pass
  const uint32_t* keys;     // later passes
  const int* order;
  int V, padding;
  __device__ __forceinline__ uint32_t key(int64_t i, int* status) const {
    return ids ? token_key(ids, i, V, padding, status) : keys[i];
  }
  __device__ __forceinline__ int position(int64_t i) const { return ids ? (int)i : order[i]; }
};

// More tokens: digit counts of each tile of kTile positions, counts[tile][digit], ..
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_count_kernel(SortIn<I> in, int* __restrict__ counts, int N, int shift, int bits, int* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ int cnt[1 << kMaxBits];
  const int bins = 1 << bits;
  if ((int)threadIdx.x < bins) cnt[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, N - t0);
  for (int i = threadIdx.x; i < n; i += kSortThreads) atomicAdd(cnt + ((in.key(t0 + i, status) >> shift) & (bins - 1u)), 1);
  __syncthreads();
  if ((int)threadIdx.x < bins) counts[(int64_t)blockIdx.x * bins + threadIdx.x] = cnt[threadIdx.x];
}

// .. then each tile finds the places of its digits from all tiles' counts (smaller digits of every tile, then the same
// digit of earlier tiles) and scatters its pairs.
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_scatter_kernel(SortIn<I> in, const int* __restrict__ counts, uint32_t* __restrict__ keys,
                         int* __restrict__ order, int N, int shift, int bits) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint32_t sm[];
  const int bins = 1 << bits;
  int* cnt = reinterpret_cast<int*>(sm);
  __shared__ int scratch[32];
  const int tiles = gridDim.x, tile = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
  const int64_t t0 = (int64_t)tile * kTile;
  const int n = (int)min((int64_t)kTile, N - t0);
  uint32_t key[kSteps], d[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int i = warp * (kTile / kSortWarps) + k * 32 + lane;
    d[k] = 0xFFFFFFFFu;
    if (i < n) {
      key[k] = in.key(t0 + i, nullptr);   // the counting kernel has reported bad ids
      d[k] = (key[k] >> shift) & (bins - 1u);
    }
  }
  int all = 0, ahead = 0;
  if ((int)threadIdx.x < bins)
    for (int t = 0; t < tiles; ++t) {
      const int c = counts[(int64_t)t * bins + threadIdx.x];
      all += c;
      if (t < tile) ahead += c;
    }
  __syncthreads();
  rank_digits(cnt + warp * bins, d);
  __syncthreads();
  const int before = exclusive_scan(all, scratch);
  warp_places(cnt, bins, before + ahead);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if (d[k] == 0xFFFFFFFFu) continue;
    const int at = cnt[warp * bins + (d[k] & 0xFFFFu)] + (int)(d[k] >> 16);
    keys[at] = key[k];
    order[at] = in.position(t0 + warp * (kTile / kSortWarps) + k * 32 + lane);
  }
}

// ---------------------------------------------------------------------------
// Sums over the runs
// ---------------------------------------------------------------------------
// First index in [lo, hi) of the ascending keys whose key is >= v (hi if there is none).
__device__ __forceinline__ int lower_bound(const uint32_t* keys, int lo, int hi, uint32_t v) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The same over [0, n) by a whole warp: 32 probes a step, three steps for 32768 keys.
__device__ __forceinline__ int lower_bound_warp(const uint32_t* keys, int n, uint32_t v) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const uint32_t less = __ballot_sync(0xffffffffu, at < hi && keys[at] < v);
    if (!less) return lo;
    const int k = 31 - __clz(less);        // probes 0 .. k are below v
    const int next = lo + (k + 1) * step;
    lo = lo + k * step + 1;
    hi = min(hi, next);
  }
  return lo;
}

// a[k][j] += sum over i < n of dy[order[i]][c + k step + j] for the PACKS packs below H, in order, eight rows'
// loads at a time.
template <int PACKS, class T, int VEC>
__device__ __forceinline__ void add_rows(const T* __restrict__ dy, int64_t lddy, const int* order, int n, int c, int step,
                                         int H, float (&a)[PACKS][VEC]) {
  auto add = [&](const Pack<T, VEC> (&p)[PACKS]) {
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
      float f[VEC];
      unpack<T, VEC>(p[k], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[k][j] += f[j];
    }
  };
  auto load = [&](Pack<T, VEC> (&p)[PACKS], int i) {
    const T* row = dy + order[i] * lddy + c;
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
      p[k] = zero_pack<T, VEC>();
      if (k == 0 || c + k * step < H) p[k] = load_pack<T, VEC>(row + k * step);
    }
  };
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    Pack<T, VEC> p[8][PACKS];
#pragma unroll
    for (int r = 0; r < 8; ++r) load(p[r], i + r);
#pragma unroll
    for (int r = 0; r < 8; ++r) add(p[r]);
  }
#pragma unroll 4
  for (; i < n; ++i) {
    Pack<T, VEC> p[PACKS];
    load(p, i);
    add(p);
  }
}
// Packs a thread sums at a time: single elements need more of them in flight.
template <int VEC>
constexpr int kPacks = VEC == 1 ? 4 : 1;
template <int VEC>
constexpr int kAddPacks = VEC == 1 ? 4 : 2;

// Piece b covers sorted places [kPiece b, kPiece (b + 1)).  A run longer than kPiece that meets the piece holds
// its first place or its last (32768 tokens of 4096 columns: 26 us): part[b][0] is the sum over the places of the run that holds the first,
// part[b][1] over those of a run that starts inside and holds the last.  Only long runs' sums are written.
template <class T, int VEC>
__global__ void __launch_bounds__(256) embed_piece_kernel(const uint32_t* __restrict__ keys,
                                                         const int* __restrict__ order, const T* __restrict__ dy,
                                                         int64_t lddy, float* __restrict__ part, int N, int V, int H) {
  pdl_wait();
  pdl_trigger();
  __shared__ int edge[4];   // run of the first place: start, end; run of the last place: start, end
  __shared__ int places[kPiece];
  const int p0 = blockIdx.x * kPiece, p1 = min(N, p0 + kPiece);
  const int warp = threadIdx.x >> 5;
  if (warp < 4) {
    const uint32_t v = keys[warp < 2 ? p0 : p1 - 1];
    const int at = v >= (uint32_t)V ? 0 : lower_bound_warp(keys, N, v + (warp & 1));
    if ((threadIdx.x & 31) == 0) edge[warp] = at;
  } else if ((int)threadIdx.x - 128 < p1 - p0) {
    places[threadIdx.x - 128] = order[p0 + threadIdx.x - 128];
  }
  __syncthreads();
  const int s0 = edge[0], e0 = edge[1], s1 = edge[2], e1 = edge[3];
  for (int which = 0; which < 2; ++which) {
    const int s = which ? s1 : s0, e = which ? e1 : e0;
    if (e - s <= kPiece || (which && s <= p0)) continue;   // short, or the first place's run again
    const int a0 = max(s, p0), a1 = min(e, p1);
    float* out = part + ((int64_t)blockIdx.x * 2 + which) * H;
    constexpr int PACKS = kPacks<VEC>;
    const int step = 256 * VEC;
    for (int c = (blockIdx.y * PACKS * 256 + threadIdx.x) * VEC; c < H; c += gridDim.y * PACKS * step) {
      float a[PACKS][VEC];
#pragma unroll
      for (int k = 0; k < PACKS; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[k][j] = 0.0f;
      add_rows<PACKS, T, VEC>(dy, lddy, places + (a0 - p0), a1 - a0, c, step, H, a);
#pragma unroll
      for (int k = 0; k < PACKS; ++k)
        if (c + k * step < H) {
          Pack<float, VEC> o;
#pragma unroll
          for (int j = 0; j < VEC; ++j) o.v[j] = a[k][j];
          store_pack<float, VEC>(out + c + k * step, o);
        }
    }
  }
}

// The row of run [s, e): its sum (of the tokens in `order`, from s on, or of its pieces), scaled and stored or added.
// `tpr` threads; thread t takes the packs t, t + tpr, .., PACKS at a time.  Four floats a pack: a warp's store is one
// run of 512 bytes.
template <int PACKS, bool ADD, class T, int VEC>
__device__ __forceinline__ void embed_row(const int* order, const T* __restrict__ dy, int64_t lddy,
                                          const float* __restrict__ part, float* __restrict__ row, int s, int e, int H,
                                          int t, int tpr, float scale) {
  const int step = tpr * VEC;
  for (int c = t * VEC; c < H; c += PACKS * step) {
    Pack<float, VEC> o[PACKS];
    float a[PACKS][VEC];
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
      if (ADD && c + k * step < H) o[k] = load_pack<float, VEC>(row + c + k * step);   // while the tokens are summed
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[k][j] = 0.0f;
    }
    if (e - s <= kPiece) {
      add_rows<PACKS, T, VEC>(dy, lddy, order, e - s, c, step, H, a);
    } else {
#pragma unroll 4
      for (int b = s / kPiece; b <= (e - 1) / kPiece; ++b) {
        const float* from = part + ((int64_t)b * 2 + (b * kPiece < s ? 1 : 0)) * H + c;
#pragma unroll
        for (int k = 0; k < PACKS; ++k)
          if (k == 0 || c + k * step < H) {
            const Pack<float, VEC> p = load_pack<float, VEC>(from + k * step);
#pragma unroll
            for (int j = 0; j < VEC; ++j) a[k][j] += p.v[j];
          }
      }
    }
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
      if (k > 0 && c + k * step >= H) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[k].v[j] = ADD ? fmaf(scale, a[k][j], o[k].v[j]) : scale * a[k][j];
      if constexpr (VEC == 4) {   // written once and not read again here: first to leave L2
        __stcs(reinterpret_cast<float4*>(row + c + k * step), make_float4(o[k].v[0], o[k].v[1], o[k].v[2], o[k].v[3]));
      } else {
        store_pack<float, VEC>(row + c + k * step, o[k]);
      }
    }
  }
}

// A dense gradient: block b owns table rows [R b, R (b + 1)).  Bound by the gradient's stores: 200000 x 4096 from 32768
// tokens 512 us, 6.6 TB/s.
template <class T, int VEC>
__global__ void __launch_bounds__(256, 4) embed_rows_kernel(const uint32_t* __restrict__ keys,
                                                        const int* __restrict__ order, const T* __restrict__ dy,
                                                        int64_t lddy, const float* __restrict__ part,
                                                        float* __restrict__ dW, int N, int V, int H, int R, int tpr,
                                                        float scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ int first[257];   // first[r]: first place of row v0 + r; R <= 256
  const int64_t v0 = (int64_t)blockIdx.x * R;
  const int rows = (int)min((int64_t)R, V - v0);
  if (threadIdx.x < 64) {
    const int r = threadIdx.x < 32 ? 0 : rows;
    const int at = lower_bound_warp(keys, N, (uint32_t)(v0 + r));
    if ((threadIdx.x & 31) == 0) first[r] = at;
  }
  __syncthreads();
  const int lo = first[0], hi = first[rows];
  if (threadIdx.x > 0 && (int)threadIdx.x < rows) first[threadIdx.x] = lower_bound(keys, lo, hi, (uint32_t)(v0 + threadIdx.x));
  __syncthreads();
  for (int r = threadIdx.x / tpr; r < rows; r += 256 / tpr)
    embed_row<kPacks<VEC>, false, T, VEC>(order + first[r], dy, lddy, part, dW + (v0 + r) * H, first[r], first[r + 1], H, threadIdx.x & (tpr - 1),
                             tpr, scale);
}

// Only the rows of tokens that occur: added into a gradient (ADD), or stored over zeros.  Block b takes the runs that start at the sorted places
// [kHeads b, kHeads (b + 1)), which it sees by itself (searching for its rows as the dense form does took
// 52 us for 16384 tokens of 2048 columns, this 44).
constexpr int kHeads = 8;
template <class T, int VEC, bool ADD>
__global__ void __launch_bounds__(256) embed_runs_kernel(const uint32_t* __restrict__ keys,
                                                       const int* __restrict__ order, const T* __restrict__ dy,
                                                       int64_t lddy, const float* __restrict__ part,
                                                       float* __restrict__ dW, int N, int V, int H, int tpr,
                                                       float scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ int run_s[kHeads], run_e[kHeads], run_v[kHeads], runs;
  __shared__ int places[kHeads][kPiece];
  const int p0 = blockIdx.x * kHeads;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, p = p0 + lane;
    const uint32_t v = p < N ? keys[p] : 0xFFFFFFFFu;
    uint32_t before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = p > 0 ? keys[p - 1] : 0xFFFFFFFEu;
    const bool head = v != before;                             // the place past the last is one too
    const uint32_t heads = __ballot_sync(0xffffffffu, head);
    const bool mine = head && lane < kHeads && v < (uint32_t)V;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    if (mine) {
      const uint32_t after = lane == 31 ? 0u : heads >> (lane + 1);
      const int i = __popc(all & ((1u << lane) - 1u));
      run_s[i] = p;
      run_e[i] = after ? p + __ffs(after) : lower_bound(keys, min(N, p0 + 32), N, v + 1);
      run_v[i] = (int)v;
    }
    if (lane == 0) runs = __popc(all);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < runs * kPiece; i += 256) {
    const int r = i / kPiece, k = i % kPiece;
    if (run_s[r] + k < run_e[r]) places[r][k] = order[run_s[r] + k];
  }
  __syncthreads();
  for (int r = threadIdx.x / tpr; r < runs; r += 256 / tpr)
    embed_row<kAddPacks<VEC>, ADD, T, VEC>(places[r], dy, lddy, part, dW + (int64_t)run_v[r] * H, run_s[r], run_e[r], H,
                            threadIdx.x & (tpr - 1), tpr, scale);
}

// out[0 .. n) = 0, from 16-byte boundary to 16-byte boundary with single elements at the ends.  late: it runs beside the
// kernel before it (the sort, which does not touch `out`, has waited for everything before it and only then lets this
// one start) and waits for that kernel at its end, so that what follows sees both complete.
__global__ void __launch_bounds__(256) embed_clear_kernel(float* __restrict__ out, int64_t n, bool late) {
  if (!late) {
    pdl_wait();
    pdl_trigger();
  }
  const int64_t head = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / 4);
  const int64_t packs = (n - head) / 4, i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  float4* body = reinterpret_cast<float4*>(out + head);
  for (int64_t i = i0; i < packs; i += (int64_t)gridDim.x * 256) __stcs(body + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  if (i0 < head) out[i0] = 0.0f;
  const int64_t tail = head + packs * 4 + i0;
  if (tail < n && i0 < 4) out[tail] = 0.0f;
  if (late) pdl_wait();
}

struct EmbedLayout {
  int tiles, passes, bits;
  size_t keys[2], order[2], counts, part, total;
};

EmbedLayout embed_layout(const moe_embed_config& c) {
  EmbedLayout L = {};
  L.tiles = (int)(((int64_t)c.N + kTile - 1) / kTile);
  int key_bits = 1;
  while (key_bits < 31 && (1u << key_bits) <= (uint32_t)c.V) ++key_bits;   // keys 0 .. V
  L.passes = (key_bits + kMaxBits - 1) / kMaxBits;
  L.bits = (key_bits + L.passes - 1) / L.passes;
  size_t o = align256(sizeof(WsHeader));
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    L.keys[i] = take((size_t)c.N * 4);
    L.order[i] = take((size_t)c.N * 4);
  }
  L.counts = take((size_t)L.tiles * (1u << L.bits) * 4);
  L.part = take((size_t)(((int64_t)c.N + kPiece - 1) / kPiece) * 2 * c.H * 4);
  L.total = o;
  return L;
}

int embed_validate(const moe_embed_config* c) {
  if (!c || c->N < 0 || c->V < 0 || c->H < 0 || c->padding_idx < -1 || !std::isfinite(c->scale))
    return MOE_ERR_INVALID_ARG;
  if (c->V < 1 || c->H < 1 || c->H > (1 << 20) || c->N > (1 << 24) || c->V >= (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

bool known_index(int t) { return t == MOE_INDEX_I32 || t == MOE_INDEX_I64; }

template <class F>
cudaError_t with_index(int id_type, F&& f) {
  return id_type == MOE_INDEX_I64 ? f(int64_t{}) : f(int32_t{});
}

template <class Kern>
cudaError_t allow_smem(Kern kern, size_t bytes) {
  return bytes > 48 * 1024
             ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
             : cudaSuccess;
}

// Sorts the positions by id; the sorted pairs end in keys / order of buffer *at.
template <class I>
cudaError_t sort_tokens(const moe_embed_config& c, const EmbedLayout& L, const I* ids, uint8_t* w, int* at,
                        cudaStream_t s) {
  int* status = reinterpret_cast<int*>(w);
  auto keys = [&](int i) { return reinterpret_cast<uint32_t*>(w + L.keys[i]); };
  auto order = [&](int i) { return reinterpret_cast<int*>(w + L.order[i]); };
  const size_t cnt = (size_t)kSortWarps * (1u << L.bits) * 4;
  if (c.N <= kCluster * kTile) {
    // a block for each 2048 tokens, up to the cluster's 8; `cap` a multiple of the warps' steps
    int blocks = 1;
    while (blocks < kCluster && c.N > blocks * 2048) blocks *= 2;
    const int cap = ((c.N + blocks - 1) / blocks + 1023) / 1024 * 1024;
    const size_t smem = (size_t)cap * 16 + cnt + (size_t)(1u << L.bits) * 4;   // at most 194 KB
    auto kern = embed_sort_cluster_kernel<I>;
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    *at = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_chain_mode() >= MOE_CHAIN_EARLY ? 2 : 1;   // the cluster attribute comes first
    e = cudaLaunchKernelEx(&cfg, kern, ids, keys(0), order(0), c.N, c.V, c.padding_idx, cap, L.passes, L.bits, status);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  const size_t smem = cnt;
  cudaError_t e = allow_smem(embed_scatter_kernel<I>, smem);
  int* counts = reinterpret_cast<int*>(w + L.counts);
  for (int p = 0; p < L.passes && e == cudaSuccess; ++p) {
    SortIn<I> in = {p == 0 ? ids : nullptr, keys((p + 1) & 1), order((p + 1) & 1), c.V, c.padding_idx};
    e = launch_pdl(embed_count_kernel<I>, dim3(L.tiles), dim3(kSortThreads), 0, s, in, counts, c.N, p * L.bits,
                   L.bits, status);
    if (e == cudaSuccess)
      e = launch_pdl(embed_scatter_kernel<I>, dim3(L.tiles), dim3(kSortThreads), smem, s, in,
                     static_cast<const int*>(counts), keys(p & 1), order(p & 1), c.N, p * L.bits, L.bits);
    *at = p & 1;
  }
  return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_embed_workspace_bytes(const moe_embed_config* cfg, size_t* fwd_bytes, size_t* bwd_bytes) {
  const int v = embed_validate(cfg);
  if (v != MOE_OK) return v;
  if (fwd_bytes) *fwd_bytes = sizeof(WsHeader);
  if (bwd_bytes) *bwd_bytes = embed_layout(*cfg).total;
  return MOE_OK;
}

int moe_embed_forward(const moe_embed_config* cfg, const void* ids, int32_t id_type, const void* table, void* y,
                      int32_t type, void* ws, size_t ws_bytes, void* stream) {
  const int v = embed_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_embed_config& c = *cfg;
  if (!known_type(type) || !known_index(id_type) || !ws || !aligned_to(ws, 16)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (c.N == 0) return MOE_OK;
  const size_t ts = type_size(type), is = id_type == MOE_INDEX_I64 ? 8 : 4;
  if (!ids || !table || !y || !aligned_to(ids, is) || !aligned_to(table, ts) || !aligned_to(y, ts))
    return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  return timed_launch(MOE_K_EMBED_FWD, "embedding", s, [&] {
    return with_type(type, [&](auto tv) {
      using T = decltype(tv);
      return with_index(id_type, [&](auto iv) {
        using I = decltype(iv);
        auto go = [&](auto vv) {
          constexpr int VEC = decltype(vv)::value;
          constexpr int kRow = 32 * kFwdPer<VEC> * VEC;
          const int pieces = (c.H + kRow - 1) / kRow;
          const int64_t units = (int64_t)c.N * pieces;
          return launch_pdl(embed_fwd_kernel<T, I, VEC>, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, s,
                            static_cast<const I*>(ids), static_cast<const T*>(table), static_cast<T*>(y), c.N, c.V,
                            c.H, pieces, c.scale, status);
        };
        constexpr int V16 = 16 / sizeof(T);
        if (c.H % V16 == 0 && aligned_to(table, 16) && aligned_to(y, 16)) return go(std::integral_constant<int, V16>{});
        return go(std::integral_constant<int, 1>{});
      });
    });
  });
}

int moe_embed_backward(const moe_embed_config* cfg, const void* ids, int32_t id_type, const void* dy, int64_t lddy,
                       int32_t type, float* dW, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  int v = embed_validate(cfg);
  if (v != MOE_OK) return v;
  const moe_embed_config& c = *cfg;
  if (!known_type(type) || !known_index(id_type) || lddy < c.H || !ws || !aligned_to(ws, 16) || !dW ||
      !aligned_to(dW, 4) || (accumulate != 0 && accumulate != 1))
    return MOE_ERR_INVALID_ARG;
  const EmbedLayout L = embed_layout(c);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.N == 0) {
    if (accumulate) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(dW, 0, (size_t)c.V * c.H * 4, s);
    return e == cudaSuccess ? MOE_OK : record_cuda_error(e, "clear dW");
  }
  const size_t ts = type_size(type), is = id_type == MOE_INDEX_I64 ? 8 : 4;
  if (!ids || !dy || !aligned_to(ids, is) || !aligned_to(dy, ts)) return MOE_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  int at = 0;
  v = timed_launch(MOE_K_EMBED_SORT, "sort tokens", s, [&] {
    return with_index(id_type, [&](auto iv) {
      return sort_tokens(c, L, static_cast<const decltype(iv)*>(ids), w, &at, s);
    });
  });
  if (v != MOE_OK) return v;
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(w + L.keys[at]);
  const int* order = reinterpret_cast<const int*>(w + L.order[at]);
  float* part = reinterpret_cast<float*>(w + L.part);
  return timed_launch(MOE_K_EMBED_BWD, "embedding gradient", s, [&] {
    return with_type(type, [&](auto tv) {
      using T = decltype(tv);
      auto go = [&](auto vv) {
        constexpr int VEC = decltype(vv)::value;
        const T* g = static_cast<const T*>(dy);
        // Rows that do not start on 16 bytes are cleared all at once, 16 bytes a store, and those that occur stored after.
        const bool clear = VEC == 1 && !accumulate;
        if (clear) {
          const cudaError_t e = launch_pdl(embed_clear_kernel, dim3(device_sm_count() * 8), dim3(256), 0, s, dW,
                                           (int64_t)c.V * c.H, launch_chain_mode() >= MOE_CHAIN_LATE);
          if (e != cudaSuccess) return e;
        }
        if (c.N > kPiece) {
          const dim3 grid((c.N + kPiece - 1) / kPiece, std::min(8, (c.H + 256 * VEC * kPacks<VEC> - 1) / (256 * VEC * kPacks<VEC>)));
          const cudaError_t e = launch_pdl(embed_piece_kernel<T, VEC>, grid, dim3(256), 0, s, keys, order, g, lddy,
                                           part, c.N, c.V, c.H);
          if (e != cudaSuccess) return e;
        }
        const float* sums = part;
        int tpr = 1;
        auto threads = [&](int packs) {   // threads a row: a power of two
          while (tpr < 256 && tpr * VEC * packs < c.H) tpr *= 2;
          return tpr;
        };
        const dim3 by_run((c.N + kHeads - 1) / kHeads);
        if (accumulate)
          return launch_pdl(embed_runs_kernel<T, VEC, true>, by_run, dim3(256), 0, s, keys, order, g, lddy, sums, dW, c.N,
                            c.V, c.H, threads(kAddPacks<VEC>), c.scale);
        if constexpr (VEC == 1) {
          return launch_pdl(embed_runs_kernel<T, VEC, false>, by_run, dim3(256), 0, s, keys, order, g, lddy, sums, dW,
                            c.N, c.V, c.H, threads(kAddPacks<VEC>), c.scale);
        } else {
          // rows a block: about 128 KB of gradient, so that the two searches of a block are paid for
          const int R = (int)std::min<int64_t>(256, std::max<int64_t>(1, 32768 / c.H));
          const dim3 grid((unsigned)(((int64_t)c.V + R - 1) / R));
          return launch_pdl(embed_rows_kernel<T, VEC>, grid, dim3(256), 0, s, keys, order, g, lddy, sums, dW, c.N, c.V,
                            c.H, R, threads(kPacks<VEC>), c.scale);
        }
      };
      if (c.H % 4 == 0 && lddy % 4 == 0 && aligned_to(dy, 4 * ts) && aligned_to(dW, 16))
        return go(std::integral_constant<int, 4>{});
      return go(std::integral_constant<int, 1>{});
    });
  });
}

}  // extern "C"

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

constexpr int kPiece = 64;          // positions of a piece of a long run
constexpr int kSortThreads = 512;   // 16 warps
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTile = 8192;         // positions sorted by one block
constexpr int kMaxBits = 10;        // bits of a digit: kSortWarps x 1024 counters are 64 KB

// ---------------------------------------------------------------------------
// Forward: one warp a 16 x 32-byte piece of a row, so a short batch still spreads over the SMs.
// ---------------------------------------------------------------------------
template <class T, class I, int VEC>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const I* __restrict__ ids, const T* __restrict__ table,
                                                       T* __restrict__ y, int N, int V, int H, int pieces,
                                                       float scale, int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t n = unit / pieces;
  const int c0 = (int)(unit - n * pieces) * (128 * VEC);
  if (n >= N) return;
  const int64_t id = ids[n];
  const bool ok = id >= 0 && id < V;
  if (!ok && c0 == 0 && lane == 0) report(status, MOE_ERR_DEVICE_CHECK, 501);
  const T* src = table + (ok ? id : 0) * H;
  T* dst = y + n * H;
  Pack<T, VEC> p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + (i * 32 + lane) * VEC;
    if (c < H) p[i] = *reinterpret_cast<const Pack<T, VEC>*>(src + c);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + (i * 32 + lane) * VEC;
    if (c >= H) continue;
    if (!ok || scale != 1.0f) {
      float f[VEC];
      unpack<T, VEC>(p[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = ok ? f[j] * scale : 0.0f;
      p[i] = pack<T, VEC>(f);
    }
    *reinterpret_cast<Pack<T, VEC>*>(dst + c) = p[i];
  }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (id, position)
// ---------------------------------------------------------------------------
// A block sorts a tile of kTile positions by one digit: warp w owns the tile's w-th consecutive
// kTile / kSortWarps positions, 32 at a time; lanes with the same digit rank themselves by lane, so equal
// digits keep their order.  cnt: [kSortWarps][bins] in shared memory, or the counters of a pass.
template <class F>
__device__ __forceinline__ void for_own_positions(int n, F&& f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kOwn = kTile / kSortWarps;
  const int end = min(n, (warp + 1) * kOwn);
  for (int b = warp * kOwn; b < end; b += 32) f(b + lane, b + lane < end);   // the whole warp takes part
}

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

// cnt[w][d] += positions of warp w with digit d.
template <class K>
__device__ __forceinline__ void count_digits(int* cnt, int bins, int n, K&& digit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for_own_positions(n, [&](int i, bool in) {
    const uint32_t d = in ? digit(i) : 0xFFFFFFFFu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    if (in && lane == __ffs(peers) - 1) cnt[warp * bins + d] += __popc(peers);
    __syncwarp();
  });
}

// Turns cnt[w][d] into the first place of warp w's digit d: the places of smaller digits, then those of the
// same digit in earlier warps.  base(d): where digit d starts, given the tile's own count in front of it.
template <class B>
__device__ __forceinline__ void digit_places(int* cnt, int* scratch, int bins, B&& base) {
  // thread t owns digits 2t and 2t + 1 (bins <= 1024)
  int sum[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = threadIdx.x * 2 + k;
    if (d < bins)
      for (int w = 0; w < kSortWarps; ++w) sum[k] += cnt[w * bins + d];
  }
  // exclusive scan of the pairs over the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = sum[0] + sum[1];
  const int own = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int before = x - own;
  for (int w = 0; w < warp; ++w) before += scratch[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = threadIdx.x * 2 + k;
    if (d < bins) {
      int at = base(d, before);
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * bins + d];
        cnt[w * bins + d] = at;
        at += c;
      }
    }
    before += sum[k];
  }
  __syncthreads();
}

// Hands each position of the tile its place: put(i, place).
template <class K, class F>
__device__ __forceinline__ void place_all(int* cnt, int bins, int n, K&& digit, F&& put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for_own_positions(n, [&](int i, bool in) {
    const uint32_t d = in ? digit(i) : 0xFFFFFFFFu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    int at = 0;
    if (in) at = cnt[warp * bins + d] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == __ffs(peers) - 1) cnt[warp * bins + d] += __popc(peers);
    __syncwarp();
    if (in) put(i, at);
  });
}

// N <= kTile: all passes in one block.  Keys and positions stay in shared memory between passes.
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_sort_one_kernel(const I* __restrict__ ids, uint32_t* __restrict__ keys, int* __restrict__ order, int N, int V,
                          int padding, int passes, int bits, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t sm[];
  uint32_t* key[2] = {sm, sm + 2 * kTile};            // key[p][i], position key[p][kTile + i]
  int* cnt = reinterpret_cast<int*>(sm + 4 * kTile);
  __shared__ int scratch[32];
  const int bins = 1 << bits;
  for (int i = threadIdx.x; i < N; i += kSortThreads) {
    key[0][i] = token_key(ids, i, V, padding, status);
    key[0][kTile + i] = i;
  }
  for (int p = 0; p < passes; ++p) {
    uint32_t *in = key[p & 1], *out = key[(p & 1) ^ 1];
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    auto digit = [&](int i) { return (in[i] >> (p * bits)) & (bins - 1u); };
    count_digits(cnt, bins, N, digit);
    __syncthreads();
    digit_places(cnt, scratch, bins, [](int, int before) { return before; });
    place_all(cnt, bins, N, digit, [&](int i, int at) {
      out[at] = in[i];
      out[kTile + at] = in[kTile + i];
    });
    __syncthreads();
  }
  const uint32_t* done = key[passes & 1];
  for (int i = threadIdx.x; i < N; i += kSortThreads) {
    keys[i] = done[i];
    order[i] = (int)done[kTile + i];
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

// Digit counts of each tile: counts[tile][digit].
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_count_kernel(SortIn<I> in, int* __restrict__ counts, int N, int shift, int bits, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t sm[];
  int* cnt = reinterpret_cast<int*>(sm);
  const int bins = 1 << bits;
  for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, N - t0);
  count_digits(cnt, bins, n, [&](int i) { return (in.key(t0 + i, status) >> shift) & (bins - 1u); });
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) {
    int s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += cnt[w * bins + d];
    counts[(int64_t)blockIdx.x * bins + d] = s;
  }
}

// Each tile finds the places of its digits from all tiles' counts (smaller digits of every tile, then the same
// digit of earlier tiles) and scatters its pairs.
template <class I>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_scatter_kernel(SortIn<I> in, const int* __restrict__ counts, uint32_t* __restrict__ keys,
                         int* __restrict__ order, int N, int shift, int bits) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t sm[];
  const int bins = 1 << bits;
  int* cnt = reinterpret_cast<int*>(sm);
  int* start = cnt + kSortWarps * bins;     // this tile's first place of each digit
  __shared__ int scratch[32], total_before[32];
  const int tiles = gridDim.x, mine = blockIdx.x;
  for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
  // start[d] = sum over d' < d of all tiles' counts + sum over earlier tiles of counts[d]
  int sum[2] = {0, 0}, ahead[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = threadIdx.x * 2 + k;
    if (d < bins)
      for (int t = 0; t < tiles; ++t) {
        const int c = counts[(int64_t)t * bins + d];
        sum[k] += c;
        if (t < mine) ahead[k] += c;
      }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = sum[0] + sum[1];
  const int own = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) total_before[warp] = x;
  __syncthreads();
  int before = x - own;
  for (int w = 0; w < warp; ++w) before += total_before[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = threadIdx.x * 2 + k;
    if (d < bins) start[d] = before + ahead[k];
    before += sum[k];
  }
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, N - t0);
  // (the counting kernel has reported bad ids)
  auto digit = [&](int i) { return (in.key(t0 + i, nullptr) >> shift) & (bins - 1u); };
  count_digits(cnt, bins, n, digit);
  __syncthreads();
  digit_places(cnt, scratch, bins, [&](int d, int) { return start[d]; });
  place_all(cnt, bins, n, digit, [&](int i, int at) {
    keys[at] = in.key(t0 + i, nullptr);
    order[at] = in.position(t0 + i);
  });
}

// ---------------------------------------------------------------------------
// Sums over the runs
// ---------------------------------------------------------------------------
// First index in [lo, hi) of the ascending keys whose key is >= v.
__device__ __forceinline__ int lower_bound(const uint32_t* keys, int lo, int hi, uint32_t v) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// a[j] += sum over sorted places [s, e) of dy[order[place]][c + j], in order, four rows' loads at a time.
template <class T, int VEC>
__device__ __forceinline__ void add_rows(const T* __restrict__ dy, int64_t lddy, const int* __restrict__ order, int s,
                                         int e, int c, float (&a)[VEC]) {
  int i = s;
  for (; i + 4 <= e; i += 4) {
    Pack<T, VEC> p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = *reinterpret_cast<const Pack<T, VEC>*>(dy + order[i + k] * lddy + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[VEC];
      unpack<T, VEC>(p[k], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[j] += f[j];
    }
  }
  for (; i < e; ++i) {
    const Pack<T, VEC> p = *reinterpret_cast<const Pack<T, VEC>*>(dy + order[i] * lddy + c);
    float f[VEC];
    unpack<T, VEC>(p, f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] += f[j];
  }
}

// Piece b covers sorted places [kPiece b, kPiece (b + 1)).  A run longer than kPiece that meets the piece holds
// its first place or its last: part[b][0] is the sum over the places of the run that holds the first,
// part[b][1] over those of a run that starts inside and holds the last.  Only long runs' sums are written.
template <class T, int VEC>
__global__ void __launch_bounds__(256) embed_piece_kernel(const uint32_t* __restrict__ keys,
                                                         const int* __restrict__ order, const T* __restrict__ dy,
                                                         int64_t lddy, float* __restrict__ part, int N, int V, int H) {
  pdl_wait();
  pdl_trigger();
  __shared__ int edge[4];   // run of the first place: start, end; run of the last place: start, end
  const int p0 = blockIdx.x * kPiece, p1 = min(N, p0 + kPiece);
  if (threadIdx.x < 4) {
    const uint32_t v = keys[threadIdx.x < 2 ? p0 : p1 - 1];
    edge[threadIdx.x] = v >= (uint32_t)V ? 0 : lower_bound(keys, 0, N, v + (threadIdx.x & 1));
  }
  __syncthreads();
  const int s0 = edge[0], e0 = edge[1], s1 = edge[2], e1 = edge[3];
  for (int which = 0; which < 2; ++which) {
    const int s = which ? s1 : s0, e = which ? e1 : e0;
    if (e - s <= kPiece || (which && s <= p0)) continue;   // short, or the first place's run again
    const int a0 = max(s, p0), a1 = min(e, p1);
    float* out = part + ((int64_t)blockIdx.x * 2 + which) * H;
    for (int c = (blockIdx.y * 256 + threadIdx.x) * VEC; c < H; c += gridDim.y * 256 * VEC) {
      float a[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[j] = 0.0f;
      add_rows<T, VEC>(dy, lddy, order, a0, a1, c, a);
#pragma unroll
      for (int j = 0; j < VEC; ++j) out[c + j] = a[j];
    }
  }
}

// Block b owns table rows [R b, R (b + 1)); its threads walk over (row, pack of columns).
template <class T, int VEC, bool ADD>
__global__ void __launch_bounds__(256) embed_rows_kernel(const uint32_t* __restrict__ keys,
                                                        const int* __restrict__ order, const T* __restrict__ dy,
                                                        int64_t lddy, const float* __restrict__ part,
                                                        float* __restrict__ dW, int N, int V, int H, int R,
                                                        float scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ int first[257];   // first[r]: first place of row v0 + r; R <= 256
  const int64_t v0 = (int64_t)blockIdx.x * R;
  const int rows = (int)min((int64_t)R, V - v0);
  if (threadIdx.x < 2) first[threadIdx.x ? rows : 0] = lower_bound(keys, 0, N, (uint32_t)(v0 + (threadIdx.x ? rows : 0)));
  __syncthreads();
  const int lo = first[0], hi = first[rows];
  if (ADD && lo == hi) return;
  if (threadIdx.x > 0 && (int)threadIdx.x < rows) first[threadIdx.x] = lower_bound(keys, lo, hi, (uint32_t)(v0 + threadIdx.x));
  __syncthreads();
  const int packs = H / VEC;
  for (int u = threadIdx.x; u < rows * packs; u += 256) {
    const int r = u / packs, c = (u - r * packs) * VEC;
    const int s = first[r], e = first[r + 1];
    if (ADD && s == e) continue;
    float a[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] = 0.0f;
    if (e - s <= kPiece) {
      add_rows<T, VEC>(dy, lddy, order, s, e, c, a);
    } else {
      for (int b = s / kPiece; b <= (e - 1) / kPiece; ++b) {
        const float* p = part + ((int64_t)b * 2 + (b * kPiece < s ? 1 : 0)) * H + c;
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] += p[j];
      }
    }
    float* out = dW + (v0 + r) * H + c;
    using Out = Pack<float, VEC>;
    Out o;
    if (ADD) {
      o = *reinterpret_cast<const Out*>(out);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = fmaf(scale, a[j], o.v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = scale * a[j];
    }
    *reinterpret_cast<Out*>(out) = o;
  }
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
  if (L.tiles == 1) {
    const size_t smem = (size_t)4 * kTile * 4 + cnt;   // at most 192 KB
    const cudaError_t e = allow_smem(embed_sort_one_kernel<I>, smem);
    if (e != cudaSuccess) return e;
    *at = 0;
    return launch_pdl(embed_sort_one_kernel<I>, dim3(1), dim3(kSortThreads), smem, s, ids, keys(0), order(0), c.N, c.V,
                      c.padding_idx, L.passes, L.bits, status);
  }
  const size_t smem = cnt + (size_t)(1u << L.bits) * 4;
  cudaError_t e = allow_smem(embed_count_kernel<I>, smem);
  if (e == cudaSuccess) e = allow_smem(embed_scatter_kernel<I>, smem);
  int* counts = reinterpret_cast<int*>(w + L.counts);
  for (int p = 0; p < L.passes && e == cudaSuccess; ++p) {
    SortIn<I> in = {p == 0 ? ids : nullptr, keys((p + 1) & 1), order((p + 1) & 1), c.V, c.padding_idx};
    e = launch_pdl(embed_count_kernel<I>, dim3(L.tiles), dim3(kSortThreads), smem, s, in, counts, c.N, p * L.bits,
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
          const int pieces = (c.H + 128 * VEC - 1) / (128 * VEC);
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
        if (c.N > kPiece) {
          const dim3 grid((c.N + kPiece - 1) / kPiece, std::min(8, (c.H + 256 * VEC - 1) / (256 * VEC)));
          const cudaError_t e = launch_pdl(embed_piece_kernel<T, VEC>, grid, dim3(256), 0, s, keys, order, g, lddy,
                                           part, c.N, c.V, c.H);
          if (e != cudaSuccess) return e;
        }
        // rows a block: about 64 KB of gradient, so that the two searches of a block are paid for
        const int R = (int)std::min<int64_t>(256, std::max<int64_t>(1, 16384 / c.H));
        const dim3 grid((unsigned)(((int64_t)c.V + R - 1) / R));
        if (accumulate)
          return launch_pdl(embed_rows_kernel<T, VEC, true>, grid, dim3(256), 0, s, keys, order, g, lddy,
                            static_cast<const float*>(part), dW, c.N, c.V, c.H, R, c.scale);
        return launch_pdl(embed_rows_kernel<T, VEC, false>, grid, dim3(256), 0, s, keys, order, g, lddy,
                          static_cast<const float*>(part), dW, c.N, c.V, c.H, R, c.scale);
      };
      constexpr int V16 = 16 / sizeof(T);
      if (c.H % V16 == 0 && lddy % V16 == 0 && aligned_to(dy, 16) && aligned_to(dW, 16))
        return go(std::integral_constant<int, V16>{});
      return go(std::integral_constant<int, 1>{});
    });
  });
}

}  // extern "C"

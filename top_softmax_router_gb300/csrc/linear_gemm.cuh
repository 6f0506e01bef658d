// Products grouped by expert on CTA pairs, for include/moe_linear.h:
//
//   LIN_Y   y  [rows of e][O] = x  [rows of e][K] W[e]^T          operands with K along the row
//   LIN_DX  dx [rows of e][K] = dy [rows of e][O] W[e]            W with its rows along the contraction
//   LIN_DW  dW [e] [O][K]     = dy [rows of e]^T x [rows of e]    both so; the contraction is as long as e has rows
//
// bf16 (tcgen05 kind::f16) or, MX, e4m3 codes with a power-of-two scale for each block of 128 (kind::mxf8f6f4, which
// multiplies each product by two e8m0 scales that lie in tensor memory).
//
// A cluster of two CTAs owns a 256 x 256 tile of one expert: each loads its 128 rows of A and half of the tile's B, 128
// bytes of the contraction at a time (64 bf16 or 128 codes; 32 KB a stage, 6 stages); the even CTA issues the MMAs
// (M = 256, N = 256, 32 bytes of the contraction each).  The tiles of the experts follow from the offsets, which every
// CTA scans for itself, so nothing is read back to the host and no other launch is needed.
//
// Few tiles (one token for each sequence, say) are shared out along the contraction: S shares of a tile go to S clusters,
// which leave their sums in the workspace; the last warp to finish a piece of 32 rows x 128 columns adds the shares up
// in their order.
//
// Warps of a CTA: 0 loads, 1 issues the MMAs (even CTA), 2..9 are the epilogue: two for each quarter of the tensor
// memory's lanes, one for each half of the tile's columns.  MX: warp 10 lays out the scales.
//
// MX: tensor memory has 512 columns; two accumulators of 256 leave no room for scales.  So the second one starts at
// column 224, and the scales lie in columns 480 .. 511.  The 32 columns that the accumulators share are drained first;
// the next tile's MMAs wait for that alone.
//
// Bound by the tensor cores where there are many rows: 16384 x 7168 x 2048 (481 GFLOP each) y 156 us, dx 171 in 8 bits
// (3.1 and 2.8 PFLOP/s), y 264, dx 262, dW 271 in bf16 (1.77 to 1.84, near the rate of a plain product; each accumulator
// over all of K: y 261, dx 254); without any copy to wait for, and with one accumulator, the MMAs alone take 127 and 146, 220
// and 219.  By tiles that are not full and by each tile's end where an expert has a few hundred rows: 128 experts,
// 63488 x 4096 x 1536 (799 GFLOP) y 358 us, dx 409, dW 678, whose tiles are eight K blocks and 64 KB of output a CTA.  By the weights' bytes where there are few: 128 rows over 128 experts of 4096 x 1536 in 8
// bits 95 us, 5.1 TB/s; one expert of 7168 x 2048 and 8 rows 16 us, of which the weights' bytes are 2 and the rest is the
// launch, the latency of a share's eight K blocks and the join of seven.
//
// Columns of the last tile past the matrix are computed and dropped: MMAs of fewer columns made 1408 of them no faster.
// Experts taken in the order of their rows, to give the clusters the same number of K blocks, did not help dW either (64
// experts 539 for 558 us, 128 experts 695 for 683), nor did shares for the last round's tiles only (246 tiles: 56 us both).
//
// Every wait is bounded (wait_bounded): a wait that runs out sets the workspace status, and both CTAs leave.
#pragma once

#include "blocks8.cuh"
#include "head_gemm.cuh"   // store_sector, tc_add16, head_settle

namespace moe {

enum LinMode : int { LIN_Y = 0, LIN_DX = 1, LIN_DW = 2 };

struct LinMaps {
  CUtensorMap a, b;
  CUtensorMap few;                      // LIN_Y, LIN_DX: A in boxes of kFewRows rows
};
// LIN_DW: both matrices in boxes of 64, 32, .. 1 rows.
struct LinDwMaps {
  CUtensorMap a[7], b[7];
};
template <int MODE>
using LinMapsOf = std::conditional_t<MODE == LIN_DW, LinDwMaps, LinMaps>;

struct LinGemm {
  int n, E;                  // rows of x and dy; experts
  const int* offsets;        // [E + 1], or NULL: all rows are one expert's
  int cols;                  // output columns
  int rows_out;              // LIN_DW: output rows (O)
  int nk;                    // LIN_Y, LIN_DX: K blocks (of 128 bytes)
  int tiles_n, tiles_m;      // column tiles; LIN_DW: row tiles
  int* status;
  int64_t limit_ns;
  // MX: scale bytes of A [n][lda_s], of B at e b_expert + (output column / 128) b_col + (contraction / 128) b_k
  const uint8_t* a_scale;
  int lda_s;
  const uint8_t* b_scale;
  int64_t b_expert;
  int b_col, b_k;
  void* out;                 // bf16, or fp32 (out32)
  bool out32;
  bool sectors;              // out lies on 32 bytes
  float* part;               // [kLinClusters][2][8][128][32]: the shares' sums
  unsigned* done;            // [kLinClusters / 2][2][8]: shares done of a piece; 0 between calls
};

constexpr int kLinClusters = 76;   // at most this many clusters run (two dies x 76 SMs in pairs)
constexpr int kLinBand = 8;        // row tiles that are worked on together: their rows and a few column tiles of W stay in L2
constexpr int kFewRows = 32;       // tiles of no more rows load no more of A (other experts' rows would come with them)
// The tensor cores cut each addition to an accumulator off towards zero, so that long sums come out too small.  An
// accumulator therefore takes so many K blocks, of four additions each, at most, and the epilogue adds a tile's
// accumulators in fp32 registers: 1024 products of bf16; 4096 of codes, whose accumulators follow each other only once the
// columns that they share are drained (and the scales of four blocks come together).
// Values of y that are not the correctly rounded ones, one accumulator over all of K -> these: bf16, K = 2048, 1.27e-3 ->
// 7.1e-4; codes, K = 7168, 2.6e-4 -> 1.6e-4; sums in fp32 alone have 2.8e-4 and 0.9e-4.  dW over 1000 rows is 9.8e-7 off,
// plain fp32 sums 6.5e-7.  What it costs: y up to 1 %, dx 2 to 3 (126976 rows over 64 experts of 2048 x 1408 433 -> 443 us).
template <bool MX>
constexpr int kAccBlocks = MX ? 32 : 16;

struct LinSmem {
  static constexpr int HALF = 128 * 128;               // 16 KB: this CTA's rows of A, or its half of B
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = 6;
  static constexpr int SF_SLOTS = 4;                   // scales of four K blocks each: 512 bytes of A, 1024 of B
  static constexpr int SF_BYTES = 1536;
  static constexpr int SF = STAGES * STAGE;
  static constexpr int BAR = SF + SF_SLOTS * SF_BYTES;
  static constexpr int EXPERTS = BAR + 256;            // offsets [E + 1], first tile [E + 1]
  static constexpr int EPI_WARPS = 8;
  static int total(int E) { return EXPERTS + 2 * (E + 1) * 4 + 1024; }
  static constexpr int threads(bool mx) { return 64 + 32 * EPI_WARPS + (mx ? 32 : 0); }
  // tensor memory columns of MX
  static constexpr int TM_ACC1 = 224, TM_SF = 480;
};

struct LinTile {
  int e, row0, rows;    // LIN_Y, LIN_DX: rows row0 .. row0 + rows - 1 of x; LIN_DW: the expert's rows
  int mt, nt;           // LIN_DW: row tile of the output; column tile
  int kb0, kb1, share;
};

// Column tiles of a row tile follow each other in bands of kLinBand row tiles, within which the row tile varies fastest.
__device__ __forceinline__ void lin_band(int w, int tiles_m, int tiles_n, int* mt, int* nt) {
  const int per = kLinBand * tiles_n, b = w / per, rem = w - b * per;
  const int in_band = min(kLinBand, tiles_m - b * kLinBand);
  *nt = rem / in_band;
  *mt = b * kLinBand + (rem - *nt * in_band);
}

// K blocks of each of a tile's shares but the last.
template <bool MX>
__device__ __forceinline__ int lin_share(int nk, int shares) {
  const int per = (nk + shares - 1) / shares;
  return MX ? (per + 3) & ~3 : per;    // the scales come four K blocks at a time
}

template <int MODE, bool MX>
__device__ __forceinline__ LinTile lin_tile(const LinGemm& p, const int* offs, const int* first, int w, int total, int shares) {
  LinTile t;
  t.share = shares > 1 ? w / total : 0;
  w -= t.share * total;
  int nk;
  if constexpr (MODE == LIN_DW) {
    const int per = p.tiles_m * p.tiles_n;
    t.e = w / per;
    lin_band(w - t.e * per, p.tiles_m, p.tiles_n, &t.mt, &t.nt);
    t.row0 = offs[t.e];
    t.rows = offs[t.e + 1] - t.row0;
    nk = (t.rows + 63) >> 6;
  } else {
    int lo = 0, hi = p.E;              // the last expert whose first tile is not past w
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= w) lo = mid;
      else hi = mid;
    }
    t.e = lo;
    const int r0 = offs[lo], n = offs[lo + 1] - r0;
    int m;
    lin_band(w - first[lo], (n + 255) >> 8, p.tiles_n, &m, &t.nt);
    t.mt = 0;
    t.row0 = r0 + 256 * m;
    t.rows = min(256, n - 256 * m);
    nk = p.nk;
  }
  const int per = lin_share<MX>(nk, shares);
  t.kb0 = min(nk, t.share * per);
  t.kb1 = min(nk, t.kb0 + per);
  return t;
}

// One lane of the (whole) warp: true there.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ void tc_mma_pair_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// 32 rows of 16 bytes from both CTAs' shared memory to four columns of their tensor memory, for each quarter of the lanes.
__device__ __forceinline__ void tc_copy_scales_pair(uint32_t taddr, uint32_t saddr) {
  // no swizzle; eight rows (128 bytes) follow each other at once, groups of eight 128 bytes apart; version 1
  const uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
// Instruction descriptor, kind::mxf8f6f4: e4m3 A and B (format 0), e8m0 scales (bit 23); the byte of a scale column that
// holds this K block's scales is set at run time (bits 4-5 for B, 29-30 for A).
__host__ __device__ constexpr uint32_t instr_desc_mx(int M, int N, bool b_mn) {
  return ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

// 16 values to a dense row: one 32-byte sector of bf16, two of fp32.
__device__ __forceinline__ void lin_store16(const LinGemm& p, int64_t at, const float* v) {
  if (p.out32) {
    float* o = static_cast<float*>(p.out) + at;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * h + j]);
      if (p.sectors) {
        store_sector(o + 8 * h, w);
      } else {
        reinterpret_cast<uint4*>(o + 8 * h)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(o + 8 * h)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    if (p.sectors) {
      store_sector(o, w);
    } else {
      reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int MODE, bool MX>
__global__ void __launch_bounds__(LinSmem::threads(MX), 1)
    linear_gemm_kernel(const __grid_constant__ LinMapsOf<MODE> maps, const LinGemm p) {
  static_assert(!(MX && MODE == LIN_DW), "dW takes bf16 operands");
  using S = LinSmem;
  constexpr bool A_MN = MODE == LIN_DW, B_MN = MODE != LIN_Y;
  constexpr int KB = MX ? 128 : 64;                 // of the contraction in a K block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + S::BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S::STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S::STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S::STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S::STAGES + 4);
  auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * S::STAGES + 5 + s); };
  auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * S::STAGES + 5 + S::SF_SLOTS + s); };
  static_assert(8 * (2 * S::STAGES + 5 + 2 * S::SF_SLOTS) + 16 <= 256, "the barriers' place");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::BAR + 8 * (2 * S::STAGES + 5 + 2 * S::SF_SLOTS));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* offs = reinterpret_cast<int*>(smem + S::EXPERTS);
  int* first = offs + p.E + 1;
  int* most = reinterpret_cast<int*>(tmem_slot + 2);   // rows of the expert that has most

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known to be uniform
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * S::EPI_WARPS);   // both CTAs' epilogue warps
    }
    mbar_init(drain_bar, 1);
    for (int s = 0; s < S::SF_SLOTS; ++s) {
      mbar_init(sfull_bar(s), 2);                   // both CTAs' scale warps
      mbar_init(sempty_bar(s), 1);
    }
    *abort_flag = 0;
    *most = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(reinterpret_cast<const CUtensorMap*>(&maps));
  }
  if (warp == 1) {
    tc_alloc_pair(smem_u32(tmem_slot), 512);
    tc_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                                   // barriers and tensor memory are ready in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();                                       // no global memory access before this point

  // The experts' rows and tiles.  Offsets that are none leave no tile (every CTA comes to the same).
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) offs[e] = p.offsets ? p.offsets[e] : e == 0 ? 0 : p.n;
  __syncthreads();
  bool bad = false;
  int my_most = 0;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    bad |= offs[e] < 0 || offs[e + 1] < offs[e] || offs[e + 1] > p.n;
    my_most = max(my_most, offs[e + 1] - offs[e]);
  }
  bad = __syncthreads_or(bad);
  if (MODE == LIN_DW && !bad && my_most > 0) atomicMax(most, my_most);
  if (MODE != LIN_DW && !bad && warp == 0) {
    int sum = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int e = b + lane;
      const int mine = e < p.E ? ((offs[e + 1] - offs[e] + 255) >> 8) * p.tiles_n : 0;
      int x = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (e < p.E) first[e] = sum + x - mine;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) first[p.E] = sum;
  }
  __syncthreads();
  if (bad && threadIdx.x == 0) report(p.status, MOE_ERR_DEVICE_CHECK, 811);
  const int total = bad ? 0 : MODE == LIN_DW ? p.E * p.tiles_m * p.tiles_n : first[p.E];
  const int blocks = MODE == LIN_DW ? (*most + 63) >> 6 : p.nk;
  // Shares of a tile: as many as there are clusters for, of four K blocks at least (of 128 bytes: 128 KB of a tile).
  int shares = total > 0 ? max(1, min(min(clusters, kLinClusters) / total, blocks >> 2)) : 1;
  if (MODE != LIN_DW && shares > 1) {              // as many as have K blocks (in dW that is each expert's own matter)
    const int per = lin_share<MX>(blocks, shares);
    shares = (blocks + per - 1) / per;
  }
  const int items = total * shares;

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = cluster; w < items && ok; w += clusters) {
        const LinTile t = lin_tile<MODE, MX>(p, offs, first, w, total, shares);
        const int col = t.nt * 256 + 128 * (int)rank;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns, p.status, 801)) {
            ok = false;
            break;
          }
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t sa = sbase + stage * S::STAGE, sb = sa + S::HALF;
          const int k0 = kb * KB;
          if constexpr (MODE == LIN_DW) {
            const int r = t.row0 + k0, left = t.rows - k0;   // rows of this K block that are the expert's
            const int orow = t.mt * 256 + 128 * (int)rank;
            if (left >= 64) {
              if (leader) mbar_expect_tx(full_bar(stage), 2 * S::STAGE);
              tma_load_2d_pair(sa, &maps.a[0], fb, orow, r);
              tma_load_2d_pair(sa + 8192, &maps.a[0], fb, orow + 64, r);
              tma_load_2d_pair(sb, &maps.b[0], fb, col, r);
              tma_load_2d_pair(sb + 8192, &maps.b[0], fb, col + 64, r);
            } else {
              // The last rows, and zeros up to a multiple of 16, an MMA's share: what follows is another expert's (or
              // nobody's, and no number).  In boxes of a power of two of rows each, the zeros from past the matrix.
              const int up = (left + 15) & ~15;
              if (leader) mbar_expect_tx(full_bar(stage), 2 * 4 * 128 * up);
              int j = 0;
              auto box = [&](const CUtensorMap* ma, const CUtensorMap* mb, int rows, int at) {
                const uint32_t da = sa + j * 128, db = sb + j * 128;
                tma_load_2d_pair(da, ma, fb, orow, at);
                tma_load_2d_pair(da + 8192, ma, fb, orow + 64, at);
                tma_load_2d_pair(db, mb, fb, col, at);
                tma_load_2d_pair(db + 8192, mb, fb, col + 64, at);
                j += rows;
              };
#pragma unroll
              for (int i = 1; i < 7; ++i)
                if (left & (64 >> i)) box(&maps.a[i], &maps.b[i], 64 >> i, r + j);
#pragma unroll
              for (int i = 6; i > 2; --i)
                if ((up - left) & (64 >> i)) box(&maps.a[i], &maps.b[i], 64 >> i, p.n);
            }
          } else {
            if (t.rows <= kFewRows) {   // the rows past them, in the even CTA and all of the odd one's, go to no output
              if (leader) {
                mbar_expect_tx(full_bar(stage), 2 * S::HALF + kFewRows * 128);
                tma_load_2d_pair(sa, &maps.few, fb, k0, t.row0);
              }
            } else {
              if (leader) mbar_expect_tx(full_bar(stage), 2 * S::STAGE);
              tma_load_2d_pair(sa, &maps.a, fb, k0, t.row0 + 128 * (int)rank);
            }
            if constexpr (!B_MN) {
              tma_load_3d_pair(sb, &maps.b, fb, k0, col, t.e);
            } else if constexpr (MX) {
              tma_load_3d_pair(sb, &maps.b, fb, col, k0, t.e);
            } else {
              tma_load_3d_pair(sb, &maps.b, fb, col, k0, t.e);
              tma_load_3d_pair(sb + 8192, &maps.b, fb, col + 64, k0, t.e);
            }
          }
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      pdl_trigger();                                // every load is issued: the next kernel may be scheduled
      if (!ok) head_settle();
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (even CTA)
    // The whole warp walks the loop, so that descriptors and addresses are computed once for all lanes in uniform
    // registers; one elected lane issues.  (Computed by a single lane of a divergent branch they cost a K block of e4m3
    // 985 cycles without any load to wait for, where its MMAs need 512.)
    if (leader) {
      const bool one = elect_one();
      int stage = 0, it = 0, slot = 0;
      uint32_t phase = 0, sphase = 0, group = 0;   // group: scales copied so far
      bool ok = true;
      for (int w = cluster; w < items && ok; w += clusters) {
        const LinTile t = lin_tile<MODE, MX>(p, offs, first, w, total, shares);
        constexpr int step = kAccBlocks<MX>;
        // one accumulator after the other (an empty share still passes its accumulator on)
        for (int k0 = t.kb0; ok && (k0 < t.kb1 || k0 == t.kb0); k0 += step, ++it) {
          const int acc = it & 1;
          bool good = true;
          if constexpr (MX) {   // the columns that the last accumulator shares with this one
            if (it > 0) good = wait_bounded(tempty_bar(0), (it - 1) & 1, abort_flag, p.limit_ns, p.status, 802);
          } else {
            good = wait_bounded(tempty_bar(acc), ((it >> 1) & 1) ^ 1u, abort_flag, p.limit_ns, p.status, 802);
          }
          if (!__all_sync(0xffffffffu, good)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tacc = tmem_base + acc * (MX ? S::TM_ACC1 : 256);
          for (int kb = k0; kb < min(t.kb1, k0 + step); ++kb) {
            good = wait_bounded(full_bar(stage), phase, abort_flag, p.limit_ns, p.status, 803);
            if (MX && (kb & 3) == 0)
              good = good && wait_bounded(sfull_bar(slot), sphase, abort_flag, p.limit_ns, p.status, 804);
            if (!__all_sync(0xffffffffu, good)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = sbase + stage * S::STAGE, sb = sa + S::HALF;
            if constexpr (MX) {
              // two sets of scale columns in turn: four of A and eight of B
              const uint32_t sfa = tmem_base + S::TM_SF + 16 * (group & 1), sfb = sfa + 8;
              const uint32_t idesc = instr_desc_mx(256, 256, B_MN) | (uint32_t)(kb & 3) << 4 | (uint32_t)(kb & 3) << 29;
              const uint64_t ad = smem_desc_sw128(sa, 0, 1024), bd = smem_desc_sw128(sb, B_MN ? 16384 : 0, 1024);
              if (one) {
                if ((kb & 3) == 0) {
                  const uint32_t from = sbase + S::SF + slot * S::SF_BYTES;
                  tc_copy_scales_pair(sfa, from);
                  tc_copy_scales_pair(sfb, from + 512);
                  tc_copy_scales_pair(sfb + 4, from + 1024);
                  tc_commit_pair(sempty_bar(slot), 0x3);
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // 32 bytes of K on, in units of 16; across it, 32 rows of 128 bytes
                  tc_mma_pair_mx(tacc, ad + 2 * kk, bd + (B_MN ? 256 : 2) * kk, idesc, sfa, sfb, kb != k0 || kk != 0 ? 1u : 0u);
                tc_commit_pair(empty_bar(stage), 0x3);
              }
            } else {
              constexpr uint32_t idesc = instr_desc_bf16(256, 256, A_MN, B_MN);
              const int steps = MODE == LIN_DW ? min(4, (t.rows - kb * 64 + 15) >> 4) : 4;
              const uint64_t ad = smem_desc_sw128(sa, A_MN ? 8192 : 0, 1024), bd = smem_desc_sw128(sb, B_MN ? 8192 : 0, 1024);
              if (one) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // 16 of K on: 32 bytes, or 16 rows of 128
                  if (kk < steps)
                    tc_mma_pair(tacc, ad + (A_MN ? 128 : 2) * kk, bd + (B_MN ? 128 : 2) * kk, idesc, kb != k0 || kk != 0 ? 1u : 0u);
                tc_commit_pair(empty_bar(stage), 0x3);
              }
            }
            __syncwarp();
            if (MX && (kb & 3) == 0 && ++slot == S::SF_SLOTS) { slot = 0; sphase ^= 1u; }
            if (MX && ((kb & 3) == 3 || kb + 1 == t.kb1)) ++group;
            if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (one) tc_commit_pair(tfull_bar(acc), 0x3);
          __syncwarp();
        }
      }
      if (one) {                                    // every MMA has completed before the tensor memory is freed
        tc_commit_pair(drain_bar, 0x1);
        volatile int no_abort = 0;
        wait_bounded(drain_bar, 0, &no_abort, max(p.limit_ns, kSettleNs), nullptr, 0);
        if (!ok) head_settle();                     // the loads it gave up on, which may all have been issued
      }
      __syncwarp();
    }
  } else if (MX && warp == 2 + S::EPI_WARPS) {
    // ------------------------------------------------------------ scales (both CTAs)
    // A tensor-memory column holds a row's scales of four K blocks; 128 rows are four columns of 32 lanes, so row
    // l + 32 i of the tile lies in word i of lane l's 16 bytes.
    // The next four K blocks' bytes are loaded while these are laid out.
    struct Bytes {
      uint32_t a[4];   // of row lane + 32 i
      uint32_t b;      // lanes 0..7: the byte of K block lane & 3, columns 128 (lane >> 2) .. of the tile
    };
    const bool words = ((reinterpret_cast<uintptr_t>(p.a_scale) | (uintptr_t)p.lda_s) & 3) == 0;
    auto fetch = [&](const LinTile& t, int kb) {
      Bytes v;
      const int left = t.kb1 - kb;
      const uint8_t* from = p.a_scale + (int64_t)(t.row0 + 128 * (int)rank + lane) * p.lda_s + kb;
#pragma unroll
      for (int i = 0; i < 4; ++i, from += (int64_t)32 * p.lda_s) {
        v.a[i] = 0x7F7F7F7Fu;
        if (128 * (int)rank + lane + 32 * i < t.rows) {
          if (words) {   // what lies past the last block is not used
            v.a[i] = *reinterpret_cast<const uint32_t*>(from);
          } else {
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = j < left ? from[j] : 127;
            v.a[i] = x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24;
          }
        }
      }
      const int h = lane >> 2, j = lane & 3;
      v.b = 127;
      if (lane < 8 && j < left && t.nt * 256 + 128 * h < p.cols)
        v.b = p.b_scale[(int64_t)t.e * p.b_expert + (int64_t)(2 * t.nt + h) * p.b_col + (int64_t)(kb + j) * p.b_k];
      return v;
    };
    int slot = 0, w = cluster, kb = 0;
    uint32_t phase = 0;
    LinTile t = {};
    // the first K block of the next tile that has one
    auto next_tile = [&] {
      for (; w < items; w += clusters) {
        t = lin_tile<MODE, MX>(p, offs, first, w, total, shares);
        kb = t.kb0;
        if (kb < t.kb1) return;
      }
    };
    next_tile();
    Bytes now = {};
    if (w < items) now = fetch(t, kb);
    while (w < items) {
      const Bytes v = now;
      kb += 4;
      if (kb >= t.kb1) {
        w += clusters;
        next_tile();
      }
      if (w < items) now = fetch(t, kb);
      uint32_t b = v.b << (8 * (lane & 3));
      b |= __shfl_xor_sync(0xffffffffu, b, 1);
      b |= __shfl_xor_sync(0xffffffffu, b, 2);
      const uint32_t b0 = __shfl_sync(0xffffffffu, b, 0), b1 = __shfl_sync(0xffffffffu, b, 4);
      const bool good = wait_bounded(sempty_bar(slot), phase ^ 1u, abort_flag, p.limit_ns, p.status, 805);
      if (!__all_sync(0xffffffffu, good)) break;
      uint4* to = reinterpret_cast<uint4*>(smem + S::SF + slot * S::SF_BYTES);
      to[lane] = make_uint4(v.a[0], v.a[1], v.a[2], v.a[3]);
      to[32 + lane] = make_uint4(b0, b0, b0, b0);
      to[64 + lane] = make_uint4(b1, b1, b1, b1);
      fence_proxy_async_smem();                     // the copies to tensor memory read them
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(sfull_bar(slot));
        else mbar_arrive_cluster(mapa_shared(sfull_bar(slot), 0));
      }
      if (++slot == S::SF_SLOTS) { slot = 0; phase ^= 1u; }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;   // the quarter of the lanes this warp may read
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    int it = 0;
    bool ok = true;
    // rows of nobody
    if (MODE != LIN_DW && !bad && p.offsets) {
      const int lead = offs[0], tail = offs[p.E], mine = cluster * 16 + (int)rank * 8 + (warp - 2);
      float z[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) z[j] = 0.0f;
      for (int i = mine; i < lead + p.n - tail; i += clusters * 16) {
        const int64_t row = i < lead ? i : tail + (i - lead);
        for (int c = lane * 16; c < p.cols; c += 512) lin_store16(p, row * p.cols + c, z);
      }
    }
    for (int w = cluster; w < items && ok; w += clusters) {
      const LinTile t = lin_tile<MODE, MX>(p, offs, first, w, total, shares);
      const int local = 128 * (int)rank + q * 32 + lane;   // row in the tile
      int64_t row;
      bool in;
      if constexpr (MODE == LIN_DW) {
        row = (int64_t)t.e * p.rows_out + t.mt * 256 + local;
        in = t.mt * 256 + local < p.rows_out;
      } else {
        row = (int64_t)t.row0 + local;
        in = local < t.rows;
      }
      const bool some = __ballot_sync(0xffffffffu, in) != 0;   // any row of this warp's 32
      const int c0 = t.nt * 256 + half * 128, width = min(128, p.cols - c0);   // a multiple of 16
      const bool none = t.kb0 == t.kb1;
      const int accs = max(1, (t.kb1 - t.kb0 + kAccBlocks<MX> - 1) / kAccBlocks<MX>);
      float sum[128];                        // of the accumulators so far
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
      // 16 columns from column c of this warp's half on: to the output, or to this share's place
      float4* part = reinterpret_cast<float4*>(p.part + ((int64_t)(w * 2 + (int)rank) * 8 + (warp - 2)) * 4096) + lane;
      auto leave = [&](int c, const float* v) {
        if (c >= width || !some) return;
        if (shares == 1) {
          if (in) lin_store16(p, row * p.cols + c0 + c, v);
        } else if (in) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            part[(c / 4 + j) * 32] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      };
      for (int a = 0; a < accs; ++a, ++it) {
        const int acc = it & 1;
        int good = 1;
        if (lane == 0) good = wait_bounded(tfull_bar(acc), (it >> 1) & 1, abort_flag, p.limit_ns, p.status, 806);
        if (!__shfl_sync(0xffffffffu, good, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tacc = tmem_base + lanes + acc * (MX ? S::TM_ACC1 : 256) + half * 128;
        auto release = [&](int bar) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(tempty_bar(bar));
            else mbar_arrive_cluster(mapa_shared(tempty_bar(bar), 0));
          }
        };
        // MX: the first accumulator's last 32 columns are the second's first 32; they go first.
        const bool shared_last = MX && half == 1 && acc == 0, shared_first = MX && half == 0 && acc == 1;
        if (MX) {
          if (!none) {
            if (shared_first) {
              tc_add16(tacc, sum);
              tc_add16(tacc + 16, sum + 16);
            }
            if (shared_last) {
              tc_add16(tacc + 96, sum + 96);
              tc_add16(tacc + 112, sum + 112);
            }
          }
          release(0);
        }
        if (!none) {
#pragma unroll
          for (int c = 0; c < 128; c += 16)
            if (!(c < 32 && shared_first) && !(c >= 96 && shared_last)) tc_add16(tacc + c, sum + c);
        }
        if (!MX) release(acc);
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 128; c += 16) leave(c, sum + c);
      if (shares > 1 && some) {
        // The last of a piece's shares adds them up, in their order.
        __threadfence();
        __syncwarp();
        const int tile = w - t.share * total;
        unsigned before = 0;
        if (lane == 0) before = atomicInc(p.done + (tile * 2 + (int)rank) * 8 + (warp - 2), (unsigned)shares - 1);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == (unsigned)shares - 1) {
          // Few rows are spread over the lanes: item i is four columns, i / wide, of row i % wide.  16 loads in flight.
          __threadfence();
          const int rows = __popc(__ballot_sync(0xffffffffu, in));     // the first ones
          const int log_wide = 32 - __clz(rows - 1), wide = 1 << log_wide;
          const int64_t row0 = row - lane;
          const float4* from = reinterpret_cast<const float4*>(p.part + ((int64_t)(tile * 2 + (int)rank) * 8 + (warp - 2)) * 4096);
          const int64_t next = (int64_t)total * 16 * 1024;             // a share further, in float4
#pragma unroll 1
          for (int k = 0; k < wide; k += 8) {
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
            for (int s = 0; s < shares; ++s) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int i = lane + 32 * (k + j), c = i >> log_wide;
                if (k + j < wide && 4 * c < width) {
                  const float4 x = __ldcg(from + s * next + c * 32 + (i & (wide - 1)));
                  v[j].x += x.x, v[j].y += x.y, v[j].z += x.z, v[j].w += x.w;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int i = lane + 32 * (k + j), c = i >> log_wide, r = i & (wide - 1);
              if (k + j < wide && 4 * c < width && r < rows) {
                const int64_t at = (row0 + r) * p.cols + c0 + 4 * c;
                if (p.out32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v[j];
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16(v[j].x, v[j].y), pack_bf16(v[j].z, v[j].w));
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  cluster_sync();                                   // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tc_dealloc_pair(tmem_base, 512);
}

template <int MODE, bool MX>
cudaError_t launch_linear_gemm(const LinMapsOf<MODE>& maps, LinGemm p, int sms, cudaStream_t s) {
  auto kern = linear_gemm_kernel<MODE, MX>;
  p.sectors = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
  const int smem = LinSmem::total(p.E);
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LinSmem::total(1024));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min(kLinClusters, sms / 2)));
  cfg.blockDim = dim3(LinSmem::threads(MX));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = launch_chain_mode() >= MOE_CHAIN_EARLY ? 2 : 1;   // the cluster attribute comes first
  err = cudaLaunchKernelEx(&cfg, kern, maps, p);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe

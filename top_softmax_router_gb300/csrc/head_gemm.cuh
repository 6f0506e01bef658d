// Dense GEMM on CTA pairs for the distillation head: C [M, N] = A [M, K] B [N, K]^T, bf16 in, fp32 accumulators in
// tensor memory, with the head's epilogues.
//
// A cluster of two CTAs owns a 256 x 256 tile: each loads its 128 rows of A and half of the tile's 256 rows of B (64
// of K at a time, 32 KB a stage, 6 stages); the even CTA issues tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16),
// which leaves rows 0..127 in its own tensor memory and rows 128..255 in its peer's.  Two accumulators of 256 columns
// let the epilogue of a tile run under the main loop of the next.
//
// Warps of a CTA (320 threads): 0 loads, 1 issues the MMAs (even CTA), 2..9 are the epilogue: two for each quarter of
// the tensor memory's lanes, one for each half of the tile's columns.
//
// Bound by the tensor cores at size (8192 x 4096 x 65536, 4.4 TFLOP each, launches apart at 2070 MHz: logits 2.67 ms,
// 1.65 PFLOP/s; d 2.53; dX 2.64; dW 2.64; in steps back to back the power cap leaves about 1730 MHz: 3.04, 2.85, 2.94,
// 2.96). Below, by whole waves of tiles on 76 clusters and the tiles' own latency (2048 x 1024 x 32000: logits 103 us,
// 1.3 PFLOP/s, the tensor pipe at work 54 % of the time; d, dX and dW 35 to 42 %), and by launch and load latency
// where there are few tiles (300 x 128 x 1000: 10 to 14 us each).
//
// Every wait is bounded (wait_bounded): a wait that runs out sets the workspace status, and both CTAs leave.
#pragma once

#include "common.cuh"
#include "gemm_kernel.cuh"   // store_bf16x32, GEMM_BK

namespace moe {

enum HeadEpi : int {
  HEAD_LSE = 0,   // (max, sum of 2^..) of each row over each 128-class half tile; the entries' logits
  HEAD_D = 1,     // d in bf16
  HEAD_OUT = 2    // C: fp32 or bf16, added to an fp32 matrix of the same shape where there is one
};

struct HeadGemm {
  int M, N, nk;              // rows, columns, K blocks of 64
  int tiles_m, tiles_n, band;
  int splits;                // HEAD_OUT: shares of K, each with its own output (1: no split)
  int* status;
  int64_t limit_ns;
  int share;                 // HEAD_LSE: K blocks that one accumulator sums (see kLseShare)
  // HEAD_LSE, HEAD_D
  float to_log2;             // log2(e) / T: logits in units of T ln 2
  int tile0;                 // class tile (of 256) of column 0
  int tiles_all, K;          // class tiles of the vocabulary; entries a row
  const int* bucket;         // [ceil(M / 32)][tiles_all + 1]: first entry of (32 rows, class tile)
  const uint32_t* entry;     // row in group | column in tile << 5 | slot << 13
  float* part_m;             // [2 tiles_n][M]
  float* part_z;
  float* entry_logit;        // [M][K]
  const float* lse;          // [M], natural
  const float* coef;         // [M]: g T / out_scale where the row has entries, else 0
  const float* q;            // [M][K]
  uint16_t* d;               // [M][ldd]
  int ldd;
  // HEAD_OUT
  const float* out_scale;    // [1]: what d was divided by
  const float* add;          // [splits][M][ldo] or NULL
  float* out32;              // [splits][M][ldo] or NULL
  uint16_t* out16;           // [M][ldo] or NULL
  int ldo;
  bool sectors;              // d and the outputs (whose rows are multiples of 64 bytes) lie on 32 bytes
};

// The tensor cores cut each addition to an accumulator off towards zero, so that a logit of H products comes out too
// small, by up to H / 16 x 2^-24 of itself, the larger the logit the more, and lse with it (H = 4096: 1.5e-6 of lse,
// against 5e-8 of fp32 sums).  The forward therefore sums 1024 products to an accumulator and adds those in fp32
// registers: the accumulators stay small, and so does what is cut off (3.6e-7; 512 products: 1.7e-7, but the logits of
// 8192 x 4096 x 65536 took 2903 us for 2689).  Unsplit they take 2580, in steps under the power cap 2930 for 3040: 4 %
// either way.  The sums cost registers too: 168 a thread, and 136 bytes are spilled.  d is rounded to bf16 and is left
// alone.
constexpr int kLseShare = 16;

struct HeadSmem {
  static constexpr int HALF = 128 * GEMM_BK * 2;       // 16 KB: this CTA's rows of A, or its half of B
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = 6;
  static constexpr int BAR = STAGES * STAGE;
  static constexpr int TOTAL = BAR + 256 + 1024;
  static constexpr int TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
};

// 2^x, relative error at most 2^-22 (PTX ex2.approx); 0 for large negative x.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four single fp32 columns of tensor memory: each thread gets its lane's values.  (The wait names the registers, so that
// nothing can use them before it.)
__device__ __forceinline__ void tc_ld_columns(const uint32_t (&taddr)[4], float (&v)[4]) {
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[k]) : "r"(taddr[k]));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])::"memory");
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(r[k]);
}

// v[j] += this thread's lane of 16 consecutive fp32 columns of tensor memory.
__device__ __forceinline__ void tc_add16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
}

// 32 lanes x 32 consecutive fp32 columns of tensor memory from the threads' values.
__device__ __forceinline__ void tc_st32(uint32_t taddr, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// 32 bytes to a 32-byte boundary in one store: a whole sector (two of 16 reach L2 as two partial writes of it, and
// dW of 53 tokens x 640 x 60341 classes went out at 2 TB/s).
__device__ __forceinline__ void store_sector(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 32 values, rounded to bf16 or as they are.  sectors: dst lies on 32 bytes.
__device__ __forceinline__ void store_row16(uint16_t* dst, const float (&v)[32], bool sectors) {
  if (!sectors) {
    store_bf16x32(dst, v);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[16 * h + 2 * j], v[16 * h + 2 * j + 1]);
    store_sector(dst + 16 * h, w);
  }
}
__device__ __forceinline__ void store_row32(float* dst, const float (&v)[32], bool sectors) {
  if (!sectors) {
    float4* o = reinterpret_cast<float4*>(dst);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    return;
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * h + j]);
    store_sector(dst + 8 * h, w);
  }
}

// What a tile's epilogue reads besides its accumulator, loaded while the main loop still runs.
struct HeadRow {
  float coef, l, q;   // HEAD_D: the row's coefficient and lse in powers of two; q of the lane's record
  int e0, e1;         // the entries of these 32 rows and this class tile
  uint32_t rec;       // the lane's among the first 32
};
template <int EPI>
__device__ __forceinline__ void load_records(const HeadGemm& p, int row0, int e0, int e1, int lane, uint32_t& rec, float& q) {
  rec = 0;
  q = 0.0f;
  if (e0 + lane < e1) {
    rec = p.entry[e0 + lane];
    if (EPI == HEAD_D) q = p.q[(int64_t)(row0 + (int)(rec & 31)) * p.K + (rec >> 13)];
  }
}
template <int EPI>
__device__ __forceinline__ HeadRow head_row(const HeadGemm& p, int row0, int nt, int lane) {
  HeadRow r = {0.0f, 0.0f, 0.0f, 0, 0, 0};
  if (EPI == HEAD_OUT || row0 >= p.M) return r;
  const int* b = p.bucket + (int64_t)(row0 >> 5) * (p.tiles_all + 1) + p.tile0 + nt;
  r.e0 = b[0];
  r.e1 = b[1];
  if (EPI == HEAD_D && row0 + lane < p.M) {
    r.coef = p.coef[row0 + lane];
    r.l = p.lse[row0 + lane] * 1.4426950408889634f;
  }
  load_records<EPI>(p, row0, r.e0, r.e1, lane, r.rec, r.q);
  return r;
}
// f(record, q, logit) for each entry in this warp's half of the columns, four of them a load of tensor memory; the whole
// warp calls it for every record, with its own lane's logit.
template <int EPI, class F>
__device__ __forceinline__ void for_entries(const HeadGemm& p, const HeadRow& pre, int row0, int half, uint32_t tacc,
                                            int lane, F&& f) {
  uint32_t recs = pre.rec;
  float qs = pre.q;
  for (int e0 = pre.e0; e0 < pre.e1; e0 += 32) {
    if (e0 != pre.e0) load_records<EPI>(p, row0, e0, pre.e1, lane, recs, qs);
    uint32_t left = __ballot_sync(0xffffffffu, e0 + lane < pre.e1 && (int)((recs >> 12) & 1) == half);
    while (left) {
      uint32_t rec[4], at[4];
      float q[4], y[4];
      const int n = min(4, __popc(left));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int src = left ? __ffs(left) - 1 : 0;
        left &= left - 1;
        rec[k] = __shfl_sync(0xffffffffu, recs, src);
        q[k] = __shfl_sync(0xffffffffu, qs, src);
        at[k] = tacc + ((rec[k] >> 5) & 255);
      }
      tc_ld_columns(at, y);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) f(rec[k], q[k], y[k]);
    }
  }
}

// The epilogue of one warp: rows row0 + lane (valid below p.M), the columns c0 .. c0 + 127 of column tile nt.  none: the
// tile's share of K is empty, and its accumulator holds nothing.
template <int EPI>
__device__ __forceinline__ void head_epilogue(const HeadGemm& p, const HeadRow& pre, int row0, int nt, int half, int split,
                                              bool none, uint32_t tacc, int lane) {
  const int row = row0 + lane;
  const bool ok = row < p.M;
  const int n0 = nt * 256;
  const int c0 = half * 128, c1 = min(c0 + 128, p.N - n0);
  float v[32];
  if constexpr (EPI == HEAD_LSE) {
    // m: running maximum of y = logit x to_log2; z: sum of 2^(y - m), rescaled when m grows
    float m = -INFINITY, z = 0.0f;
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {
      tc_ld32(tacc + c, v);
      const int valid = c1 - c;
      float cm = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < valid) cm = fmaxf(cm, v[j]);
      const float mn = fmaxf(m, cm * p.to_log2);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < valid) s += exp2_fast(fmaf(v[j], p.to_log2, -mn));
      z = fmaf(z, exp2_fast(m - mn), s);
      m = mn;
    }
    if (ok) {
      p.part_m[(int64_t)(2 * nt + half) * p.M + row] = m;
      p.part_z[(int64_t)(2 * nt + half) * p.M + row] = z;
    }
  } else if constexpr (EPI == HEAD_D) {
    const float coef = pre.coef, l = pre.l;
    uint16_t* d = p.d + (int64_t)row * p.ldd + n0;
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {
      tc_ld32(tacc + c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = coef == 0.0f ? 0.0f : coef * exp2_fast(fmaf(v[j], p.to_log2, -l));
      if (ok) store_row16(d + c, v, p.sectors);
    }
    for_entries<EPI>(p, pre, row0, half, tacc, lane, [&](uint32_t rec, float q, float y) {
      if (ok && lane == (int)(rec & 31))                // this thread wrote the element above
        d[(rec >> 5) & 255] = __bfloat16_as_ushort(__float2bfloat16_rn(coef * (exp2_fast(fmaf(y, p.to_log2, -l)) - q)));
    });
  } else {
    const int64_t at = ((int64_t)split * p.M + row) * p.ldo + n0;
    const float scale = *p.out_scale;
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {               // N is a multiple of 32 here
      tc_ld32(tacc + c, v);
      if (!ok) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = none ? 0.0f : v[j] * scale;
      if (p.add) {
        const float4* a = reinterpret_cast<const float4*>(p.add + at + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 x = a[j];
          v[4 * j] += x.x, v[4 * j + 1] += x.y, v[4 * j + 2] += x.z, v[4 * j + 3] += x.w;
        }
      }
      if (p.out32) store_row32(p.out32 + at + c, v, p.sectors);
      if (p.out16) store_row16(p.out16 + at + c, v, p.sectors);
    }
  }
  if constexpr (EPI == HEAD_LSE)
    for_entries<EPI>(p, pre, row0, half, tacc, lane, [&](uint32_t rec, float, float y) {
      if (ok && lane == (int)(rec & 31)) p.entry_logit[(int64_t)row * p.K + (rec >> 13)] = y;
    });
}

// Tile w: bands of p.band row tiles; within a band the row tile varies fastest, so that the clusters at work share a
// few tiles of A and of B, which stay in L2.  K blocks [kb0, kb1); with splits, all tiles of a share come before the
// next share's.
__device__ __forceinline__ void head_tile(const HeadGemm& p, int w, int* mt, int* nt, int* kb0, int* kb1, int* split) {
  const int tiles = p.tiles_m * p.tiles_n, per_split = (p.nk + p.splits - 1) / p.splits;
  *split = w / tiles;
  w -= *split * tiles;
  *kb0 = min(p.nk, *split * per_split);
  *kb1 = min(p.nk, *kb0 + per_split);
  const int per_band = p.band * p.tiles_n;
  const int b = w / per_band, rem = w - b * per_band;
  const int in_band = min(p.band, p.tiles_m - b * p.band);
  *nt = rem / in_band;
  *mt = b * p.band + (rem - *nt * in_band);
}

// A wait ran out: the copies in flight (this CTA's and the peer's) complete on the even CTA's barriers in an order that no
// longer says when the last one has landed, so both CTAs stay (they leave together) for far longer than a copy takes.
__device__ __forceinline__ void head_settle() {
  const uint64_t t0 = globaltimer();
  while ((int64_t)(globaltimer() - t0) < kSettleNs) {}
}

// A_MN / B_MN: the operand lies with its rows along K ([K][M] or [K][N] in memory).
template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(HeadSmem::THREADS, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const HeadGemm p) {
  using S = HeadSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S::STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S::STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S::STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S::STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::BAR + 8 * (2 * S::STAGES + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  if (warp == 1) {
    tc_alloc_pair(smem_u32(tmem_slot), S::TMEM_COLS);
    tc_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                                   // barriers and tensor memory are ready in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();                                       // no global memory access before this point

  const int total = p.tiles_m * p.tiles_n * p.splits;
  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = cluster; w < total && ok; w += clusters) {
        int mt, nt, kb0, kb1, split;
        head_tile(p, w, &mt, &nt, &kb0, &kb1, &split);
        const int row = mt * 256 + 128 * (int)rank, col = nt * 256 + 128 * (int)rank;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns, p.status, 701)) {
            ok = false;
            break;
          }
          if (leader) mbar_expect_tx(full_bar(stage), 2 * S::STAGE);
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t sa = sbase + stage * S::STAGE, sb = sa + S::HALF;
          const int k0 = kb * GEMM_BK;
          if constexpr (A_MN) {
            tma_load_2d_pair(sa, &ta, fb, row, k0);
            tma_load_2d_pair(sa + 8192, &ta, fb, row + 64, k0);
          } else {
            tma_load_2d_pair(sa, &ta, fb, k0, row);
          }
          if constexpr (B_MN) {
            tma_load_2d_pair(sb, &tb, fb, col, k0);
            tma_load_2d_pair(sb + 8192, &tb, fb, col + 64, k0);
          } else {
            tma_load_2d_pair(sb, &tb, fb, k0, col);
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
    if (leader) {
      constexpr uint32_t idesc = instr_desc_bf16(256, 256, A_MN, B_MN);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = cluster; w < total && ok; w += clusters) {
        int mt, nt, kb0, kb1, split;
        head_tile(p, w, &mt, &nt, &kb0, &kb1, &split);
        const int step = EPI == HEAD_LSE ? p.share : max(1, kb1 - kb0);
        // one accumulator after the other (an empty share of K still passes its accumulator on)
        for (int k0 = kb0; ok && (k0 < kb1 || k0 == kb0); k0 += step, ++it) {
          const int acc = it & 1;
          int good = 1;
          if (lane == 0)
            good = wait_bounded(tempty_bar(acc), ((it >> 1) & 1) ^ 1u, abort_flag, p.limit_ns, p.status, 702);
          if (!__shfl_sync(0xffffffffu, good, 0)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tacc = tmem_base + acc * 256;
          for (int kb = k0; kb < min(kb1, k0 + step); ++kb) {
            if (lane == 0) good = wait_bounded(full_bar(stage), phase, abort_flag, p.limit_ns, p.status, 703);
            if (!__shfl_sync(0xffffffffu, good, 0)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = sbase + stage * S::STAGE, sb = sa + S::HALF;
            if (lane == 0) {
#pragma unroll
              for (int kk = 0; kk < GEMM_BK / 16; ++kk) {
                const uint64_t ad = A_MN ? smem_desc_sw128(sa + kk * 2048, 8192, 1024) : smem_desc_sw128(sa + kk * 32, 0, 1024);
                const uint64_t bd = B_MN ? smem_desc_sw128(sb + kk * 2048, 8192, 1024) : smem_desc_sw128(sb + kk * 32, 0, 1024);
                tc_mma_pair(tacc, ad, bd, idesc, kb != k0 || kk != 0 ? 1u : 0u);
              }
              tc_commit_pair(empty_bar(stage), 0x3);
            }
            __syncwarp();
            if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (lane == 0) tc_commit_pair(tfull_bar(acc), 0x3);
          __syncwarp();
        }
      }
      if (lane == 0) {                              // every MMA has completed before the tensor memory is freed
        tc_commit_pair(drain_bar, 0x1);
        volatile int no_abort = 0;
        wait_bounded(drain_bar, 0, &no_abort, max(p.limit_ns, kSettleNs), nullptr, 0);
        if (!ok) head_settle();                     // the loads it gave up on, which may all have been issued
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;   // the quarter of the lanes this warp may read
    int it = 0;
    bool ok = true;
    for (int w = cluster; w < total && ok; w += clusters) {
      int mt, nt, kb0, kb1, split;
      head_tile(p, w, &mt, &nt, &kb0, &kb1, &split);
      const int row0 = mt * 256 + 128 * (int)rank + q * 32;
      const HeadRow pre = head_row<EPI>(p, row0, nt, lane);
      const int accs = EPI == HEAD_LSE ? (p.nk + p.share - 1) / p.share : 1;
      float sum[EPI == HEAD_LSE ? 128 : 1];   // of the accumulators so far
      if constexpr (EPI == HEAD_LSE) {
#pragma unroll
        for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
      }
      for (int a = 0; a < accs; ++a, ++it) {
        const int acc = it & 1;
        int good = 1;
        if (lane == 0) good = wait_bounded(tfull_bar(acc), (it >> 1) & 1, abort_flag, p.limit_ns, p.status, 704);
        if (!__shfl_sync(0xffffffffu, good, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
        if constexpr (EPI == HEAD_LSE) {
          if (accs > 1) {
#pragma unroll
            for (int c = 0; c < 128; c += 16) tc_add16(tacc + half * 128 + c, sum + c);
            if (a + 1 == accs) {   // the sums take the last accumulator's place
#pragma unroll
              for (int c = 0; c < 128; c += 32) tc_st32(tacc + half * 128 + c, sum + c);
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
          }
        }
        if (a + 1 == accs)
          head_epilogue<EPI>(p, pre, row0, nt, half, split, kb0 == kb1, tacc, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(tempty_bar(acc));
          else mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
        }
      }
    }
  }

  tc_fence_before();
  cluster_sync();                                   // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tc_dealloc_pair(tmem_base, S::TMEM_COLS);
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t launch_head_gemm(const CUtensorMap& a, const CUtensorMap& b, HeadGemm p, int sms, cudaStream_t s) {
  auto kern = head_gemm_kernel<EPI, A_MN, B_MN>;
  p.tiles_m = (p.M + 255) / 256;
  p.tiles_n = (p.N + 255) / 256;
  if (p.splits < 1) p.splits = 1;
  p.sectors = ((reinterpret_cast<uintptr_t>(p.out16) | reinterpret_cast<uintptr_t>(p.out32) |
               reinterpret_cast<uintptr_t>(p.d)) & 31) == 0;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.splits;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, HeadSmem::TOTAL);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(tiles, sms / 2)));
  cfg.blockDim = dim3(HeadSmem::THREADS);
  cfg.dynamicSmemBytes = HeadSmem::TOTAL;
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
  err = cudaLaunchKernelEx(&cfg, kern, a, b, p);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe

// gated_ff.cuh -- the gated feed-forward of the UNet's transformer block, both
// projections, the activation and the product in one kernel, and its backward
// pass.
//
//   h = x Wh^T + bh,  g = x Wg^T + bg        W [2F][C]: Wh its first F rows, Wg its last
//   y = h GELU(g)                            GELU(g) = g Phi(g), exact (erf) form
//
//   backward, from x, W, b and dy alone (h and g are computed again: for the
//   UNet's widths the product is cheaper than writing and reading them back):
//   dh = dy GELU(g),  dg = dy h (Phi(g) + g phi(g)),   P = [dh, dg]   [T][2F]
//   dx = P W,  dW = P^T x,  db = column sums of P
//
// gated_kernel     x, W (, dy) -> y, or P in 16 bits and partial sums of db
// product_kernel   P, W, x -> dx and dW, one launch for both products
// finish_kernel    partial products of a split contraction -> dx, dW; partial sums -> db
//
// All products run on the tensor cores (fp32 accumulators in tensor memory);
// bias, activation and gradients are fp32.  Roundings to 16 bits: y, dx, dW
// once; P once, because it is the tensor cores' operand in the two products
// that follow (a relative 2^-9 / 2^-12 on average per entry, random, which the
// products average out to about that of their own output rounding).  db is
// summed from the unrounded fp32 entries of P.
//
// The pair of columns (h_f, g_f) must meet in one thread: a tile is 128 rows
// by HN columns of h and the matching HN columns of g, both in one B operand
// of 2 HN rows (two TMA boxes one under the other), so one tcgen05.mma of
// N = 2 HN per 16 columns of C computes both and the epilogue finds h_f and
// g_f in the same tensor-memory lane, HN columns apart.
#pragma once

#include "layer_norm.cuh"
#include "pipeline.cuh"
#include "unet_ops.cuh"

namespace sdattn {

// Measured (C = 320, F = 1280): forward of 8192 rows 14.5 us, of 65536 rows 81 us
// alone (1.3 PFLOP/s, 82% of a library product's best rate) and 113 us in a row,
// where the power cap holds the clock at 1250 MHz.  With the epilogue left out
// the latter took 70 us: the operands' way to the SMs, 32 KB a step at 43 bytes
// a clock (the MMAs are 512 clocks of a step's 730).  With the products left out
// it took 73 us, some 4000 clocks a tile: latency, with no pipe above a third of
// its rate and 43% of issue slots used.  Backward of 8192 rows 57 us (cold, under
// a profiler, 35 us here and 29 us in product_kernel).

// GELU of a pair of gates on packed fp32 pairs (half the instructions of two
// scalars).  With q = erfc(|g| / sqrt 2) / 2, the normal tail,
//   Phi(g) = 1 - q for g >= 0 and q below,  so  GELU(g) = max(g, 0) - |g| q.
// log2 q is smooth: q = 2^P(-|g|), P of degree 7, fitted on [-5.6, 0] in
// gelu_tail_fit.py for the least largest error of q and |g| q (1e-7 in fp32
// arithmetic) and still falling at -8, where q is 2^-48.  That is one exponential and
// seven FMAs; gelu_erf's form takes an exponential, a reciprocal and as many
// FMAs, and two MUFU operations a column were slower (16 images at 64x64 100 us,
// this way 95 us).
constexpr float kTailBound = 8.f;
constexpr float kTail0 = -0.9999998211860657f, kTail1 = 1.1511149406433105f, kTail2 = -0.4591203033924103f,
                kTail3 = 0.05278468504548073f, kTail4 = 0.0075082783587276936f, kTail5 = 0.000494707899633795f,
                kTail6 = -3.2478859793627635e-05f, kTail7 = -6.1192795328679495e-06f;

// max(x, 0) that keeps a not-a-number (max.NaN).
__device__ __forceinline__ float nan_max0(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// Takes half the gates, u = g / 2 (an exact scaling, folded into the bias's
// addition): max(g, 0) = u + |u| costs what a maximum does, and at a gate of
// -infinity it is the formula's not-a-number.
__device__ __forceinline__ uint64_t gelu_pair(uint64_t u) {
  const auto both = [](float c) { return f2_pack(c, c); };
  float u0, u1, e0, e1;
  f2_unpack(u, u0, u1);
  // the bound keeps a gate of +infinity from meeting q = 0
  const uint64_t m = f2_pack(fmaxf(-fabsf(u0), -0.5f * kTailBound), fmaxf(-fabsf(u1), -0.5f * kTailBound));
  uint64_t y = f2_fma(m, both(128.f * kTail7), both(64.f * kTail6));
  y = f2_fma(m, y, both(32.f * kTail5));
  y = f2_fma(m, y, both(16.f * kTail4));
  y = f2_fma(m, y, both(8.f * kTail3));
  y = f2_fma(m, y, both(4.f * kTail2));
  y = f2_fma(m, y, both(2.f * kTail1));
  y = f2_fma(m, y, both(1.f + kTail0));      // log2 of 2 q
  f2_unpack(y, e0, e1);
  return f2_fma(m, f2_pack(ex2_approx(e0), ex2_approx(e1)), f2_pack(u0 + fabsf(u0), u1 + fabsf(u1)));
}

// GELU and its slope Phi(g) + g phi(g) for a pair of gates, for the backward
// pass.  phi needs exp(-g^2 / 2), which also gives the tail by gelu_erf's
// approximation (Abramowitz and Stegun 7.1.26):
//   q = t (a1 + t (a2 + ...)) / 2 exp(-g^2 / 2),  t = 1 / (1 + p |g| / sqrt 2),
// again one exponential and one reciprocal a column; gelu_pair's tail beside
// its own exponential was 4% slower over the whole pass.
struct GeluGrad {
  uint64_t gelu, slope;
};

__device__ __forceinline__ GeluGrad gelu_grad_pair(uint64_t g) {
  constexpr float kP = 0.3275911f * 0.7071067811865476f, kA1 = -0.5f * 0.254829592f, kA2 = 0.5f * 0.284496736f,
                  kA3 = -0.5f * 1.421413741f, kA4 = 0.5f * 1.453152027f, kA5 = -0.5f * 1.061405429f;
  constexpr float kE = -0.5f * 1.4426950408889634f;
  const auto both = [](float c) { return f2_pack(c, c); };
  float g0, g1, d0, d1, e0, e1, t0, t1, s0, s1;
  f2_unpack(g, g0, g1);
  // q is 0 far below 64: the bound keeps a gate of +infinity from meeting it
  // (-infinity meets it and gives the formula's not-a-number)
  const uint64_t mag = f2_pack(fmaxf(fminf(fabsf(g0), 64.f), -g0), fmaxf(fminf(fabsf(g1), 64.f), -g1));
  f2_unpack(f2_fma(mag, both(kP), both(1.f)), d0, d1);
  f2_unpack(f2_mul(f2_mul(g, g), both(kE)), e0, e1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(d1));
  const uint64_t bell = f2_pack(ex2_approx(e0), ex2_approx(e1)), t = f2_pack(t0, t1);
  uint64_t y = f2_fma(t, both(kA5), both(kA4));
  y = f2_fma(t, y, both(kA3));
  y = f2_fma(t, y, both(kA2));
  y = f2_fma(t, y, both(kA1));
  const uint64_t nq = f2_mul(f2_mul(t, y), bell);   // -q
  GeluGrad r;
  r.gelu = f2_fma(mag, nq, f2_pack(nan_max0(g0), nan_max0(g1)));
  // Phi = 1/2 + (1/2 - q) with g's sign
  f2_unpack(f2_add(nq, both(0.5f)), s0, s1);
  const uint64_t s = f2_add(f2_pack(copysignf(s0, g0), copysignf(s1, g1)), both(0.5f));
  r.slope = f2_fma(f2_mul(g, both(0.3989422804014327f)), bell, s);
  return r;
}

// Sums v[i] over the warp's lanes for N columns at once (N a power of two up
// to 32): each exchange halves the columns a lane still holds.  Lane l ends
// with the total of column l / (32 / N); the order is fixed.
template <int N>
__device__ __forceinline__ float warp_column_sums(float* v, int lane) {
  int s = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  float t = v[0];
  for (; s >= 1; s >>= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
  return t;
}

struct GatedCfg {
  static constexpr int BK = 64;                     // columns of C per stage
  static constexpr int A_BYTES = 128 * 128;         // 128 rows of x
  static constexpr int HN = 128;                    // most columns of h (and of g) per tile
  static constexpr int EPI = 16;                    // epilogue warps
  static constexpr int NTHREADS = (4 + EPI) * 32;   // TMA, MMA, bias, one idle warp, epilogue
  static constexpr uint32_t TMEM_COLS = 512;        // two accumulators of 2 HN columns
};

// PAIR: a stage is 64 columns of C of the CTA's 128 rows of x and the h or the
// g half of W's tile.  Otherwise it is 128 columns (two halves) of tm rows of x
// and hn rows each of Wh and Wg, as many as the ring holds.
template <bool BWD, bool PAIR>
struct GatedSmem {
  static constexpr int STAGE = 2 * 128 * 128;       // PAIR
  static constexpr int STAGES = BWD ? 4 : 5;        // PAIR
  static constexpr int RING = PAIR ? STAGES * STAGE : 212992;
  static constexpr int SLACK = 16384;               // kept behind the stages when x's tile is short: its products read up to 16 KB
  static constexpr int MAX_STAGES = 12;
  // an epilogue warp's staging (PAIR): 32 rows x 32 columns of y; backward: of
  // dy, which dh replaces in place, and of dg
  static constexpr int WSTG = PAIR ? (BWD ? 4096 : 2048) : 0;
  static constexpr int OFF_STG = RING;
  static constexpr int OFF_BIAS = OFF_STG + GatedCfg::EPI * WSTG;   // [2 tiles][h, g][HN] fp32
  static constexpr int OFF_BAR = OFF_BIAS + 2 * 2 * GatedCfg::HN * 4;
  static constexpr int NBAR = 2 * MAX_STAGES + 4 + 4 + 1 + (PAIR && BWD ? GatedCfg::EPI : 0);
  static constexpr int BYTES = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(BYTES <= 232448, "shared memory budget");
};

struct GatedParams {
  const float* bias;    // [2F] or null
  const void* dY;       // [T][F]      (backward)
  void* Y;              // [T][F]; backward: P [T][2F]
  float* part;          // [ceil(T / 32)][2F] partial sums of db, or null
  int T, F;
  int hn;               // columns of h per tile: a multiple of 16, at most 128
  int tm;               // rows of x loaded per CTA: 128, or all rows of a shorter x rounded up to 8
  int stages, stage;    // of the ring without pairs: how many, bytes of one
  int rts, fts;         // row tiles (of 256 rows in a pair), column tiles
  int ksteps;           // ceil(C / 64)
  int chains;           // accumulators a tile's contraction is dealt over: 1, or 2 (backward, long contractions)
};

// y (or dh and dg) of 8 columns of one row, from the accumulators and the
// columns' biases in shared memory (the same address in every lane; forward, the
// gates' are halved).
template <bool BWD, bool BF16>
__device__ __forceinline__ void gated_columns8(const uint32_t* h, const uint32_t* g, const float* bh, const float* bg,
                                               const uint4& dy, float* o0, float* o1) {
  float d[8];
  if constexpr (BWD) unpack8<BF16>(dy, d);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 bv = reinterpret_cast<const float4*>(bh)[q], gv = reinterpret_cast<const float4*>(bg)[q];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = 4 * q + 2 * k;
      const uint64_t hp = f2_add(f2_pack(__uint_as_float(h[e]), __uint_as_float(h[e + 1])),
                                 k ? f2_pack(bv.z, bv.w) : f2_pack(bv.x, bv.y));
      const uint64_t ga = f2_pack(__uint_as_float(g[e]), __uint_as_float(g[e + 1]));
      const uint64_t gb = k ? f2_pack(gv.z, gv.w) : f2_pack(gv.x, gv.y);
      if constexpr (BWD) {
        const GeluGrad a = gelu_grad_pair(f2_add(ga, gb));
        const uint64_t dp = f2_pack(d[e], d[e + 1]);
        f2_unpack(f2_mul(dp, a.gelu), o0[e], o0[e + 1]);
        f2_unpack(f2_mul(f2_mul(dp, hp), a.slope), o1[e], o1[e + 1]);
      } else {
        f2_unpack(f2_mul(hp, gelu_pair(f2_fma(ga, f2_pack(0.5f, 0.5f), gb))), o0[e], o0[e + 1]);
      }
    }
  }
}

// Roles: warp 0 TMA (a ring of x / W stages), warp 1 MMA (tcgen05 SS,
// 128 or, in a pair, 256 x 2 hn x 16; two accumulators so that a tile's
// epilogue overlaps the next tile's products), warp 2 the tiles' biases, warps
// 4..19 epilogue: four warps per quarter of the CTA's 128 rows, dividing the
// tile's columns.  (More warps hide more of the epilogue's latency: eight took
// 123 us for 16 images at 64x64 where sixteen took 95; two groups of eight on
// alternate tiles lose where a CTA has an odd handful of tiles.)
// PAIR: tiles of 256 rows by 128 columns of h, a CTA of the pair holding the h
// rows of W's tile and the other the g rows; the results leave through shared
// memory and TMA stores of 32 rows x 32 columns of y, or of dh and of dg, which
// also clip at the edges.  Backward: a warp's dy arrives by TMA while it waits
// for the products (read from global memory where it was used, its latency set
// the pace: 37 us for the 64x64 pair).
// Otherwise tiles of 128 rows by hn columns, stored 16 bytes per thread.
template <bool BF16, bool BWD, bool PAIR>
__global__ void __launch_bounds__(GatedCfg::NTHREADS, 1)
    gated_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmDY,
                 const __grid_constant__ CUtensorMap tmDG, const GatedParams p) {
  using C = GatedCfg;
  using S = GatedSmem<BWD, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
  uint64_t* full = bars;                     // [stages] TMA -> MMA (the leader's; both CTAs' loads)
  uint64_t* empty = full + S::MAX_STAGES;    // [stages] MMA -> TMA
  uint64_t* acc_full = empty + S::MAX_STAGES;   // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;        // [2] epilogue -> MMA (the leader's; both CTAs' warps)
  uint64_t* bias_full = acc_empty + 2;       // [2] bias warp -> epilogue
  uint64_t* bias_empty = bias_full + 2;      // [2] back
  uint64_t* drain_bar = bias_empty + 2;
  uint64_t* dy_full = drain_bar + 1;         // backward pairs: [EPI] each epilogue warp's dy
  float* sbias = reinterpret_cast<float*>(smem + S::OFF_BIAS);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + S::NBAR);   // [0] tensor memory, [1] abort
  volatile uint32_t* abort_flag = misc + 1;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int hn = PAIR ? 128 : p.hn;
  const int tiles = p.rts * p.fts;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
  const int u0 = PAIR ? blockIdx.x / 2 : blockIdx.x, ustep = PAIR ? gridDim.x / 2 : gridDim.x;
  constexpr int TROWS = PAIR ? 256 : 128;    // rows per tile
  constexpr int SUB = PAIR ? 1 : 2;          // contraction steps of 64 per stage
  const int nstages = PAIR ? S::STAGES : p.stages, stage = PAIR ? S::STAGE : p.stage;
  const int off_w = PAIR ? C::A_BYTES : p.tm * 128, sub = off_w + (PAIR ? 128 : 2 * hn) * 128;   // bytes of a step

  if (threadIdx.x == 0) {
    for (int i = 0; i < nstages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], (PAIR ? 2 : 1) * C::EPI);
      mbar_init(&bias_full[i], 1);
      mbar_init(&bias_empty[i], C::EPI);
    }
    mbar_init(drain_bar, 1);
    if (PAIR && BWD)
      for (int i = 0; i < C::EPI; ++i) mbar_init(&dy_full[i], 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    if (PAIR) tma_prefetch_desc(&tmY);
    if (PAIR && BWD) {
      tma_prefetch_desc(&tmDY);
      tma_prefetch_desc(&tmDG);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&misc[0], C::TMEM_COLS);
    } else {
      tmem_alloc(&misc[0], C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();        // both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = misc[0];
  grid_dependency_wait();
  grid_launch_dependents();

  const uint32_t sbase = smem_u32(smem), bfull = smem_u32(full), bempty = smem_u32(empty);
  const uint32_t bacc_full = smem_u32(acc_full), bacc_empty = smem_u32(acc_empty);
  const int chains = BWD ? p.chains : 1;

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    const uint32_t lfull = PAIR ? cluster_addr(bfull, 0) : bfull;
    RingWalk ring(bempty, nstages, 1);
    uint32_t c = 0;
    bool live = true;
    for (int u = u0; u < tiles && live; u += ustep) {
      const int rt = u / p.fts, ft = u - rt * p.fts;
      for (int ks = 0; ks < p.ksteps; ks += SUB, ++c) {
        uint32_t st;
        live = ring.take(st, kSiteKEmpty, abort_flag);
        if (!live) break;
        const uint32_t s = sbase + st * stage, bar = lfull + 8 * st;
        const bool two = SUB == 2 && ks + 1 < p.ksteps;
        if (rank == 0) expect_tx_elect(bfull + 8 * st, PAIR ? 2 * S::STAGE : two ? 2 * sub : sub);
        if constexpr (PAIR) {
          load_elect_pair(s, &tmX, ks * C::BK, rt * TROWS + rank * 128, 0, bar);
          load_elect_pair(s + C::A_BYTES, &tmW, ks * C::BK, ft * hn, rank, bar);
        } else {
          load_elect(s, &tmX, ks * C::BK, rt * TROWS, 0, bar);
          load_elect(s + off_w, &tmW, ks * C::BK, ft * hn, 0, bar);
          load_elect(s + off_w + hn * 128, &tmW, ks * C::BK, ft * hn, 1, bar);
          if (two) {
            load_elect(s + sub, &tmX, (ks + 1) * C::BK, rt * TROWS, 0, bar);
            load_elect(s + sub + off_w, &tmW, (ks + 1) * C::BK, ft * hn, 0, bar);
            load_elect(s + sub + off_w + hn * 128, &tmW, (ks + 1) * C::BK, ft * hn, 1, bar);
          }
        }
      }
    }
    drain_ring(rank == 0 ? bfull : bempty, nstages, c, rank == 0 ? kSiteKFull : kSiteKEmpty);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------ MMA issuer --------------------------------
    const uint32_t idesc = idesc_f16(TROWS, 2 * hn, BF16, false, false);
    const uint64_t adesc = sdesc_sw128(sbase, 16, 1024), bdesc = sdesc_sw128(sbase + off_w, 16, 1024);
    RingWalk ring(bfull, nstages, 0);
    uint32_t ui = 0;
    bool live = true;
    for (int u = u0; u < tiles && live; u += ustep, ++ui) {
      const uint32_t ab = ui & 1, na = ui >> 1;
      // one chain: tiles alternate between the accumulators, and this one was
      // the tile's before last; two: every tile takes both, after the last one
      if (chains == 1) {
        live = wait_warp(bacc_empty + 8 * ab, (na & 1) ^ 1, kSiteAccEmpty, abort_flag);
      } else if (ui > 0) {
        live = wait_warp(bacc_empty + 8 * (ab ^ 1), ((ui - 1) >> 1) & 1, kSiteAccEmpty, abort_flag);
      }
      if (!live) break;
      tc_fence_after();
      // the step where the second chain begins: a whole stage's first
      const int turn = chains == 1 ? p.ksteps : (p.ksteps + 3) / 4 * 2;
      uint32_t d = tmem + (chains == 1 ? ab * 256 : 0), acc = 0;
      for (int ks = 0; ks < p.ksteps; ks += SUB) {
        uint32_t st;
        live = ring.take(st, kSiteKFull, abort_flag);
        if (!live) break;
        tc_fence_after();
        if (BWD && ks == turn) {
          d = tmem + 256;
          acc = 0;
        }
        const uint64_t off = st * (static_cast<uint32_t>(stage) >> 4);
        if constexpr (PAIR) {
          mma_ss4_pair(d, adesc + off, bdesc + off, idesc, acc, 2, 2);
          mma_commit_pair(bempty + 8 * st);
        } else {
          mma_ss4(d, adesc + off, bdesc + off, idesc, acc, 2, 2);
          if (ks + 1 < p.ksteps) {
            const uint64_t off2 = off + (static_cast<uint32_t>(sub) >> 4);
            mma_ss4(d, adesc + off2, bdesc + off2, idesc, 1, 2, 2);
          }
          mma_commit_at(bempty + 8 * st);
        }
        acc = 1;
      }
      if (live) {
        if constexpr (PAIR) {
          mma_commit_pair(bacc_full + 8 * ab);
        } else {
          mma_commit_at(bacc_full + 8 * ab);
        }
      }
    }
    volatile uint32_t never = 0;
    if constexpr (PAIR) {
      mma_commit_pair(smem_u32(drain_bar));
    } else {
      mma_commit_at(smem_u32(drain_bar));
    }
    wait_warp(smem_u32(drain_bar), 0, kSiteAccFull, &never);
  } else if (warp == 2) {
    // ------------------------------ biases ------------------------------------
    uint32_t ui = 0;
    for (int u = u0; u < tiles; u += ustep, ++ui) {
      const uint32_t ab = ui & 1, na = ui >> 1;
      if (!wait_warp(smem_u32(&bias_empty[ab]), (na & 1) ^ 1, kSiteVEmpty, abort_flag)) break;
      const int f = (u % p.fts) * hn;
      for (int j = lane; j < hn; j += 32) {
        const bool ok = p.bias != nullptr && f + j < p.F;   // columns past F take none: their products are zero
        sbias[ab * 256 + j] = ok ? __ldg(p.bias + f + j) : 0.f;
        sbias[ab * 256 + 128 + j] = ok ? __ldg(p.bias + p.F + f + j) * (BWD ? 1.f : 0.5f) : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bias_full[ab]);
    }
  } else if (warp >= 4) {
    // ------------------------------ epilogue ----------------------------------
    constexpr int CW = PAIR ? 16 : 8;             // columns per pass
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stg = smem + S::OFF_STG + (warp - 4) * S::WSTG;
    const uint32_t dyb = smem_u32(&dy_full[warp - 4]), dys = smem_u32(stg);
    uint32_t loads = 0;
    // this warp's dy of tile u: 32 columns of its 32 rows
    auto load_dy = [&](int u) {
      const int rt = u / p.fts, ft = u - rt * p.fts;
      expect_tx_elect(dyb, 2048);
      load_elect(dys, &tmDY, ft * hn + part * 32, rt * TROWS + rank * 128 + quarter * 32, 0, dyb);
      ++loads;
    };
    uint32_t ui = 0;
    if (PAIR && BWD && u0 < tiles) load_dy(u0);
    for (int u = u0; u < tiles; u += ustep, ++ui) {
      const int rt = u / p.fts, ft = u - rt * p.fts;
      const uint32_t ab = ui & 1, na = ui >> 1;
      const int r0 = rt * TROWS + rank * 128 + quarter * 32, row = r0 + lane;
      const bool row_ok = row < p.T;
      const uint16_t* dy_row = static_cast<const uint16_t*>(p.dY) + static_cast<int64_t>(row) * p.F + ft * hn;
      // PAIR: this warp's 32 columns; otherwise every fourth 8 columns
      const int first = PAIR ? part * 32 : part * 8, step = PAIR ? CW : 32, last = PAIR ? first + 32 : hn;
      uint4 next_dy = make_uint4(0, 0, 0, 0);     // without pairs: loaded one pass ahead
      if (BWD && !PAIR && row_ok && ft * hn + first < p.F) next_dy = __ldg(reinterpret_cast<const uint4*>(dy_row + first));
      if (!wait_warp(smem_u32(&bias_full[ab]), na & 1, kSiteVFull, abort_flag) ||
          !wait_warp(bacc_full + 8 * ab, na & 1, kSiteAccFull, abort_flag))
        break;
      tc_fence_after();
      if (PAIR && BWD && !wait_warp(dyb, ui & 1, kSiteQFull, abort_flag)) break;
      if (PAIR && !BWD) {
        if (lane == 0) bulk_wait_read<0>();       // the buffer's previous store has read it
        __syncwarp();
      }
      // The accumulator is free once the warp's last columns are in registers:
      // the next tile but one's products wait for it, not for the arithmetic.
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) {
            arrive_cluster(cluster_addr(bacc_empty + 8 * ab, 0));
          } else {
            mbar_arrive(&acc_empty[ab]);
          }
        }
      };
      if (first >= last) release();               // a narrow tile without columns for this warp
#pragma unroll 1
      for (int c0 = first; c0 < last; c0 += step) {
        const int f = ft * hn + c0;
        uint4 dy[CW / 8];
        if constexpr (BWD && PAIR) {
#pragma unroll
          for (int q = 0; q < CW / 8; ++q)        // zeros past T and F
            dy[q] = *reinterpret_cast<const uint4*>(stg + lane * 64 + ((((c0 & 31) / 8 + q) ^ (lane >> 1 & 3)) << 4));
        } else if constexpr (BWD) {
          dy[0] = next_dy;
          next_dy = row_ok && c0 + step < last && f + step < p.F ? __ldg(reinterpret_cast<const uint4*>(dy_row + c0 + step))
                                                                 : make_uint4(0, 0, 0, 0);
        }
        uint32_t h[CW], g[CW];
        const uint32_t at = tmem + (chains == 1 ? ab * 256 : 0) + c0 + lane_off;
        if constexpr (PAIR) {
          tmem_ld_x16(at, h);
          tmem_ld_x16(at + hn, g);
        } else {
          tmem_ld_x8(at, h);
          tmem_ld_x8(at + hn, g);
        }
        tmem_wait_ld();
        reg_fence<CW>(h);
        reg_fence<CW>(g);
        if (BWD && chains == 2) {                 // the second chain's sums
          uint32_t h2[CW], g2[CW];
          if constexpr (PAIR) {
            tmem_ld_x16(at + 256, h2);
            tmem_ld_x16(at + 256 + hn, g2);
          } else {
            tmem_ld_x8(at + 256, h2);
            tmem_ld_x8(at + 256 + hn, g2);
          }
          tmem_wait_ld();
          reg_fence<CW>(h2);
          reg_fence<CW>(g2);
#pragma unroll
          for (int j = 0; j < CW; ++j) {
            h[j] = __float_as_uint(__uint_as_float(h[j]) + __uint_as_float(h2[j]));
            g[j] = __float_as_uint(__uint_as_float(g[j]) + __uint_as_float(g2[j]));
          }
        }
        if (c0 + step >= last) release();
        const float* bh = sbias + ab * 256 + c0;
        float o0[CW], o1[CW];
#pragma unroll
        for (int q = 0; q < CW / 8; ++q)
          gated_columns8<BWD, BF16>(h + 8 * q, g + 8 * q, bh + 8 * q, bh + 128 + 8 * q, dy[q], o0 + 8 * q, o1 + 8 * q);
        if constexpr (PAIR) {
#pragma unroll
          for (int q = 0; q < CW / 8; ++q) {
            // rows of 64 bytes, 64-byte swizzle: chunk ^ row / 2
            const int ch = (((c0 & 31) / 8 + q) ^ (lane >> 1 & 3)) << 4;
            *reinterpret_cast<uint4*>(stg + lane * 64 + ch) = pack8<BF16>(o0 + 8 * q);
            if constexpr (BWD) *reinterpret_cast<uint4*>(stg + 2048 + lane * 64 + ch) = pack8<BF16>(o1 + 8 * q);
          }
          if (c0 + CW == last) {
            fence_proxy_async_smem();
            __syncwarp();
            // stores start inside the tensor; what runs over its edges is clipped
            const int fs = ft * hn + first;
            if (lane == 0 && r0 < p.T && fs < p.F) {
              tma_store_3d(&tmY, stg, fs, r0, 0);
              if constexpr (BWD) tma_store_3d(&tmDG, stg + 2048, fs, r0, 0);
              bulk_commit();
            }
          }
        } else if (row_ok && f < p.F) {
          uint16_t* dst = static_cast<uint16_t*>(p.Y) + static_cast<int64_t>(row) * (BWD ? 2 * p.F : p.F) + f;
          *reinterpret_cast<uint4*>(dst) = pack8<BF16>(o0);
          if constexpr (BWD) *reinterpret_cast<uint4*>(dst + p.F) = pack8<BF16>(o1);
        }
        if constexpr (BWD) {
          if (p.part != nullptr) {
            if (r0 + 32 > p.T) {                  // rows past T add nothing, whatever their biases are
#pragma unroll
              for (int j = 0; j < CW; ++j) {
                o0[j] = row_ok ? o0[j] : 0.f;
                o1[j] = row_ok ? o1[j] : 0.f;
              }
            }
            const float s0 = warp_column_sums<CW>(o0, lane), s1 = warp_column_sums<CW>(o1, lane);
            const int j = lane / (32 / CW);
            if (lane % (32 / CW) == 0 && f + j < p.F && r0 < p.T) {
              float* dst = p.part + static_cast<int64_t>(r0 / 32) * 2 * p.F + f + j;
              dst[0] = s0;
              dst[p.F] = s1;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bias_empty[ab]);
      if (PAIR && BWD && u + ustep < tiles) {     // the next tile's dy, over dh once its store has read it
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        load_dy(u + ustep);
      }
    }
    if (PAIR && BWD && loads > 0) {               // the last dy has landed, also where the loop gave up
      volatile uint32_t never = 0;
      wait_warp(dyb, (loads - 1) & 1, kSiteQFull, &never);
    }
    if (PAIR && lane == 0) bulk_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) pair_exit(smem_u32(drain_bar));
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) {
      tmem_dealloc_pair(tmem, C::TMEM_COLS);
    } else {
      tmem_dealloc(tmem, C::TMEM_COLS);
    }
  }
}

// ---------------------------------------------------------------------------
// dx = P W and dW = P^T x in one launch, on CTA pairs.  A unit is a 256-row
// tile of one of the two results, up to 320 of its columns, over one split of
// the contraction; units of both results are dealt out together, so that
// neither product leaves SMs idle while the other runs.
//   dx: A = P [T][2F], K-major;  B = W [2F][C], N-major (its rows run along N)
//   dW: A = P, M-major (P^T);    B = x [T][C], N-major
// Each CTA of a pair holds its 128 rows of A and half of the tile's columns of
// B.  M- and N-major tiles are slabs of 64 columns x 64 contraction rows,
// 128-byte swizzled.  A result whose contraction is split goes to fp32
// partials that finish_kernel adds in split order.
//
// Bound by operand loads: a step of a 320-column tile brings 40 KB to each SM,
// some 900 clocks at the 45 bytes per clock that L2 gives every SM at once,
// against 640 clocks of products.  (8192 rows, C = 320, F = 1280: both products,
// 26.8 GFLOP, in 29 us cold; a warp each for A's and B's loads changed nothing.)
// ---------------------------------------------------------------------------
struct ProductCfg {
  static constexpr int BK = 64;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int SLAB = 64 * 128;             // 64 columns x 64 contraction rows
  static constexpr int BN = 320;                    // most columns of a tile, half of them in each CTA
  static constexpr int STAGE = A_BYTES + 3 * SLAB;
  static constexpr int STAGES = 4;
  static constexpr int EPI = 16;                    // epilogue warps
  static constexpr int OFF_STG = STAGES * STAGE;    // [EPI] 32 rows x 32 columns of up to 4 bytes
  static constexpr int OFF_BAR = OFF_STG + EPI * 4096;
  static constexpr int NBAR = 2 * STAGES + 4 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr int NTHREADS = (4 + EPI) * 32;
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct ProductSide {
  int M, N;           // the result's rows and columns
  int bn;             // columns per tile, a multiple of 64 up to 320
  int nts;            // column tiles
  int mn;             // row tiles (of 256) x column tiles
  int splits;         // of the contraction
  int ksteps, kper;   // contraction steps of 64: in all, per split
  int units;          // mn * splits
};

struct ProductParams {
  ProductSide s[2];   // 0: dx, 1: dW
  int first;          // the side whose units are longer
  int wide;           // tiles of more than 256 columns: one accumulator
  // The long units go to the pairs in turn; the pairs [heavy, pairs) then have
  // one fewer and get up to `fill` short units each, at most a long one's worth
  // and no more than their even share; the others go to all pairs in turn.
  int heavy, fill;
};

// The k-th unit of a pair, or -1.
__device__ __forceinline__ int product_deal(const ProductParams& p, int pair, int pairs, int k) {
  const int n1 = p.s[p.first].units, n2 = p.s[1 - p.first].units;
  const int longs = (n1 - pair + pairs - 1) / pairs;
  if (k < longs) return pair + k * pairs;
  k -= longs;
  if (pair >= p.heavy) {
    const int own = min(max(n2 - (pair - p.heavy) * p.fill, 0), p.fill);
    if (k < own) return n1 + (pair - p.heavy) * p.fill + k;
    k -= own;
  }
  const int u = min(n2, (pairs - p.heavy) * p.fill) + pair + k * pairs;
  return u < n2 ? n1 + u : -1;
}

struct ProductUnit {
  int side, m0, n0, cols, half, split, k0, k1;
};

__device__ __forceinline__ ProductUnit product_unit(const ProductParams& p, int u) {
  ProductUnit r;
  const int n1 = p.s[p.first].units;
  r.side = u < n1 ? p.first : 1 - p.first;
  if (u >= n1) u -= n1;
  const ProductSide& s = p.s[r.side];
  r.split = u / s.mn;
  const int t = u - r.split * s.mn, mt = t / s.nts, nt = t - mt * s.nts;
  r.m0 = mt * 256;
  r.n0 = nt * s.bn;
  r.cols = min(s.bn, s.N - r.n0);
  r.half = r.cols > 256 ? 160 : (r.cols + 31) / 32 * 16;   // columns of B in each CTA
  r.k0 = r.split * s.kper;
  r.k1 = min(s.ksteps, r.k0 + s.kper);
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(ProductCfg::NTHREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmPk, const __grid_constant__ CUtensorMap tmPm,
                   const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmO0, const __grid_constant__ CUtensorMap tmO1,
                   const __grid_constant__ ProductParams p) {
  using C = ProductCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                     // [STAGES] both CTAs' loads -> MMA (the leader's)
  uint64_t* empty = full + C::STAGES;        // [STAGES] MMA -> TMA
  uint64_t* acc_full = empty + C::STAGES;    // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;        // [2] both CTAs' epilogues -> MMA (the leader's)
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = misc + 1;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * C::EPI);
    }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmPk);
    tma_prefetch_desc(&tmPm);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmO0);
    tma_prefetch_desc(&tmO1);
  }
  if (warp == 1) tmem_alloc_pair(&misc[0], C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint32_t sbase = smem_u32(smem), bfull = smem_u32(full), bempty = smem_u32(empty);
  const uint32_t bacc_full = smem_u32(acc_full), bacc_empty = smem_u32(acc_empty);
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    const uint32_t lfull = cluster_addr(bfull, 0);
    RingWalk ring(bempty, C::STAGES, 1);
    uint32_t c = 0;
    bool live = true;
    for (int ui = 0; live; ++ui) {
      const int u = product_deal(p, pair, pairs, ui);
      if (u < 0) break;
      const ProductUnit t = product_unit(p, u);
      const int slabs = (t.half + 63) / 64, m = t.m0 + rank * 128, n = t.n0 + rank * t.half;
      for (int ks = t.k0; ks < t.k1; ++ks, ++c) {
        uint32_t st;
        live = ring.take(st, kSiteKEmpty, abort_flag);
        if (!live) break;
        const uint32_t s = sbase + st * C::STAGE, bar = lfull + 8 * st;
        const int k = ks * C::BK;
        if (rank == 0) expect_tx_elect(bfull + 8 * st, 2 * (C::A_BYTES + slabs * C::SLAB));
        if (t.side == 0) {
          load_elect_pair(s, &tmPk, k, m, 0, bar);
          load_elect_pair(s + C::A_BYTES, &tmW, n, k, 0, bar);
          if (slabs > 1) load_elect_pair(s + C::A_BYTES + C::SLAB, &tmW, n + 64, k, 0, bar);
          if (slabs > 2) load_elect_pair(s + C::A_BYTES + 2 * C::SLAB, &tmW, n + 128, k, 0, bar);
        } else {
          load_elect_pair(s, &tmPm, m, k, 0, bar);
          load_elect_pair(s + C::SLAB, &tmPm, m + 64, k, 0, bar);
          load_elect_pair(s + C::A_BYTES, &tmX, n, k, 0, bar);
          if (slabs > 1) load_elect_pair(s + C::A_BYTES + C::SLAB, &tmX, n + 64, k, 0, bar);
          if (slabs > 2) load_elect_pair(s + C::A_BYTES + 2 * C::SLAB, &tmX, n + 128, k, 0, bar);
        }
      }
    }
    drain_ring(rank == 0 ? bfull : bempty, C::STAGES, c, rank == 0 ? kSiteKFull : kSiteKEmpty);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------ MMA issuer --------------------------------
    RingWalk ring(bfull, C::STAGES, 0);
    bool live = true;
    for (uint32_t ui = 0; live; ++ui) {
      const int u = product_deal(p, pair, pairs, ui);
      if (u < 0) break;
      const ProductUnit t = product_unit(p, u);
      const uint32_t ab = p.wide ? 0 : ui & 1, na = p.wide ? ui : ui >> 1;
      const uint32_t idesc = idesc_f16(256, 2 * min(t.half, 128), BF16, t.side == 1, true);
      const uint32_t idesc2 = idesc_f16(256, 64, BF16, t.side == 1, true);   // each CTA's columns from 128 on
      // A: 32 bytes along a K-major row, or 16 contraction rows of an M-major slab, per 16 of K
      const uint64_t adesc = sdesc_sw128(sbase, t.side == 1 ? C::SLAB : 16, 1024), astep = t.side == 1 ? 128 : 2;
      const uint64_t bdesc = sdesc_sw128(sbase + C::A_BYTES, C::SLAB, 1024);
      live = wait_warp(bacc_empty + 8 * ab, (na & 1) ^ 1, kSiteAccEmpty, abort_flag);
      if (!live) break;
      tc_fence_after();
      uint32_t acc = 0;
      for (int ks = t.k0; ks < t.k1; ++ks) {
        uint32_t st;
        live = ring.take(st, kSiteKFull, abort_flag);
        if (!live) break;
        tc_fence_after();
        const uint64_t off = st * (C::STAGE >> 4);
        mma_ss4_pair(tmem + ab * 256, adesc + off, bdesc + off, idesc, acc, astep, 128);
        if (t.half > 128) mma_ss4_pair(tmem + 256, adesc + off, bdesc + off + 2 * (C::SLAB >> 4), idesc2, acc, astep, 128);
        mma_commit_pair(bempty + 8 * st);
        acc = 1;
      }
      if (live) mma_commit_pair(bacc_full + 8 * ab);
    }
    volatile uint32_t never = 0;
    mma_commit_pair(smem_u32(drain_bar));
    wait_warp(smem_u32(drain_bar), 0, kSiteAccFull, &never);
  } else if (warp >= 4) {
    // ------------------------------ epilogue ----------------------------------
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stg = smem + C::OFF_STG + (warp - 4) * 4096;
    for (uint32_t ui = 0;; ++ui) {
      const int u = product_deal(p, pair, pairs, ui);
      if (u < 0) break;
      const ProductUnit t = product_unit(p, u);
      const ProductSide& sd = p.s[t.side];
      const CUtensorMap* tmO = t.side == 0 ? &tmO0 : &tmO1;
      const uint32_t ab = p.wide ? 0 : ui & 1, na = p.wide ? ui : ui >> 1;
      const int r0 = t.m0 + rank * 128 + quarter * 32;
      if (!wait_warp(bacc_full + 8 * ab, na & 1, kSiteAccFull, abort_flag)) break;
      tc_fence_after();
      const bool f32 = sd.splits > 1;
      auto release = [&]() {                    // as in gated_kernel
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(bacc_empty + 8 * ab, 0));
      };
      // pieces of 32 columns, the four warps of a quarter in turn; TMA clips at
      // the result's edges
      if (part * 32 >= t.cols || r0 >= sd.M) release();
#pragma unroll 1
      for (int c0 = part * 32; c0 < t.cols && r0 < sd.M; c0 += 128) {
        // where a wide tile's column lies: each CTA's first 128, then the others
        const int q = c0 >= t.half ? 1 : 0, l = c0 - q * t.half;
        const int at = t.half <= 128 ? c0 : l < 128 ? q * 128 + l : 256 + q * 32 + l - 128;
        uint32_t v[32];
        tmem_ld_x32(tmem + ab * 256 + at + lane_off, v);
        tmem_wait_ld();
        reg_fence<32>(v);
        if (c0 + 128 >= t.cols) release();
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        if (f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
                pack8<BF16>(reinterpret_cast<const float*>(v) + 8 * j);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(tmO, stg, t.n0 + c0, r0, t.split);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  pair_exit(smem_u32(drain_bar));
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM_COLS);
  }
}

// What remains after the products, in one launch: the split results' sums, out[i]
// = sum over splits of part[split][i] in split order (n a multiple of 8), and db
// from its partial rows (blocks from `first` on, as in column_sum_kernel).
struct FinishParams {
  const float* part[2];   // null where a side was not split
  void* out[2];
  int64_t n[2];
  int splits[2];
  const float* db_part;   // [rows][cols], or null
  float* db;
  int64_t rows;
  int cols;
  int first;              // blocks of the split results
};

template <bool BF16>
__global__ void __launch_bounds__(1024) finish_kernel(const FinishParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.first) {
    column_sum_block(p.db_part, p.rows, p.cols, p.cols, p.db, p.db, blockIdx.x - p.first);
    return;
  }
  const int64_t stride = static_cast<int64_t>(p.first) * blockDim.x;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (p.part[side] == nullptr) continue;
    const int64_t n = p.n[side];
    // a warp's 32 pieces together, warps dealt over the blocks
    const int64_t i0 = (static_cast<int64_t>(threadIdx.x >> 5) * p.first + blockIdx.x) * 32 + (threadIdx.x & 31);
    for (int64_t i = i0; i < n / 8; i += stride) {
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int s = 0; s < p.splits[side]; ++s) {
        const float4* src = reinterpret_cast<const float4*>(p.part[side] + s * n) + 2 * i;
        const float4 u = __ldcs(src), v = __ldcs(src + 1);
        a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
        a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
      }
      reinterpret_cast<uint4*>(p.out[side])[i] = pack8<BF16>(a);
    }
  }
}

}  // namespace sdattn

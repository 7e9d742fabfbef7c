// adapter.cuh -- a projection shared by all requests with a low-rank adapter
// of its own for each, in one kernel:
//
//   y[t] = x[t] W^T + bias + s_i (x[t] D_i^T) U_i^T,      i = ids[t / rows]
//
// x [T][C], W [K][C], D [L][R][C] (down), U [L][K][R] (up), s [L]; a row whose
// id is outside 0 .. L-1 takes the projection alone.  These are the
// projections around the UNet's attention, with one style adapter per image of
// the batch.
//
// A tile is 128 rows by bn columns.  The D rows of the tile's adapters lie
// behind W's in shared memory, so one product of bn + 16 .. 64 columns gives
// x W^T and z = x D^T side by side, with no second pass over x; z goes
// from tensor memory through registers (scaled by s in fp32, then as two 16-bit
// parts, the next product's operands) back to tensor memory, and as the A operand
// of z U^T adds onto the same fp32 accumulator as x W^T, in the lanes of that
// adapter's rows alone: a request never meets another's U, infinities included.
// Nothing but x, W, the adapters in use and y touches global memory, and W and x
// are never copied per request.
//
// Rows of different adapters may share a tile.  The planner warp lists a
// tile's distinct adapters; each contributes ceil(R / 64) slots of rc ranks
// (R rounded up to 16, at most 64), and 64 / rc slots fit a phase.  Phase 0
// runs with x W^T; a tile of more slots runs through x again, once per phase,
// against D alone.  The MMA warp starts the next phase's (or tile's) x
// products and adds the last one's z U^T half way through them, so that the
// conversion of z passes under products.
//
// Few rows with an adapter each (the time embedding's projection, single
// tokens) would cost a phase for every few rows.  There the adapters are
// per-row work, bound by reading D and U once for each row: adapter_z_kernel
// computes z with plain fp32 sums (a warp per row and two ranks); in the
// projection's kernel the epilogue's warps compute z U^T while the products
// run (a thread per row and two columns) and leave it in shared memory.
//
// Measured: 16 images at 64x64 (65536 rows, C = K = 320, 8 adapters of rank 16)
// 31.5 us, 2.7 TB/s, the plain projection 19.5 us (a library product: 18.4 us;
// 16384 x 1280 to 1280: 52 us and 40 us); 154 rows of 768 to 320, 2 adapters,
// 6.6 us; 48 single rows of 1280, 12 adapters of rank 32, 9.0 us.  Few rows are
// chains of latencies.  Many rows are
// bound by the operands' way to each SM, x and W's tile anew for every tile
// (36 KB a step, 45 bytes per clock at best); D's third box adds 6 us to the
// first figure whatever its size, and U and the hand-off of z 7 us.
#pragma once

#include "pipeline.cuh"
#include "unet_ops.cuh"

namespace sdattn {

enum : int { kAdapterNone = 0, kAdapterRows = 1, kAdapterMma = 2 };

struct AdapterCfg {
  static constexpr int BK = 64;
  static constexpr int BN = 160;                    // most columns per tile
  static constexpr int BN_ROWS = 64;                // with per-row adapters
  static constexpr int ZN = 64;                     // ranks per phase
  static constexpr int MAX_STAGES = 12;
  static constexpr int SLACK = 16384;               // kept behind the stages when x's tile is short: its products read up to 16 KB
  static constexpr int RING = 180224;               // bytes of the ring of stages, and with per-row adapters of z U^T behind it
  static constexpr int CORR = 128 * (BN_ROWS + 4) * 4;
  static constexpr int EPI = 16;                    // epilogue warps, four per quarter of a tile's rows
  static constexpr int PW = 40;                     // most columns of an epilogue warp
  static constexpr int OFF_STG = RING;              // [EPI] 32 rows of up to PW columns of y
  static constexpr int STG = 32 * PW * 2;
  static constexpr int PLANS = 3;                   // tiles the planner may run ahead
  static constexpr int PLAN = 128 * 4 + 128 * 4 + 128 * 4 + 16;   // adapters, rows' places, rows' scales, count
  static constexpr int OFF_PLAN = OFF_STG + EPI * STG;
  static constexpr int OFF_BIAS = OFF_PLAN + PLANS * PLAN;   // [EPI] biases of up to PW columns
  static constexpr int OFF_BAR = OFF_BIAS + EPI * PW * 4;
  static constexpr int NBAR = 2 * MAX_STAGES + 4 + 4 + 2 * PLANS + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr int NTHREADS = (8 + EPI) * 32;   // TMA, MMA, planner, TMA, epilogue, four that convert z
  static constexpr int CORR_THREADS = (4 + EPI) * 32;   // that compute z U^T of single rows
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int TM_TILE = 256;               // tensor-memory columns of a tile: its accumulator, then z
  __host__ __device__ static constexpr int ring(int mode) { return mode == kAdapterRows ? RING - CORR : RING; }
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct AdapterParams {
  const float* bias;      // [K], on 16 bytes, or null
  const int32_t* ids;     // [T / rows], or null: no adapters
  const float* scale;     // [L], or null: ones
  const float* z;         // ROWS: [T][R], scaled
  const void* U;          // ROWS: [L][K][R]
  void* Y;                // [T][K]
  int T, K, L, R, rows;   // rows: rows per id
  int bn;                 // columns per tile: a multiple of 16 up to 160
  int pw;                 // columns per epilogue warp: a multiple of 8 up to 40 that divides bn, bn / pw <= 4
  int tm;                 // rows per tile: 128, or all rows of a shorter x rounded up to 8
  int rts, nts;           // row tiles, column tiles
  int ksteps;             // ceil(C / 64)
  int rc;                 // ranks per slot: 16, 32, 48 or 64
  int chunks;             // slots per adapter: ceil(R / 64)
  int stages, stage;      // of the ring: how many, bytes of one (each step: x, then W or U, then D)
  int sub;                // contraction steps of 64 per stage: two (half the waits per step) where three such stages fit, else one
};

// z[t][r] = s_i x[t] . D_i[r], one warp per row and pair of ranks.
template <bool BF16>
__global__ void __launch_bounds__(256) adapter_z_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ D,
                                                        const float* __restrict__ scale, const int32_t* __restrict__ ids,
                                                        float* __restrict__ z, int T, int C, int L, int R, int rows) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / (R / 2)), r = static_cast<int>(w - static_cast<int64_t>(t) * (R / 2)) * 2;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= T) return;
  const int id = __ldg(ids + t / rows);
  if (id < 0 || id >= L) return;                    // nobody reads this row of z
  const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(t) * C);
  const uint4* d0 = reinterpret_cast<const uint4*>(D + (static_cast<int64_t>(id) * R + r) * C);
  const uint4* d1 = reinterpret_cast<const uint4*>(D + (static_cast<int64_t>(id) * R + r + 1) * C);
  float a = 0.f, b = 0.f;
#pragma unroll 5
  for (int i = lane; i < C / 8; i += 32) {
    float fx[8], f0[8], f1[8];
    unpack8<BF16>(__ldg(x + i), fx);
    unpack8<BF16>(__ldg(d0 + i), f0);
    unpack8<BF16>(__ldg(d1 + i), f1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a = fmaf(fx[e], f0[e], a);
      b = fmaf(fx[e], f1[e], b);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    b += __shfl_xor_sync(0xffffffffu, b, off);
  }
  if (lane == 0) {
    const float s = scale != nullptr ? __ldg(scale + id) : 1.f;
    *reinterpret_cast<float2*>(z + static_cast<int64_t>(t) * R + r) = make_float2(a * s, b * s);
  }
}

// a as the sum of two values of the element type, right to 2^-13 (bf16) or 2^-19
// (fp16) of a: rounded once, z would add as much again to y's error as y's own
// rounding, and a request's y would depend on which form its call takes.  hi is
// a little below a in magnitude, so that lo is never zero beside it and has its
// sign: both parts' products with an infinite U are the formula's infinity.
template <bool BF16>
__device__ __forceinline__ void split_z(float a, float& hi, float& lo) {
  if constexpr (BF16) {
    hi = __uint_as_float(__float_as_uint(a * (1.f - 0x1p-7f)) & 0xffff0000u);
  } else {
    hi = __half2float(__float2half_rz(a * (1.f - 0x1p-10f)));
  }
  lo = fabsf(a) < __int_as_float(0x7f800000) ? a - hi : a;   // an infinity twice
}

// One tile's plan in shared memory.
struct AdapterPlan {
  int32_t adapter[128];   // the distinct adapters, in order of first appearance
  int32_t place[128];     // each row's place in that list, -1 without one
  float scale[128];       // each row's scale
  int32_t count;          // adapters
  int32_t slots, phases;  // count * chunks, and the phases they fill (at least one)
  int32_t pad;
};
static_assert(sizeof(AdapterPlan) == AdapterCfg::PLAN, "plan layout");

// z U^T of the tile's rows and columns into corr, by the threads of the
// warps from 4 on: a thread takes a row and two columns at a time.  Rows without an
// adapter get zeros.
template <bool BF16>
__device__ __forceinline__ void adapter_corr(const AdapterParams& p, float* corr, int row0, int n0) {
  const int pairs = p.bn / 2, rows = min(p.tm, p.T - row0);
  for (int i = threadIdx.x - 128; i < rows * pairs; i += AdapterCfg::CORR_THREADS) {
    const int r = i / pairs, c = (i - r * pairs) * 2, row = row0 + r, n = n0 + c;
    float a = 0.f, b = 0.f;
    const int id = __ldg(p.ids + row / p.rows);
    if (id >= 0 && id < p.L && n < p.K) {
      const float4* z = reinterpret_cast<const float4*>(p.z + static_cast<int64_t>(row) * p.R);
      const uint4* u0 = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.U) + (static_cast<int64_t>(id) * p.K + n) * p.R);
      const uint4* u1 = u0 + p.R / 8;
#pragma unroll 4
      for (int q = 0; q < p.R / 8; ++q) {
        const float4 z0 = __ldg(z + 2 * q), z1 = __ldg(z + 2 * q + 1);
        const float zz[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
        float w0[8], w1[8];
        unpack8<BF16>(__ldg(u0 + q), w0);
        unpack8<BF16>(__ldg(u1 + q), w1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a = fmaf(zz[e], w0[e], a);
          b = fmaf(zz[e], w1[e], b);
        }
      }
    }
    *reinterpret_cast<float2*>(corr + r * (p.bn + 4) + c) = make_float2(a, b);
  }
}

template <bool BF16, int MODE>
__global__ void __launch_bounds__(AdapterCfg::NTHREADS, 1)
    adapter_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmU,
                   const __grid_constant__ CUtensorMap tmY, const AdapterParams p) {
  using C = AdapterCfg;
  constexpr bool MMA = MODE == kAdapterMma, ROWS = MODE == kAdapterRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                      // [stages] TMA -> MMA
  uint64_t* empty = full + C::MAX_STAGES;     // [stages] MMA -> TMA
  uint64_t* acc_full = empty + C::MAX_STAGES; // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;         // [2] epilogue -> MMA
  uint64_t* z_full = acc_empty + 2;           // [2] MMA -> conversion: z is complete
  uint64_t* p_full = z_full + 2;              // [2] conversion -> MMA
  uint64_t* plan_full = p_full + 2;           // [PLANS] planner -> both TMA, MMA, conversion
  uint64_t* plan_empty = plan_full + C::PLANS;   // [PLANS] back
  uint64_t* drain_bar = plan_empty + C::PLANS;
  uint32_t* misc = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = misc + 1;
  AdapterPlan* plans = reinterpret_cast<AdapterPlan*>(smem + C::OFF_PLAN);
  float* corr = reinterpret_cast<float*>(smem + C::ring(MODE));   // ROWS: [128][bn + 4], z U^T of the tile
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int tiles = p.rts * p.nts;
  const int spp = C::ZN / p.rc;               // slots per phase
  const uint32_t NS = p.stages;
  const uint32_t sbase = smem_u32(smem), bfull = smem_u32(full), bempty = smem_u32(empty);
  const int off_w = p.tm * 128, off_d = off_w + p.bn * 128;
  const int sub = off_d + (MMA ? C::ZN * 128 : 0);   // bytes of a step
  const int mid = p.ksteps / 2 / p.sub * p.sub;   // the step of x's products after which the last phase's z U^T goes

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], C::EPI);
      mbar_init(&z_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    for (int i = 0; i < C::PLANS; ++i) {
      mbar_init(&plan_full[i], 1);
      mbar_init(&plan_empty[i], 7);
    }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmY);
    if (MMA) {
      tma_prefetch_desc(&tmD);
      tma_prefetch_desc(&tmU);
    }
  }
  if (warp == 1) {
    tmem_alloc(&misc[0], C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  grid_dependency_wait();
  grid_launch_dependents();

  // slots of phase ph of a tile
  auto slots_of = [&](int slots, int ph) { return min(spp, slots - ph * spp); };

  if (warp == 2) {
    // ------------------------------ planner -----------------------------------
    uint32_t ui = 0;
    for (int u = blockIdx.x; MMA && u < tiles; u += gridDim.x, ++ui) {
      const uint32_t pb = ui % C::PLANS, n = ui / C::PLANS;
      if (!wait_warp(smem_u32(&plan_empty[pb]), (n & 1) ^ 1, kSiteTicket, abort_flag)) break;
      AdapterPlan* pl = &plans[pb];
      const int r0 = u / p.nts * p.tm;
      int id[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = lane + 32 * q;
        id[q] = -1;
        if (r < p.tm && r0 + r < p.T) {
          const int v = __ldg(p.ids + (r0 + r) / p.rows);
          if (v >= 0 && v < p.L) id[q] = v;
        }
        pl->scale[r] = id[q] >= 0 ? (p.scale != nullptr ? __ldg(p.scale + id[q]) : 1.f) : 0.f;
        pl->place[r] = -1;
      }
      int count = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        for (;;) {
          const uint32_t m = __ballot_sync(0xffffffffu, id[q] >= 0);
          if (m == 0) break;
          const int a = __shfl_sync(0xffffffffu, id[q], __ffs(m) - 1);
          if (lane == 0) pl->adapter[count] = a;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (id[j] == a) {
              pl->place[lane + 32 * j] = count;
              id[j] = -1;
            }
          ++count;
        }
      }
      if (lane == 0) {
        pl->count = count;
        pl->slots = count * p.chunks;
        pl->phases = max(1, (count * p.chunks + spp - 1) / spp);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&plan_full[pb]);
    }
  } else if (warp == 0 || warp == 3) {
    // ------------------------------ TMA producers -----------------------------
    // Warp 0 loads x, warp 3 W, D and U, both walking the same stages (16 images at
    // 64x64 with 8 adapters: 34.5 us from one warp, 32.8 from two).
    const bool lead = warp == 0;
    RingWalk ring(bempty, NS, 1);
    uint32_t c = 0, ui = 0;
    bool live = true, pend = false, pend_last = false;
    int pend_ph = 0, pend_n0 = 0;
    uint32_t pend_pb = 0, pend_zr = 0;
    for (int u = blockIdx.x; live && (MMA || u < tiles); u += gridDim.x, ++ui) {
      const bool more = !MMA || u < tiles;      // one turn past the last tile: its last phase's U tiles
      if (MMA && u >= tiles && !pend) break;
      const int rt = u / p.nts, n0 = (u - rt * p.nts) * p.bn;
      const uint32_t pb = ui % C::PLANS;
      int slots = 0, nph = 1;
      if (MMA && more) {
        live = wait_warp(smem_u32(&plan_full[pb]), (ui / C::PLANS) & 1, kSiteTicket, abort_flag);
        if (!live) break;
        slots = plans[pb].slots;
        nph = plans[pb].phases;
      }
      const int steps = more ? p.ksteps : 1;
      for (int ph = 0; ph < nph && live; ++ph) {
        const int ns = MMA && more ? slots_of(slots, ph) : 0;
        const uint32_t zr = (ui + ph) & 1;        // the tensor memory of this phase's z
        // the last phase's U tiles: half way through this one's steps, or before
        // them where this one's z takes the last one's place (after a tile of an
        // even number of phases)
        const int when = pend && pend_zr == zr ? -1 : mid;
        const uint32_t bytes = p.tm * 128 + (ph == 0 ? p.bn * 128 : 0) + ns * p.rc * 128;
        int da[4], dr[4];                         // the slots' adapters and first ranks
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int sl = ph * spp + j;
          da[j] = j < ns ? plans[pb].adapter[sl / p.chunks] : 0;
          dr[j] = sl % p.chunks * 64;
        }
        for (int ks = when < 0 ? -p.sub : 0; ks < steps; ks += p.sub) {
          if (more && ks >= 0) {
            uint32_t st;
            live = ring.take(st, kSiteKEmpty, abort_flag);
            if (!live) break;
            const uint32_t s = sbase + st * p.stage, bar = bfull + 8 * st;
            const bool two = p.sub == 2 && ks + 1 < steps;
            if (lead) {
              expect_tx_elect(bar, two ? 2 * bytes : bytes);
              load_elect(s, &tmX, ks * C::BK, rt * p.tm, 0, bar);
              if (two) load_elect(s + sub, &tmX, (ks + 1) * C::BK, rt * p.tm, 0, bar);
            } else {
              if (ph == 0) {
                load_elect(s + off_w, &tmW, ks * C::BK, n0, 0, bar);
                if (two) load_elect(s + sub + off_w, &tmW, (ks + 1) * C::BK, n0, 0, bar);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j < ns) {
                  load_elect(s + off_d + j * p.rc * 128, &tmD, ks * C::BK, dr[j], da[j], bar);
                  if (two) load_elect(s + sub + off_d + j * p.rc * 128, &tmD, (ks + 1) * C::BK, dr[j], da[j], bar);
                }
              }
            }
            ++c;
          }
          if (MMA && pend && (ks == mid || ks < 0 || !more)) {
            // the U tiles of the last phase, one stage per slot
            const AdapterPlan* pl = &plans[pend_pb];
            const int nu = slots_of(pl->slots, pend_ph);
            for (int j = 0; j < nu; ++j) {
              uint32_t st;
              live = ring.take(st, kSiteKEmpty, abort_flag);
              if (!live) break;
              const int sl = pend_ph * spp + j;
              const uint32_t bar = bfull + 8 * st;
              if (lead) {
                expect_tx_elect(bar, p.bn * 128);
              } else {
                load_elect(sbase + st * p.stage + off_w, &tmU, sl % p.chunks * 64, pend_n0, pl->adapter[sl / p.chunks], bar);
              }
              ++c;
            }
            if (!live) break;
            if (pend_last) arrive_elect(smem_u32(&plan_empty[pend_pb]));
            pend = false;
          }
        }
        if (ns > 0) {
          pend = true;
          pend_ph = ph;
          pend_n0 = n0;
          pend_pb = pb;
          pend_zr = zr;
          pend_last = ph == nph - 1;
        } else if (MMA && more) {
          arrive_elect(smem_u32(&plan_empty[pb]));   // a tile without adapters
        }
      }
      if (!more) break;
    }
    drain_ring(bfull, NS, c, kSiteKFull);
  } else if (warp == 1) {
    // ------------------------------ MMA issuer --------------------------------
    const uint32_t idesc_w = idesc_f16(128, p.bn, BF16, false, false);
    const uint64_t xdesc = sdesc_sw128(sbase, 16, 1024), wdesc = sdesc_sw128(sbase + off_w, 16, 1024);
    const uint64_t ddesc = sdesc_sw128(sbase + off_d, 16, 1024);   // W's rows, then D's: one operand
    RingWalk ring(bfull, NS, 0);
    uint32_t ui = 0, zc = 0;                    // tiles, phases with adapters
    bool live = true, pend = false, pend_last = false;
    int pend_ph = 0, pend_slots = 0;
    uint32_t pend_pb = 0, pend_ab = 0, pend_z = 0, pend_zr = 0;
    for (int u = blockIdx.x; live && (MMA || u < tiles); u += gridDim.x, ++ui) {
      const bool more = !MMA || u < tiles;      // as in the producer
      if (MMA && u >= tiles && !pend) break;
      const uint32_t ab = ui & 1, na = ui >> 1, pb = ui % C::PLANS;
      int slots = 0, nph = 1;
      if (more) {
        if (MMA) {
          live = wait_warp(smem_u32(&plan_full[pb]), (ui / C::PLANS) & 1, kSiteTicket, abort_flag);
          if (!live) break;
          slots = plans[pb].slots;
          nph = plans[pb].phases;
        }
        live = wait_warp(smem_u32(&acc_empty[ab]), (na & 1) ^ 1, kSiteAccEmpty, abort_flag);
        if (!live) break;
        tc_fence_after();
      }
      const int steps = more ? p.ksteps : 1;
      for (int ph = 0; ph < nph && live; ++ph) {
        const int ns = MMA && more ? slots_of(slots, ph) : 0;
        const uint32_t zb = zc & 1, zr = (ui + ph) & 1;
        const int when = pend && pend_zr == zr ? -1 : mid;   // as in the producer
        // phase 0: W's columns and the adapters' in one product; later ones: the adapters' alone
        const uint32_t idesc = idesc_f16(128, ph == 0 ? p.bn + ns * p.rc : max(ns, 1) * p.rc, BF16, false, false);
        const uint32_t dst = tmem + zr * C::TM_TILE + (ph == 0 ? 0 : p.bn);
        const uint64_t opdesc = ph == 0 ? wdesc : ddesc;
        for (int ks = when < 0 ? -p.sub : 0; ks < steps; ks += p.sub) {
          if (more && ks >= 0) {
            uint32_t st;
            live = ring.take(st, kSiteKFull, abort_flag);
            if (!live) break;
            tc_fence_after();
            const uint64_t off = st * (static_cast<uint32_t>(p.stage) >> 4);
            mma_ss4(dst, xdesc + off, opdesc + off, idesc, ks > 0, 2, 2);
            if (p.sub == 2 && ks + 1 < steps) {
              const uint64_t off2 = off + (static_cast<uint32_t>(sub) >> 4);
              mma_ss4(dst, xdesc + off2, opdesc + off2, idesc, 1, 2, 2);
            }
            mma_commit_at(bempty + 8 * st);
          }
          if (MMA && pend && (ks == mid || ks < 0 || !more)) {
            // z U^T of the last phase onto its tile's accumulator
            const uint32_t pz = pend_z & 1;
            live = wait_warp(smem_u32(&p_full[pz]), (pend_z >> 1) & 1, kSitePFull, abort_flag);
            if (!live) break;
            tc_fence_after();
            const int nu = slots_of(pend_slots, pend_ph);
            for (int j = 0; j < nu; ++j) {
              uint32_t st, others[4];           // rows of other adapters
#pragma unroll
              for (int q = 0; q < 4; ++q)
                others[q] = __ballot_sync(0xffffffffu, plans[pend_pb].place[lane + 32 * q] != (pend_ph * spp + j) / p.chunks);
              live = ring.take(st, kSiteVFull, abort_flag);
              if (!live) break;
              tc_fence_after();
              const uint64_t ud = wdesc + st * (p.stage >> 4);
              for (int kk = 0; kk < p.rc / 16; ++kk) {
                const int r = j * p.rc + kk * 16;   // rank within the phase: two per tensor-memory column, 32 ranks' parts together
                const uint32_t z = tmem + pend_zr * C::TM_TILE + p.bn + r / 32 * 32 + r % 32 / 2;
                mma_ts_lanes(tmem + pend_ab * C::TM_TILE, z, ud + 2 * kk, idesc_w, others);
                mma_ts_lanes(tmem + pend_ab * C::TM_TILE, z + 16, ud + 2 * kk, idesc_w, others);
              }
              mma_commit_at(bempty + 8 * st);
            }
            if (!live) break;
            if (pend_last) {
              mma_commit_at(smem_u32(&acc_full[pend_ab]));
              arrive_elect(smem_u32(&plan_empty[pend_pb]));
            }
            pend = false;
          }
        }
        if (!live || !more) break;
        if (ns > 0) {
          mma_commit_at(smem_u32(&z_full[zb]));
          pend = true;
          pend_ph = ph;
          pend_slots = slots;
          pend_pb = pb;
          pend_ab = ab;
          pend_z = zc++;
          pend_zr = zr;
          pend_last = ph == nph - 1;
        } else {
          mma_commit_at(smem_u32(&acc_full[ab]));
          if (MMA) arrive_elect(smem_u32(&plan_empty[pb]));
        }
      }
      if (!more) break;
    }
    volatile uint32_t never = 0;
    mma_commit_at(smem_u32(drain_bar));
    wait_warp(smem_u32(drain_bar), 0, kSiteAccFull, &never);
  } else if (ROWS && warp >= 4 + C::EPI) {
    // ------------------------------ z U^T -------------------------------------
    for (int u = blockIdx.x; u < tiles; u += gridDim.x) {
      const int rt = u / p.nts;
      adapter_corr<BF16>(p, corr, rt * p.tm, (u - rt * p.nts) * p.bn);
      named_bar_sync(1, C::CORR_THREADS);                   // z U^T is complete
      named_bar_sync(2, C::CORR_THREADS);                   // and has been read
    }
  } else if (MMA && warp >= 4 + C::EPI) {
    // ------------------------------ conversion of z ---------------------------
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;
    uint32_t ui = 0, zc = 0;
    bool live = MMA;
    for (int u = blockIdx.x; u < tiles && live; u += gridDim.x, ++ui) {
      const uint32_t pb = ui % C::PLANS;
      live = wait_warp(smem_u32(&plan_full[pb]), (ui / C::PLANS) & 1, kSiteTicket, abort_flag);
      if (!live) break;
      const AdapterPlan* pl = &plans[pb];
      const int count = pl->count, slots = pl->slots, tile_phases = pl->phases;
      const float scale = pl->scale[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&plan_empty[pb]);
      const int nph = count > 0 ? tile_phases : 0;
      for (int ph = 0; ph < nph; ++ph, ++zc) {
        const uint32_t zb = zc & 1;
        live = wait_warp(smem_u32(&z_full[zb]), (zc >> 1) & 1, kSiteSFull, abort_flag);
        if (!live) break;
        tc_fence_after();
        const int ranks = slots_of(slots, ph) * p.rc;
#pragma unroll 1
        for (int j0 = 0; j0 < ranks; j0 += 32) {
          const uint32_t zt = tmem + ((ui + ph) & 1) * C::TM_TILE + p.bn + j0 + lane_off;
          uint32_t v[32], w[16], x[16];
          tmem_ld_x32(zt, v);
          tmem_wait_ld();
          reg_fence<32>(v);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // ranks past R: zeros also where x is not finite
            const int at = j0 + 8 * g, slot = ph * spp + at / p.rc;
            const bool rank = slot % p.chunks * 64 + at % p.rc < p.R;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float ah, al, bh, bl;
              split_z<BF16>(rank ? __uint_as_float(v[8 * g + 2 * j]) * scale : 0.f, ah, al);
              split_z<BF16>(rank ? __uint_as_float(v[8 * g + 2 * j + 1]) * scale : 0.f, bh, bl);
              w[4 * g + j] = pack2<BF16>(ah, bh);
              x[4 * g + j] = pack2<BF16>(al, bl);
            }
          }
          tmem_st_x16(zt, w);                   // over z's own columns: the upper parts, then the lower
          tmem_st_x16(zt + 16, x);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[zb]);
      }
    }
  } else if (warp >= 4 && warp < 4 + C::EPI) {
    // ------------------------------ epilogue ----------------------------------
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stg = smem + C::OFF_STG + (warp - 4) * C::STG;
    float* sb = reinterpret_cast<float*>(smem + C::OFF_BIAS) + (warp - 4) * C::PW;
    const int c0 = part * p.pw;                 // this warp's columns of a tile
    uint32_t ui = 0;
    for (int u = blockIdx.x; u < tiles; u += gridDim.x, ++ui) {
      const uint32_t ab = ui & 1, na = ui >> 1;
      const int rt = u / p.nts, n0 = (u - rt * p.nts) * p.bn;
      const int r = quarter * 32 + lane;
      const int rows = min(min(p.tm - quarter * 32, 32), p.T - rt * p.tm - quarter * 32);   // of this warp
      const bool mine = c0 < p.bn && n0 + c0 < p.K && rows > 0;
      __syncwarp();
      for (int i = lane; mine && i < p.pw; i += 32)
        sb[i] = p.bias != nullptr && n0 + c0 + i < p.K ? __ldg(p.bias + n0 + c0 + i) : 0.f;
      if constexpr (ROWS) {
        adapter_corr<BF16>(p, corr, rt * p.tm, n0);
        named_bar_sync(1, C::CORR_THREADS);
      }
      __syncwarp();
      const bool live = wait_warp(smem_u32(&acc_full[ab]), na & 1, kSiteAccFull, abort_flag);
      // a CTA that gives up keeps its barriers' company to the last tile
      if (!live && !ROWS) break;
      tc_fence_after();
      // The sums come into registers first, so that the next tile but one can
      // have their place while they are stored: its products wait for that.
      constexpr int PW = ROWS ? C::BN_ROWS / 4 : C::PW;
      uint32_t v[PW];
      if (mine) {
#pragma unroll
        for (int j = 0; j < PW; j += 8)
          if (j < p.pw) tmem_ld_x8(tmem + ab * C::TM_TILE + c0 + j + lane_off, v + j);
        tmem_wait_ld();
        reg_fence<PW>(v);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
      if (mine && live) {
        if (lane == 0) bulk_wait_read<0>();     // the piece before has been read
        __syncwarp();
        // rows of 2 pw bytes as TMA takes them
#pragma unroll
        for (int j = 0; j < PW; j += 8) {
          if (j < p.pw) {
            float f[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 b = reinterpret_cast<const float4*>(sb + j)[q];
              f[4 * q] = __uint_as_float(v[j + 4 * q]) + b.x;
              f[4 * q + 1] = __uint_as_float(v[j + 4 * q + 1]) + b.y;
              f[4 * q + 2] = __uint_as_float(v[j + 4 * q + 2]) + b.z;
              f[4 * q + 3] = __uint_as_float(v[j + 4 * q + 3]) + b.w;
            }
            if constexpr (ROWS) {
              if (lane < rows) {
                const float4* cr = reinterpret_cast<const float4*>(corr + r * (p.bn + 4) + c0 + j);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const float4 b = cr[q];
                  f[4 * q] += b.x;
                  f[4 * q + 1] += b.y;
                  f[4 * q + 2] += b.z;
                  f[4 * q + 3] += b.w;
                }
              }
            }
            *reinterpret_cast<uint4*>(stg + lane * 2 * p.pw + 2 * j) = pack8<BF16>(f);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tmY, stg, n0 + c0, rt * p.tm + quarter * 32, 0);   // clipped at T and K
          bulk_commit();
        }
      }
      if constexpr (ROWS) named_bar_sync(2, C::CORR_THREADS);
    }
    if (lane == 0) bulk_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace sdattn

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
// A tile is 128 rows by bn columns.  While x's tile of 64 columns of C is in
// shared memory for x W^T it also meets the D rows of the tile's adapters, so
// z = x D^T costs 16 .. 64 more MMA columns and no second pass over x; z goes
// from tensor memory through registers (scaled by s in fp32, zeroed in the
// rows of other adapters, rounded to 16 bits: the next product's operand) back
// to tensor memory, and as the A operand of z U^T adds onto the same fp32
// accumulator as x W^T.  Nothing but x, W, the adapters in use and y touches
// global memory, and W and x are never copied per request.
//
// Rows of different adapters may share a tile.  The planner warp lists a
// tile's distinct adapters; each contributes ceil(R / 64) slots of rc ranks
// (R rounded up to 16, at most 64), and 64 / rc slots fit a phase.  Phase 0
// runs with x W^T; a tile of more slots runs through x again, once per phase,
// against D alone.  The MMA warp issues the next phase's (or tile's) x
// products before it waits for the conversion of the last one's z, so the
// conversion is hidden except at the end.
#pragma once

#include "unet_ops.cuh"

namespace sdattn {

struct AdapterCfg {
  static constexpr int BK = 64;
  static constexpr int X_BYTES = 128 * 128;
  static constexpr int BN = 192;                    // most columns per tile
  static constexpr int W_BYTES = BN * 128;
  static constexpr int ZN = 64;                     // ranks per phase
  static constexpr int D_BYTES = ZN * 128;
  static constexpr int STAGE = X_BYTES + W_BYTES + D_BYTES;
  static constexpr int STAGES = 4;
  static constexpr int OFF_PLAN = STAGES * STAGE;
  static constexpr int PLAN = 128 * 4 + 128 * 4 + 128 * 4 + 16;   // adapters, rows' adapters, rows' scales, count
  static constexpr int OFF_BAR = OFF_PLAN + 2 * PLAN;
  static constexpr int NBAR = 2 * STAGES + 4 + 4 + 4 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr int NTHREADS = 384;              // TMA, MMA, planner, idle, eight epilogue warps
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int TM_Z = 2 * BN;               // accumulators at 0 and BN, z at 384 and 448
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct AdapterParams {
  const float* bias;      // [K], on 16 bytes, or null
  const int32_t* ids;     // [T / rows], or null: no adapters
  const float* scale;     // [L], or null: ones
  void* Y;                // [T][K]
  int T, K, L, rows;      // rows: rows per id
  int bn;                 // columns per tile: a multiple of 16 up to 192
  int tm;                 // rows per tile, up to 128
  int rts, nts;           // row tiles, column tiles
  int ksteps;             // ceil(C / 64)
  int rc;                 // ranks per slot: 16, 32, 48 or 64
  int chunks;             // slots per adapter: ceil(R / 64)
};

// One tile's plan in shared memory.
struct AdapterPlan {
  int32_t adapter[128];   // the distinct adapters, in order of first appearance
  int32_t place[128];     // each row's place in that list, -1 without one
  float scale[128];       // each row's scale
  int32_t count;
  int32_t pad[3];
};
static_assert(sizeof(AdapterPlan) == AdapterCfg::PLAN, "plan layout");

template <bool BF16>
__global__ void __launch_bounds__(AdapterCfg::NTHREADS, 1)
    adapter_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmU,
                   const AdapterParams p) {
  using C = AdapterCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                      // [STAGES] TMA -> MMA
  uint64_t* empty = full + C::STAGES;         // [STAGES] MMA -> TMA
  uint64_t* acc_full = empty + C::STAGES;     // [2] MMA -> epilogue
  uint64_t* acc_empty = acc_full + 2;         // [2] epilogue -> MMA
  uint64_t* z_full = acc_empty + 2;           // [2] MMA -> epilogue: z is complete
  uint64_t* p_full = z_full + 2;              // [2] epilogue -> MMA: z is converted
  uint64_t* plan_full = p_full + 2;           // [2] planner -> TMA, MMA, epilogue
  uint64_t* plan_empty = plan_full + 2;       // [2] back
  uint64_t* drain_bar = plan_empty + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = misc + 1;
  AdapterPlan* plans = reinterpret_cast<AdapterPlan*>(smem + C::OFF_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = p.rts * p.nts;
  const int spp = C::ZN / p.rc;               // slots per phase

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);
      mbar_init(&z_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&plan_full[i], 1);
      mbar_init(&plan_empty[i], 10);
    }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    if (p.ids != nullptr) {
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

  // Phases of a tile of `count` adapters, and the slots of phase ph.
  auto phases = [&](int count) { return max(1, (count * p.chunks + spp - 1) / spp); };
  auto slots_of = [&](int count, int ph) { return min(spp, count * p.chunks - ph * spp); };

  if (warp == 2) {
    // ------------------------------ planner -----------------------------------
    uint32_t ui = 0;
    for (int u = blockIdx.x; u < tiles; u += gridDim.x, ++ui) {
      const uint32_t pb = ui & 1, n = ui >> 1;
      if (!mbar_wait_warp(&plan_empty[pb], (n & 1) ^ 1, kSiteTicket, abort_flag)) break;
      AdapterPlan* pl = &plans[pb];
      const int r0 = u / p.nts * p.tm;
      int id[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = lane + 32 * q;
        id[q] = -1;
        if (p.ids != nullptr && r < p.tm && r0 + r < p.T) {
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
      if (lane == 0) pl->count = count;
      __syncwarp();
      if (lane == 0) mbar_arrive(&plan_full[pb]);
    }
  } else if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      uint32_t c = 0, ui = 0;
      bool live = true, pend = false;
      int pend_ph = 0, pend_n0 = 0;
      uint32_t pend_pb = 0;
      bool pend_last = false;
      // the U tiles of a phase, one stage per slot
      auto load_up = [&]() {
        const AdapterPlan* pl = &plans[pend_pb];
        const int ns = slots_of(pl->count, pend_ph);
        for (int j = 0; j < ns && live; ++j, ++c) {
          const int s = pend_ph * spp + j, a = pl->adapter[s / p.chunks], ch = s % p.chunks;
          const uint32_t st = c % C::STAGES, n = c / C::STAGES;
          if (!mbar_wait(&empty[st], (n & 1) ^ 1, kSiteKEmpty, abort_flag)) { live = false; break; }
          mbar_arrive_expect_tx(&full[st], p.bn * 128);
          tma_load_3d(smem + st * C::STAGE + C::X_BYTES, &tmU, ch * 64, pend_n0, a, &full[st]);
        }
        if (pend_last) mbar_arrive(&plan_empty[pend_pb]);
        pend = false;
      };
      for (int u = blockIdx.x; u < tiles && live; u += gridDim.x, ++ui) {
        const int rt = u / p.nts, n0 = (u - rt * p.nts) * p.bn;
        const uint32_t pb = ui & 1;
        if (!mbar_wait(&plan_full[pb], (ui >> 1) & 1, kSiteTicket, abort_flag)) { live = false; break; }
        const AdapterPlan* pl = &plans[pb];
        const int count = pl->count, nph = phases(count);
        for (int ph = 0; ph < nph && live; ++ph) {
          const int ns = slots_of(count, ph);
          const uint32_t bytes = p.tm * 128 + (ph == 0 ? p.bn * 128 : 0) + max(ns, 0) * p.rc * 128;
          for (int ks = 0; ks < p.ksteps; ++ks, ++c) {
            const uint32_t st = c % C::STAGES, n = c / C::STAGES;
            if (!mbar_wait(&empty[st], (n & 1) ^ 1, kSiteKEmpty, abort_flag)) { live = false; break; }
            uint8_t* s = smem + st * C::STAGE;
            mbar_arrive_expect_tx(&full[st], bytes);
            tma_load_3d(s, &tmX, ks * C::BK, rt * p.tm, 0, &full[st]);
            if (ph == 0) tma_load_3d(s + C::X_BYTES, &tmW, ks * C::BK, n0, 0, &full[st]);
            for (int j = 0; j < ns; ++j) {
              const int sl = ph * spp + j;
              tma_load_3d(s + C::X_BYTES + C::W_BYTES + j * p.rc * 128, &tmD, ks * C::BK, sl % p.chunks * 64,
                          pl->adapter[sl / p.chunks], &full[st]);
            }
          }
          if (pend && live) load_up();
          if (ns > 0) {
            pend = true;
            pend_ph = ph;
            pend_n0 = n0;
            pend_pb = pb;
            pend_last = ph == nph - 1;
          } else {
            mbar_arrive(&plan_empty[pb]);   // a tile without adapters
          }
        }
      }
      if (pend && live) load_up();
      // every load this thread issued lands before the CTA can exit
      volatile uint32_t never = 0;
      for (uint32_t st = 0; st < C::STAGES && st < c; ++st) {
        const uint32_t uses = (c - st + C::STAGES - 1) / C::STAGES;
        mbar_wait(&full[st], (uses - 1) & 1, kSiteKFull, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer --------------------------------
    const uint32_t idesc_w = idesc_f16(128, p.bn, BF16, false, false);
    const uint32_t base = smem_u32(smem);
    uint32_t c = 0, ui = 0, zc = 0;             // stages, tiles, phases with adapters
    bool live = true, pend = false;
    int pend_ph = 0, pend_count = 0;
    uint32_t pend_pb = 0, pend_ab = 0, pend_z = 0;
    bool pend_last = false;
    // z U^T of a phase onto its tile's accumulator
    auto mma_up = [&]() {
      const uint32_t zb = pend_z & 1;
      if (!mbar_wait_warp(&p_full[zb], (pend_z >> 1) & 1, kSitePFull, abort_flag)) { live = false; return; }
      tc_fence_after();
      const int ns = slots_of(pend_count, pend_ph);
      for (int j = 0; j < ns; ++j, ++c) {
        const uint32_t st = c % C::STAGES, n = c / C::STAGES;
        if (!mbar_wait_warp(&full[st], n & 1, kSiteVFull, abort_flag)) { live = false; return; }
        tc_fence_after();
        const uint32_t su = base + st * C::STAGE + C::X_BYTES;
        for (int kk = 0; kk < p.rc / 16; ++kk) {
          const int r = j * p.rc + kk * 16;     // rank within the phase: two per tensor-memory column
          mma_ts(tmem + pend_ab * C::BN, tmem + C::TM_Z + zb * C::ZN + r / 32 * 32 + r % 32 / 2,
                 sdesc_sw128(su + kk * 32, 16, 1024), idesc_w, 1u);
        }
        mma_commit(&empty[st]);
      }
      if (pend_last) {
        mma_commit(&acc_full[pend_ab]);
        if (lane == 0) mbar_arrive(&plan_empty[pend_pb]);
      }
      pend = false;
    };
    for (int u = blockIdx.x; u < tiles && live; u += gridDim.x, ++ui) {
      const uint32_t ab = ui & 1, na = ui >> 1;
      if (!mbar_wait_warp(&plan_full[ab], na & 1, kSiteTicket, abort_flag)) { live = false; break; }
      const int count = plans[ab].count, nph = phases(count);
      if (!mbar_wait_warp(&acc_empty[ab], (na & 1) ^ 1, kSiteAccEmpty, abort_flag)) { live = false; break; }
      tc_fence_after();
      for (int ph = 0; ph < nph && live; ++ph) {
        const int ns = slots_of(count, ph);
        const uint32_t zb = zc & 1;
        const uint32_t idesc_d = idesc_f16(128, max(ns, 1) * p.rc, BF16, false, false);
        for (int ks = 0; ks < p.ksteps; ++ks, ++c) {
          const uint32_t st = c % C::STAGES, n = c / C::STAGES;
          if (!mbar_wait_warp(&full[st], n & 1, kSiteKFull, abort_flag)) { live = false; break; }
          tc_fence_after();
          const uint32_t s = base + st * C::STAGE;
#pragma unroll
          for (int kk = 0; kk < C::BK / 16; ++kk) {
            const uint64_t xd = sdesc_sw128(s + kk * 32, 16, 1024);
            const uint32_t acc = (ks > 0 || kk > 0) ? 1u : 0u;
            if (ph == 0) mma_ss(tmem + ab * C::BN, xd, sdesc_sw128(s + C::X_BYTES + kk * 32, 16, 1024), idesc_w, acc);
            if (ns > 0)
              mma_ss(tmem + C::TM_Z + zb * C::ZN, xd, sdesc_sw128(s + C::X_BYTES + C::W_BYTES + kk * 32, 16, 1024),
                     idesc_d, acc);
          }
          mma_commit(&empty[st]);
        }
        if (!live) break;
        if (ns > 0) {
          mma_commit(&z_full[zb]);
        } else {
          mma_commit(&acc_full[ab]);
          if (lane == 0) mbar_arrive(&plan_empty[ab]);
        }
        if (pend) mma_up();
        if (ns > 0) {
          pend = true;
          pend_ph = ph;
          pend_count = count;
          pend_pb = ab;
          pend_ab = ab;
          pend_z = zc++;
          pend_last = ph == nph - 1;
        }
      }
    }
    if (pend && live) mma_up();
    volatile uint32_t never = 0;
    mma_commit(drain_bar);
    mbar_wait_warp(drain_bar, 0, kSiteAccFull, &never);
  } else if (warp >= 4) {
    // ------------------------------ epilogue ----------------------------------
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t ui = 0, zc = 0;
    bool live = true;
    for (int u = blockIdx.x; u < tiles && live; u += gridDim.x, ++ui) {
      const uint32_t ab = ui & 1, na = ui >> 1;
      const int rt = u / p.nts, n0 = (u - rt * p.nts) * p.bn;
      const int r = quarter * 32 + lane, row = rt * p.tm + r;
      live = mbar_wait_warp(&plan_full[ab], na & 1, kSiteTicket, abort_flag);
      if (!live) break;
      const AdapterPlan* pl = &plans[ab];
      const int count = pl->count, place = pl->place[r];
      const float scale = pl->scale[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&plan_empty[ab]);
      if (count > 0) {
        const int nph = phases(count);
        for (int ph = 0; ph < nph; ++ph, ++zc) {
          const uint32_t zb = zc & 1;
          live = mbar_wait_warp(&z_full[zb], (zc >> 1) & 1, kSiteSFull, abort_flag);
          if (!live) break;
          tc_fence_after();
          const uint32_t zt = tmem + C::TM_Z + zb * C::ZN + half * 32 + lane_off;
          uint32_t v[32], w[16];
          tmem_ld_x32(zt, v);
          tmem_wait_ld();
          reg_fence<32>(v);
#pragma unroll
          for (int g = 0; g < 2; ++g) {         // 16 ranks belong to one slot
            const int slot = ph * spp + (half * 32 + g * 16) / p.rc;
            const bool mine = slot / p.chunks == place;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float a = mine ? __uint_as_float(v[16 * g + 2 * j]) * scale : 0.f;
              const float b = mine ? __uint_as_float(v[16 * g + 2 * j + 1]) * scale : 0.f;
              w[8 * g + j] = pack2<BF16>(a, b);
            }
          }
          tmem_st_x16(zt, w);                   // over the warp's own columns of z
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[zb]);
        }
        if (!live) break;
      }
      live = mbar_wait_warp(&acc_full[ab], na & 1, kSiteAccFull, abort_flag);
      if (!live) break;
      tc_fence_after();
      // 16 columns at a time, the two warps of a quarter in turn
#pragma unroll 1
      for (int c0 = half * 16; c0 < p.bn && n0 + c0 < p.K; c0 += 32) {
        uint32_t v[16];
        tmem_ld_x16(tmem + ab * C::BN + c0 + lane_off, v);
        tmem_wait_ld();
        reg_fence<16>(v);
        if (r < p.tm && row < p.T) {
          uint16_t* dst = static_cast<uint16_t*>(p.Y) + static_cast<int64_t>(row) * p.K + n0 + c0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (n0 + c0 + 8 * q >= p.K) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * q + e]);
            if (p.bias != nullptr) {
              const float4* bs = reinterpret_cast<const float4*>(p.bias + n0 + c0 + 8 * q);
              const float4 b0 = __ldg(bs), b1 = __ldg(bs + 1);
              f[0] += b0.x; f[1] += b0.y; f[2] += b0.z; f[3] += b0.w;
              f[4] += b1.x; f[5] += b1.y; f[6] += b1.z; f[7] += b1.w;
            }
            reinterpret_cast<uint4*>(dst)[q] = pack8<BF16>(f);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace sdattn

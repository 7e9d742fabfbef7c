// pipeline.cuh -- what the transformer block's tensor-core kernels share: waits,
// loads and products issued by one warp in a short loop, and CTA pairs.
//
// A k-step of such a kernel (64 columns of the contraction) is 4 MMAs of 16; a
// 128 x 256 tile spends 512 clocks on it, a narrow one a few dozen.  One warp
// issues loads and another products, so what bounds narrow tiles is the code
// those warps run per step: with every wait's slow path inlined, descriptors
// built for each MMA and the ring's stage found by division, a step took 480 to
// 1030 clocks whatever its width.  So here a wait is one try and a call,
// the four MMAs of a step are one asm block that advances its
// descriptors, and stages are counted.  The warps stay converged (elect.sync picks the issuing
// lane), which keeps operands in uniform registers.
//
// Waits have sm100.cuh's limits: a second, then the error word and the CTA's
// abort flag.
#pragma once

#include "sm100.cuh"

namespace sdattn {

// The clock is read only after a good many tries: a read of it costs more than
// most waits last.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t site, volatile uint32_t* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 127u) == 0u) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *abort_flag = 1u;
        atomicCAS(&g_error_word, 0u, 0x100u + site);
        return false;
      }
    }
  }
}

// Waits for the phase of the barrier at shared address `bar` with parity
// `parity`; the same result in every lane of the (converged) warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t site, volatile uint32_t* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, site, abort_flag));
}

// One warp's walk around a ring of n stages with a barrier each: take() waits
// for the next stage.  `parity`: 0 for the consumer of full stages, 1 for the
// producer, whose first turn finds them empty.
struct RingWalk {
  uint32_t bars, n, st, parity;
  __device__ __forceinline__ RingWalk(uint32_t bars_, uint32_t n_, uint32_t parity_)
      : bars(bars_), n(n_), st(0), parity(parity_) {}
  __device__ __forceinline__ bool take(uint32_t& stage, uint32_t site, volatile uint32_t* abort_flag) {
    const bool ok = wait_warp(bars + 8 * st, parity, site, abort_flag);
    stage = st;
    if (++st == n) {
      st = 0;
      parity ^= 1u;
    }
    return ok;
  }
};

// Waits for the last phase of every stage that c turns of a ring used, so that
// what still arrives in this CTA's shared memory lands before the CTA exits: a
// CTA's own loads; in a pair, the leader waits for both CTAs' loads and the
// other CTA for the leader's commits that empty its stages.  An abort elsewhere
// does not cut it short; its own limit is one second in all.
__device__ __forceinline__ void drain_ring(uint32_t bars, uint32_t n, uint32_t c, uint32_t site) {
  volatile uint32_t never = 0;
  for (uint32_t st = 0; st < n && st < c; ++st) {
    const uint32_t uses = (c - st + n - 1) / n;
    wait_warp(bars + 8 * st, (uses - 1) & 1, site, &never);
  }
}

// --------------------------- issued by a converged warp ---------------------------
__device__ __forceinline__ void expect_tx_elect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void arrive_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void load_elect(uint32_t sdst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(sdst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem]^T over 64 of K: four MMAs, the descriptors
// advancing by astep and bstep (in 16-byte units); `accumulate` is the first's.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                        uint64_t astep, uint64_t bstep) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(astep), "l"(bstep)
      : "memory");
}

// D[tmem] += A[tmem] B[smem]^T over 16 of K in the lanes whose bit of `off` is
// clear; the other lanes of D keep their values, whatever their products are.
__device__ __forceinline__ void mma_ts_lanes(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, const uint32_t (&off)[4]) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}

// ---------------------------------------------------------------------------
// CTA pairs (cta_group::2): the two CTAs of a cluster, on neighbouring SMs,
// run one tcgen05.mma of twice the rows.  Each holds its own 128 rows of A and
// half of B's rows, so a tile of 256 rows reads B from L2 once instead of
// twice.  The even CTA (the leader) issues the MMAs; barriers that the other
// CTA signals are addressed in the leader's shared memory.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  return remote;
}

// A TMA load into this CTA's shared memory that signals the leader's barrier.
__device__ __forceinline__ void load_elect_pair(uint32_t sdst, const CUtensorMap* map, int x, int y, int z,
                                                uint32_t leader_bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(sdst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(leader_bar)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_result, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_result)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// mma_ss4 on both CTAs' shared and tensor memory, issued by the leader.
__device__ __forceinline__ void mma_ss4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                             uint64_t astep, uint64_t bstep) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(astep), "l"(bstep)
      : "memory");
}

// Arrives once on the barrier at this offset in both CTAs when every MMA the
// elected thread issued so far has completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void mma_commit_at(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// The end of a pair's work, by all threads of both CTAs.  The leader's last
// commit arrives on `drain` in both CTAs, after all its products and earlier
// commits; the leader's issuing warp has waited for its own.  The other CTA
// waits for its copy, which would otherwise be on its way to shared memory that
// the CTA has left.  Then neither CTA leaves while the other's products read
// its memory.
__device__ __forceinline__ void pair_exit(uint32_t drain) {
  if (threadIdx.x >> 5 == 1 && cluster_rank() != 0) {
    volatile uint32_t never = 0;
    wait_warp(drain, 0, kSiteAccFull, &never);
  }
  cluster_sync();
}

// An arrival on a barrier of either CTA.  (Released at cluster scope it costs
// a full memory barrier, 12% of the gated kernel; what it hands over is tensor
// memory, ordered by tcgen05.fence.)
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

}  // namespace sdattn

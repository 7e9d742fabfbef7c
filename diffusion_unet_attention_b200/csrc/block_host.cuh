// block_host.cuh -- argument checks, plans and launches of the transformer
// block's operators around attention (layer norm).  Included by sdattn.cu
// after its launch helpers, inside its anonymous namespace.
#pragma once

// --------------------------------------------------------------------------
// Layer norm (layer_norm.cuh)
// --------------------------------------------------------------------------
constexpr int kLNMaxC = 8192;   // a CTA of 512 threads holds such a row in registers, with its column sums

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sdattn_status check_ln(const sdattn_ln_desc* d) {
  if (!d) return SDATTN_ERR_INVALID_ARG;
  if (d->T < 0 || d->C < 1) return SDATTN_ERR_INVALID_ARG;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return SDATTN_ERR_INVALID_ARG;
  if (d->dtype != SDATTN_F16 && d->dtype != SDATTN_BF16 && d->dtype != SDATTN_F32) return SDATTN_ERR_UNSUPPORTED;
  if (d->C > kLNMaxC || d->T >= (int64_t(1) << 31)) return SDATTN_ERR_UNSUPPORTED;
  return SDATTN_OK;
}

int ln_elem(const sdattn_ln_desc* d) {
  return d->dtype == SDATTN_F32 ? sdattn::kElemF32 : d->dtype == SDATTN_BF16 ? sdattn::kElemBF16 : sdattn::kElemF16;
}

struct LNPlan {
  bool vec, cta;
  int U;         // accesses per lane (a compiled count)
  int L;         // lanes per row
  int threads;   // per CTA
};

// The compiled access counts; a count is rounded up to the next one.
int ln_round_u(int u, bool vec) {
  if (vec) return u;   // 1 .. 5
  int r = 1;
  while (r < u) r *= 2;
  return r;            // 1 .. 16
}

// Rows go to 8, 16 or 32 lanes of a warp, whichever leaves the fewest lanes
// idle in the row's last access; with too few rows to give every SM a CTA of
// 8-lane rows, to 32 lanes (the row's chain is shorter).  The backward pass
// keeps two sums per column in registers beside x and dy: more than 24
// columns per lane leave room for one CTA per SM only, which counts as half as
// much again.  Rows past a warp's registers take a CTA.
LNPlan plan_ln(const sdattn_ln_desc* d, bool vec, bool backward, int nsm) {
  LNPlan pl;
  pl.vec = vec;
  const int E = !vec ? 1 : d->dtype == SDATTN_F32 ? 4 : 8;
  const int nch = d->C / E, umax = vec ? 5 : 16;
  if (nch > 32 * umax) {
    pl.cta = true;
    int u = 1;
    while (u * sdattn::kLNRowThreads < nch) ++u;
    pl.U = ln_round_u(u, vec);
    pl.threads = std::min(sdattn::kLNRowThreads, ((nch + pl.U - 1) / pl.U + 31) / 32 * 32);
    pl.L = pl.threads;
    return pl;
  }
  pl.cta = false;
  pl.threads = sdattn::kLNThreads;
  const bool few = d->T * 8 / sdattn::kLNThreads < nsm;
  double best = 1e30;
  for (int L = few ? 32 : 8; L <= 32; L *= 2) {
    const int u = ln_round_u((nch + L - 1) / L, vec);
    if (u > umax) continue;
    double cost = static_cast<double>(L) * u;
    if (backward && u * E > 24) cost *= 1.5;
    if (cost < best) {
      best = cost;
      pl.L = L;
      pl.U = u;
    }
  }
  return pl;
}

// Whether a plan can ask for this CTA kernel: rows above 32 * 5 (16-byte
// accesses) or 32 * 16 (single elements) and up to kLNMaxC, over 512 threads.
constexpr bool ln_cta_u(int dt, bool vec, int u) {
  return vec ? u <= kLNMaxC / (dt == sdattn::kElemF32 ? 4 : 8) / sdattn::kLNRowThreads : u >= 2;
}

template <int DT, bool VEC, int U>
sdattn_status launch_ln_u(const sdattn::LNParams& p, const LNPlan& pl, bool backward, int64_t grid, cudaStream_t s) {
  const int g = static_cast<int>(grid);
  bool ok = false;
  if (!pl.cta) {
    ok = backward ? launch(sdattn::layer_norm_bwd_kernel<DT, VEC, U, false>, g, pl.threads, 2 * p.C * 4, s, p)
                  : launch(sdattn::layer_norm_kernel<DT, VEC, U, false>, g, pl.threads, 0, s, p);
  } else if constexpr (ln_cta_u(DT, VEC, U)) {
    ok = backward ? launch(sdattn::layer_norm_bwd_kernel<DT, VEC, U, true>, g, pl.threads, 0, s, p)
                  : launch(sdattn::layer_norm_kernel<DT, VEC, U, true>, g, pl.threads, 0, s, p);
  }
  return ok ? SDATTN_OK : SDATTN_ERR_CUDA;
}

template <int DT>
sdattn_status launch_ln_dt(const sdattn::LNParams& p, const LNPlan& pl, bool backward, int64_t grid, cudaStream_t s) {
  if (pl.vec) {
    switch (pl.U) {
      case 1: return launch_ln_u<DT, true, 1>(p, pl, backward, grid, s);
      case 2: return launch_ln_u<DT, true, 2>(p, pl, backward, grid, s);
      case 3: return launch_ln_u<DT, true, 3>(p, pl, backward, grid, s);
      case 4: return launch_ln_u<DT, true, 4>(p, pl, backward, grid, s);
      case 5: return launch_ln_u<DT, true, 5>(p, pl, backward, grid, s);
    }
  } else {
    switch (pl.U) {
      case 1: return launch_ln_u<DT, false, 1>(p, pl, backward, grid, s);
      case 2: return launch_ln_u<DT, false, 2>(p, pl, backward, grid, s);
      case 4: return launch_ln_u<DT, false, 4>(p, pl, backward, grid, s);
      case 8: return launch_ln_u<DT, false, 8>(p, pl, backward, grid, s);
      case 16: return launch_ln_u<DT, false, 16>(p, pl, backward, grid, s);
    }
  }
  return SDATTN_ERR_UNSUPPORTED;
}

sdattn_status launch_ln(const sdattn_ln_desc* d, sdattn::LNParams p, const LNPlan& pl, bool backward, int64_t grid,
                        cudaStream_t s) {
  const int E = !pl.vec ? 1 : d->dtype == SDATTN_F32 ? 4 : 8;
  p.T = d->T;
  p.C = d->C;
  p.eps = d->eps;
  p.L = pl.L;
  p.nch = d->C / E;
  switch (ln_elem(d)) {
    case sdattn::kElemF32: return launch_ln_dt<sdattn::kElemF32>(p, pl, backward, grid, s);
    case sdattn::kElemBF16: return launch_ln_dt<sdattn::kElemBF16>(p, pl, backward, grid, s);
    default: return launch_ln_dt<sdattn::kElemF16>(p, pl, backward, grid, s);
  }
}

// Whole 16-byte accesses: rows of whole accesses, every pointer on 16 bytes
// (null parameters need none).
bool ln_vec(const sdattn_ln_desc* d, std::initializer_list<const void*> ps) {
  if (d->C % (d->dtype == SDATTN_F32 ? 4 : 8) != 0) return false;
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

// CTAs of the backward pass: two per SM (four when a row takes a small CTA),
// but at least four rows for each lane group, since every CTA costs a partial
// row of sums that the second kernel reads.
int64_t ln_bwd_grid(const sdattn_ln_desc* d, const LNPlan& pl, int nsm) {
  const int64_t rpc = pl.cta ? 1 : pl.threads / pl.L;
  const int64_t per_sm = pl.cta && pl.threads <= 256 ? 4 : 2;
  return std::min((d->T + 4 * rpc - 1) / (4 * rpc), static_cast<int64_t>(nsm) * per_sm);
}

bool launch_column_sum(const float* part, int64_t P, int n, int n0, float* out0, float* out1, cudaStream_t s) {
  return launch(sdattn::column_sum_kernel, (n + 31) / 32, 1024, 0, s, part, P, n, n0, out0, out1);
}

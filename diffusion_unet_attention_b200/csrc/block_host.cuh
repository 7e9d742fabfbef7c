// block_host.cuh -- argument checks, plans and launches of the transformer
// block's operators around attention (layer norm, gated feed-forward,
// projections with adapters).  Included by sdattn.cu
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
    ok = backward ? launch(sdattn::layer_norm_bwd_kernel<DT, VEC, U, false>, g, pl.threads, pl.threads / 32 * p.C * 4, s, p)
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
// but at least two rows for each lane group, since every CTA costs a partial
// row of sums that the second kernel reads.
int64_t ln_bwd_grid(const sdattn_ln_desc* d, const LNPlan& pl, int nsm) {
  const int64_t rpc = pl.cta ? 1 : pl.threads / pl.L;
  const int64_t per_sm = pl.cta && pl.threads <= 256 ? 4 : 2;
  return std::min((d->T + 2 * rpc - 1) / (2 * rpc), static_cast<int64_t>(nsm) * per_sm);
}

bool launch_column_sum(const float* part, int64_t P, int n, int n0, float* out0, float* out1, cudaStream_t s) {
  return launch(sdattn::column_sum_kernel, (n + 31) / 32, 1024, 0, s, part, P, n, n0, out0, out1);
}

// --------------------------------------------------------------------------
// Gated feed-forward (gated_ff.cuh)
// --------------------------------------------------------------------------
sdattn_status check_ff(const sdattn_ff_desc* d) {
  if (!d) return SDATTN_ERR_INVALID_ARG;
  if (d->T < 0 || d->C < 1 || d->F < 1) return SDATTN_ERR_INVALID_ARG;
  if (d->dtype != SDATTN_F16 && d->dtype != SDATTN_BF16) return SDATTN_ERR_UNSUPPORTED;
  // rows of x, W and y are whole 16-byte units, as TMA needs; the bounds keep
  // every tile count in 32 bits
  if (d->C % 8 != 0 || d->F % 8 != 0 || d->C > 65536 || d->F > 65536 || d->T >= (int64_t(1) << 27))
    return SDATTN_ERR_UNSUPPORTED;
  return SDATTN_OK;
}

CUtensorMapDataType elem16(int dtype) {
  return dtype == SDATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Pairs of CTAs on tiles of 256 rows by 128 columns of h, or single CTAs on
// 128 rows by hn columns (a multiple of 16 up to 128): the fewest waves of the
// longest of a tile's products (2 clocks per accumulator column and 64 of C),
// issue (300 clocks a step), loads (45 bytes per clock and SM, measured with the
// epilogue left out) and epilogue, plus one tile's epilogue at the end.  Many rows take pairs, which
// read W's tile once for 256 rows; few rows narrower tiles, until there is
// about one per SM.
struct GatedPlan {
  bool pair;
  int hn;
};

GatedPlan plan_gated(const sdattn_ff_desc* d, bool backward, int nsm) {
  const double ksteps = (d->C + 63) / 64;
  const double epi = backward ? 40.0 : 20.0;      // clocks per column of a 128-row tile
  auto cost = [&](int64_t tiles, int64_t slots, int hn, double bytes) {
    const double waves = static_cast<double>((tiles + slots - 1) / slots);
    return waves * std::max(ksteps * std::max(std::max(4.0 * hn, 300.0), bytes / 45.0), epi * hn) + epi * hn;
  };
  GatedPlan best{true, 128};
  double least = 1e300;
  if (d->T > 128) least = cost((d->T + 255) / 256 * ((d->F + 127) / 128), nsm / 2, 128, 16384.0 + 16384.0);
  for (int hn = 128; hn >= 16; hn -= 16) {
    // the narrow form's stores cost it about half as much again
    const double c = cost((d->T + 127) / 128 * ((d->F + hn - 1) / hn), nsm, hn, 16384.0 + 256.0 * hn) + 0.5 * epi * hn;
    if (c < least) {
      least = c;
      best = {false, hn};
    }
  }
  return best;
}

template <bool BF16, bool BWD>
sdattn_status launch_gated(const sdattn_ff_desc* d, const void* X, const void* W, const float* bias, const void* dY,
                           void* Y, float* part, cudaStream_t s) {
  const int dev = current_device();
  if (dev < 0) return SDATTN_ERR_CUDA;
  const int nsm = sm_count(dev);
  const uint64_t T = d->T, C = d->C, F = d->F;
  sdattn::GatedParams p;
  p.bias = bias;
  p.dY = dY;
  p.Y = Y;
  p.part = part;
  p.T = static_cast<int>(T);
  p.F = d->F;
  const GatedPlan plan = plan_gated(d, BWD, nsm);
  p.hn = plan.hn;
  p.rts = static_cast<int>(plan.pair ? (T + 255) / 256 : (T + 127) / 128);
  p.fts = (d->F + p.hn - 1) / p.hn;
  p.ksteps = (d->C + 63) / 64;
  p.tm = plan.pair ? 128 : static_cast<int>(std::min<uint64_t>(128, (T + 7) / 8 * 8));
  using Smem = sdattn::GatedSmem<BWD, false>;
  p.stage = 2 * (p.tm + 2 * p.hn) * 128;
  p.stages = std::min(Smem::MAX_STAGES, (Smem::RING - (p.tm < 128 ? Smem::SLACK : 0)) / p.stage);
  // The tensor cores' fp32 sums truncate: an entry of h or g comes out low by
  // about 1.2e-9 of its terms per column of C, which all rows share and db
  // adds up (1.5e-6 of db at C = 1280).  Past C = 640 the backward pass halves
  // that with two chains per tile, whose sums are rounded once.
  p.chains = BWD && p.ksteps > 10 ? 2 : 1;
  const CUtensorMapDataType dt = elem16(d->dtype);
  CUtensorMap mx, mw, my;
  if (!make_map_3d(&mx, X, dt, C, T, 1, C * 2, T * C * 2, 64, static_cast<uint32_t>(p.tm))) return SDATTN_ERR_CUDA;
  if (!make_map_3d(&mw, W, dt, C, F, 2, C * 2, F * C * 2, 64, static_cast<uint32_t>(p.hn))) return SDATTN_ERR_CUDA;
  // y, or the two halves of P = [dh, dg], and dy as the pairs' warps move them
  const uint64_t ldy = BWD ? 4 * F : 2 * F;
  CUtensorMap mdy, mdg;
  constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_map_3d(&my, Y, dt, F, T, 1, ldy, T * ldy, 32, 32, sw)) return SDATTN_ERR_CUDA;
  if (BWD) {
    if (!make_map_3d(&mdy, dY, dt, F, T, 1, F * 2, T * F * 2, 32, 32, sw)) return SDATTN_ERR_CUDA;
    if (!make_map_3d(&mdg, static_cast<uint16_t*>(Y) + F, dt, F, T, 1, ldy, T * ldy, 32, 32, sw))
      return SDATTN_ERR_CUDA;
  } else {
    mdy = mdg = my;   // never read
  }
  const int64_t tiles = int64_t(p.rts) * p.fts;
  if (plan.pair) {
    auto kern = sdattn::gated_kernel<BF16, BWD, true>;
    constexpr int smem = sdattn::GatedSmem<BWD, true>::BYTES;
    static std::atomic<uint64_t> done{0};
    if (!ensure_smem(kern, smem, done, dev)) return SDATTN_ERR_CUDA;
    const int grid = static_cast<int>(std::min<int64_t>(nsm / 2, tiles)) * 2;
    return launch_cluster(kern, grid, 2, sdattn::GatedCfg::NTHREADS, smem, s, mx, mw, my, mdy, mdg, p) ? SDATTN_OK : SDATTN_ERR_CUDA;
  }
  auto kern = sdattn::gated_kernel<BF16, BWD, false>;
  constexpr int smem = sdattn::GatedSmem<BWD, false>::BYTES;
  static std::atomic<uint64_t> done{0};
  if (!ensure_smem(kern, smem, done, dev)) return SDATTN_ERR_CUDA;
  const int grid = static_cast<int>(std::min<int64_t>(nsm, tiles));
  return launch(kern, grid, sdattn::GatedCfg::NTHREADS, smem, s, mx, mw, my, mdy, mdg, p) ? SDATTN_OK : SDATTN_ERR_CUDA;
}

// dx = P W and dW = P^T x: tiles, splits and where their partials lie.
struct FFBwdPlan {
  sdattn::ProductParams pp;
  size_t p_bytes, db_bytes, part_bytes[2];
  size_t total;
  int pairs;          // CTA pairs of the products' launch
};

// Up to 320 columns of a result are one tile; more are cut into the fewest
// tiles of at most 256, rounded up to whole slabs of 64 (at 640 columns two
// wide tiles took 4 us more than three with two accumulators).  With L the contraction steps a pair of SMs would run
// if both products were shared out evenly, a contraction longer than 5/4 L is
// split into pieces of at most L (at least 8 steps: a piece costs a partial
// result that is written and read again).
FFBwdPlan plan_ff_bwd(const sdattn_ff_desc* d, int nsm) {
  FFBwdPlan pl;
  const int pairs = std::max(1, nsm / 2);
  const int M[2] = {static_cast<int>(d->T), 2 * d->F}, K[2] = {2 * d->F, static_cast<int>(d->T)};
  double total = 0;
  for (int i = 0; i < 2; ++i) {
    sdattn::ProductSide& s = pl.pp.s[i];
    s.M = M[i];
    s.N = d->C;
    const int most = s.N <= sdattn::ProductCfg::BN ? sdattn::ProductCfg::BN : 256, n = (s.N + most - 1) / most;
    s.bn = ((s.N + n - 1) / n + 63) / 64 * 64;
    s.nts = (s.N + s.bn - 1) / s.bn;
    s.mn = (s.M + 255) / 256 * s.nts;
    s.ksteps = (K[i] + 63) / 64;
    total += static_cast<double>(s.mn) * s.ksteps;
  }
  const double L = total / pairs;
  size_t at = 0;
  auto place = [&](size_t bytes) { at += (bytes + 255) / 256 * 256; return bytes; };
  pl.p_bytes = place(static_cast<size_t>(d->T) * 2 * d->F * 2);
  pl.db_bytes = place(static_cast<size_t>((d->T + 31) / 32) * 2 * d->F * 4);
  for (int i = 0; i < 2; ++i) {
    sdattn::ProductSide& s = pl.pp.s[i];
    s.splits = 1;
    if (s.ksteps > 1.25 * L) s.splits = std::max(1, std::min(s.ksteps / 8, static_cast<int>(std::ceil(s.ksteps / L))));
    s.kper = (s.ksteps + s.splits - 1) / s.splits;
    s.splits = (s.ksteps + s.kper - 1) / s.kper;
    s.units = s.mn * s.splits;
    pl.part_bytes[i] = s.splits > 1 ? place(static_cast<size_t>(s.splits) * s.M * s.N * 4) : 0;
  }
  sdattn::ProductParams& pp = pl.pp;
  pp.first = pp.s[1].kper >= pp.s[0].kper ? 1 : 0;
  pp.wide = pp.s[0].bn > 256 ? 1 : 0;           // both results have C columns
  pl.pairs = std::min(pairs, pp.s[0].units + pp.s[1].units);
  pp.heavy = pp.s[pp.first].units % pl.pairs;
  const int light = pl.pairs - pp.heavy, n2 = pp.s[1 - pp.first].units;
  pp.fill = pp.heavy == 0 ? 0 : std::min(pp.s[pp.first].kper / pp.s[1 - pp.first].kper, (n2 + light - 1) / light);
  pl.total = at;
  return pl;
}

template <bool BF16>
sdattn_status launch_ff_bwd(const sdattn_ff_desc* d, const FFBwdPlan& pl, const void* dY, const void* X, const void* W,
                            const float* bias, void* dX, void* dW, float* dbias, void* ws, cudaStream_t s) {
  const int dev = current_device();
  if (dev < 0) return SDATTN_ERR_CUDA;
  const int nsm = sm_count(dev);
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  void* P = take(pl.p_bytes);
  float* db_part = reinterpret_cast<float*>(take(pl.db_bytes));
  float* parts[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i)
    if (pl.part_bytes[i] > 0) parts[i] = reinterpret_cast<float*>(take(pl.part_bytes[i]));

  sdattn_status st = launch_gated<BF16, true>(d, X, W, bias, dY, P, dbias ? db_part : nullptr, s);
  if (st != SDATTN_OK) return st;

  const uint64_t T = d->T, C = d->C, F2 = 2 * uint64_t(d->F);
  const CUtensorMapDataType dt = elem16(d->dtype);
  CUtensorMap mpk, mpm, mw, mx, mo[2];
  if (!make_map_3d(&mpk, P, dt, F2, T, 1, F2 * 2, T * F2 * 2, 64, 128)) return SDATTN_ERR_CUDA;
  if (!make_map_3d(&mpm, P, dt, F2, T, 1, F2 * 2, T * F2 * 2, 64, 64)) return SDATTN_ERR_CUDA;
  if (!make_map_3d(&mw, W, dt, C, F2, 1, C * 2, F2 * C * 2, 64, 64)) return SDATTN_ERR_CUDA;
  if (!make_map_3d(&mx, X, dt, C, T, 1, C * 2, T * C * 2, 64, 64)) return SDATTN_ERR_CUDA;
  void* outs[2] = {dX, dW};
  for (int i = 0; i < 2; ++i) {
    const sdattn::ProductSide& sd = pl.pp.s[i];
    const uint64_t M = sd.M;
    const bool ok = sd.splits > 1
                        ? make_map_3d(&mo[i], parts[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, C, M, sd.splits, C * 4, M * C * 4, 32, 32)
                        : make_map_3d(&mo[i], outs[i], dt, C, M, 1, C * 2, M * C * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return SDATTN_ERR_CUDA;
  }
  auto kern = sdattn::product_kernel<BF16>;
  static std::atomic<uint64_t> done{0};
  if (!ensure_smem(kern, sdattn::ProductCfg::SMEM, done, dev)) return SDATTN_ERR_CUDA;
  if (!launch_cluster(kern, pl.pairs * 2, 2, sdattn::ProductCfg::NTHREADS, sdattn::ProductCfg::SMEM, s, mpk, mpm, mw, mx, mo[0], mo[1], pl.pp))
    return SDATTN_ERR_CUDA;
  sdattn::FinishParams f = {};
  int64_t work = 0;
  for (int i = 0; i < 2; ++i) {
    const sdattn::ProductSide& sd = pl.pp.s[i];
    if (sd.splits == 1) continue;
    f.part[i] = parts[i];
    f.out[i] = outs[i];
    f.n[i] = static_cast<int64_t>(sd.M) * sd.N;
    f.splits[i] = sd.splits;
    work = std::max(work, f.n[i] / 8);
  }
  f.first = static_cast<int>(std::min<int64_t>((work + 127) / 128, int64_t(nsm) * 2));
  if (dbias) {
    f.db_part = db_part;
    f.db = dbias;
    f.rows = (d->T + 31) / 32;
    f.cols = 2 * d->F;
  }
  const int blocks = f.first + (dbias ? (f.cols + 31) / 32 : 0);
  if (blocks == 0) return SDATTN_OK;
  return launch(sdattn::finish_kernel<BF16>, blocks, 1024, 0, s, f) ? SDATTN_OK : SDATTN_ERR_CUDA;
}

// --------------------------------------------------------------------------
// Projection with low-rank adapters (adapter.cuh)
// --------------------------------------------------------------------------
sdattn_status check_adapter(const sdattn_adapter_desc* d) {
  if (!d) return SDATTN_ERR_INVALID_ARG;
  if (d->T < 0 || d->C < 1 || d->K < 1 || d->L < 0 || d->R < 0 || d->rows < 1 || d->T % d->rows != 0)
    return SDATTN_ERR_INVALID_ARG;
  if ((d->L == 0) != (d->R == 0)) return SDATTN_ERR_INVALID_ARG;
  if (d->dtype != SDATTN_F16 && d->dtype != SDATTN_BF16) return SDATTN_ERR_UNSUPPORTED;
  // whole 16-byte units along C, K and R, as TMA needs; the bounds keep every
  // tile count in 32 bits
  if (d->C % 8 != 0 || d->K % 8 != 0 || d->R % 8 != 0 || d->C > 65536 || d->K > 65536 || d->R > 256 ||
      d->T >= (int64_t(1) << 27))
    return SDATTN_ERR_UNSUPPORTED;
  return SDATTN_OK;
}

// Ranks per slot of a phase, and slots per adapter (adapter.cuh).
int adapter_rc(const sdattn_adapter_desc* d) { return std::max(16, std::min(64, (d->R + 15) / 16 * 16)); }
int adapter_chunks(const sdattn_adapter_desc* d) { return std::max(1, (d->R + 63) / 64); }

// Columns per tile (16, 48, or a multiple of 32, up to `most`, so that equal
// pieces of whole 16-byte units go to at most four warps): the fewest waves of the
// longest of a tile's products (2 clocks per column and 64 of C, the adapters'
// ranks included), issue (300 clocks a step), loads (45 bytes per clock and SM)
// and epilogue, plus one epilogue at the end.
struct AdapterTiles {
  int bn;
  double waves, clocks;
};

AdapterTiles plan_adapter(const sdattn_adapter_desc* d, int tm, int rc, int most, int nsm) {
  const int64_t rts = (d->T + tm - 1) / tm;
  const double ksteps = (d->C + 63) / 64;
  AdapterTiles best{most, 0, 1e300};
  for (int bn = most; bn >= 16; bn -= 16) {
    if (bn % 32 != 0 && bn != 16 && bn != 48) continue;
    const int64_t tiles = rts * ((d->K + bn - 1) / bn);
    const double waves = static_cast<double>((tiles + nsm - 1) / nsm);
    const double step = std::max(std::max(2.0 * (bn + rc), 300.0), 128.0 * (tm + bn + rc) / 45.0);
    const double clocks = waves * std::max(ksteps * step, 12.0 * bn) + 12.0 * bn;
    if (clocks < best.clocks) best = {bn, waves, clocks};
  }
  return best;
}

int adapter_tm(const sdattn_adapter_desc* d) { return static_cast<int>(std::min<int64_t>(128, (d->T + 7) / 8 * 8)); }

// Whether the adapters are per-row work: requests of fewer than 16 rows whose
// adapters could fill three phases or more of a tile, where that is expected
// to be the cheaper form.  Which adapters meet in a tile is on the device; the
// one-launch form costs between one adapter a tile (best) and as many as its
// rows allow (worst): a phase past the first another pass over x and D (380
// clocks a step, or its loads), a slot past the first 1400 clocks, a tile's
// hand-off 4000.  The per-row form costs a launch and D and U read for every
// row (2000 bytes a clock).  It is taken where rows^2 < best * worst, so that
// neither form can lose by more than the square root of worst / best.  One
// adapter a tile, random ids, per-row form, measured: 64 rows of 1600 to 2560,
// 32 adapters of rank 128: 19, 340, 35 us (per row); 300 rows of 1280, 200 of
// rank 64: 13, 499, 39 (per row); 48 rows of 1280, 12 of rank 32: 10, 41, 9
// (per row); 64 requests of 8 rows of 1280, 32 of rank 64: 15, 111, 44 (one
// launch); 16384 rows of 320, 16 of rank 8: 16, 45, 64 (one launch).
bool adapter_rows(const sdattn_adapter_desc* d, int nsm) {
  if (d->L == 0 || d->T == 0 || d->rows >= 16) return false;
  if (d->T * d->R > (int64_t(1) << 24)) return false;   // z: 64 MB of workspace at most
  const int rc = adapter_rc(d), spp = sdattn::AdapterCfg::ZN / rc, chunks = adapter_chunks(d), tm = adapter_tm(d);
  const int64_t distinct = std::min<int64_t>(std::min<int64_t>(d->T / d->rows, (128 + d->rows - 1) / d->rows + 1), d->L);
  if (distinct * chunks <= 2 * spp) return false;
  const AdapterTiles mma = plan_adapter(d, tm, rc, sdattn::AdapterCfg::BN, nsm);
  const AdapterTiles plain = plan_adapter(d, tm, 0, sdattn::AdapterCfg::BN_ROWS, nsm);
  const double pass = (d->C + 63) / 64 * std::max(380.0, 128.0 * (tm + sdattn::AdapterCfg::ZN) / 45.0);
  auto launch = [&](int64_t adapters) {
    const int64_t slots = adapters * chunks, phases = (slots + spp - 1) / spp;
    return 4000.0 + mma.clocks + mma.waves * (4000.0 + (phases - 1) * pass + (slots - 1) * 1400.0);
  };
  const double rows = 8000.0 + plain.clocks + static_cast<double>(d->T) * d->R * (d->C + d->K) * 2.0 / 2000.0;
  return rows * rows < launch(1) * launch(distinct);
}

size_t adapter_ws_bytes(const sdattn_adapter_desc* d, int nsm) {
  return adapter_rows(d, nsm) ? static_cast<size_t>(d->T) * d->R * sizeof(float) : 0;
}

template <bool BF16, int MODE>
sdattn_status launch_adapter(const sdattn_adapter_desc* d, const void* X, const void* W, const float* bias,
                             const void* D, const void* U, const float* scale, const int32_t* ids, void* Y, void* ws,
                             cudaStream_t s) {
  using Cfg = sdattn::AdapterCfg;
  constexpr bool MMA = MODE == sdattn::kAdapterMma, ROWS = MODE == sdattn::kAdapterRows;
  const int dev = current_device();
  if (dev < 0) return SDATTN_ERR_CUDA;
  const int nsm = sm_count(dev);
  const uint64_t T = d->T, C = d->C, K = d->K, L = d->L, R = d->R;
  sdattn::AdapterParams p;
  p.bias = bias;
  p.ids = ids;
  p.scale = scale;
  p.z = static_cast<const float*>(ws);
  p.U = U;
  p.Y = Y;
  p.T = static_cast<int>(T);
  p.K = d->K;
  p.L = d->L;
  p.R = d->R;
  p.rows = d->rows;
  p.rc = adapter_rc(d);
  p.chunks = adapter_chunks(d);
  p.tm = adapter_tm(d);
  p.bn = plan_adapter(d, p.tm, MMA ? p.rc : 0, ROWS ? Cfg::BN_ROWS : Cfg::BN, nsm).bn;
  p.rts = static_cast<int>((T + p.tm - 1) / p.tm);
  p.nts = (d->K + p.bn - 1) / p.bn;
  p.ksteps = (d->C + 63) / 64;
  const int step = p.tm * 128 + p.bn * 128 + (MMA ? Cfg::ZN * 128 : 0);
  const int room = Cfg::ring(MODE) - (p.tm < 128 ? Cfg::SLACK : 0);
  p.sub = room / (2 * step) >= 3 ? 2 : 1;
  p.stage = p.sub * step;
  p.stages = std::min(Cfg::MAX_STAGES, room / p.stage);
  const CUtensorMapDataType dt = elem16(d->dtype);
  CUtensorMap mx, mw, md, mu, my;
  if (!make_map_3d(&mx, X, dt, C, T, 1, C * 2, T * C * 2, 64, static_cast<uint32_t>(p.tm))) return SDATTN_ERR_CUDA;
  if (!make_map_3d(&mw, W, dt, C, K, 1, C * 2, K * C * 2, 64, static_cast<uint32_t>(p.bn))) return SDATTN_ERR_CUDA;
  p.pw = (p.bn + 31) / 32 * 8;
  if (!make_map_3d(&my, Y, dt, K, T, 1, K * 2, T * K * 2, static_cast<uint32_t>(p.pw), 32, CU_TENSOR_MAP_SWIZZLE_NONE))
    return SDATTN_ERR_CUDA;
  if (MMA) {
    if (!make_map_3d(&md, D, dt, C, R, L, C * 2, R * C * 2, 64, static_cast<uint32_t>(p.rc))) return SDATTN_ERR_CUDA;
    if (!make_map_3d(&mu, U, dt, R, K, L, R * 2, K * R * 2, 64, static_cast<uint32_t>(p.bn))) return SDATTN_ERR_CUDA;
  } else {
    md = mu = mw;   // never read
  }
  if constexpr (ROWS) {
    const int64_t warps = d->T * (d->R / 2);
    if (!launch(sdattn::adapter_z_kernel<BF16>, static_cast<int>((warps + 7) / 8), 256, 0, s,
                static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(D), scale, ids, static_cast<float*>(ws),
                p.T, d->C, d->L, d->R, d->rows))
      return SDATTN_ERR_CUDA;
  }
  auto kern = sdattn::adapter_kernel<BF16, MODE>;
  static std::atomic<uint64_t> done{0};
  if (!ensure_smem(kern, Cfg::SMEM, done, dev)) return SDATTN_ERR_CUDA;
  const int grid = static_cast<int>(std::min<int64_t>(nsm, int64_t(p.rts) * p.nts));
  return launch(kern, grid, Cfg::NTHREADS, Cfg::SMEM, s, mx, mw, md, mu, my, p) ? SDATTN_OK : SDATTN_ERR_CUDA;
}

template <bool BF16>
sdattn_status dispatch_adapter(const sdattn_adapter_desc* d, bool rows, const void* X, const void* W, const float* bias,
                               const void* D, const void* U, const float* scale, const int32_t* ids, void* Y, void* ws,
                               cudaStream_t s) {
  if (!ids) return launch_adapter<BF16, sdattn::kAdapterNone>(d, X, W, bias, D, U, scale, ids, Y, ws, s);
  if (rows) return launch_adapter<BF16, sdattn::kAdapterRows>(d, X, W, bias, D, U, scale, ids, Y, ws, s);
  return launch_adapter<BF16, sdattn::kAdapterMma>(d, X, W, bias, D, U, scale, ids, Y, ws, s);
}

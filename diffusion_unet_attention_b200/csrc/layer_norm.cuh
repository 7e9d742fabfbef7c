// layer_norm.cuh -- the transformer block's layer normalisation, forward and
// backward.
//
//   forward   m = mean(x), r = 1 / sqrt(var(x) + eps) (biased variance),
//             z = (x - m) r,  y = z gamma + beta            per row of C values
//   backward  e = dy gamma,
//             dx = r (e - mean(e) - z mean(e z)),
//             dgamma = sum over rows of dy z,  dbeta = sum over rows of dy
//
// Both passes are bound by memory: x (and dy) are read once, y (dx) written
// once; everything between is held in registers.  A row belongs to L lanes of
// a warp (L = 8, 16 or 32; several rows per warp when rows are short) or to a
// whole CTA when it is too long for a warp's registers, so its sums are a few
// shuffles.  The variance is the mean of squared deviations from the mean
// (two passes over registers, no cancellation).  Where the mean is above eight
// deviations a third pass takes what its rounding left off them (a constant row
// of 2000: 1e-4, which r = 316 would make 0.04; taken off in every row it cost
// rows of a CTA 10%).  All arithmetic is fp32; y and dx are rounded once to the
// element type.
//
// The weight's gradients: every CTA runs over rows b, b + grid, ... and keeps
// the sums of its columns in registers (a lane owns the same columns of every
// row it sees), adds its warps' sums in warp order and writes one partial
// row of 2C floats; a second kernel adds the partial rows in a fixed order
// (with one CTA its sums are the result).
// No atomics: repeated calls give identical bits.
//
// Measured: backward, 65536 rows of 320 fp32 values (252 MB), 48 us, 5.2 TB/s,
// 78% of a copy's rate; what is left is the column sums' arithmetic and the
// chain load, two sums, store of each row, which two CTAs per SM overlap.
// Reading x and dy a second time (from L1) instead of holding them took 51 us,
// loading the next row ahead 56 us (registers: one CTA per SM).  Forward, the same
// rows, 27 us (6.2 TB/s), of fp16 20 us.  Forward and backward of 8192 rows of
// 320 16-bit values take 5.4 and 9.0 us, one and two dependent launches on data
// that is in L2.  Element by element (319 fp16 values, 65536 rows) 54 and 186 us.
#pragma once

#include "unet_ops.cuh"

namespace sdattn {

enum : int { kElemF16 = 0, kElemBF16 = 1, kElemF32 = 2 };

// E consecutive elements as loaded (RawT) and as floats.  VEC: one 16-byte
// access (8 16-bit or 4 fp32 elements); otherwise one element at a time.
template <int DT, bool VEC>
struct LNElem {
  static constexpr int E = VEC ? (DT == kElemF32 ? 4 : 8) : 1;
  using Scalar = typename std::conditional<DT == kElemF32, float, uint16_t>::type;
  using Raw = typename std::conditional<VEC, uint4, Scalar>::type;

  __device__ static __forceinline__ Raw load(const void* base, int64_t at) {
    return __ldcs(reinterpret_cast<const Raw*>(static_cast<const Scalar*>(base) + at));
  }
  __device__ static __forceinline__ Raw zero() {
    if constexpr (VEC) {
      return make_uint4(0, 0, 0, 0);
    } else {
      return Raw(0);
    }
  }
  __device__ static __forceinline__ void unpack(const Raw& r, float* f) {
    if constexpr (VEC && DT == kElemF32) {
      f[0] = __uint_as_float(r.x);
      f[1] = __uint_as_float(r.y);
      f[2] = __uint_as_float(r.z);
      f[3] = __uint_as_float(r.w);
    } else if constexpr (VEC) {
      unpack8<DT == kElemBF16>(r, f);
    } else if constexpr (DT == kElemF32) {
      f[0] = r;
    } else if constexpr (DT == kElemBF16) {
      f[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
    } else {
      f[0] = __half2float(__ushort_as_half(r));
    }
  }
  __device__ static __forceinline__ void store(void* base, int64_t at, const float* f) {
    Raw* p = reinterpret_cast<Raw*>(static_cast<Scalar*>(base) + at);
    if constexpr (VEC && DT == kElemF32) {
      __stcs(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    } else if constexpr (VEC) {
      __stcs(p, pack8<DT == kElemBF16>(f));
    } else if constexpr (DT == kElemF32) {
      *p = f[0];
    } else if constexpr (DT == kElemBF16) {
      *p = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
      *p = __half_as_ushort(__float2half_rn(f[0]));
    }
  }
  // E fp32 parameters at column c; `dflt` where there are none
  __device__ static __forceinline__ void params(const float* p, int c, float dflt, float* f) {
    if (p == nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = dflt;
    } else if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + c) + q);
        f[4 * q] = v.x;
        f[4 * q + 1] = v.y;
        f[4 * q + 2] = v.z;
        f[4 * q + 3] = v.w;
      }
    } else {
      f[0] = __ldg(p + c);
    }
  }
};

constexpr int kLNThreads = 256;      // rows shared by lanes of a warp
constexpr int kLNRowThreads = 512;   // a whole CTA per row

struct LNParams {
  const void* X;
  void* Y;              // forward
  const void* dY;       // backward
  void* dX;
  const float* gamma;   // may be null (ones)
  const float* beta;    // may be null (zeros)
  float* stats;         // [T][2]: mean, 1 / sqrt(var + eps)  (forward: may be null)
  float* part0;         // backward: partial sums of dgamma and dbeta, CTA b's at + b * pitch
  float* part1;
  int64_t pitch;
  int64_t T;
  int C;
  int nch;              // accesses of E elements per row
  int L;                // lanes per row (CTA kernels: all threads)
  float eps;
};

// Sums a and b over the row's lanes; every lane gets both totals.
template <bool CTA>
__device__ __forceinline__ void ln_row_sums(float& a, float& b, int L, float* red) {
  if constexpr (CTA) {
    a = block_sum(a, red);
    b = block_sum(b, red);
  } else {
    for (int off = L >> 1; off >= 1; off >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, off);
      b += __shfl_xor_sync(0xffffffffu, b, off);
    }
  }
}

template <bool CTA>
__device__ __forceinline__ float ln_row_sum(float a, int L, float* red) {
  if constexpr (CTA) {
    return block_sum(a, red);
  } else {
    for (int off = L >> 1; off >= 1; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    return a;
  }
}

template <int DT, bool VEC, int U, bool CTA>
__global__ void __launch_bounds__(CTA ? kLNRowThreads : kLNThreads) layer_norm_kernel(const LNParams p) {
  using El = LNElem<DT, VEC>;
  constexpr int E = El::E;
  __shared__ float red[32];
  const int lane = CTA ? threadIdx.x : threadIdx.x & (p.L - 1);
  const int rpc = CTA ? 1 : blockDim.x / p.L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rpc + (CTA ? 0 : threadIdx.x / p.L);
  const bool live = row < p.T;
  const int64_t at = row * p.C;
  grid_dependency_wait();
  grid_launch_dependents();
  typename El::Raw r[U];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = lane + u * p.L;
    r[u] = live && i < p.nch ? El::load(p.X, at + static_cast<int64_t>(i) * E) : El::zero();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[E];
    El::unpack(r[u], f);   // zeros past the row's end add nothing
#pragma unroll
    for (int e = 0; e < E; ++e) sum += f[e];
  }
  const float inv = 1.f / static_cast<float>(p.C);
  const float mean = ln_row_sum<CTA>(sum, p.L, red) * inv;
  float sq = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (lane + u * p.L < p.nch) {
      float f[E];
      El::unpack(r[u], f);
#pragma unroll
      for (int e = 0; e < E; ++e) sq = fmaf(f[e] - mean, f[e] - mean, sq);
    }
  }
  float squares = ln_row_sum<CTA>(sq, p.L, red);
  // The mean's rounding matters where it is large beside the deviations: their
  // own mean is what it left.  (All rows of a warp together; a CTA has one row.)
  const bool far = live && squares * inv * 64.f < mean * mean;
  float shift = 0.f;
  if (__builtin_expect(CTA ? far : __any_sync(0xffffffffu, far), 0)) {
    float dev = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (lane + u * p.L < p.nch) {
        float f[E];
        El::unpack(r[u], f);
#pragma unroll
        for (int e = 0; e < E; ++e) dev += f[e] - mean;
      }
    }
    dev = ln_row_sum<CTA>(dev, p.L, red);
    shift = dev * inv;
    if (!far) shift = 0.f;                    // whatever rows share its warp, a row's result is the same
    squares = fmaxf(squares - shift * dev, 0.f);
  }
  const float rstd = 1.f / sqrtf(fmaf(squares, inv, p.eps)), offset = -shift * rstd;
  if (!live) return;
  if (p.stats != nullptr && lane == 0) *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(mean + shift, rstd);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = lane + u * p.L;
    if (i < p.nch) {
      float f[E], g[E], b[E];
      El::unpack(r[u], f);
      El::params(p.gamma, i * E, 1.f, g);
      El::params(p.beta, i * E, 0.f, b);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf(fmaf(f[e] - mean, rstd, offset), g[e], b[e]);
      El::store(p.Y, at + static_cast<int64_t>(i) * E, f);
    }
  }
}

template <int DT, bool VEC, int U, bool CTA>
__global__ void __launch_bounds__(CTA ? kLNRowThreads : kLNThreads) layer_norm_bwd_kernel(const LNParams p) {
  using El = LNElem<DT, VEC>;
  constexpr int E = El::E;
  __shared__ float red[32];
  extern __shared__ __align__(16) float colsum[];   // [warps][C], warp kernels only
  const int lane = CTA ? threadIdx.x : threadIdx.x & (p.L - 1);
  const int rpc = CTA ? 1 : blockDim.x / p.L;
  const int grp = CTA ? 0 : threadIdx.x / p.L;
  const float inv = 1.f / static_cast<float>(p.C);
  float ag[U][E], ab[U][E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) ag[u][e] = ab[u][e] = 0.f;
  grid_dependency_wait();
  grid_launch_dependents();
  // the loop's bound is the CTA's, so every lane takes part in every sum
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpc; row0 < p.T; row0 += static_cast<int64_t>(gridDim.x) * rpc) {
    const int64_t row = row0 + grp;
    const bool live = row < p.T;
    const int64_t at = row * p.C;
    typename El::Raw rx[U], rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = lane + u * p.L;
      const bool ok = live && i < p.nch;
      rx[u] = ok ? El::load(p.X, at + static_cast<int64_t>(i) * E) : El::zero();
      rd[u] = ok ? El::load(p.dY, at + static_cast<int64_t>(i) * E) : El::zero();
    }
    const float2 st = live ? __ldg(reinterpret_cast<const float2*>(p.stats + 2 * row)) : make_float2(0.f, 0.f);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = lane + u * p.L;
      if (live && i < p.nch) {
        float x[E], d[E], g[E];
        El::unpack(rx[u], x);
        El::unpack(rd[u], d);
        El::params(p.gamma, i * E, 1.f, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float z = (x[e] - st.x) * st.y;
          ag[u][e] = fmaf(d[e], z, ag[u][e]);
          ab[u][e] += d[e];
          const float w = d[e] * g[e];
          s1 += w;
          s2 = fmaf(w, z, s2);
        }
      }
    }
    ln_row_sums<CTA>(s1, s2, p.L, red);
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = lane + u * p.L;
      if (live && i < p.nch) {
        float x[E], d[E], g[E];
        El::unpack(rx[u], x);
        El::unpack(rd[u], d);
        El::params(p.gamma, i * E, 1.f, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float z = (x[e] - st.x) * st.y;
          d[e] = st.y * (fmaf(d[e], g[e], -s1) - z * s2);
        }
        El::store(p.dX, at + static_cast<int64_t>(i) * E, d);
      }
    }
  }
  float* out0 = p.part0 + blockIdx.x * p.pitch;
  float* out1 = p.part1 + blockIdx.x * p.pitch;
  if constexpr (CTA) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = lane + u * p.L;
      if (i < p.nch)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          out0[i * E + e] = ag[u][e];
          out1[i * E + e] = ab[u][e];
        }
    }
  } else {
    // rows of one warp first (lanes L apart own the same columns), then the
    // warps in order
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e)
        for (int off = 16; off >= p.L; off >>= 1) {
          ag[u][e] += __shfl_xor_sync(0xffffffffu, ag[u][e], off);
          ab[u][e] += __shfl_xor_sync(0xffffffffu, ab[u][e], off);
        }
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int side = 0; side < 2; ++side) {        // dgamma's sums, then dbeta's
      if (static_cast<int>(threadIdx.x & 31) < p.L) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = lane + u * p.L;
          if (i < p.nch) {
            const float* a = side ? ab[u] : ag[u];
            float* d = colsum + warp * p.C + i * E;
            if constexpr (VEC) {
#pragma unroll
              for (int q = 0; q < E / 4; ++q)
                reinterpret_cast<float4*>(d)[q] = make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
            } else {
              *d = a[0];
            }
          }
        }
      }
      __syncthreads();
      for (int j = threadIdx.x; j < p.C; j += blockDim.x) {
        float t = colsum[j];
        for (int w = 1; w < nw; ++w) t += colsum[w * p.C + j];
        (side ? out1 : out0)[j] = t;
      }
      __syncthreads();
    }
  }
}

// Adds P partial rows of n floats, column by column and in a fixed order: 32
// columns per block of 1024 threads, 32 threads per column over rows r, r + 32,
// ..., then the 32 sums in order.  The first n0 columns go to out0, the others
// to out1.
__device__ __forceinline__ void column_sum_block(const float* part, int64_t P, int n, int n0, float* out0, float* out1,
                                                 int block) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int j = block * 32 + cx;
  float a = 0.f;
  if (j < n) {
#pragma unroll 8
    for (int64_t r = ry; r < P; r += 32) a += __ldcg(part + r * n + j);
  }
  s[ry][cx] = a;
  __syncthreads();
  // warp ry now owns column ry of the block: its 32 lanes add the 32 sums
  float t = s[cx][ry];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  const int jj = block * 32 + ry;
  if (cx == 0 && jj < n) {
    if (jj < n0) {
      out0[jj] = t;
    } else {
      out1[jj - n0] = t;
    }
  }
}

__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int64_t P, int n, int n0, float* out0,
                                                          float* out1) {
  grid_dependency_wait();
  grid_launch_dependents();
  column_sum_block(part, P, n, n0, out0, out1, blockIdx.x);
}

}  // namespace sdattn

// Layer normalisation over the channel axis of x [outer][C][inner], forward and
// backward.  A point is one (outer, inner) pair; its C values lie `inner`
// elements apart.
//   mean = sum_c x / C,  var = sum_c (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh gamma + beta
//   g = dy gamma,  dx = rstd (g - mean_c(g) - xh mean_c(g xh))
//   dgamma[c] = sum_points dy xh,  dbeta[c] = sum_points dy
// All sums are float32 (over many channels compensated: Sum).  The variance is taken
// about a first mean m0 in a second sweep over the values, which also gives
// e = mean(x - m0), the rounding of m0: mean = m0 + e, var = mean((x - m0)^2) - e^2,
// xh = ((x - m0) - e) rstd, so a common offset far above the spread costs no more than
// the offset's own storage.
//
// Times beside these kernels (norm*.cu) are device times: calls in a captured graph on
// inputs used in turn, which exceed L2 together where the case is large (one B200 at 1965
// MHz).  A pass on fresh inputs through the binding takes up to 10 % more, a small one
// its host time (about 7 us forward, 10 backward).
//
// The kernels here serve what no other one takes (many channels on a grid, very long
// rows).  They read the values again in each sweep, and on grids a thread walks its
// point's channels alone: 2 x 2100 x 600 float32 forward 503 us, backward 686.
#include "norm_common.cuh"

namespace fno {

namespace {

constexpr int LT = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// sum over the CTA of LT threads, the same value in every thread
__device__ __forceinline__ float cta_sum(float v, float *sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < LT / 32; ++i) t += sh[i];
  __syncthreads();
  return t;
}

// ---------------------------------------------------------------------------
// any channel count: the values are read again in each sweep
// ---------------------------------------------------------------------------

// A thread's sum of many values with the rounding of every addition kept beside it and
// made good by the next (Kahan, "Further remarks on reducing truncation errors"): off by
// two units of 2^-24 of the sum of the values' sizes, however many they are.  (One
// float32 chain of 4099 equal values was off by 690 units, one of 2^20 values by 1 %.)
struct Sum {
  float s = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float w = v - lost, t = s + w;
    lost = (t - s) - w;
    s = t;
  }
};

// thread per point (inner > 1: neighbouring threads read neighbouring points)
template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_fwd_point(const T *x, const T *__restrict__ gamma, const T *__restrict__ beta, T *y,
                   float *__restrict__ mean, float *__restrict__ rstd, long long points, int C,
                   long long inner, float inv_c, float eps) {
  const long long stride = (long long)gridDim.x * LT;
  for (long long p = (long long)blockIdx.x * LT + threadIdx.x; p < points; p += stride) {
    const long long b = p / inner, base = b * C * inner + (p - b * inner);
    Sum m, es, q;
    for (int c = 0; c < C; ++c) m.add(to_f<T>(x[base + c * inner]));
    const float m0 = m.s * inv_c;
    for (int c = 0; c < C; ++c) {
      const float d = to_f<T>(x[base + c * inner]) - m0;
      es.add(d);
      q.add(d * d);
    }
    const float e = es.s * inv_c, r = ln_rstd(q.s * inv_c, e, eps);
    if (mean) {
      mean[p] = m0 + e;
      rstd[p] = r;
    }
    for (int c = 0; c < C; ++c) {
      const float xh = ((to_f<T>(x[base + c * inner]) - m0) - e) * r;
      y[base + c * inner] = from_f<T>(fmaf(xh, gamma ? to_f<T>(gamma[c]) : 1.f,
                                           beta ? to_f<T>(beta[c]) : 0.f));
    }
  }
}

// The values of channels c .. c + 7 of a point, all on their way before the first is
// used; beyond the last channel that one again.
template <typename T>
__device__ __forceinline__ void next8(const T *p, long long hop, int c, int C, float *v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f<T>(p[(c + i < C ? c + i : C - 1) * hop]);
}

template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_bwd_point(const T *__restrict__ x, const T *__restrict__ gamma,
                   const float *__restrict__ mean, const float *__restrict__ rstd, const T *dy,
                   T *dx, long long points, int C, long long inner, float inv_c) {
  const long long stride = (long long)gridDim.x * LT;
  for (long long p = (long long)blockIdx.x * LT + threadIdx.x; p < points; p += stride) {
    const long long b = p / inner, base = b * C * inner + (p - b * inner);
    const float mu = mean[p], r = rstd[p];
    Sum gs, gx;
    float v[8], w[8], ga[8];
    for (int c = 0; c < C; c += 8) {
      next8<T>(x + base, inner, c, C, v);
      next8<T>(dy + base, inner, c, C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) ga[i] = gamma ? to_f<T>(gamma[c + i < C ? c + i : C - 1]) : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = c + i < C ? w[i] * ga[i] : 0.f;
        gs.add(g);
        gx.add(g * ((v[i] - mu) * r));
      }
    }
    const float c1 = gs.s * inv_c, c2 = gx.s * inv_c;
    for (int c = 0; c < C; ++c) {
      const float g = to_f<T>(dy[base + c * inner]) * (gamma ? to_f<T>(gamma[c]) : 1.f);
      const float xh = (to_f<T>(x[base + c * inner]) - mu) * r;
      dx[base + c * inner] = from_f<T>(r * (g - c1 - xh * c2));
    }
  }
}

// CTA per (channel, slice of the points): partial[slice][c] = (dgamma, dbeta)
template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_dparam_point(const T *__restrict__ x, const float *__restrict__ mean,
                      const float *__restrict__ rstd, const T *__restrict__ dy,
                      float *__restrict__ partial, long long points, int C, long long inner) {
  __shared__ float sh[LT / 32];
  const int c = blockIdx.x, slices = gridDim.y, sl = blockIdx.y;
  float dg = 0.f, db = 0.f;
  for (long long p = (long long)sl * LT + threadIdx.x; p < points; p += (long long)slices * LT) {
    const long long b = p / inner, i = (b * C + c) * inner + (p - b * inner);
    const float d = to_f<T>(dy[i]);
    dg = fmaf(d, (to_f<T>(x[i]) - mean[p]) * rstd[p], dg);
    db += d;
  }
  dg = cta_sum(dg, sh);
  db = cta_sum(db, sh);
  if (threadIdx.x == 0) {
    partial[((long long)sl * C + c) * 2] = dg;
    partial[((long long)sl * C + c) * 2 + 1] = db;
  }
}

// CTA per row (inner == 1)
template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_fwd_row(const T *x, const T *__restrict__ gamma, const T *__restrict__ beta, T *y,
                 float *__restrict__ mean, float *__restrict__ rstd, long long rows, int C,
                 float inv_c, float eps) {
  __shared__ float sh[LT / 32];
  for (long long p = blockIdx.x; p < rows; p += gridDim.x) {
    const T *xr = x + p * C;
    T *yr = y + p * C;
    Sum m, es, q;
    for (int c = threadIdx.x; c < C; c += LT) m.add(to_f<T>(xr[c]));
    const float m0 = cta_sum(m.s, sh) * inv_c;
    for (int c = threadIdx.x; c < C; c += LT) {
      const float d = to_f<T>(xr[c]) - m0;
      es.add(d);
      q.add(d * d);
    }
    const float e = cta_sum(es.s, sh) * inv_c;
    const float r = ln_rstd(cta_sum(q.s, sh) * inv_c, e, eps);
    if (mean && threadIdx.x == 0) {
      mean[p] = m0 + e;
      rstd[p] = r;
    }
    for (int c = threadIdx.x; c < C; c += LT) {
      const float xh = ((to_f<T>(xr[c]) - m0) - e) * r;
      yr[c] = from_f<T>(fmaf(xh, gamma ? to_f<T>(gamma[c]) : 1.f, beta ? to_f<T>(beta[c]) : 0.f));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_bwd_row(const T *__restrict__ x, const T *__restrict__ gamma,
                 const float *__restrict__ mean, const float *__restrict__ rstd, const T *dy,
                 T *dx, long long rows, int C, float inv_c) {
  __shared__ float sh[LT / 32];
  for (long long p = blockIdx.x; p < rows; p += gridDim.x) {
    const float mu = mean[p], r = rstd[p];
    Sum gs, gx;
    for (int c = threadIdx.x; c < C; c += LT) {
      const float g = to_f<T>(dy[p * C + c]) * (gamma ? to_f<T>(gamma[c]) : 1.f);
      gs.add(g);
      gx.add(g * ((to_f<T>(x[p * C + c]) - mu) * r));
    }
    const float c1 = cta_sum(gs.s, sh) * inv_c, c2 = cta_sum(gx.s, sh) * inv_c;
    for (int c = threadIdx.x; c < C; c += LT) {
      const float g = to_f<T>(dy[p * C + c]) * (gamma ? to_f<T>(gamma[c]) : 1.f);
      const float xh = (to_f<T>(x[p * C + c]) - mu) * r;
      dx[p * C + c] = from_f<T>(r * (g - c1 - xh * c2));
    }
  }
}

// thread per channel over a slice of the rows
template <typename T>
__global__ void __launch_bounds__(LT)
    k_ln_dparam_row(const T *__restrict__ x, const float *__restrict__ mean,
                    const float *__restrict__ rstd, const T *__restrict__ dy,
                    float *__restrict__ partial, long long rows, int C) {
  const int c = blockIdx.x * LT + threadIdx.x;
  if (c >= C) return;
  float dg = 0.f, db = 0.f;
  for (long long p = blockIdx.y; p < rows; p += gridDim.y) {
    const float d = to_f<T>(dy[p * C + c]);
    dg = fmaf(d, (to_f<T>(x[p * C + c]) - mean[p]) * rstd[p], dg);
    db += d;
  }
  partial[((long long)blockIdx.y * C + c) * 2] = dg;
  partial[((long long)blockIdx.y * C + c) * 2 + 1] = db;
}

unsigned capped(long long want, long long cap) {
  return (unsigned)(want < 1 ? 1 : want < cap ? want : cap);
}

// slices of the points, each a partial row
int dparam_row_slices(long long rows) { return (int)capped((rows + 15) / 16, kLnParts); }
int dparam_point_slices(long long points) {
  return (int)capped((points + 4 * LT - 1) / (4 * LT), kLnParts);
}

// dgamma and dbeta of the kernels' partial rows [nparts][C][2].  A CTA takes COLS
// neighbouring values, neighbouring threads neighbouring values of a row and the
// CTA's 1024 threads as many rows as they reach; their sums meet in a fixed order.
// Launched while the kernel before it runs (launch_dependent).  With reduce_partials
// after a normal launch the backward took 18.2 us at 4099 x 1001 float32 (16.1 now).
// Eight values a CTA while all CTAs run at once
// (4 x 20 x 4096: 4.2 us, with 32 values 4.7; 4096 x 8192 bfloat16: 88.9 and 78.7).
template <int COLS>
__global__ void __launch_bounds__(1024)
    k_ln_reduce(const float *partial, int nparts, int n, float *dgamma, float *dbeta) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * COLS + threadIdx.x % COLS;
  cudaGridDependencySynchronize();
  float s = 0.f;
  if (e < n) {
    const float *src = partial + e;
#pragma unroll 8
    for (int p = threadIdx.x / COLS; p < nparts; p += 1024 / COLS)
      s += __ldcg(src + (long long)p * n);
  }
#pragma unroll
  for (int o = COLS; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  sh[warp][lane] = s;
  __syncthreads();
  const int out = blockIdx.x * COLS + warp;
  if (warp >= COLS || out >= n) return;
  s = warp_sum(sh[lane][warp]);
  float *to = out & 1 ? dbeta : dgamma;
  if (lane == 0 && to) to[out >> 1] = s;
}

cudaError_t reduce_params(const Launch &L, const float *partial, int nparts, int C, float *dgamma,
                          float *dbeta) {
  const int n = 2 * C, cols = n <= 8 * 2 * L.num_sms ? 8 : 32;
  launch_begin(L);
  const cudaError_t err =
      launch_dependent(L, (n + cols - 1) / cols, 1024, cols == 8 ? k_ln_reduce<8> : k_ln_reduce<32>,
                       partial, nparts, n, dgamma, dbeta);
  launch_end(L, "ln_dparam_sum");
  return err;
}

}  // namespace

// The partial rows that no kernel exceeds for this shape on any device: a row is the work
// of one CTA, and no CTA of the grid kernels has fewer than 32 points of a sample (the
// pipelines and the odd grids) or of all (the register kernels).  A larger outer never
// needs fewer rows, whichever kernels it goes to, so that a workspace serves every
// smaller batch.
size_t ln_partial_bytes(const NormShape &s, int dtype) {
  const long long points = s.outer * s.inner;
  long long rows;
  if (ln_rows_supported(s, dtype, true)) rows = ln_rows_parts(s, dtype);
  else if (s.inner == 1) rows = dparam_row_slices(points);
  else if (s.C > kGridBwdChannels) rows = dparam_point_slices(points);
  else rows = capped(s.outer * ((s.inner + 31) / 32), kLnParts);
  return sizeof(float) * 2 * (size_t)s.C * (size_t)rows;
}

cudaError_t launch_ln_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                          const void *gamma, const void *beta, void *y, float *mean,
                          float *rstd) {
  if (ln_pipe_supported(s, dtype, false))
    return launch_ln_pipe_fwd(L, s, dtype, x, gamma, beta, y, mean, rstd);
  if (ln_rows_supported(s, dtype, false))
    return launch_ln_rows_fwd(L, s, dtype, x, gamma, beta, y, mean, rstd);
  if (ln_odd_supported(s, dtype, false))
    return launch_ln_odd(L, s, dtype, x, gamma, beta, nullptr, y, mean, rstd, nullptr, nullptr,
                         nullptr, nullptr);
  if (ln_grid_supported(s, dtype, false))
    return launch_ln_grid_fwd(L, s, dtype, x, gamma, beta, y, mean, rstd);
  const long long points = s.outer * s.inner;
  const float inv_c = 1.0f / (float)s.C;
  launch_begin(L);
  if (s.inner == 1) {
    const unsigned grid = capped(points, 8LL * L.num_sms);
    FNO_DISPATCH_T(dtype, k_ln_fwd_row<T><<<grid, LT, 0, L.stream>>>(
                              (const T *)x, (const T *)gamma, (const T *)beta, (T *)y, mean, rstd,
                              points, s.C, inv_c, s.eps));
  } else {
    const unsigned grid = capped((points + LT - 1) / LT, 8LL * L.num_sms);
    FNO_DISPATCH_T(dtype, k_ln_fwd_point<T><<<grid, LT, 0, L.stream>>>(
                              (const T *)x, (const T *)gamma, (const T *)beta, (T *)y, mean, rstd,
                              points, s.C, s.inner, inv_c, s.eps));
  }
  const cudaError_t err = cudaGetLastError();
  launch_end(L, "ln_fwd");
  return err;
}

cudaError_t launch_ln_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                          const void *gamma, const float *mean, const float *rstd, const void *dy,
                          void *dx, float *dgamma, float *dbeta, float *partial) {
  const long long points = s.outer * s.inner;
  const float inv_c = 1.0f / (float)s.C;
  cudaError_t err;
  const bool params = dgamma || dbeta;
  float *part = params ? partial : nullptr;
  int nparts = 0;
  bool done = true;
  if (ln_pipe_supported(s, dtype, true))
    err = launch_ln_pipe_bwd(L, s, dtype, x, gamma, mean, rstd, dy, dx, part, &nparts);
  else if (ln_rows_supported(s, dtype, true))
    err = launch_ln_rows_bwd(L, s, dtype, x, gamma, mean, rstd, dy, dx, part, &nparts);
  else if (ln_odd_supported(s, dtype, true))
    err = launch_ln_odd(L, s, dtype, x, gamma, nullptr, dy, dx, nullptr, nullptr, mean, rstd,
                        part, &nparts);
  else if (ln_grid_supported(s, dtype, true))
    err = launch_ln_grid_bwd(L, s, dtype, x, gamma, mean, rstd, dy, dx, part, &nparts);
  else
    done = false;
  if (done) {
    if (err != cudaSuccess || !params) return err;
    return reduce_params(L, partial, nparts, s.C, dgamma, dbeta);
  }
  // the parameter gradients first: dx may overwrite dy
  if (params) {
    int slices;
    launch_begin(L);
    if (s.inner == 1) {
      slices = dparam_row_slices(points);
      const dim3 grid((s.C + LT - 1) / LT, slices);
      FNO_DISPATCH_T(dtype, k_ln_dparam_row<T><<<grid, LT, 0, L.stream>>>(
                                (const T *)x, mean, rstd, (const T *)dy, partial, points, s.C));
    } else {
      slices = dparam_point_slices(points);
      const dim3 grid(s.C, slices);
      FNO_DISPATCH_T(dtype, k_ln_dparam_point<T><<<grid, LT, 0, L.stream>>>(
                                (const T *)x, mean, rstd, (const T *)dy, partial, points, s.C,
                                s.inner));
    }
    err = cudaGetLastError();
    launch_end(L, "ln_dparam");
    if (err != cudaSuccess) return err;
    err = reduce_params(L, partial, slices, s.C, dgamma, dbeta);
    if (err != cudaSuccess) return err;
  }
  launch_begin(L);
  if (s.inner == 1) {
    const unsigned grid = capped(points, 8LL * L.num_sms);
    FNO_DISPATCH_T(dtype, k_ln_bwd_row<T><<<grid, LT, 0, L.stream>>>(
                              (const T *)x, (const T *)gamma, mean, rstd, (const T *)dy, (T *)dx,
                              points, s.C, inv_c));
  } else {
    const unsigned grid = capped((points + LT - 1) / LT, 8LL * L.num_sms);
    FNO_DISPATCH_T(dtype, k_ln_bwd_point<T><<<grid, LT, 0, L.stream>>>(
                              (const T *)x, (const T *)gamma, mean, rstd, (const T *)dy, (T *)dx,
                              points, s.C, s.inner, inv_c));
  }
  err = cudaGetLastError();
  launch_end(L, "ln_bwd");
  return err;
}

}  // namespace fno

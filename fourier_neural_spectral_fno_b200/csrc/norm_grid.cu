// Layer norm over the channels of grid activations (inner > 1), one pass: every
// value is read once, kept in registers and written once.
//
// A warp owns LP x V neighbouring points.  With groups of V = 4 or 8 points (inner
// a multiple of V) LP lanes cover 128 contiguous bytes of a channel row and the
// warp's 32 / LP lane groups take different channels, so a lane holds CPL
// channels of V points and the channel sums are CPL - 1 additions and a few
// shuffles.  Where inner is no such multiple the rows start at any element: 32
// lanes then read one element each of a channel row.  Channels beyond one
// warp's registers are spread over up to MW warps of a CTA, whose sums meet in
// shared memory.
//
// Both directions are bound by HBM (the arithmetic is about 7 and 14 operations
// per value); the design aims at bytes in flight: all CPL loads of a lane are
// issued before the first is used.  16 x 32 x 65536 float32 forward 44.5 us, 96 % of
// the copy rate; 1 x 20 x 256 float32 2.6 us; 4 x 20 x 4096 float32 backward 4.2 with its
// parameters' sums.  Where the channels are spread over a CTA's warps it is at half that
// rate (8 x 256 x 65536 bfloat16 forward 169 us, 50 %; backward 415, 30 %).
#include "norm_common.cuh"

namespace fno {

namespace {

constexpr int GT = 128;          // threads per CTA where one warp holds all channels

template <typename T, int V> struct Lanes {
  // lanes along the points: 128 contiguous bytes of a channel row
  static constexpr int LP = V > 1 ? 128 / (V * sizeof(T)) : 32;
  static constexpr int G = 32 / LP;           // channel groups in a warp
};

// sum over the channel groups of a warp: lanes LP apart
template <typename T, int V> __device__ __forceinline__ void group_sum(float *s) {
#pragma unroll
  for (int o = Lanes<T, V>::LP; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
}

// sum over the warps of a CTA: buf [W][LP V], each warp's group 0 writes
template <typename T, int V>
__device__ __forceinline__ void warps_sum(float *s, float *buf, int warp, int warps, int pl,
                                          int grp) {
  constexpr int P = Lanes<T, V>::LP * V;
  if (grp == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) buf[warp * P + pl * V + i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += buf[w * P + pl * V + i];
}

// element offset of channel 0 of point p
__device__ __forceinline__ long long point_base(long long p, long long inner, int C,
                                                long long points) {
  if (points <= 0x7fffffffLL) {   // 32-bit division
    const unsigned b = (unsigned)p / (unsigned)inner;
    return (long long)b * (C - 1) * inner + p;
  }
  return (p / inner) * (C - 1) * inner + p;
}

// MW: most warps that the channels are spread over, one tile per CTA; 0: every
// warp has a tile of its own.
template <typename T, int V, int CPL, int MW>
__global__ void __launch_bounds__(MW ? 32 * MW : GT)
    k_ln_fwd_grid(const T *x, const T *__restrict__ gamma, const T *__restrict__ beta, T *y,
                  float *__restrict__ mean, float *__restrict__ rstd, long long points, int C,
                  long long inner, float inv_c, float eps) {
  constexpr int LP = Lanes<T, V>::LP, G = Lanes<T, V>::G, P = LP * V;
  __shared__ float red[MW ? 2 * MW * P : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int pl = lane % LP, grp = lane / LP;
  const long long tile = MW ? (long long)blockIdx.x : (long long)blockIdx.x * warps + warp;
  const long long p0 = tile * P + pl * V;
  const bool in = p0 < points;
  // channel of slot j: c0 + j step
  const int c0 = MW ? warp * G + grp : grp, step = MW ? warps * G : G;
  const long long base = in ? point_base(p0, inner, C, points) : 0;
  const T *xp = x + base + c0 * inner;
  Pack<T, V> v[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    v[j].zero();
    const int c = c0 + j * step;
    if (in && c < C) v[j] = *reinterpret_cast<const Pack<T, V> *>(xp);
    xp += step * inner;
  }
  float m0[V], e[V], q[V], f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) m0[i] = e[i] = q[i] = 0.f;
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    v[j].get(f);
#pragma unroll
    for (int i = 0; i < V; ++i) m0[i] += f[i];
    v[j].keep();
  }
  group_sum<T, V>(m0);
  if (MW) warps_sum<T, V>(m0, red, warp, warps, pl, grp);
#pragma unroll
  for (int i = 0; i < V; ++i) m0[i] *= inv_c;
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    if (c0 + j * step < C) {
      v[j].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = f[i] - m0[i];
        e[i] += d;
        q[i] = fmaf(d, d, q[i]);
      }
      v[j].keep();
    }
  }
  group_sum<T, V>(e);
  group_sum<T, V>(q);
  if (MW) {
    warps_sum<T, V>(e, red + MW * P, warp, warps, pl, grp);
    warps_sum<T, V>(q, red, warp, warps, pl, grp);   // every warp has read red by now
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    e[i] *= inv_c;
    q[i] = ln_rstd(q[i] * inv_c, e[i], eps);
  }
  if (!in) return;
  if (mean && c0 == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mean[p0 + i] = m0[i] + e[i];
      rstd[p0 + i] = q[i];
    }
  }
  T *yp = y + base + again(c0 * inner);
  const long long hop = again(step * inner);
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = c0 + j * step;
    if (c < C) {
      const float ga = gamma ? ldf(gamma + c) : 1.f, be = beta ? ldf(beta + c) : 0.f;
      v[j].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = fmaf(((f[i] - m0[i]) - e[i]) * q[i], ga, be);
      v[j].set(f);
      *reinterpret_cast<Pack<T, V> *>(yp) = v[j];
      yp += hop;
    }
  }
}

// Persistent over the tiles: a lane keeps its channels' dgamma and dbeta sums in
// registers; at the end lanes along the points meet by shuffles, the CTA's warps
// in shared memory, and the CTA writes one row of partial sums.
template <typename T, int V, int CPL, int MW>
__global__ void __launch_bounds__(MW ? 32 * MW : GT)
    k_ln_bwd_grid(const T *__restrict__ x, const T *__restrict__ gamma,
                  const float *__restrict__ mean, const float *__restrict__ rstd, const T *dy,
                  T *dx, float *__restrict__ partial, long long points, int C, long long inner,
                  float inv_c) {
  constexpr int LP = Lanes<T, V>::LP, G = Lanes<T, V>::G, P = LP * V;
  __shared__ float red[MW ? 2 * MW * P : 2 * (GT / 32) * CPL * G];
  cudaTriggerProgrammaticLaunchCompletion();   // the sum of the partial rows is set up meanwhile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int pl = lane % LP, grp = lane / LP;
  const int c0 = MW ? warp * G + grp : grp, step = MW ? warps * G : G;
  const long long tiles = (points + P - 1) / P;
  const long long first = MW ? (long long)blockIdx.x : (long long)blockIdx.x * warps + warp;
  const long long stride = MW ? (long long)gridDim.x : (long long)gridDim.x * warps;
  float dg[CPL], db[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) dg[j] = db[j] = 0.f;
  for (long long tile = first; tile < tiles; tile += stride) {
    const long long p0 = tile * P + pl * V;
    const bool in = p0 < points;
    const long long base = in ? point_base(p0, inner, C, points) : 0;
    const T *xp = x + base + c0 * inner, *yp = dy + base + c0 * inner;
    Pack<T, V> a[CPL], b[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      a[j].zero();
      b[j].zero();
      const int c = c0 + j * step;
      if (in && c < C) {
        a[j] = *reinterpret_cast<const Pack<T, V> *>(xp);
        b[j] = *reinterpret_cast<const Pack<T, V> *>(yp);
      }
      xp += step * inner;
      yp += step * inner;
    }
    float mu[V], r[V], c1[V], c2[V], f[V], g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mu[i] = in ? mean[p0 + i] : 0.f;
      r[i] = in ? rstd[p0 + i] : 0.f;
      c1[i] = c2[i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = c0 + j * step;
      const float ga = gamma && c < C ? ldf(gamma + c) : 1.f;
      a[j].get(f);
      b[j].get(g);
#pragma unroll
      for (int i = 0; i < V; ++i) {   // dy is 0 where there is nothing
        const float xh = (f[i] - mu[i]) * r[i], gg = g[i] * ga;
        c1[i] += gg;
        c2[i] = fmaf(gg, xh, c2[i]);
        dg[j] = fmaf(g[i], xh, dg[j]);
        db[j] += g[i];
      }
      a[j].keep();
      b[j].keep();
    }
    group_sum<T, V>(c1);
    group_sum<T, V>(c2);
    if (MW) {
      warps_sum<T, V>(c1, red, warp, warps, pl, grp);
      warps_sum<T, V>(c2, red + MW * P, warp, warps, pl, grp);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c1[i] *= inv_c;
      c2[i] *= inv_c;
    }
    T *op = dx + base + again(c0 * inner);
    const long long hop = again(step * inner);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = c0 + j * step;
      if (in && c < C) {
        const float ga = gamma ? ldf(gamma + c) : 1.f;
        a[j].get(f);
        b[j].get(g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (f[i] - mu[i]) * r[i];
          g[i] = r[i] * (fmaf(g[i], ga, -c1[i]) - xh * c2[i]);
        }
        b[j].set(g);
        *reinterpret_cast<Pack<T, V> *>(op) = b[j];
        op += hop;
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int j = 0; j < CPL; ++j)
#pragma unroll
    for (int o = 1; o < LP; o <<= 1) {
      dg[j] += __shfl_xor_sync(0xffffffffu, dg[j], o);
      db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
    }
  float *row = partial + (long long)blockIdx.x * 2 * C;
  if (MW) {   // every warp has channels of its own
    if (pl == 0)
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const int c = c0 + j * step;
        if (c < C) {
          row[2 * c] = dg[j];
          row[2 * c + 1] = db[j];
        }
      }
    return;
  }
  if (pl == 0)
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      red[(warp * CPL * G + j * G + grp) * 2] = dg[j];
      red[(warp * CPL * G + j * G + grp) * 2 + 1] = db[j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C; i += GT) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) s += red[w * CPL * G * 2 + i];
    row[i] = s;
  }
}

// groups of four values (the forward) stay inside a channel row
bool vec_ok(const NormShape &s) { return s.inner % 4 == 0; }

// Channels per lane for which kernels exist.  A lane's 16-byte groups cost four
// registers each (the backward holds two arrays); single elements cost one, and
// the backward two sums more per channel.
#define LN_FWD_CASES(CALL)                                         \
  do {                                                             \
    if (vec_ok(s)) {                                        \
      const int need = (s.C + Lanes<T, 4>::G - 1) / Lanes<T, 4>::G; \
      if (need <= 2) CALL(4, 2, 0);                                \
      else if (need <= 4) CALL(4, 4, 0);                           \
      else if (need <= 6) CALL(4, 6, 0);                           \
      else if (need <= 8) CALL(4, 8, 0);                           \
      else if (need <= 10) CALL(4, 10, 0);                         \
      else if (need <= 12) CALL(4, 12, 0);                         \
      else if (need <= 16) CALL(4, 16, 0);                         \
      else CALL(4, 16, 16);                                        \
    } else {                                                       \
      if (s.C <= 8) CALL(1, 8, 0);                                 \
      else if (s.C <= 16) CALL(1, 16, 0);                          \
      else if (s.C <= 24) CALL(1, 24, 0);                          \
      else if (s.C <= 32) CALL(1, 32, 0);                          \
      else CALL(1, 32, 16);                                        \
    }                                                              \
  } while (0)

#define LN_BWD_CASES(CALL)                                        \
  do {                                                            \
    constexpr int VN = VecOf<T>::N;                               \
    if (s.inner % VN == 0) {                                       \
      const int need = (s.C + Lanes<T, VN>::G - 1) / Lanes<T, VN>::G;   \
      if (need <= 2) CALL(VN, 2, 0);                              \
      else if (need <= 4) CALL(VN, 4, 0);                         \
      else if (VN == 4 && need <= 6) CALL(VN, 6, 0);              \
      else if (VN == 4 && need <= 8) CALL(VN, 8, 0);              \
      else CALL(VN, 4, 16);                         \
    } else {                                                      \
      if (s.C <= 8) CALL(1, 8, 0);                                \
      else if (s.C <= 16) CALL(1, 16, 0);                         \
      else if (s.C <= 24) CALL(1, 24, 0);                         \
      else CALL(1, 16, 16);                                       \
    }                                                             \
  } while (0)

template <typename T, int V, int CPL, int MW> int grid_threads(const NormShape &s) {
  if (!MW) return GT;
  const int per = CPL * Lanes<T, V>::G;
  return 32 * ((s.C + per - 1) / per);
}

template <typename T, int V, int MW> long long grid_tiles(const NormShape &s, int threads) {
  const long long tiles = (s.outer * s.inner + Lanes<T, V>::LP * V - 1) / (Lanes<T, V>::LP * V);
  return MW ? tiles : (tiles + threads / 32 - 1) / (threads / 32);
}

template <typename T, int V, int CPL, int MW>
cudaError_t fwd_t(const Launch &L, const NormShape &s, const void *x, const void *gamma,
                  const void *beta, void *y, float *mean, float *rstd) {
  const int threads = grid_threads<T, V, CPL, MW>(s);
  const long long grid = grid_tiles<T, V, MW>(s, threads);
  k_ln_fwd_grid<T, V, CPL, MW><<<(unsigned)grid, threads, 0, L.stream>>>(
      (const T *)x, (const T *)gamma, (const T *)beta, (T *)y, mean, rstd, s.outer * s.inner, s.C,
      s.inner, 1.0f / (float)s.C, s.eps);
  return cudaGetLastError();
}

template <typename T, int V, int CPL, int MW>
cudaError_t bwd_t(const Launch &L, const NormShape &s, const void *x, const void *gamma,
                  const float *mean, const float *rstd, const void *dy, void *dx, float *partial,
                  int *nparts) {
  const int threads = grid_threads<T, V, CPL, MW>(s);
  long long grid = grid_tiles<T, V, MW>(s, threads);
  if (grid > kLnParts) grid = kLnParts;
  *nparts = (int)grid;
  k_ln_bwd_grid<T, V, CPL, MW><<<(unsigned)grid, threads, 0, L.stream>>>(
      (const T *)x, (const T *)gamma, mean, rstd, (const T *)dy, (T *)dx, partial,
      s.outer * s.inner, s.C, s.inner, 1.0f / (float)s.C);
  return cudaGetLastError();
}

}  // namespace

// the channels that the widest kernels hold (16 warps), and a grid that fits its
// 31 bits
bool ln_grid_supported(const NormShape &s, int dtype, bool bwd) {
  if (s.inner == 1 || s.outer * s.inner > 32LL * 0x7fffffffLL) return false;
  // 16 warps of four lane groups of 4 channels, or of single elements of 16
  static_assert(kGridBwdChannels == 16 * 16, "channels of the widest backward");
  if (bwd) return s.C <= kGridBwdChannels;
  if (vec_ok(s)) return s.C <= (dtype == DT_F32 ? 4 : 2) * 16 * 16;
  return s.C <= 32 * 16;
}

cudaError_t launch_ln_grid_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd) {
  cudaError_t err = cudaSuccess;
#define LN_FWD(V, CPL, MW) \
  err = fwd_t<T, V, CPL, MW>(L, s, x, gamma, beta, y, mean, rstd)
  launch_begin(L);
  FNO_DISPATCH_T(dtype, LN_FWD_CASES(LN_FWD));
  launch_end(L, "ln_fwd");
#undef LN_FWD
  return err;
}

cudaError_t launch_ln_grid_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts) {
  cudaError_t err = cudaSuccess;
#define LN_BWD(V, CPL, MW) \
  err = bwd_t<T, V, CPL, MW>(L, s, x, gamma, mean, rstd, dy, dx, partial, nparts)
  launch_begin(L);
  FNO_DISPATCH_T(dtype, LN_BWD_CASES(LN_BWD));
  launch_end(L, "ln_bwd");
#undef LN_BWD
  return err;
}

}  // namespace fno

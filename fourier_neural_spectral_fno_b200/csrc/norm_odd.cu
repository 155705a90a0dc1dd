// Layer norm over the channels of grid activations whose rows start anywhere (odd
// grid sides: the number of points is no multiple of a 16-byte piece), at most 128
// channels.
//
// A warp takes 32 PPL neighbouring points of one sample, a lane the points lane,
// lane + 32, ...: single values, but neighbouring lanes read neighbouring ones and
// a channel's address, coefficients and loop are shared by PPL points.  Up to 32
// channels forward and 24 backward a lane walks all of them itself, so the sums
// need no exchange; beyond that the KW warps of a CTA share the points, each with
// its part of the channels in registers, and add up their sums in shared memory.
// Lanes beyond the row's end repeat its last point and store nothing.
// The work per value, not HBM, bounds this form with 16-bit types; the element
// kernels of norm_grid.cu, one point per lane with coefficients read from global
// memory, took 48 instructions a value.  Copying a tile's whole 16-byte pieces
// through shared memory, each row at its own offset, measured slower (29 us at 12 x
// 20 x 48323 float16).  Measured there, against the element kernels: forward 13.4
// and 19.3 us, backward 23.7 and 37.9; float32 forward 18.9 and 19.4, backward 28.5 and
// 34.1.  4 x 64 x 44521: float16 forward 16.2 and 26.4, backward 29.0 and 43.6, float32
// 19.6 and 25.6, 30.3 and 39.5; 4 x 128 x 44521: 37.4 and 50.5, 63.0 and 86.1, 37.0
// and 47.5, 62.9 and 79.2.
#include "norm_common.cuh"

namespace fno {

namespace {

constexpr int OT = 128;   // threads per CTA where a warp holds all channels

constexpr int odd_threads(int KW) { return KW > 1 ? 32 * KW : OT; }
// Forward CTAs an SM that the compiler plans for; 0: it chooses the registers by itself
// (held to one CTA it takes up to 24 more: 4 x 128 x 44521 float32 41.1 us against 36.7).
// With 20 channels seven, since by itself it then fits 63 registers by loading in turns
// (12 x 20 x 48323 float16 16.4 us a pass on fresh inputs against 14.8, float32 19.4
// against 18.9).
constexpr int odd_ctas(int CM, int KW) { return KW == 1 && CM == 20 ? 7 : 0; }

struct OddArgs {
  const void *x, *dy, *gamma, *beta;
  const float *mean_in, *rstd_in;
  float *mean_out, *rstd_out;
  void *out;
  float *partial;
  long long inner;
  unsigned tiles, segs;
  int C;
  float inv_c, eps;
};

// a warp's tile: where the lane's points lie
template <int PPL> struct Spot {
  long long base, point;   // element of channel 0, and point, of the lane's first one
  int off[PPL];            // its points from there on
  bool in[PPL];
  __device__ __forceinline__ Spot(const OddArgs &a, unsigned tile) {
    const unsigned b = tile / a.segs;
    const int lane = threadIdx.x & 31;
    const long long n = (long long)(tile - b * a.segs) * (32 * PPL) + lane;
    const long long n0 = n < a.inner ? n : a.inner - 1;
    base = (long long)b * a.C * a.inner + n0;
    point = (long long)b * a.inner + n0;
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      in[k] = n + 32 * k < a.inner;
      off[k] = in[k] ? 32 * k : 0;
    }
  }
};

template <typename T> __device__ __forceinline__ void coefs(const OddArgs &a, int n, float2 *coef) {
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    const T *g = static_cast<const T *>(a.gamma), *h = static_cast<const T *>(a.beta);
    coef[c] = c < a.C ? make_float2(g ? ldf(g + c) : 1.f, h ? ldf(h + c) : 0.f)
                      : make_float2(0.f, 0.f);
  }
  __syncthreads();
}

// The KW warps' values v[0 .. M-1] of each lane added up in a fixed order, the same
// in every warp.  `turn` alternates: a slow warp still reads what a fast one does not
// overwrite.
template <int KW, int M>
__device__ __forceinline__ void join(float (*sh)[KW][M][32], int turn, float *v) {
  if constexpr (KW > 1) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < M; ++k) sh[turn][threadIdx.x >> 5][k][lane] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < M; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) v[k] += sh[turn][w][k][lane];
    }
  }
}

// KW = 1: a warp's tile has all channels.  Else the CTA's KW warps share a tile, each
// with C / KW neighbouring channels, rounded down or up: at least one (C >= KW), at
// most CM.
template <int KW> __device__ __forceinline__ int first_channel(int C, int warp) {
  return KW > 1 ? warp * C / KW : 0;
}

// CLO: the fewest channels of a warp that CM is used for.  The correction of the mean as
// in norm_rows.cu (4 x 128 x 44521 float16 37.3 us, as a sum 40.3).
template <typename T, int CM, int CLO, int PPL, int KW>
__global__ void __launch_bounds__(odd_threads(KW), odd_ctas(CM, KW)) k_ln_fwd_odd(const __grid_constant__ OddArgs a) {
  constexpr bool kResidual = CM * KW <= ResidualChannels<T>::N;
  constexpr int M = kResidual ? PPL : 2 * PPL;   // sums of the second sweep
  __shared__ float2 coef[CM * KW];
  __shared__ float sums[1][KW][PPL][32], sums2[1][KW][M][32];
  coefs<T>(a, CM * KW, coef);
  const int warp = threadIdx.x >> 5, c0 = first_channel<KW>(a.C, warp);
  const unsigned tile = KW > 1 ? blockIdx.x : blockIdx.x * (OT / 32) + warp;
  if (KW == 1 && tile >= a.tiles) return;
  const Spot<PPL> sp(a, tile);
  const int C = KW > 1 ? first_channel<KW>(a.C, warp + 1) - c0 : a.C;   // the warp's
  const long long base = sp.base + c0 * a.inner;
  float v[CM][PPL], m[PPL], e[PPL], q[PPL];
  {
    const T *p = static_cast<const T *>(a.x) + base;
#pragma unroll
    for (int c = 0; c < CM; ++c) {
#pragma unroll
      for (int k = 0; k < PPL; ++k) v[c][k] = c < CLO || c < C ? to_f<T>(p[sp.off[k]]) : 0.f;
      p += a.inner;
    }
  }
#pragma unroll
  for (int k = 0; k < PPL; ++k) m[k] = e[k] = q[k] = 0.f;
#pragma unroll
  for (int c = 0; c < CM; ++c)
#pragma unroll
    for (int k = 0; k < PPL; ++k) m[k] += v[c][k];
  join<KW, PPL>(sums, 0, m);
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    const float sum = m[k];
    m[k] = sum * a.inv_c;
    if (kResidual) e[k] = ln_residual(sum, m[k], a.C, a.inv_c);
  }
#pragma unroll
  for (int c = 0; c < CM; ++c)
    if (c < CLO || c < C)
#pragma unroll
      for (int k = 0; k < PPL; ++k) {
        v[c][k] -= m[k];
        if (!kResidual) e[k] += v[c][k];
        q[k] = fmaf(v[c][k], v[c][k], q[k]);
      }
  if (KW > 1) {
    float qe[M];
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      qe[k] = q[k];
      if (!kResidual) qe[PPL + k] = e[k];
    }
    join<KW, M>(sums2, 0, qe);
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      q[k] = qe[k];
      if (!kResidual) e[k] = qe[PPL + k];
    }
  }
  T *p = static_cast<T *>(a.out) + base;
  const long long hop = again(a.inner);
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    if (!kResidual) e[k] *= a.inv_c;
    q[k] = ln_rstd(q[k] * a.inv_c, e[k], a.eps);
    if (a.mean_out && sp.in[k] && c0 == 0) {
      a.mean_out[sp.point + sp.off[k]] = m[k] + e[k];
      a.rstd_out[sp.point + sp.off[k]] = q[k];
    }
    e[k] *= -q[k];   // xh = (x - m) q - e q
  }
#pragma unroll
  for (int c = 0; c < CM; ++c) {
    if (c < CLO || c < C) {
      const float2 gb = coef[c0 + c];
#pragma unroll
      for (int k = 0; k < PPL; ++k)
        if (sp.in[k]) p[sp.off[k]] = from_f<T>(fmaf(fmaf(v[c][k], q[k], e[k]), gb.x, gb.y));
    }
    p += hop;
  }
}

// Persistent: the channels' dgamma and dbeta sums stay in registers.  One point per
// lane: with two the values of 20 channels cost half the warps (and half again the time
// at 12 x 20 x 48323 float16).  EACH: CTAs an SM; where warps share the channels the
// registers are held to what so many CTAs leave (4 x 64 x 44521 float32: 30.3 us,
// without that 40.4).
template <typename T, int CM, int CLO, int KW, int EACH>
__global__ void __launch_bounds__(odd_threads(KW), KW > 1 ? EACH : 1)
    k_ln_bwd_odd(const __grid_constant__ OddArgs a) {
  __shared__ float2 coef[CM * KW];
  __shared__ float red[KW > 1 ? 1 : OT / 32][KW > 1 ? 1 : 2 * CM];
  __shared__ float sums[2][KW][2][32];
  cudaTriggerProgrammaticLaunchCompletion();   // the sum of the partial rows is set up meanwhile
  coefs<T>(a, CM * KW, coef);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = first_channel<KW>(a.C, warp);
  const int C = KW > 1 ? first_channel<KW>(a.C, warp + 1) - c0 : a.C;   // the warp's
  int turn = 0;
  float dg[CM], db[CM];
#pragma unroll
  for (int c = 0; c < CM; ++c) dg[c] = db[c] = 0.f;
  constexpr int W = KW > 1 ? 1 : OT / 32;   // tiles at a time
  for (unsigned tile = blockIdx.x * W + (KW > 1 ? 0 : warp); tile < a.tiles;
       tile += gridDim.x * W) {
    const Spot<1> sp(a, tile);
    const long long base = sp.base + c0 * a.inner;
    const float mu = a.mean_in[sp.point], r = a.rstd_in[sp.point];
    float xh[CM], g[CM], c1[2] = {0.f, 0.f}, c2[2] = {0.f, 0.f};
    const T *px = static_cast<const T *>(a.x) + base;
    const T *py = static_cast<const T *>(a.dy) + base;
    // every load on its way before the first is used; beyond the warp's channels its
    // last one once more (a condition around loads and conversions became branches
    // that waited for each: 222 us against 80 at 4 x 128 x 44521 float16)
    long long off = 0;
#pragma unroll
    for (int c = 0; c < CM; ++c) {
      xh[c] = to_f<T>(px[off]);
      g[c] = to_f<T>(py[off]);
      off += c + 1 < CLO || c + 1 < C ? a.inner : 0;
    }
#pragma unroll
    for (int c = 0; c < CM; ++c) {
      const bool in = sp.in[0] && (c < CLO || c < C);
      const float d = in ? g[c] : 0.f;
      xh[c] = in ? (xh[c] - mu) * r : 0.f;
      dg[c] = fmaf(d, xh[c], dg[c]);
      db[c] += d;
      g[c] = d * coef[c0 + c].x;
      c1[c & 1] += g[c];
      c2[c & 1] = fmaf(g[c], xh[c], c2[c & 1]);
    }
    float c12[2] = {c1[0] + c1[1], c2[0] + c2[1]};
    join<KW, 2>(sums, turn, c12);
    turn ^= 1;
    const float k1 = c12[0] * a.inv_c, k2 = c12[1] * a.inv_c;
    T *po = static_cast<T *>(a.out) + base;
    const long long hop = again(a.inner);
#pragma unroll
    for (int c = 0; c < CM; ++c) {
      const T z = from_f<T>(r * ((g[c] - k1) - xh[c] * k2));
      if (sp.in[0] && (c < CLO || c < C)) *po = z;
      po += hop;
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int c = 0; c < CM; ++c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      dg[c] += __shfl_xor_sync(0xffffffffu, dg[c], o);
      db[c] += __shfl_xor_sync(0xffffffffu, db[c], o);
    }
    if (KW > 1) {
      if (lane == 0 && c < C)
        *reinterpret_cast<float2 *>(a.partial + ((long long)blockIdx.x * a.C + c0 + c) * 2) =
            make_float2(dg[c], db[c]);
    } else if (lane == 0) {
      red[warp][2 * c] = dg[c];
      red[warp][2 * c + 1] = db[c];
    }
  }
  if (KW > 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C; i += OT) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < OT / 32; ++w) s += red[w][i];
    a.partial[(long long)blockIdx.x * 2 * C + i] = s;
  }
}

template <typename T, int CM, int CLO, int PPL, int KW = 1>
cudaError_t fwd_t(const Launch &L, const NormShape &s, OddArgs a) {
  constexpr int W = KW > 1 ? 1 : OT / 32;
  a.segs = (unsigned)((s.inner + 32 * PPL - 1) / (32 * PPL));
  a.tiles = (unsigned)s.outer * a.segs;
  k_ln_fwd_odd<T, CM, CLO, PPL, KW>
      <<<(a.tiles + W - 1) / W, odd_threads(KW), 0, L.stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int CM, int CLO, int KW = 1, int EACH = 4>
cudaError_t bwd_t(const Launch &L, const NormShape &s, OddArgs a, int *nparts) {
  constexpr int W = KW > 1 ? 1 : OT / 32;
  a.segs = (unsigned)((s.inner + 31) / 32);
  a.tiles = (unsigned)s.outer * a.segs;
  unsigned grid = (a.tiles + W - 1) / W;
  const unsigned cap = EACH * L.num_sms < kLnParts ? EACH * L.num_sms : kLnParts;
  if (grid > cap) grid = cap;
  *nparts = (int)grid;
  k_ln_bwd_odd<T, CM, CLO, KW, EACH><<<grid, odd_threads(KW), 0, L.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Rows that fill most of their tiles, tile numbers of 32 bits.  Backward float16 with up
// to 8 channels, where a lane has few loads on their way, goes to the element kernels
// (15 x 8 x 48323: 20.4 us; 27.9 here, when that was tried; float32 23.1 there, 19.2
// here).  With 16 channels float16 takes 33.4 us here and 39.1 there; float32, which
// would gain a little there (32.9 against 37.4), follows the rule for 8 and for 20.
bool ln_odd_supported(const NormShape &s, int dtype, bool bwd) {
  if (s.inner % (bwd && dtype != DT_F32 ? 8 : 4) == 0) return false;
  const long long segs = (s.inner + 31) / 32;
  if (bwd && dtype != DT_F32 && s.C <= 8) return false;
  return s.C <= 128 && s.inner >= 256 && segs <= 0x7fffffffLL &&
         s.outer <= 0x7fffffffLL / segs;
}

cudaError_t launch_ln_odd(const Launch &L, const NormShape &s, int dtype, const void *x,
                          const void *gamma, const void *beta, const void *dy, void *out,
                          float *mean_out, float *rstd_out, const float *mean_in,
                          const float *rstd_in, float *partial, int *nparts) {
  OddArgs a{};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.out = out;
  a.mean_out = mean_out;
  a.rstd_out = rstd_out;
  a.mean_in = mean_in;
  a.rstd_in = rstd_in;
  a.partial = partial;
  a.inner = s.inner;
  a.C = s.C;
  a.inv_c = 1.0f / (float)s.C;
  a.eps = s.eps;
  cudaError_t err = cudaSuccess;
  launch_begin(L);
  FNO_DISPATCH_T(dtype, {
    if (dy) {
      constexpr int kLeast = sizeof(T) == 4 ? 8 : 16;   // 16-bit types: more than 8 channels
      if (s.C <= kLeast) err = bwd_t<T, kLeast, kLeast == 8 ? 1 : 9>(L, s, a, nparts);
      else if (s.C <= 16) err = bwd_t<T, 16, 9>(L, s, a, nparts);
      else if (s.C <= 20) err = bwd_t<T, 20, 17>(L, s, a, nparts);
      else if (s.C <= 24) err = bwd_t<T, 24, 21>(L, s, a, nparts);
      else if (s.C <= 32) err = bwd_t<T, 8, 0, 4, 4>(L, s, a, nparts);
      else if (s.C <= 48) err = bwd_t<T, 12, 0, 4, 4>(L, s, a, nparts);
      else if (s.C <= 64) err = bwd_t<T, 8, 0, 8, 4>(L, s, a, nparts);
      else if (s.C <= 96) err = bwd_t<T, 12, 0, 8, 2>(L, s, a, nparts);
      else err = bwd_t<T, 8, 0, 16, 2>(L, s, a, nparts);
    } else {
      // with shared channels one point a lane where the values are 4 bytes wide (16 x 64 x
      // 19881: float16 26.0 us with two, 34.0 with one; float32 32.2 and 30.7; 4 x 90 x
      // 44521: float16 24.9 and 28.9, float32 30.7 and 29.3), and in every type from 97
      // channels on (4 x 128 x 44521 float32: 38.4 with two, 37.0 with one; float16,
      // which two points would serve better, 29.9 and 37.4)
      if (s.C <= 8) err = fwd_t<T, 8, 1, 4>(L, s, a);
      else if (s.C <= 16) err = fwd_t<T, 16, 9, 4>(L, s, a);
      else if (s.C <= 20) err = fwd_t<T, 20, 17, 2>(L, s, a);
      else if (s.C <= 24) err = fwd_t<T, 24, 21, 2>(L, s, a);
      else if (s.C <= 32) err = fwd_t<T, 32, 25, 2>(L, s, a);
      else if (s.C <= 48) err = fwd_t<T, 12, 0, 2, 4>(L, s, a);
      else if (s.C <= 64) err = fwd_t<T, 16, 0, sizeof(T) == 4 ? 1 : 2, 4>(L, s, a);
      else if (s.C <= 96) err = fwd_t<T, 12, 0, sizeof(T) == 4 ? 1 : 2, 8>(L, s, a);
      else err = fwd_t<T, 16, 0, 1, 8>(L, s, a);
    }
  });
  launch_end(L, dy ? "ln_bwd_odd" : "ln_fwd_odd");
  return err;
}

}  // namespace fno

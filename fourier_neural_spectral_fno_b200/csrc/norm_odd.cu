// Layer norm over the channels of grid activations whose rows start anywhere (odd
// grid sides: the number of points is no multiple of a 16-byte piece), at most 48
// channels forward and 32 backward.
//
// A warp takes 32 PPL neighbouring points of one sample, a lane the points lane,
// lane + 32, ...: single values, but neighbouring lanes read neighbouring ones and
// a channel's address, coefficients and loop are shared by PPL points.  A lane
// walks all channels itself, so the sums need no exchange.  Lanes beyond the row's
// end repeat its last point and store nothing.
// The work per value, not HBM, bounds this form with 16-bit types; the element
// kernels of norm_grid.cu, one point per lane with coefficients read from global
// memory, took 48 instructions a value.  Copying a tile's whole 16-byte pieces
// through shared memory, each row at its own offset, measured slower (29 us at 12 x
// 20 x 48323 float16).  Measured there, against the element kernels: forward 14.2
// and 19.6 us, backward 27.8 and 41.2; float32 19.2 and 19.5, 32.1 and 37.5 (backward
// with a sum of the partial rows that took 3 us more than now).
#include "norm_common.cuh"

namespace fno {

namespace {

constexpr int OT = 128;   // threads per CTA

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

template <typename T> __device__ __forceinline__ void coefs(const OddArgs &a, float2 *coef) {
  for (int c = threadIdx.x; c < a.C; c += OT) {
    const T *g = static_cast<const T *>(a.gamma), *h = static_cast<const T *>(a.beta);
    coef[c] = make_float2(g ? ldf(g + c) : 1.f, h ? ldf(h + c) : 0.f);
  }
  __syncthreads();
}

// CLO: the fewest channels CM is used for
template <typename T, int CM, int CLO, int PPL>
__global__ void __launch_bounds__(OT) k_ln_fwd_odd(const __grid_constant__ OddArgs a) {
  constexpr bool kCorrect = sizeof(T) == 4;   // as in norm_pipe.cu
  __shared__ float2 coef[CM];
  coefs<T>(a, coef);
  const unsigned tile = blockIdx.x * (OT / 32) + (threadIdx.x >> 5);
  if (tile >= a.tiles) return;
  const Spot<PPL> sp(a, tile);
  const int C = a.C;
  float v[CM][PPL], m[PPL], e[PPL], q[PPL];
  {
    const T *p = static_cast<const T *>(a.x) + sp.base;
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
#pragma unroll
  for (int k = 0; k < PPL; ++k) m[k] *= a.inv_c;
#pragma unroll
  for (int c = 0; c < CM; ++c)
    if (c < CLO || c < C)
#pragma unroll
      for (int k = 0; k < PPL; ++k) {
        v[c][k] -= m[k];
        if (kCorrect) e[k] += v[c][k];
        q[k] = fmaf(v[c][k], v[c][k], q[k]);
      }
  T *p = static_cast<T *>(a.out) + sp.base;
  const long long hop = again(a.inner);
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    e[k] *= a.inv_c;
    q[k] = ln_rstd(q[k] * a.inv_c, e[k], a.eps);
    if (a.mean_out && sp.in[k]) {
      a.mean_out[sp.point + sp.off[k]] = m[k] + e[k];
      a.rstd_out[sp.point + sp.off[k]] = q[k];
    }
  }
#pragma unroll
  for (int c = 0; c < CM; ++c) {
    if (c < CLO || c < C) {
      const float2 gb = coef[c];
#pragma unroll
      for (int k = 0; k < PPL; ++k) {
        const float d = kCorrect ? v[c][k] - e[k] : v[c][k];
        if (sp.in[k]) p[sp.off[k]] = from_f<T>(fmaf(d * q[k], gb.x, gb.y));
      }
    }
    p += hop;
  }
}

// Persistent: the channels' dgamma and dbeta sums stay in registers.  One point per
// lane: with two the values of 20 channels cost half the warps (42 us against 28 in
// the case above).
template <typename T, int CM, int CLO>
__global__ void __launch_bounds__(OT) k_ln_bwd_odd(const __grid_constant__ OddArgs a) {
  __shared__ float2 coef[CM];
  __shared__ float red[OT / 32][2 * CM];
  cudaTriggerProgrammaticLaunchCompletion();   // the sum of the partial rows is set up meanwhile
  coefs<T>(a, coef);
  const int C = a.C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float dg[CM], db[CM];
#pragma unroll
  for (int c = 0; c < CM; ++c) dg[c] = db[c] = 0.f;
  for (unsigned tile = blockIdx.x * (OT / 32) + warp; tile < a.tiles;
       tile += gridDim.x * (OT / 32)) {
    const Spot<1> sp(a, tile);
    const float mu = a.mean_in[sp.point], r = a.rstd_in[sp.point];
    float xh[CM], g[CM], c1[2] = {0.f, 0.f}, c2[2] = {0.f, 0.f};
    const T *px = static_cast<const T *>(a.x) + sp.base;
    const T *py = static_cast<const T *>(a.dy) + sp.base;
#pragma unroll
    for (int c = 0; c < CM; ++c) {   // every load on its way before the first is used
      if (c < CLO || c < C) {
        xh[c] = to_f<T>(*px);
        g[c] = to_f<T>(*py);
      }
      px += a.inner;
      py += a.inner;
    }
#pragma unroll
    for (int c = 0; c < CM; ++c) {
      if (c < CLO || c < C) {
        const float d = sp.in[0] ? g[c] : 0.f;
        xh[c] = sp.in[0] ? (xh[c] - mu) * r : 0.f;
        dg[c] = fmaf(d, xh[c], dg[c]);
        db[c] += d;
        g[c] = d * coef[c].x;
        c1[c & 1] += g[c];
        c2[c & 1] = fmaf(g[c], xh[c], c2[c & 1]);
      }
    }
    const float k1 = (c1[0] + c1[1]) * a.inv_c, k2 = (c2[0] + c2[1]) * a.inv_c;
    T *po = static_cast<T *>(a.out) + sp.base;
    const long long hop = again(a.inner);
#pragma unroll
    for (int c = 0; c < CM; ++c) {
      if (c < CLO || c < C)
        if (sp.in[0]) *po = from_f<T>(r * ((g[c] - k1) - xh[c] * k2));
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
    if (lane == 0) {
      red[warp][2 * c] = dg[c];
      red[warp][2 * c + 1] = db[c];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C; i += OT) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < OT / 32; ++w) s += red[w][i];
    a.partial[(long long)blockIdx.x * 2 * C + i] = s;
  }
}

template <typename T, int CM, int CLO, int PPL>
cudaError_t fwd_t(const Launch &L, const NormShape &s, OddArgs a) {
  a.segs = (unsigned)((s.inner + 32 * PPL - 1) / (32 * PPL));
  a.tiles = (unsigned)s.outer * a.segs;
  const unsigned grid = (a.tiles + OT / 32 - 1) / (OT / 32);
  k_ln_fwd_odd<T, CM, CLO, PPL><<<grid, OT, 0, L.stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int CM, int CLO>
cudaError_t bwd_t(const Launch &L, const NormShape &s, OddArgs a, int *nparts) {
  a.segs = (unsigned)((s.inner + 31) / 32);
  a.tiles = (unsigned)s.outer * a.segs;
  unsigned grid = (a.tiles + OT / 32 - 1) / (OT / 32);
  const unsigned cap = 4 * L.num_sms < kLnParts ? 4 * L.num_sms : kLnParts;
  if (grid > cap) grid = cap;
  *nparts = (int)grid;
  k_ln_bwd_odd<T, CM, CLO><<<grid, OT, 0, L.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Rows that fill most of their tiles, tile numbers of 32 bits.  Against the element
// kernels, us, rows of 48323 points: forward with C = 48 float32 11.2 and 13.1, with
// C = 64 29.5 and 25.4; backward with C = 32 24.4 and 31.8, with C = 48 the values of
// a point no longer fit the registers (59.8 and 28.2); float16 with C = 16 17.3 and
// 23.6, with C = 8, where a lane has few loads on their way, 27.9 and 23.2 (float32
// 23.5 and 26.1).
bool ln_odd_supported(const NormShape &s, int dtype, bool bwd) {
  if (s.inner % (bwd && dtype != DT_F32 ? 8 : 4) == 0) return false;
  const long long segs = (s.inner + 31) / 32;
  if (bwd && dtype != DT_F32 && s.C <= 8) return false;
  return s.C <= (bwd ? 32 : 48) && s.inner >= 256 && segs <= 0x7fffffffLL &&
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
      else err = bwd_t<T, 32, 25>(L, s, a, nparts);
    } else {
      if (s.C <= 8) err = fwd_t<T, 8, 1, 4>(L, s, a);
      else if (s.C <= 16) err = fwd_t<T, 16, 9, 4>(L, s, a);
      else if (s.C <= 20) err = fwd_t<T, 20, 17, 2>(L, s, a);
      else if (s.C <= 24) err = fwd_t<T, 24, 21, 2>(L, s, a);
      else if (s.C <= 32) err = fwd_t<T, 32, 25, 2>(L, s, a);
      else err = fwd_t<T, 48, 33, 2>(L, s, a);
    }
  });
  launch_end(L, dy ? "ln_bwd_odd" : "ln_fwd_odd");
  return err;
}

}  // namespace fno

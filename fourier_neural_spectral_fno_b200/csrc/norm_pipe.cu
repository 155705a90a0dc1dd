// Layer norm over the channels of grid activations as a TMA pipeline: at most 128
// channels, grids whose rows start on 16-byte boundaries.
//
// A team of warps is a pipeline of its own.  Its tile is every channel of SG
// columns of 32 W four-byte words of neighbouring points, [CM][SG 128 W bytes],
// which one tiled TMA copy brings into the team's ring of NS stages: the first
// warp's lane 0 issues, every lane waits on the stage's mbarrier.  Wide rows
// matter to HBM: 128 bytes of each of 64 channel rows at a time reached 80 % of
// the copy rate even without the arithmetic, whatever the ring.  A lane owns its
// words' points (one or two per word) and walks the channels in shared memory, so
// the channel sums need no exchange between lanes, and what is in flight is held
// by shared memory, not by registers.  The KW warps of a column take every KW-th
// pair of channels each and add up their sums through shared memory.  The results
// are written over the tile, which a TMA store brings out (no addresses or bounds
// per channel: those alone cost more instructions than the arithmetic); the stage
// is filled again one tile later, when the store has read it.  Arithmetic runs on
// packed pairs of channels (f32x2).
//
// CM is the channel count rounded up to a count for which a kernel exists: the
// box is CM rows high.  Rows beyond C are filled with zeros, which add nothing to
// the backward's sums (the forward's squares leave them out), and are not stored.
//
// Bound by HBM: 32 x 64 x 65536 bfloat16 backward 128.2 us with its parameters'
// sums, 99 % of the copy rate; 2 x 20 x 128^3 float32 169.3 us, 95 %.
#include <cuda.h>

#include "norm_common.cuh"
#include "tc_util.cuh"
#include "tma_util.cuh"

namespace fno {

namespace {

constexpr int kRingBytes = 224 * 1024;   // stages and exchange of a CTA

// The shape of a pipeline: element type, channels, arrays copied per tile, words
// per lane, warps per column, columns per tile, most teams
template <typename T_, int CM_, int CLO_, int ARRAYS_, int W_, int KW_, int SG_, int MT>
struct Shape {
  using T = T_;
  // CLO: the fewest channels this CM is used for
  static constexpr int CM = CM_, CLO = CLO_, ARRAYS = ARRAYS_, W = W_, KW = KW_, SG = SG_;
  static constexpr int E = 4 / sizeof(T);      // points per word
  static constexpr int N = W * E;              // points per lane
  static constexpr int P = 32 * N * SG;        // points per tile
  static constexpr int column = 128 * W;       // bytes of a channel in a column
  static constexpr int row = column * SG;      // bytes of a channel in the tile
  static constexpr int array = CM * row;
  static constexpr int stage = array * ARRAYS;
  // the team's exchange of sums: [SG][2][KW][2 N][32] floats
  static constexpr int xch_group = KW > 1 ? 2 * KW * 2 * N * 128 : 0;
  static constexpr int fit = kRingBytes / (3 * stage + SG * xch_group);
  static constexpr int NT = fit < MT ? fit : MT;               // teams per CTA, one CTA per SM
  static constexpr int deep = (kRingBytes / NT - SG * xch_group) / stage;
  static constexpr int NS = deep > 5 ? 5 : deep;               // stages per team
  static constexpr int warps = NT * SG * KW;
  static constexpr int threads = warps * 32;
  static constexpr int pairs = CM / 2 / KW;                    // channel pairs of a warp
  static constexpr int coef = NT * NS * stage;                 // float4 [CM / 2]
  static constexpr int xch = coef + CM / 2 * 16;
  static constexpr int bars = xch + NT * SG * xch_group;       // full, done [NT][NS]
  static constexpr int flags = bars + NT * NS * 16;            // [NT][SG][2][KW] waits that held
  static constexpr int total = flags + NT * SG * 2 * KW * 4;
  static_assert(CLO <= CM && CM % (2 * KW) == 0 && NS >= 3 && total <= 227 * 1024 && P <= 256 &&
                    (KW == 1 || NT * SG <= 15) && warps <= 32,
                "shape");
};

struct PipeArgs {
  const void *gamma, *beta;
  const float *mean_in, *rstd_in;
  float *mean_out, *rstd_out;
  void *out;
  float *partial;
  long long inner;
  unsigned tiles, segs;       // tiles in all, tiles along inner
  int C;
  float inv_c, eps;
  int *err;
};

// the lane's points of channels c, c + 1 as pairs over the channels
template <typename S> __device__ __forceinline__ void ld_pairs(const unsigned char *at, f32x2 *v) {
  using T = typename S::T;
#pragma unroll
  for (int w = 0; w < S::W; ++w) {
    const unsigned a = reinterpret_cast<const unsigned *>(at)[32 * w];
    const unsigned b = reinterpret_cast<const unsigned *>(at + S::row)[32 * w];
    if constexpr (sizeof(T) == 4) {
      v[w] = f2pack(__uint_as_float(a), __uint_as_float(b));
    } else {
      float a0, a1, b0, b1;
      word_get<T>(a, a0, a1);
      word_get<T>(b, b0, b1);
      v[2 * w] = f2pack(a0, b0);
      v[2 * w + 1] = f2pack(a1, b1);
    }
  }
}

// the results back in their places
template <typename S> __device__ __forceinline__ void st_pairs(unsigned char *at, const f32x2 *v) {
  using T = typename S::T;
#pragma unroll
  for (int w = 0; w < S::W; ++w) {
    float a[2], b[2];
    unsigned r0, r1;
    f2unpack(v[S::E * w], a[0], a[1]);
    if constexpr (sizeof(T) == 4) {
      r0 = __float_as_uint(a[0]);
      r1 = __float_as_uint(a[1]);
    } else {
      f2unpack(v[2 * w + 1], b[0], b[1]);
      r0 = word_set<T>(a[0], b[0]);
      r1 = word_set<T>(a[1], b[1]);
    }
    reinterpret_cast<unsigned *>(at)[32 * w] = r0;
    reinterpret_cast<unsigned *>(at + S::row)[32 * w] = r1;
  }
}

// In front of every sweep over the tile: without an ordering point the compiler
// keeps the values of the sweep before in registers (and spills them).
__device__ __forceinline__ void sweep() { __syncwarp(); }

// A place in a team's walk over its tiles: the walk's tile `it` is
// first + it stride, sample b, tile `seg` of its row of segs.
struct Cursor {
  unsigned it, b, seg;
};

template <typename S> struct Walk {
  unsigned char *ring;
  uint64_t *full, *done;
  float *xch;
  int *flags;
  const CUtensorMap *m0, *m1, *mo;
  int *err;
  unsigned count, segs, step_b, step_seg;   // tiles of the team; stride as (b, seg)
  int lane, team, col, part;                // column of the tile, share of its channels
  Cursor load;                              // the next tile to load (the leader's)
  unsigned issued;                          // tiles loaded so far (the leader's)

  __device__ __forceinline__ void advance(Cursor &c) const {
    ++c.it;
    c.b += step_b;
    c.seg += step_seg;
    if (c.seg >= segs) {
      c.seg -= segs;
      ++c.b;
    }
  }
  __device__ __forceinline__ bool leads() const { return part == 0 && col == 0 && lane == 0; }
  // the leader: the next tile into its stage
  __device__ __forceinline__ void issue() {
    if (load.it < count) {
      const unsigned s = load.it % S::NS;
      unsigned char *to = ring + s * S::stage;
      const int n = (int)(load.seg * S::P), b = (int)load.b;
      tma::arrive_expect_tx(&full[s], S::stage);
      tma::load_4d(to, m0, &full[s], n, 0, b, 0);
      if (S::ARRAYS == 2) tma::load_4d(to + S::array, m1, &full[s], n, 0, b, 0);
      issued = load.it + 1;
    }
    advance(load);
  }
  // every lane waits; false (in all lanes) once a wait has expired.  A column's
  // warps agree on it in their exchange.
  __device__ __forceinline__ bool wait(unsigned it) const {
    const bool ok = tc::mbar_wait(&full[it % S::NS], (it / S::NS) & 1, err);
    return __all_sync(0xffffffffu, ok);
  }
  // the results lie in `from`: once the whole team has written them the leader
  // stores them, and fills the stage of the tile before (its store has been read).
  // A team that does not come in time gets no further tiles, so its next waits
  // expire too.  (One path for every warp, and no result: a branch of their own
  // for the others, or leaving the loop from here, cost the backward 15 %.)
  __device__ __forceinline__ void store(const Cursor &c, const unsigned char *from) {
    constexpr bool kTeam = S::KW * S::SG > 1;
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (kTeam && lane == 0 && part + col != 0) tma::arrive(&done[c.it % S::NS]);
    if (leads()) {
      bool ok = true;
      if (kTeam) ok = tc::mbar_wait(&done[c.it % S::NS], (c.it / S::NS) & 1, err);
      if (ok) tma::store_4d(mo, from, (int)(c.seg * S::P), 0, (int)c.b, 0);
      tma::store_commit();
      tma::store_wait_read<1>();
      if (!ok) load.it = count;
      if (c.it > 0) issue();
    }
    __syncwarp();
  }
  // after an expired wait for `it`: what the leader has in flight lands first
  __device__ __forceinline__ void drain(unsigned it) const {
    if (!leads()) return;
    for (unsigned j = it; j < issued; ++j)
      tc::mbar_wait(&full[j % S::NS], (j / S::NS) & 1, nullptr);
  }
  // the leader's stores have left shared memory and are written
  __device__ __forceinline__ void finish() const {
    if (leads()) tma::store_wait_all();
  }
  // add the M values of the column's warps, lane by lane, in a fixed order; `turn`
  // alternates, so a slow warp still reads what a fast one does not overwrite.
  // Returns whether every warp of the column passed ok.
  template <int M> __device__ __forceinline__ bool exchange(float *v, unsigned turn, bool ok) const {
    if (S::KW == 1) return ok;
    float *buf = xch + (turn & 1) * (S::KW * 2 * S::N * 32);
    int *fl = flags + (turn & 1) * S::KW;
#pragma unroll
    for (int k = 0; k < M; ++k) buf[(part * M + k) * 32 + lane] = v[k];
    if (lane == 0) fl[part] = ok;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team * S::SG + col), "n"(32 * S::KW) : "memory");
#pragma unroll
    for (int k = 0; k < M; ++k) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < S::KW; ++p) s += buf[(p * M + k) * 32 + lane];
      v[k] = s;
    }
    bool all = true;
#pragma unroll
    for (int p = 0; p < S::KW; ++p) all = all && fl[p];
    return all;
  }
};

template <typename S>
__device__ __forceinline__ Walk<S> pipe_begin(unsigned char *smem, const PipeArgs &a,
                                              const CUtensorMap *m0, const CUtensorMap *m1,
                                              const CUtensorMap *mo, Cursor &at) {
  using T = typename S::T;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::bars);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::NT * S::NS; ++i) {
      tc::mbar_init(&bars[i], 1);
      tc::mbar_init(&bars[S::NT * S::NS + i], S::KW * S::SG > 1 ? S::KW * S::SG - 1 : 1);
    }
    tma::fence_barrier_init();
  }
  float *coef = reinterpret_cast<float *>(smem + S::coef);
  for (int c = threadIdx.x; c < S::CM; c += S::threads) {
    const bool in = c < a.C;
    const T *g = static_cast<const T *>(a.gamma), *h = static_cast<const T *>(a.beta);
    coef[(c >> 1) * 4 + (c & 1)] = in ? (g ? ldf(g + c) : 1.f) : 0.f;
    coef[(c >> 1) * 4 + 2 + (c & 1)] = in && h ? ldf(h + c) : 0.f;
  }
  __syncthreads();
  Walk<S> w;
  w.lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  w.part = warp % S::KW;
  w.col = warp / S::KW % S::SG;
  w.team = warp / (S::KW * S::SG);
  const int column = w.team * S::SG + w.col;
  w.ring = smem + w.team * S::NS * S::stage;
  w.full = bars + w.team * S::NS;
  w.done = bars + (S::NT + w.team) * S::NS;
  w.xch = reinterpret_cast<float *>(smem + S::xch + column * S::xch_group);
  w.flags = reinterpret_cast<int *>(smem + S::flags) + column * 2 * S::KW;
  w.m0 = m0;
  w.m1 = m1;
  w.mo = mo;
  w.err = a.err;
  const unsigned first = blockIdx.x * S::NT + w.team, stride = gridDim.x * S::NT;
  w.count = first < a.tiles ? (a.tiles - first + stride - 1) / stride : 0;
  w.segs = a.segs;
  w.step_b = stride / a.segs;
  w.step_seg = stride - w.step_b * a.segs;
  at.it = 0;
  at.b = first / a.segs;
  at.seg = first - at.b * a.segs;
  w.load = at;
  w.issued = 0;
  if (w.leads())
    for (int i = 0; i < S::NS; ++i) w.issue();
  return w;
}

// The converted values stay in registers from the first sweep on (a word is read
// and converted once).  The correction of the mean (norm.cu) serves the 16-bit types
// as well: a point of equal values has no step of its own to outweigh the rounding.  For
// them it comes from the residual (norm_common.cuh): 19 x 99 x 2704 float16 7.6 us, as a
// sum over the deviations 7.9; but for 33 to 64 channels, where many points are slower
// with it (32 x 64 x 65536 bfloat16 101.5 against 92.1 us, 32 x 48 x 65536 76.7 against
// 70.1; 40 x 41 x 20000 float16 29.1 against 30.2).
template <typename S>
__global__ void __launch_bounds__(S::threads, 1)
    k_ln_fwd_pipe(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                  const __grid_constant__ PipeArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int N = S::N;
  constexpr bool kResidual =
      S::CM <= ResidualChannels<typename S::T>::N && (S::CM < 48 || S::CM > 64);
  constexpr int M = kResidual ? N : 2 * N;   // sums of the second sweep
  Cursor at;
  Walk<S> w = pipe_begin<S>(smem, a, &mx, nullptr, &my, at);
  const float4 *coef = reinterpret_cast<const float4 *>(smem + S::coef) + w.part;
  const int C = a.C;
  unsigned turn = 0;
  for (; at.it < w.count; w.advance(at)) {
    bool ok = w.wait(at.it);
    if (S::KW == 1 && !ok) {
      w.drain(at.it);
      break;
    }
    unsigned char *tile = w.ring + (at.it % S::NS) * S::stage;
    unsigned char *st = tile + 2 * w.part * S::row + w.col * S::column + w.lane * 4;
    f32x2 v[S::pairs][N], s[N], e[N], m[N];
    float sum[M];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = f2splat(0.f);
#pragma unroll
    for (int i = 0; i < S::pairs; ++i) {
      ld_pairs<S>(st + 2 * S::KW * i * S::row, v[i]);
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] = f2add(s[k], v[i][k]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = pair_sum(s[k]);
    ok = w.template exchange<N>(sum, turn++, ok);
    if (S::KW > 1 && !ok) {
      w.drain(at.it);
      break;
    }
    float mean[N], res[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      mean[k] = sum[k] * a.inv_c;
      if (kResidual) res[k] = ln_residual(sum[k], mean[k], C, a.inv_c);
      m[k] = f2splat(-mean[k]);
      s[k] = e[k] = f2splat(0.f);
    }
#pragma unroll
    for (int i = 0; i < S::pairs; ++i) {
      const int c = 2 * (S::KW * i + w.part);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[i][k] = f2add(v[i][k], m[k]);
        if (2 * (S::KW * i + S::KW) > S::CLO) {   // rows of zeros beyond the channels
          float d0, d1;
          f2unpack(v[i][k], d0, d1);
          v[i][k] = f2pack(c < C ? d0 : 0.f, c + 1 < C ? d1 : 0.f);
        }
        if (!kResidual) e[k] = f2add(e[k], v[i][k]);
        s[k] = f2fma(v[i][k], v[i][k], s[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      sum[k] = pair_sum(s[k]);
      if (!kResidual) sum[N + k] = pair_sum(e[k]);
    }
    w.template exchange<M>(sum, turn++, true);
    const long long n = (long long)at.seg * S::P + (w.col * 32 * S::W + w.lane) * S::E;
    float r[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float ek = kResidual ? res[k] : sum[N + k] * a.inv_c;
      r[k] = ln_rstd(sum[k] * a.inv_c, ek, a.eps);
      m[k] = f2splat(r[k]);
      mean[k] += ek;
      e[k] = f2splat(-ek * r[k]);   // xh = (x - mean) r - e r
    }
    if (a.mean_out && w.part == 0) {
#pragma unroll
      for (int k = 0; k < S::W; ++k)
        if (n + 32 * S::E * k < a.inner) {   // the points of a word
          const long long p = at.b * a.inner + n + 32 * S::E * k;
          if constexpr (S::E == 2) {
            *reinterpret_cast<float2 *>(a.mean_out + p) = make_float2(mean[2 * k], mean[2 * k + 1]);
            *reinterpret_cast<float2 *>(a.rstd_out + p) = make_float2(r[2 * k], r[2 * k + 1]);
          } else {
            a.mean_out[p] = mean[k];
            a.rstd_out[p] = r[k];
          }
        }
    }
#pragma unroll
    for (int i = 0; i < S::pairs; ++i) {
      const float4 gb = coef[S::KW * i];
      const f32x2 ga = f2pack(gb.x, gb.y), be = f2pack(gb.z, gb.w);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[i][k] = f2fma(f2fma(v[i][k], m[k], e[k]), ga, be);
      }
      st_pairs<S>(st + 2 * S::KW * i * S::row, v[i]);
    }
    w.store(at, tile);
  }
  w.finish();
}

// Per point: first sweep c1 = sum g, c2 = sum g xh (g = dy gamma) and the
// channels' dgamma += dy xh, dbeta += dy in registers; second sweep
//   dx = rstd ((g - c1 / C) - xh c2 / C)
// (rstd^2 c2 / C, one product less, leaves float32's range long before dx does)
template <typename S>
__global__ void __launch_bounds__(S::threads, 1)
    k_ln_bwd_pipe(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mdy,
                  const __grid_constant__ CUtensorMap mdx, const __grid_constant__ PipeArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int N = S::N;
  cudaTriggerProgrammaticLaunchCompletion();   // the sum of the partial rows is set up meanwhile
  Cursor at;
  Walk<S> w = pipe_begin<S>(smem, a, &mx, &mdy, &mdx, at);
  const float4 *coef = reinterpret_cast<const float4 *>(smem + S::coef) + w.part;
  const int C = a.C;
  f32x2 dg[S::pairs], db[S::pairs];
#pragma unroll
  for (int i = 0; i < S::pairs; ++i) dg[i] = db[i] = f2splat(0.f);
  // a tile's statistics are fetched one tile ahead
  float mu[N], r[N];
  auto fetch = [&](const Cursor &c) {
    const long long n = (long long)c.seg * S::P + (w.col * 32 * S::W + w.lane) * S::E;
    const bool live = c.it < w.count;
#pragma unroll
    for (int k = 0; k < S::W; ++k) {
      const bool in = live && n + 32 * S::E * k < a.inner;
      const long long p = c.b * a.inner + n + 32 * S::E * k;
      if (S::E == 2) {
        const float2 z = make_float2(0.f, 0.f);
        const float2 u = in ? __ldg(reinterpret_cast<const float2 *>(a.mean_in + p)) : z;
        const float2 q = in ? __ldg(reinterpret_cast<const float2 *>(a.rstd_in + p)) : z;
        mu[2 * k] = u.x;
        mu[2 * k + 1] = u.y;
        r[2 * k] = q.x;
        r[2 * k + 1] = q.y;
      } else {
        mu[k] = in ? __ldg(a.mean_in + p) : 0.f;
        r[k] = in ? __ldg(a.rstd_in + p) : 0.f;
      }
    }
  };
  fetch(at);
  while (at.it < w.count) {
    bool ok = w.wait(at.it);
    if (S::KW == 1 && !ok) {
      w.drain(at.it);
      break;
    }
    unsigned char *tile = w.ring + (at.it % S::NS) * S::stage;
    const unsigned char *sx =
        tile + 2 * w.part * S::row + w.col * S::column + w.lane * 4;
    unsigned char *sy = tile + S::array + 2 * w.part * S::row + w.col * S::column + w.lane * 4;
    f32x2 m[N], rr[N], c1[N], c2[N], x[N], y[N];
    float sums[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      m[k] = f2splat(-mu[k]);
      rr[k] = f2splat(r[k]);
      c1[k] = c2[k] = f2splat(0.f);
    }
    Cursor now = at;
    w.advance(at);
    fetch(at);
#pragma unroll
    for (int i = 0; i < S::pairs; ++i) {
      if (i == 0) sweep();
      ld_pairs<S>(sx + 2 * S::KW * i * S::row, x);
      ld_pairs<S>(sy + 2 * S::KW * i * S::row, y);
      const float4 gb = coef[S::KW * i];
      const f32x2 ga = f2pack(gb.x, gb.y);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const f32x2 xh = f2mul(f2add(x[k], m[k]), rr[k]), g = f2mul(y[k], ga);
        c1[k] = f2add(c1[k], g);
        c2[k] = f2fma(g, xh, c2[k]);
        dg[i] = f2fma(y[k], xh, dg[i]);
        db[i] = f2add(db[i], y[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      sums[2 * k] = pair_sum(c1[k]);
      sums[2 * k + 1] = pair_sum(c2[k]);
    }
    ok = w.template exchange<2 * N>(sums, now.it, ok);
    if (S::KW > 1 && !ok) {
      w.drain(now.it);
      break;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      c1[k] = f2splat(-(sums[2 * k] * a.inv_c));
      c2[k] = f2splat(-(sums[2 * k + 1] * a.inv_c));
    }
#pragma unroll
    for (int i = 0; i < S::pairs; ++i) {
      if (i == 0) sweep();
      ld_pairs<S>(sx + 2 * S::KW * i * S::row, x);
      ld_pairs<S>(sy + 2 * S::KW * i * S::row, y);
      const float4 gb = coef[S::KW * i];
      const f32x2 ga = f2pack(gb.x, gb.y);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const f32x2 xh = f2mul(f2add(x[k], m[k]), rr[k]);
        x[k] = f2mul(f2fma(xh, c2[k], f2fma(y[k], ga, c1[k])), rr[k]);
      }
      st_pairs<S>(sy + 2 * S::KW * i * S::row, x);
    }
    w.store(now, tile + S::array);
  }
  w.finish();
  if (!a.partial) return;
  __syncthreads();   // no copy is under way and every stage has been read
  // The lanes' sums through the team's ring, column after column: value
  // v = 2 c + {0 dgamma, 1 dbeta} in row v of 32 lanes, the row's sum beside them;
  // then the columns' sums, in order.
  constexpr int kCol = 2 * S::CM * 33;   // floats
  static_assert(S::SG * kCol * 4 <= S::NS * S::stage, "the sums fit the ring");
  float *fl = reinterpret_cast<float *>(w.ring) + w.col * kCol;
#pragma unroll
  for (int i = 0; i < S::pairs; ++i) {
    float g0, g1, h0, h1;
    f2unpack(dg[i], g0, g1);
    f2unpack(db[i], h0, h1);
    float *at4 = fl + 4 * (S::KW * i + w.part) * 33 + w.lane;
    at4[0] = g0;
    at4[33] = h0;
    at4[66] = g1;
    at4[99] = h1;
  }
  __syncthreads();
  for (int v = w.part * 32 + w.lane; v < 2 * S::CM; v += 32 * S::KW) {
    float s = 0.f;
#pragma unroll
    for (int l = 0; l < 32; ++l) s += fl[v * 33 + l];
    fl[v * 33 + 32] = s;
  }
  __syncthreads();
  for (int v = threadIdx.x; v < 2 * C; v += S::threads) {
    float s = 0.f;
    for (int k = 0; k < S::NT * S::SG; ++k)
      s += reinterpret_cast<const float *>(smem + k / S::SG * S::NS *
                                                      S::stage)[k % S::SG * kCol + v * 33 + 32];
    a.partial[(long long)blockIdx.x * 2 * C + v] = s;
  }
}

template <typename T> CUtensorMapDataType map_type();
template <> CUtensorMapDataType map_type<float>() { return CU_TENSOR_MAP_DATA_TYPE_FLOAT32; }
template <> CUtensorMapDataType map_type<__half>() { return CU_TENSOR_MAP_DATA_TYPE_FLOAT16; }
template <> CUtensorMapDataType map_type<__nv_bfloat16>() {
  return CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <typename S> bool encode(CUtensorMap *map, const NormShape &s, const void *base) {
  const uint64_t row = (uint64_t)s.inner * sizeof(typename S::T);
  const uint64_t dims[4] = {(uint64_t)s.inner, (uint64_t)s.C, (uint64_t)s.outer, 1};
  const uint64_t strides[3] = {row, row * s.C, row * s.C * s.outer};
  const uint32_t box[4] = {S::P, S::CM, 1, 1};
  return encode_tmap_4d(map, map_type<typename S::T>(), base, dims, strides, box);
}

template <typename S> int pipe_args(const Launch &L, const NormShape &s, PipeArgs *a) {
  a->inner = s.inner;
  a->C = s.C;
  a->inv_c = 1.0f / (float)s.C;
  a->eps = s.eps;
  a->err = L.err;
  a->segs = (unsigned)((s.inner + S::P - 1) / S::P);
  a->tiles = (unsigned)(s.outer * a->segs);
  const unsigned ctas = (a->tiles + S::NT - 1) / S::NT;
  const unsigned cap = L.num_sms < kLnParts ? L.num_sms : kLnParts;
  return (int)(ctas < cap ? ctas : cap);
}

template <typename S>
cudaError_t fwd_t(const Launch &L, const NormShape &s, const void *x, PipeArgs a) {
  CUtensorMap mx, my;
  if (!encode<S>(&mx, s, x) || !encode<S>(&my, s, a.out)) return cudaErrorInvalidValue;
  const int grid = pipe_args<S>(L, s, &a);
  const auto kern = k_ln_fwd_pipe<S>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  if (e != cudaSuccess) return e;
  kern<<<grid, S::threads, S::total, L.stream>>>(mx, my, a);
  return cudaGetLastError();
}

template <typename S>
cudaError_t bwd_t(const Launch &L, const NormShape &s, const void *x, const void *dy, PipeArgs a,
                  int *nparts) {
  CUtensorMap mx, my, md;
  if (!encode<S>(&mx, s, x) || !encode<S>(&my, s, dy) || !encode<S>(&md, s, a.out))
    return cudaErrorInvalidValue;
  const int grid = pipe_args<S>(L, s, &a);
  *nparts = grid;
  const auto kern = k_ln_bwd_pipe<S>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  if (e != cudaSuccess) return e;
  kern<<<grid, S::threads, S::total, L.stream>>>(mx, my, md, a);
  return cudaGetLastError();
}

// Per channel count: CM, words per lane, warps per column, columns per tile, most
// teams; chosen by a sweep over these at 64 M (32-bit) and 128 M bytes (16-bit)
// per array.  Rows of 512 bytes and one or two columns' worth of warps per team
// were best nearly everywhere, the neighbours within 5 %; above 64 channels tiles
// that leave room for two teams (8 x 100 x 65536 bfloat16: forward 39.1 us with two
// teams of two columns, 42.7 with one of four; 16 warps a column 95 us backward,
// four 65).
struct Cfg {
  int cm, w, kw, sg, mt;
};
constexpr Cfg kFwd[] = {{8, 2, 1, 2, 12}, {16, 2, 1, 2, 8}, {20, 2, 1, 2, 6}, {24, 2, 1, 2, 6},
                        {32, 1, 1, 4, 4}, {48, 1, 4, 4, 2}, {64, 1, 4, 4, 2}, {96, 1, 4, 2, 2},
                        {128, 1, 4, 2, 2}};
constexpr Cfg kBwd[] = {{8, 2, 1, 2, 8}, {16, 2, 2, 2, 4}, {20, 2, 2, 2, 3}, {24, 2, 2, 2, 3},
                        {32, 1, 2, 2, 4}, {48, 1, 4, 2, 3}, {64, 1, 4, 2, 2}, {96, 1, 4, 1, 2},
                        {128, 1, 4, 1, 2}};
template <typename T, int I, int ARRAYS> struct ShapeOf {
  static constexpr Cfg c = ARRAYS == 1 ? kFwd[I] : kBwd[I];
  static constexpr int lo = I ? kFwd[I ? I - 1 : 0].cm + 1 : 1;
  using type = Shape<T, c.cm, lo, ARRAYS, c.w, c.kw, c.sg, c.mt>;
};

#define LN_PIPE_CASES(CALL)          \
  do {                               \
    if (s.C <= 8) CALL(0);           \
    else if (s.C <= 16) CALL(1);     \
    else if (s.C <= 20) CALL(2);     \
    else if (s.C <= 24) CALL(3);     \
    else if (s.C <= 32) CALL(4);     \
    else if (s.C <= 48) CALL(5);     \
    else if (s.C <= 64) CALL(6);     \
    else if (s.C <= 96) CALL(7);     \
    else CALL(8);                    \
  } while (0)

}  // namespace

// Rows on 16-byte boundaries (the maps' strides), at most 128 channels, tile
// numbers of 31 bits, strides the maps can hold; rows that fill most of their
// tiles of up to 256 points; and enough work that the pipelines' start does not
// show.  Against the register kernels (norm_grid.cu), us, with up to 64 channels:
// backward float32 20 x 4096 at batch 8 / 16 / 32: 5.7 / 7.3 / 9.7 against
// 5.0 / 6.2 / 9.1, 64 x 4096 at 2 / 4: 6.1 / 6.6 against 5.1 / 6.4; bfloat16
// 20 x 4096 at 8 / 16: 6.1 / 6.3 against 5.5 / 7.5: from a million values on (20
// channels of float32 gain later).
// Forward bfloat16 20 x 4096 at 32 / 64: 5.4 / 7.4 against 4.5 / 7.5: from four
// million; float32 never (16 x 32 x 65536: 51 against 44.5, 96 % of the copy rate).
// With more channels, where the register kernels split a point's channels over a
// CTA's warps, from a million values on in every direction and type: at 128 x 4096,
// batch 4, and 128 x 65536, batch 8, forward bfloat16 5.5 and 49.9 against 7.2 and
// 74.7, float32 5.1 and 97.4 against 8.6 and 113; backward bfloat16 7.3 and 71.4
// against 7.9 and 139, float32 8.5 and 130 against 10.1 and 208.
bool ln_pipe_supported(const NormShape &s, int dtype, bool bwd) {
  if (!bwd && dtype == DT_F32 && s.C <= 64) return false;
  const long long es = dtype == DT_F32 ? 4 : 2, n = s.outer * s.C * s.inner;
  if (s.C > 128 || s.inner * es % 16 != 0 || (s.inner < 512 && s.inner != 256) ||
      n < (bwd || s.C > 64 ? 1 << 20 : 1 << 22))
    return false;
  const long long segs = (s.inner + 31) / 32;
  return s.inner <= 0x7fffffffLL && s.outer <= 0x7fffffffLL / segs && n * es < (1LL << 40);
}

cudaError_t launch_ln_pipe_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd) {
  PipeArgs a{};
  a.gamma = gamma;
  a.beta = beta;
  a.mean_out = mean;
  a.rstd_out = rstd;
  a.out = y;
  cudaError_t err = cudaSuccess;
#define LN_FWD(I) err = fwd_t<typename ShapeOf<T, I, 1>::type>(L, s, x, a)
  launch_begin(L);
  if (dtype == DT_F16) {
    using T = __half;
    LN_PIPE_CASES(LN_FWD);
  } else if (dtype == DT_BF16) {
    using T = __nv_bfloat16;
    LN_PIPE_CASES(LN_FWD);
  } else {
    using T = float;
    if (s.C <= 96) LN_FWD(7);
    else LN_FWD(8);
  }
  launch_end(L, "ln_fwd_pipe");
#undef LN_FWD
  return err;
}

cudaError_t launch_ln_pipe_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts) {
  PipeArgs a{};
  a.gamma = gamma;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.out = dx;
  a.partial = partial;
  cudaError_t err = cudaSuccess;
#define LN_BWD(I) err = bwd_t<typename ShapeOf<T, I, 2>::type>(L, s, x, dy, a, nparts)
  launch_begin(L);
  FNO_DISPATCH_T(dtype, LN_PIPE_CASES(LN_BWD));
  launch_end(L, "ln_bwd_pipe");
#undef LN_BWD
  return err;
}

}  // namespace fno

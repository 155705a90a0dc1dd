// Layer norm of rows [outer][C] (inner = 1), one pass: every value is read once,
// kept in registers and written once.
//
// A row belongs to a group of TPR neighbouring threads (8 to 512, a power of two),
// thread t taking the 16-byte pieces t, t + TPR, ... of the row.  Where C is no
// multiple of a piece, rows start inside one: a group then takes rows that are a
// multiple of V apart (V values to a piece), which all start `shift` values into
// a piece, so its threads keep their columns from row to row; pieces that reach
// over a row's ends are read and written value by value.  Sums go by shuffles
// inside a warp and through shared memory between a row's warps (a named barrier
// per group).  Groups walk over the rows: gamma and beta, and the backward's sums
// of dgamma and dbeta, stay in registers.  20011 x 768 bfloat16 forward 18.1 us (53 %
// of the copy rate), 262144 x 64 float32 24.7 (85 %); 4099 x 1001 float32 backward
// 16.1: what is in flight, held by 16 warps an SM, bounds the rows, and HBM the rest.
#include "norm_common.cuh"

namespace fno {

namespace {

constexpr int kRowThreads = 256;
constexpr int kPackedAbove = 32 * 24;   // 16-bit rows of whole pieces with more: packed

// a group's place in its CTA and the sums over its threads
struct Group {
  float *red;   // [2][16][16 values]: the warps' parts; alternating, so that one
                // barrier serves a sum
  int tpr, t, r, turn;
  template <int M> __device__ __forceinline__ void sum(float *v) {
    const int half = (tpr < 32 ? tpr : 32) >> 1;
    for (int o = half; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < M; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr <= 32) return;
    float *buf = red + (turn & 1) * 256;
    ++turn;
    const int warp = threadIdx.x >> 5, first = warp & ~(tpr / 32 - 1);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < M; ++k) buf[warp * 16 + k] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + r), "r"(tpr) : "memory");
#pragma unroll
    for (int k = 0; k < M; ++k) v[k] = 0.f;
    for (int w = 0; w < tpr / 32; ++w)
#pragma unroll
      for (int k = 0; k < M; ++k) v[k] += buf[(first + w) * 16 + k];
  }
};

template <typename T> struct Rows {
  static constexpr int V = VecOf<T>::N;
  using P = Pack<T, V>;
};

// piece j of a row: columns lo .. lo + V - 1, lo = (j tpr + t) V - shift
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_piece(typename Rows<T>::P &p, const T *row, int lo, int C,
                                           bool in) {
  constexpr int V = Rows<T>::V;
  p.zero();
  if (!in) return;
  if (lo >= 0 && lo + V <= C) {
    p = *reinterpret_cast<const typename Rows<T>::P *>(row + lo);
  } else if (SHIFT) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      f[i] = (unsigned)(lo + i) < (unsigned)C ? to_f<T>(row[lo + i]) : 0.f;
    p.set(f);   // exact: the values are of the type
  }
}

template <typename T, bool SHIFT>
__device__ __forceinline__ void store_piece(const f32x2 *f, T *row, int lo, int C) {
  constexpr int V = Rows<T>::V;
  if (lo >= 0 && lo + V <= C) {
    typename Rows<T>::P p;
    p.set2(f);
    *reinterpret_cast<typename Rows<T>::P *>(row + lo) = p;
  } else if (SHIFT) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      float a, b;
      f2unpack(f[i / 2], a, b);
      if ((unsigned)(lo + i) < (unsigned)C) row[lo + i] = from_f<T>(a);
      if ((unsigned)(lo + i + 1) < (unsigned)C) row[lo + i + 1] = from_f<T>(b);
    }
  }
}

// per-channel values of a piece (NULL: `none`)
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_coef(f32x2 *p, const T *w, int lo, int C, float none) {
  constexpr int V = Rows<T>::V;
  if (w && lo >= 0 && lo + V <= C && (!SHIFT || lo % V == 0)) {
    typename Rows<T>::P q = *reinterpret_cast<const typename Rows<T>::P *>(w + lo);
    q.get2(p);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float a = w && (unsigned)(lo + i) < (unsigned)C ? to_f<T>(w[lo + i]) : none;
    const float b = w && (unsigned)(lo + i + 1) < (unsigned)C ? to_f<T>(w[lo + i + 1]) : none;
    p[i / 2] = f2pack(a, b);
  }
}

// a pair's halves where their columns lie in the row, else 0
__device__ __forceinline__ f32x2 masked(f32x2 v, int c, int C) {
  float a, b;
  f2unpack(v, a, b);
  return f2pack((unsigned)c < (unsigned)C ? a : 0.f, (unsigned)(c + 1) < (unsigned)C ? b : 0.f);
}

// The converted values stay in registers (each is converted once); the next row's
// pieces are on their way meanwhile.  The correction of the mean (norm.cu) comes from a
// residual for 16-bit types where no row of the kernel has more channels than that is
// exact for; as a sum over the deviations, as float32 needs it, it cost 2 to 5 % (20011
// x 768 18.6 us against 18.0, 262144 x 64 20.2 against 19.5).
template <typename T, int NV, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS)
    k_ln_fwd_rows(const T *x, const T *__restrict__ gamma, const T *__restrict__ beta, T *y,
                  float *__restrict__ mean, float *__restrict__ rstd, long long rows, int C,
                  int tpr, float inv_c, float eps) {
  constexpr int V = Rows<T>::V, H = V / 2;
  constexpr int kMost = V == 8 && !SHIFT ? kPackedAbove : 24 * THREADS;   // channels
  constexpr bool kResidual = kMost <= ResidualChannels<T>::N;
  __shared__ float red[512];
  Group gr{red, tpr, (int)(threadIdx.x & (tpr - 1)), (int)(threadIdx.x / tpr), 0};
  const int R = blockDim.x / tpr;
  const long long G = (long long)gridDim.x * R, first = (long long)blockIdx.x * R + gr.r;
  const int shift = SHIFT ? (int)(first * C % V) : 0, lo0 = gr.t * V - shift, hop = tpr * V;
  // a warp's groups make the same number of rounds: as many as its first one
  const long long lag = tpr < 32 ? gr.r % (32 / tpr) : 0;
  typename Rows<T>::P nx[NV];
  f32x2 ga[NV][H], be[NV][H], v[NV][H];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_piece<T, SHIFT>(nx[j], x + first * C, lo0 + j * hop, C, first < rows);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_coef<T, SHIFT>(ga[j], gamma, lo0 + j * hop, C, 1.f);
    load_coef<T, SHIFT>(be[j], beta, lo0 + j * hop, C, 0.f);
  }
  for (long long row = first; row - lag < rows; row += G) {
    f32x2 s[2], e[2];   // two chains of each sum
    s[0] = s[1] = e[0] = e[1] = f2splat(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      nx[j].get2(v[j]);
#pragma unroll
      for (int i = 0; i < H; ++i) s[i & 1] = f2add(s[i & 1], v[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      load_piece<T, SHIFT>(nx[j], x + (row + G) * C, lo0 + j * hop, C, row + G < rows);
    float sum = pair_sum(f2add(s[0], s[1]));
    gr.sum<1>(&sum);
    const float m0 = sum * inv_c;
    const f32x2 m = f2splat(-m0);
    s[0] = s[1] = f2splat(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int lo = lo0 + j * hop;
      const bool whole = lo >= 0 && lo + V <= C;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        v[j][i] = f2add(v[j][i], m);
        if (!whole) v[j][i] = masked(v[j][i], lo + 2 * i, C);
        if (!kResidual) e[i & 1] = f2add(e[i & 1], v[j][i]);
        s[i & 1] = f2fma(v[j][i], v[j][i], s[i & 1]);
      }
    }
    float q[2] = {pair_sum(f2add(s[0], s[1])), kResidual ? 0.f : pair_sum(f2add(e[0], e[1]))};
    gr.sum<kResidual ? 1 : 2>(q);
    const float ek = kResidual ? ln_residual(sum, m0, C, inv_c) : q[1] * inv_c;
    const float r = ln_rstd(q[0] * inv_c, ek, eps);
    if (row < rows) {
      if (mean && gr.t == 0) {
        mean[row] = m0 + ek;
        rstd[row] = r;
      }
      const f32x2 rr = f2splat(r), er = f2splat(-ek * r);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < H; ++i)
          v[j][i] = f2fma(f2fma(v[j][i], rr, er), ga[j][i], be[j][i]);
        store_piece<T, SHIFT>(v[j], y + row * C, lo0 + j * hop, C);
      }
    }
  }
}

// The forward of long rows (use_packed): one row per group and many warps, the row
// in its packed form (converted in each sweep), gamma and beta read where they are
// used (they stay in L1).
template <typename T, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, (NV <= 4 ? 1280 : 1024) / THREADS)
    k_ln_fwd_rows_packed(const T *x, const T *__restrict__ gamma, const T *__restrict__ beta,
                         T *y, float *__restrict__ mean, float *__restrict__ rstd, long long rows,
                         int C, int tpr, float inv_c, float eps) {
  constexpr int V = Rows<T>::V, H = V / 2;
  constexpr bool kResidual = 4 * V * THREADS <= ResidualChannels<T>::N;
  __shared__ float red[512];
  Group gr{red, tpr, (int)(threadIdx.x & (tpr - 1)), (int)(threadIdx.x / tpr), 0};
  const long long row = (long long)blockIdx.x * (THREADS / tpr) + gr.r;
  const int lo0 = gr.t * V, hop = tpr * V;
  typename Rows<T>::P p[NV];
  f32x2 v[H], s[2], e[2];   // two chains of each sum
#pragma unroll
  for (int j = 0; j < NV; ++j) load_piece<T, false>(p[j], x + row * C, lo0 + j * hop, C, row < rows);
  s[0] = s[1] = e[0] = e[1] = f2splat(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    p[j].get2(v);
#pragma unroll
    for (int i = 0; i < H; ++i) s[i & 1] = f2add(s[i & 1], v[i]);
    p[j].keep();
  }
  float sum = pair_sum(f2add(s[0], s[1]));
  gr.sum<1>(&sum);
  const float m0 = sum * inv_c;
  const f32x2 m = f2splat(-m0);
  s[0] = s[1] = f2splat(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (lo0 + j * hop < C) {
      p[j].get2(v);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        v[i] = f2add(v[i], m);
        if (!kResidual) e[i & 1] = f2add(e[i & 1], v[i]);
        s[i & 1] = f2fma(v[i], v[i], s[i & 1]);
      }
      p[j].keep();
    }
  }
  float q[2] = {pair_sum(f2add(s[0], s[1])), kResidual ? 0.f : pair_sum(f2add(e[0], e[1]))};
  gr.sum<kResidual ? 1 : 2>(q);
  const float ek = kResidual ? ln_residual(sum, m0, C, inv_c) : q[1] * inv_c;
  const float r = ln_rstd(q[0] * inv_c, ek, eps);
  if (row >= rows) return;
  if (mean && gr.t == 0) {
    mean[row] = m0 + ek;
    rstd[row] = r;
  }
  const f32x2 rr = f2splat(r), er = f2splat(-ek * r);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int lo = lo0 + j * hop;
    if (lo < C) {
      f32x2 ga[H], be[H];
      load_coef<T, false>(ga, gamma, lo, C, 1.f);
      load_coef<T, false>(be, beta, lo, C, 0.f);
      p[j].get2(v);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        v[i] = f2fma(f2add(v[i], m), rr, er);
        v[i] = f2fma(v[i], ga[i], be[i]);
      }
      store_piece<T, false>(v, y + row * C, lo, C);
    }
  }
}

template <typename T, int NV, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
    k_ln_bwd_rows(const T *__restrict__ x, const T *__restrict__ gamma,
                  const float *__restrict__ mean, const float *__restrict__ rstd, const T *dy,
                  T *dx, float *__restrict__ partial, long long rows, int C, int tpr,
                  float inv_c) {
  constexpr int V = Rows<T>::V, H = V / 2;
  extern __shared__ float acc[];   // [groups][C][2], where a CTA has several
  __shared__ float red[512];
  cudaTriggerProgrammaticLaunchCompletion();   // the sum of the partial rows is set up meanwhile
  Group gr{red, tpr, (int)(threadIdx.x & (tpr - 1)), (int)(threadIdx.x / tpr), 0};
  const int R = blockDim.x / tpr;
  const long long G = (long long)gridDim.x * R, first = (long long)blockIdx.x * R + gr.r;
  const int shift = SHIFT ? (int)(first * C % V) : 0, lo0 = gr.t * V - shift, hop = tpr * V;
  const long long lag = tpr < 32 ? gr.r % (32 / tpr) : 0;
  typename Rows<T>::P na[NV], nb[NV];
  f32x2 ga[NV][H], dg[NV][H], db[NV][H], xh[NV][H], g[NV][H];
  float nmu = 0.f, nr = 0.f;
  auto fetch = [&](long long row) {
    const bool in = row < rows;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_piece<T, SHIFT>(na[j], x + row * C, lo0 + j * hop, C, in);
      load_piece<T, SHIFT>(nb[j], dy + row * C, lo0 + j * hop, C, in);
    }
    nmu = in ? mean[row] : 0.f;
    nr = in ? rstd[row] : 0.f;
  };
  // The next row on its way where a thread has fewer than 16 values (262144 x 64:
  // float32 37.8 us, without it 41.9; bfloat16 28.1 and 34.3).  With 16, float32's
  // registers give more as a second CTA's (4099 x 1001: 16.1 us, with the next row
  // 19.0); packed 16-bit rows could hold it (16384 x 1024 bfloat16 30.5 us, with the
  // next row 25.9), which this rule leaves out.
  constexpr bool kAhead = NV * V < 16;
  if (kAhead) fetch(first);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_coef<T, SHIFT>(ga[j], gamma, lo0 + j * hop, C, 1.f);
#pragma unroll
    for (int i = 0; i < H; ++i) dg[j][i] = db[j][i] = f2splat(0.f);
  }
  for (long long row = first; row - lag < rows; row += G) {
    if (!kAhead) fetch(row);
    const float r = nr;
    const f32x2 m = f2splat(-nmu), rr = f2splat(r);
    f32x2 c1[2], c2[2];   // two chains of each sum
    c1[0] = c1[1] = c2[0] = c2[1] = f2splat(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {   // dy is 0 where there is nothing
      na[j].get2(xh[j]);
      nb[j].get2(g[j]);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        xh[j][i] = f2mul(f2add(xh[j][i], m), rr);
        dg[j][i] = f2fma(g[j][i], xh[j][i], dg[j][i]);
        db[j][i] = f2add(db[j][i], g[j][i]);
        g[j][i] = f2mul(g[j][i], ga[j][i]);
        c1[i & 1] = f2add(c1[i & 1], g[j][i]);
        c2[i & 1] = f2fma(g[j][i], xh[j][i], c2[i & 1]);
      }
    }
    if (kAhead) fetch(row + G);
    float c12[2] = {pair_sum(f2add(c1[0], c1[1])), pair_sum(f2add(c2[0], c2[1]))};
    gr.sum<2>(c12);
    if (row < rows) {
      const f32x2 k1 = f2splat(-(c12[0] * inv_c)), k2 = f2splat(-(c12[1] * inv_c));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < H; ++i)
          g[j][i] = f2mul(f2fma(xh[j][i], k2, f2add(g[j][i], k1)), rr);
        store_piece<T, SHIFT>(g[j], dx + row * C, lo0 + j * hop, C);
      }
    }
  }
  if (!partial) return;
  // the groups' sums side by side in shared memory, then added in order
  float *out = partial + (long long)blockIdx.x * 2 * C, *to = R > 1 ? acc + gr.r * 2 * C : out;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int c = lo0 + j * hop + 2 * i;
      float g0, g1, h0, h1;
      f2unpack(dg[j][i], g0, g1);
      f2unpack(db[j][i], h0, h1);
      if ((unsigned)c < (unsigned)C) *reinterpret_cast<float2 *>(to + 2 * c) = make_float2(g0, h0);
      if ((unsigned)(c + 1) < (unsigned)C)
        *reinterpret_cast<float2 *>(to + 2 * c + 2) = make_float2(g1, h1);
    }
  if (R == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C; i += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < R; ++k) s += acc[k * 2 * C + i];
    out[i] = s;
  }
}

// Threads per row: as few (8 at least, 512 at most) as hold the row with at most
// `most` pieces each; 0: it does not fit.
int pick_tpr(int pieces, int most) {
  for (int tpr = 8; tpr <= 2 * kRowThreads; tpr *= 2)
    if (pieces <= tpr * most) return tpr;
  return 0;
}

// pieces that a row may reach into
template <typename T> int row_pieces(const NormShape &s) {
  constexpr int V = Rows<T>::V;
  return s.C % V == 0 ? s.C / V : (s.C + V - 2) / V + 1;
}

// Rows for the packed forward: those that a warp does not hold, where it measured
// faster than the one with converted values (bfloat16 16384 x 1024: 20.4 against
// 24.0 us, 4096 x 8192: 37.0 against 53.5; 20011 x 768: 19.3 against 18.1), in
// float32 only those of 512 threads (4096 x 8192: 66.7 against 76.0 us, 8192 x 4096:
// 58.4 against 55.5).
template <typename T> bool use_packed(const NormShape &s) {
  constexpr int V = Rows<T>::V;
  return s.C % V == 0 && s.C > (V == 8 ? kPackedAbove : 256 * 24);
}

// most pieces per thread: 24 values of a row forward (the packed form four 16-bit
// pieces), 16 backward, where each costs five registers
template <typename T, bool BWD> int most(const NormShape &s) {
  constexpr int V = Rows<T>::V;
  return BWD ? 16 / V : V == 8 && use_packed<T>(s) ? 4 : 24 / V;
}

#define LN_ROW_NV(CALL, SHIFT)                           \
  do {                                                   \
    if (nv == 1) CALL(1, SHIFT);                         \
    else if (nv == 2) CALL(2, SHIFT);                    \
    else if (nv == 3) CALL(3, SHIFT);                    \
    else if (nv == 4) CALL(4, SHIFT);                    \
    else CALL(6, SHIFT);                                 \
  } while (0)
#define LN_ROW_CASES(CALL, BWD)                          \
  do {                                                   \
    const int pieces = row_pieces<T>(s);                 \
    const int tpr = pick_tpr(pieces, most<T, BWD>(s));   \
    const int nv = (pieces + tpr - 1) / tpr;             \
    if (s.C % Rows<T>::V == 0) LN_ROW_NV(CALL, false);   \
    else LN_ROW_NV(CALL, true);                          \
  } while (0)

int row_threads(int tpr) { return tpr > kRowThreads ? tpr : kRowThreads; }

// CTAs for that many groups of work, at most `cap`; with shifted rows the number
// of groups is a multiple of V (a divisor of cap's multiples of eight)
unsigned row_grid(long long groups, int R, int V, bool shifted, long long cap) {
  const long long unit = shifted && R < V ? V / R : 1;
  long long n = (groups + R - 1) / R;
  if (n > cap) n = cap;
  n = (n + unit - 1) / unit * unit;
  if (n > cap) n -= unit;
  return (unsigned)n;
}

template <typename T, int NV, bool SHIFT>
cudaError_t fwd_t(const Launch &L, const NormShape &s, int tpr, const void *x, const void *gamma,
                  const void *beta, void *y, float *mean, float *rstd) {
  const int threads = row_threads(tpr), R = threads / tpr;
  const float inv_c = 1.0f / (float)s.C;
  if (SHIFT || !use_packed<T>(s)) {
    constexpr int N = NV * Rows<T>::V > 24 ? 24 / Rows<T>::V : NV;
    const unsigned grid = row_grid(s.outer, R, Rows<T>::V, SHIFT, 4LL * L.num_sms);
    const auto kern = threads == kRowThreads ? k_ln_fwd_rows<T, N, SHIFT, kRowThreads>
                                             : k_ln_fwd_rows<T, N, SHIFT, 2 * kRowThreads>;
    kern<<<grid, threads, 0, L.stream>>>((const T *)x, (const T *)gamma, (const T *)beta, (T *)y,
                                         mean, rstd, s.outer, s.C, tpr, inv_c, s.eps);
  } else {
    constexpr int N = sizeof(T) == 2 && NV > 4 ? 4 : NV;
    const unsigned grid = (unsigned)((s.outer + R - 1) / R);
    const auto kern = threads == kRowThreads ? k_ln_fwd_rows_packed<T, N, kRowThreads>
                                             : k_ln_fwd_rows_packed<T, N, 2 * kRowThreads>;
    kern<<<grid, threads, 0, L.stream>>>((const T *)x, (const T *)gamma, (const T *)beta, (T *)y,
                                         mean, rstd, s.outer, s.C, tpr, inv_c, s.eps);
  }
  return cudaGetLastError();
}

template <typename T, int NV, bool SHIFT>
cudaError_t bwd_t(const Launch &L, const NormShape &s, int tpr, const void *x, const void *gamma,
                  const float *mean, const float *rstd, const void *dy, void *dx, float *partial,
                  int *nparts) {
  constexpr int N = NV * Rows<T>::V > 16 ? 16 / Rows<T>::V : NV;
  const int threads = row_threads(tpr), R = threads / tpr;
  long long cap = 2LL * L.num_sms;
  if (cap > kLnParts) cap = kLnParts;
  const unsigned grid = row_grid(s.outer, R, Rows<T>::V, SHIFT, cap);
  *nparts = (int)grid;
  // R C <= 256 16: at most 32 KB
  const size_t smem = R > 1 ? sizeof(float) * 2 * s.C * R : 0;
  const auto kern = threads == kRowThreads ? k_ln_bwd_rows<T, N, SHIFT, kRowThreads>
                                           : k_ln_bwd_rows<T, N, SHIFT, 2 * kRowThreads>;
  kern<<<grid, threads, smem, L.stream>>>((const T *)x, (const T *)gamma, mean, rstd,
                                          (const T *)dy, (T *)dx, partial, s.outer, s.C, tpr,
                                          1.0f / (float)s.C);
  return cudaGetLastError();
}

// the backward's grid under the cap of every device
template <typename T> int most_parts(const NormShape &s) {
  const int tpr = pick_tpr(row_pieces<T>(s), most<T, true>(s));
  return (int)row_grid(s.outer, row_threads(tpr) / tpr, Rows<T>::V, s.C % Rows<T>::V != 0, kLnParts);
}

template <typename T> bool fits(const NormShape &s, bool bwd) {
  return pick_tpr(row_pieces<T>(s), bwd ? most<T, true>(s) : most<T, false>(s)) != 0;
}

}  // namespace

bool ln_rows_supported(const NormShape &s, int dtype, bool bwd) {
  if (s.inner != 1 || s.outer > 0x7fffffffLL) return false;
  return dtype == DT_F32 ? fits<float>(s, bwd) : fits<__half>(s, bwd);
}

int ln_rows_parts(const NormShape &s, int dtype) {
  return dtype == DT_F32 ? most_parts<float>(s) : most_parts<__half>(s);
}

cudaError_t launch_ln_rows_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd) {
  cudaError_t err = cudaSuccess;
#define LN_FWD(NV, SHIFT) err = fwd_t<T, NV, SHIFT>(L, s, tpr, x, gamma, beta, y, mean, rstd)
  launch_begin(L);
  FNO_DISPATCH_T(dtype, LN_ROW_CASES(LN_FWD, false));
  launch_end(L, "ln_fwd_rows");
#undef LN_FWD
  return err;
}

cudaError_t launch_ln_rows_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts) {
  cudaError_t err = cudaSuccess;
#define LN_BWD(NV, SHIFT) \
  err = bwd_t<T, NV, SHIFT>(L, s, tpr, x, gamma, mean, rstd, dy, dx, partial, nparts)
  launch_begin(L);
  FNO_DISPATCH_T(dtype, LN_ROW_CASES(LN_BWD, true));
  launch_end(L, "ln_bwd_rows");
#undef LN_BWD
  return err;
}

}  // namespace fno

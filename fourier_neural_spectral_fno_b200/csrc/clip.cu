// The 2-norm of many gradients together, the clipping factor, and the clipped
// gradients:
//   norm = |grad_scale| sqrt(sum over all tensors of g^2)
//   factor = 1 if norm <= max_norm, else max_norm / norm
//   out = g (grad_scale factor)
// Every sum beyond one 16-byte group is float64: tens of millions of squares
// spread over many orders of magnitude keep their full float32 accuracy, and
// squares that float32 cannot hold are summed as float64 (sq_group).  The order
// of the sums is fixed by the sizes alone, so results do not vary from call to
// call.
//
// The tensors' pointers and sizes travel in the launch's parameters (nothing to
// upload, and a captured graph holds them).  The tensors are cut into chunks of
// 4 KB, one for a warp at a time (many short parameters then still spread over
// the GPU); a warp finds its chunk's tensor by bisection over the running chunk
// counts, once per tensor.
//
// At most one chunk for each warp of a CTA: one launch of one CTA.  Else one
// launch for the sums, which runs from the last chunk to the first so that the
// next reader of the gradients, from the first on, finds them in L2, and one that
// adds up the sums and scales (or only writes the norm); the second is launched
// while the first runs (programmatic dependent launch).  A cluster of eight CTAs
// for up to 4 MB in one launch measured slower (18 parameters of 0.9 M float32:
// 9.1 us against 3.5; 320 short bfloat16 ones, clipped: 29 against 6.3).
//
// Bound by HBM for many bytes (25.5 us for 37.8 M float32, 92 % of the copy rate;
// clipped they no longer fit L2 and are read twice: 73.8 us), by the two launches
// for few.  A tensor off the 16-byte boundaries goes value by value: the same 37.8 M with
// every tensor one value off take 25.9 us for the norm and 164 clipped into other
// tensors (74 on the boundaries), in bfloat16 30 us and 202 (19 and 42).
#include <math.h>

#include "fno_common.cuh"
#include "fno_kernels.cuh"

namespace fno {

namespace {

constexpr int CT = 256;                      // threads per CTA
constexpr int kVecs = 8;                     // 16-byte groups per lane and chunk
constexpr int kChunkBytes = 32 * kVecs * 16;
constexpr int ST = 1024;                     // threads of the one-CTA form

template <int N> struct TensorTable {
  const void *in[N];
  void *out[N];
  long long n[N];
  int first[N + 1];                          // chunks before each tensor
  int count;
};

// A warp's place in the table: the tensor of its last chunk.
struct Place {
  int t = 0, lo = 0, hi = 0;                 // tensor t has the chunks lo .. hi - 1
};

// a chunk's tensor, first element and elements
template <int N>
__device__ __forceinline__ void find(const TensorTable<N> &tab, int chunk, int elems, Place &p,
                                     long long &off, int &n) {
  if (chunk < p.lo || chunk >= p.hi) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= chunk) lo = mid;
      else hi = mid - 1;
    }
    p.t = lo;
    p.lo = tab.first[lo];
    p.hi = tab.first[lo + 1];
  }
  off = (long long)(chunk - p.lo) * elems;
  const long long left = tab.n[p.t] - off;
  n = (int)(left < elems ? left : elems);
}

template <typename T> struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float get(int i) const {
    return to_f<T>(reinterpret_cast<const T *>(&raw)[i]);
  }
  __device__ __forceinline__ void set(int i, float v) {
    reinterpret_cast<T *>(&raw)[i] = from_f<T>(v);
  }
};

// Sum of the squares of one 16-byte group: in float32 where that sum lies well
// inside float32's range (a few roundings of 2^-24, then averaged over the
// groups), else in float64 (very small, zero, very large or not finite).
template <typename T> __device__ __forceinline__ double sq_group(const Vec16<T> &v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < Vec16<T>::N; ++i) s = fmaf(v.get(i), v.get(i), s);
  if (s >= 1e-18f && s <= 1e37f) return (double)s;
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < Vec16<T>::N; ++i) d = fma((double)v.get(i), (double)v.get(i), d);
  return d;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the CTA's sum, in every thread
template <int THREADS> __device__ __forceinline__ double cta_sum(double v, double *sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += sh[i];
  return t;
}

// the lane's share of a chunk's squares
template <typename T, int N>
__device__ __forceinline__ double chunk_sq(const TensorTable<N> &tab, int chunk, Place &p) {
  constexpr int VN = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  long long off;
  int n, done = 0;
  find(tab, chunk, kChunkBytes / (int)sizeof(T), p, off, n);
  const T *src = static_cast<const T *>(tab.in[p.t]) + off;
  double acc = 0.0;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
    const uint4 *v = reinterpret_cast<const uint4 *>(src);
    const int nv = n / VN;
    done = nv * VN;
    Vec16<T> g[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = lane + j * 32;
      g[j].raw = i < nv ? v[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (lane + j * 32 < nv) acc += sq_group<T>(g[j]);
  }
  for (int i = done + lane; i < n; i += 32) {
    const double g = (double)to_f<T>(src[i]);
    acc = fma(g, g, acc);
  }
  return acc;
}

// out = g f over a chunk; in place and with f == 1 nothing changes and nothing is
// written
template <typename T, int N>
__device__ __forceinline__ void chunk_scale(const TensorTable<N> &tab, int chunk, Place &p,
                                            float f) {
  constexpr int VN = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  long long off;
  int n, done = 0;
  find(tab, chunk, kChunkBytes / (int)sizeof(T), p, off, n);
  if (f == 1.f && tab.in[p.t] == tab.out[p.t]) return;
  const T *src = static_cast<const T *>(tab.in[p.t]) + off;
  T *dst = static_cast<T *>(tab.out[p.t]) + off;
  if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
    const int nv = n / VN;
    done = nv * VN;
    Vec16<T> g[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = lane + j * 32;
      if (i < nv) g[j].raw = reinterpret_cast<const uint4 *>(src)[i];
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = lane + j * 32;
      if (i < nv) {
#pragma unroll
        for (int k = 0; k < VN; ++k) g[j].set(k, g[j].get(k) * f);
        reinterpret_cast<uint4 *>(dst)[i] = g[j].raw;
      }
    }
  }
  for (int i = done + lane; i < n; i += 32) dst[i] = from_f<T>(to_f<T>(src[i]) * f);
}

// norm[0] = the norm, norm[1] = the factor, of a sum of squares
__device__ __forceinline__ float2 norm_of(double sum, double scale, double max_norm) {
  const double nm = sqrt(sum) * scale;
  return make_float2((float)nm, nm <= max_norm ? 1.f : (float)(max_norm / nm));
}

// partial[blockIdx] = sum of the squares of the CTA's chunks
template <typename T, int N>
__global__ void __launch_bounds__(CT)
    k_grad_sumsq(const __grid_constant__ TensorTable<N> tab, double *__restrict__ partial) {
  __shared__ double sh[CT / 32];
  cudaTriggerProgrammaticLaunchCompletion();   // the next launch may be set up meanwhile
  const int chunks = tab.first[tab.count], step = gridDim.x * (CT / 32);
  double acc = 0.0;
  Place p;
  for (int ch = chunks - 1 - (int)(blockIdx.x * (CT / 32) + (threadIdx.x >> 5)); ch >= 0; ch -= step)
    acc += chunk_sq<T>(tab, ch, p);
  acc = cta_sum<CT>(acc, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// the sum of all partial sums, in every thread; `partial` comes from the launch
// before
__device__ __forceinline__ double all_parts(const double *partial, int nparts, double *sh) {
  cudaGridDependencySynchronize();
  double acc = 0.0;
  for (int i = threadIdx.x; i < nparts; i += CT) acc += __ldcg(partial + i);
  return cta_sum<CT>(acc, sh);
}

__global__ void __launch_bounds__(CT)
    k_grad_norm(const double *partial, int nparts, double scale, double max_norm, float *norm) {
  __shared__ double sh[CT / 32];
  const float2 r = norm_of(all_parts(partial, nparts, sh), scale, max_norm);
  if (threadIdx.x == 0) {
    norm[0] = r.x;
    norm[1] = r.y;
  }
}

// every CTA adds up the partial sums for itself; CTA 0 writes the norm
template <typename T, int N>
__global__ void __launch_bounds__(CT)
    k_grad_scale(const __grid_constant__ TensorTable<N> tab, const double *partial, int nparts,
                 double scale, double max_norm, float grad_scale, float *norm) {
  __shared__ double sh[CT / 32];
  const float2 r = norm_of(all_parts(partial, nparts, sh), scale, max_norm);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = r.x;
    norm[1] = r.y;
  }
  const float f = r.y * grad_scale;
  const int chunks = tab.first[tab.count], step = gridDim.x * (CT / 32);
  Place p;
  for (int ch = blockIdx.x * (CT / 32) + (threadIdx.x >> 5); ch < chunks; ch += step)
    chunk_scale<T>(tab, ch, p, f);
}

// all of it by one CTA
template <typename T, int N, bool SCALE>
__global__ void __launch_bounds__(ST)
    k_grad_one(const __grid_constant__ TensorTable<N> tab, double scale, double max_norm,
               float grad_scale, float *norm) {
  __shared__ double sh[ST / 32];
  const int chunk = threadIdx.x >> 5;
  const bool in = chunk < tab.first[tab.count];
  Place p;
  double acc = in ? chunk_sq<T>(tab, chunk, p) : 0.0;
  acc = cta_sum<ST>(acc, sh);
  const float2 r = norm_of(acc, scale, max_norm);
  if (threadIdx.x == 0) {
    norm[0] = r.x;
    norm[1] = r.y;
  }
  if (SCALE && in) chunk_scale<T>(tab, chunk, p, r.y * grad_scale);
}

// Fill `tab` from tensor `at` on, passing over empty ones; returns the tensor
// after the last one taken.
template <int N>
int fill(TensorTable<N> &tab, int at, int n, const void *const *in, void *const *out,
         const int64_t *sizes, int elem) {
  const long long ce = kChunkBytes / elem;
  int chunks = 0;   // at most 2^40 elements in all: below 2^30 chunks and one a tensor
  tab.count = 0;
  int i = at;
  for (; i < n && tab.count < N; ++i) {
    if (sizes[i] == 0) continue;
    tab.in[tab.count] = in[i];
    tab.out[tab.count] = out ? out[i] : const_cast<void *>(in[i]);
    tab.n[tab.count] = sizes[i];
    tab.first[tab.count] = chunks;
    chunks += (int)((sizes[i] + ce - 1) / ce);
    ++tab.count;
  }
  tab.first[tab.count] = chunks;
  return i;
}

int clip_grid(const Launch &L, int chunks) {
  const int ctas = (chunks + CT / 32 - 1) / (CT / 32);
  int cap = 4 * L.num_sms;
  if (cap > kNormCTAs) cap = kNormCTAs;
  return ctas < cap ? ctas : cap;
}

template <typename T, int N>
cudaError_t run(const Launch &L, int n, const void *const *grads, void *const *out, bool scale_too,
                const int64_t *sizes, float grad_scale, float max_norm, float *norm,
                double *partial) {
  const double scale = fabs((double)grad_scale), limit = (double)max_norm;
  TensorTable<N> tab;
  int at = fill(tab, 0, n, grads, out, sizes, sizeof(T));
  if (at == n && tab.first[tab.count] <= ST / 32) {
    launch_begin(L);
    if (scale_too)
      k_grad_one<T, N, true><<<1, ST, 0, L.stream>>>(tab, scale, limit, grad_scale, norm);
    else
      k_grad_one<T, N, false><<<1, ST, 0, L.stream>>>(tab, scale, limit, grad_scale, norm);
    const cudaError_t err = cudaGetLastError();
    launch_end(L, scale_too ? "grad_clip" : "grad_norm");
    return err;
  }
  int nparts = 0;
  for (int from = 0; from < n;) {
    if (from > 0 || at == 0) at = fill(tab, from, n, grads, out, sizes, sizeof(T));
    from = at;
    if (tab.count == 0) continue;
    const int grid = clip_grid(L, tab.first[tab.count]);
    launch_begin(L);
    k_grad_sumsq<T, N><<<grid, CT, 0, L.stream>>>(tab, partial + nparts);
    const cudaError_t err = cudaGetLastError();
    launch_end(L, "grad_sumsq");
    if (err != cudaSuccess) return err;
    nparts += grid;
  }
  if (!scale_too) {
    launch_begin(L);
    const cudaError_t err =
        launch_dependent(L, 1, CT, k_grad_norm, (const double *)partial, nparts, scale, limit, norm);
    launch_end(L, "grad_norm");
    return err;
  }
  bool first = true;
  for (int from = 0; from < n;) {
    // a single table is still filled
    if (n > N || !first) from = fill(tab, from, n, grads, out, sizes, sizeof(T));
    else from = n;
    if (tab.count == 0) continue;
    launch_begin(L);
    const int grid = clip_grid(L, tab.first[tab.count]);
    const cudaError_t err =
        launch_dependent(L, grid, CT, k_grad_scale<T, N>, tab, (const double *)partial, nparts, scale,
                         limit, grad_scale, first ? norm : nullptr);
    launch_end(L, "grad_scale");
    if (err != cudaSuccess) return err;
    first = false;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_grad_norm(const Launch &L, int n, const void *const *grads, void *const *out,
                             bool scale_too, const int64_t *sizes, int dtype, float grad_scale,
                             float max_norm, float *norm, double *partial) {
  cudaError_t err;
  if (n <= kFewTensors)
    FNO_DISPATCH_T(dtype, err = run<T, kFewTensors>(L, n, grads, out, scale_too, sizes, grad_scale,
                                                    max_norm, norm, partial));
  else if (n <= kSomeTensors)
    FNO_DISPATCH_T(dtype, err = run<T, kSomeTensors>(L, n, grads, out, scale_too, sizes,
                                                     grad_scale, max_norm, norm, partial));
  else
    FNO_DISPATCH_T(dtype, err = run<T, kClipTensors>(L, n, grads, out, scale_too, sizes,
                                                     grad_scale, max_norm, norm, partial));
  return err;
}

}  // namespace fno

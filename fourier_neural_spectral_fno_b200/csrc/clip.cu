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
// kChunkBytes; a CTA takes every gridDim-th chunk and finds its tensor by
// bisection over the running chunk counts.
#include <math.h>

#include "fno_common.cuh"
#include "fno_kernels.cuh"

namespace fno {

namespace {

constexpr int CT = 256;                      // threads per CTA
constexpr int kVecs = 8;                     // 16-byte groups per thread and chunk
constexpr int kChunkBytes = CT * kVecs * 16;

struct TensorTable {
  const void *in[kClipTensors];
  void *out[kClipTensors];
  long long n[kClipTensors];
  int first[kClipTensors + 1];               // chunks before each tensor
  int count;
};

// tensor of a chunk: the last one with first[t] <= chunk (empty ones excluded)
__device__ __forceinline__ int find_tensor(const TensorTable &tab, int chunk) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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

// the CTA's sum, in thread 0
__device__ __forceinline__ double cta_sum(double v, double *sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < CT / 32; ++i) t += sh[i];
  return t;
}

// partial[blockIdx] = sum of the squares of the CTA's chunks
template <typename T>
__global__ void __launch_bounds__(CT)
    k_grad_sumsq(const __grid_constant__ TensorTable tab, double *__restrict__ partial) {
  __shared__ double sh[CT / 32];
  constexpr int VN = Vec16<T>::N;
  constexpr long long CE = kChunkBytes / sizeof(T);
  const int chunks = tab.first[tab.count];
  double acc = 0.0;
  for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    const int t = find_tensor(tab, ch);
    const long long off = (ch - tab.first[t]) * CE;
    const long long left = tab.n[t] - off;
    const int n = (int)(left < CE ? left : CE);
    const T *src = static_cast<const T *>(tab.in[t]) + off;
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
      const uint4 *v = reinterpret_cast<const uint4 *>(src);
      const int nv = n / VN;
      done = nv * VN;
      Vec16<T> g[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int i = threadIdx.x + j * CT;
        g[j].raw = i < nv ? __ldg(v + i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (threadIdx.x + j * CT < nv) acc += sq_group<T>(g[j]);
    }
    for (int i = done + threadIdx.x; i < n; i += CT) {
      const double g = (double)to_f<T>(src[i]);
      acc = fma(g, g, acc);
    }
  }
  acc = cta_sum(acc, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// norm[0] = the norm, norm[1] = the factor
__global__ void __launch_bounds__(CT)
    k_grad_norm(const double *__restrict__ partial, int nparts, double scale, double max_norm,
                float *__restrict__ norm) {
  __shared__ double sh[CT / 32];
  double acc = 0.0;
  for (int i = threadIdx.x; i < nparts; i += CT) acc += partial[i];
  acc = cta_sum(acc, sh);
  if (threadIdx.x == 0) {
    const double nm = sqrt(acc) * scale;
    norm[0] = (float)nm;
    norm[1] = nm <= max_norm ? 1.f : (float)(max_norm / nm);
  }
}

// out = g (scale factor); in place and with a multiplier of one nothing changes
// and nothing is written
template <typename T>
__global__ void __launch_bounds__(CT)
    k_grad_scale(const __grid_constant__ TensorTable tab, const float *__restrict__ norm,
                 float scale) {
  constexpr int VN = Vec16<T>::N;
  constexpr long long CE = kChunkBytes / sizeof(T);
  const int chunks = tab.first[tab.count];
  const float f = norm[1] * scale;
  for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    const int t = find_tensor(tab, ch);
    if (f == 1.f && tab.in[t] == tab.out[t]) continue;
    const long long off = (ch - tab.first[t]) * CE;
    const long long left = tab.n[t] - off;
    const int n = (int)(left < CE ? left : CE);
    const T *src = static_cast<const T *>(tab.in[t]) + off;
    T *dst = static_cast<T *>(tab.out[t]) + off;
    int done = 0;
    if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
      const int nv = n / VN;
      done = nv * VN;
      Vec16<T> g[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int i = threadIdx.x + j * CT;
        if (i < nv) g[j].raw = reinterpret_cast<const uint4 *>(src)[i];
      }
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int i = threadIdx.x + j * CT;
        if (i < nv) {
#pragma unroll
          for (int k = 0; k < VN; ++k) g[j].set(k, g[j].get(k) * f);
          reinterpret_cast<uint4 *>(dst)[i] = g[j].raw;
        }
      }
    }
    for (int i = done + threadIdx.x; i < n; i += CT) dst[i] = from_f<T>(to_f<T>(src[i]) * f);
  }
}

// Fill `tab` from tensor `at` on; returns the tensors taken (empty ones are
// passed over, so it may take more than it lists), and false where the chunks
// do not fit an int.
int fill(TensorTable &tab, int at, int n, const void *const *in, void *const *out,
         const int64_t *sizes, int elem) {
  const long long ce = kChunkBytes / elem;
  long long chunks = 0;
  tab.count = 0;
  int i = at;
  for (; i < n && tab.count < kClipTensors; ++i) {
    if (sizes[i] == 0) continue;
    const long long c = (sizes[i] + ce - 1) / ce;
    if (chunks + c > 0x7fffffffLL - kNormCTAs) break;
    tab.in[tab.count] = in[i];
    tab.out[tab.count] = out ? out[i] : const_cast<void *>(in[i]);
    tab.n[tab.count] = sizes[i];
    tab.first[tab.count] = (int)chunks;
    chunks += c;
    ++tab.count;
  }
  tab.first[tab.count] = (int)chunks;
  return i - at;
}

#define FNO_DISPATCH_T(dtype, ...)                                \
  do {                                                            \
    if ((dtype) == DT_F32) {                                      \
      using T = float;                                            \
      __VA_ARGS__;                                                \
    } else if ((dtype) == DT_F16) {                               \
      using T = __half;                                           \
      __VA_ARGS__;                                                \
    } else {                                                      \
      using T = __nv_bfloat16;                                    \
      __VA_ARGS__;                                                \
    }                                                             \
  } while (0)

int clip_grid(const Launch &L, int chunks) {
  long long cap = 4LL * L.num_sms;
  if (cap > kNormCTAs) cap = kNormCTAs;
  return (int)(chunks < cap ? chunks : cap);
}

}  // namespace

cudaError_t launch_grad_norm(const Launch &L, int n, const void *const *grads,
                             const int64_t *sizes, int dtype, float grad_scale, float max_norm,
                             float *norm, double *partial) {
  TensorTable tab;
  int nparts = 0;
  for (int at = 0; at < n;) {
    at += fill(tab, at, n, grads, nullptr, sizes, dtype == DT_F32 ? 4 : 2);
    if (tab.count == 0) continue;
    const int grid = clip_grid(L, tab.first[tab.count]);
    launch_begin(L);
    FNO_DISPATCH_T(dtype, k_grad_sumsq<T><<<grid, CT, 0, L.stream>>>(tab, partial + nparts));
    const cudaError_t err = cudaGetLastError();
    launch_end(L, "grad_sumsq");
    if (err != cudaSuccess) return err;
    nparts += grid;
  }
  launch_begin(L);
  k_grad_norm<<<1, CT, 0, L.stream>>>(partial, nparts, fabs((double)grad_scale),
                                      (double)max_norm, norm);
  const cudaError_t err = cudaGetLastError();
  launch_end(L, "grad_norm");
  return err;
}

cudaError_t launch_grad_scale(const Launch &L, int n, const void *const *grads, void *const *out,
                              const int64_t *sizes, int dtype, float grad_scale,
                              const float *norm) {
  TensorTable tab;
  for (int at = 0; at < n;) {
    at += fill(tab, at, n, grads, out, sizes, dtype == DT_F32 ? 4 : 2);
    if (tab.count == 0) continue;
    const int grid = clip_grid(L, tab.first[tab.count]);
    launch_begin(L);
    FNO_DISPATCH_T(dtype, k_grad_scale<T><<<grid, CT, 0, L.stream>>>(tab, norm, grad_scale));
    const cudaError_t err = cudaGetLastError();
    launch_end(L, "grad_scale");
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace fno

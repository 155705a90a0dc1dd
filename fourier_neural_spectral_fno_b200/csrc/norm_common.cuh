// Helpers shared by the layer norm kernels.
#pragma once

#include "fno_common.cuh"
#include "fno_kernels.cuh"

namespace fno {

// the two values of a four-byte word of a 16-bit type
template <typename T> __device__ __forceinline__ void word_get(unsigned w, float &a, float &b);
template <> __device__ __forceinline__ void word_get<__half>(unsigned w, float &a, float &b) {
  const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  a = t.x;
  b = t.y;
}
template <>
__device__ __forceinline__ void word_get<__nv_bfloat16>(unsigned w, float &a, float &b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <typename T> __device__ __forceinline__ unsigned word_set(float a, float b);
template <> __device__ __forceinline__ unsigned word_set<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const unsigned *>(&h);
}
template <> __device__ __forceinline__ unsigned word_set<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned *>(&h);
}

// V consecutive values of the storage type as one memory access of V sizeof(T)
// bytes (16, or one element).  keep() hides the values' origin from the compiler:
// a later sweep converts the packed registers again instead of holding the
// converted ones, which for 16-bit types take twice as many.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ void keep() {
    asm volatile("" : "+f"(r.x), "+f"(r.y), "+f"(r.z), "+f"(r.w));
  }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float *f) const { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
  __device__ __forceinline__ void set(const float *f) { r = make_float4(f[0], f[1], f[2], f[3]); }
  __device__ __forceinline__ void get2(f32x2 *p) const {
    p[0] = f2pack(r.x, r.y);
    p[1] = f2pack(r.z, r.w);
  }
  __device__ __forceinline__ void set2(const f32x2 *p) {
    f2unpack(p[0], r.x, r.y);
    f2unpack(p[1], r.z, r.w);
  }
};
template <> struct Pack<__half, 8> {
  uint4 r;
  __device__ __forceinline__ void keep() {
    asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w));
  }
  __device__ __forceinline__ void get2(f32x2 *p) const {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      word_get<__half>(w[i], a, b);
      p[i] = f2pack(a, b);
    }
  }
  __device__ __forceinline__ void set2(const f32x2 *p) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2unpack(p[i], a, b);
      w[i] = word_set<__half>(a, b);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float *f) const {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ __forceinline__ void set(const float *f) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Pack<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void keep() {
    asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w));
  }
  __device__ __forceinline__ void get2(f32x2 *p) const {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      word_get<__nv_bfloat16>(w[i], a, b);
      p[i] = f2pack(a, b);
    }
  }
  __device__ __forceinline__ void set2(const f32x2 *p) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2unpack(p[i], a, b);
      w[i] = word_set<__nv_bfloat16>(a, b);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  // a bfloat16 is the upper half of the float32 of the same value
  __device__ __forceinline__ void get(float *f) const {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float *f) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T> struct Pack<T, 4> {   // 16-bit types: 8 bytes
  uint2 r;
  __device__ __forceinline__ void keep() { asm volatile("" : "+r"(r.x), "+r"(r.y)); }
  __device__ __forceinline__ void zero() { r = make_uint2(0, 0); }
  __device__ __forceinline__ void get(float *f) const {
    word_get<T>(r.x, f[0], f[1]);
    word_get<T>(r.y, f[2], f[3]);
  }
  __device__ __forceinline__ void set(const float *f) {
    r = make_uint2(word_set<T>(f[0], f[1]), word_set<T>(f[2], f[3]));
  }
};
template <typename T> struct Pack<T, 1> {
  T r;
  __device__ __forceinline__ void keep() {}
  __device__ __forceinline__ void zero() { r = from_f<T>(0.f); }
  __device__ __forceinline__ void get(float *f) const { f[0] = to_f<T>(r); }
  __device__ __forceinline__ void set(const float *f) { r = from_f<T>(f[0]); }
};

// hides a value's origin, so that what depends on it is computed again (inside a
// loop: in each round) rather than held in registers: multiples of a channel's
// stride, above all
__device__ __forceinline__ long long again(long long v) {
  asm volatile("" : "+l"(v));
  return v;
}

// the sum of a pair's halves
__device__ __forceinline__ float pair_sum(f32x2 v) {
  float a, b;
  f2unpack(v, a, b);
  return a + b;
}

template <typename T> struct VecOf { static constexpr int N = 16 / sizeof(T); };

// 1 / sqrt(var + eps) with var = q / C - e^2 from the deviations about a first
// mean: never below zero by rounding, and a NaN stays one
__device__ __forceinline__ float ln_rstd(float q_mean, float e, float eps) {
  const float var = fmaf(-e, e, q_mean);
  return 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

// e = mean(x - m0) of a first mean m0 = sum / C of 16-bit values, from the residual of
// that division in place of a sum over the deviations.  It leaves out what the sum itself
// has lost.  That is nothing where it would show, for values within a factor of two: they
// are whole multiples of one step, with 12 bits (float16) or 9 (bfloat16), and a sum of
// ResidualChannels of them keeps within float32's 24.  Values farther apart have a
// spread of at least |x| / (2 C^1/2), against which a sum's rounding is small.
template <typename T> struct ResidualChannels { static constexpr int N = 0; };
template <> struct ResidualChannels<__half> { static constexpr int N = 1 << 12; };
template <> struct ResidualChannels<__nv_bfloat16> { static constexpr int N = 1 << 15; };
__device__ __forceinline__ float ln_residual(float sum, float m0, int C, float inv_c) {
  return fmaf(-(float)C, m0, sum) * inv_c;
}

// ---- per-layout kernels -----------------------------------------------------
// grid layout (inner > 1), values held in registers (norm_grid.cu)
constexpr int kGridBwdChannels = 256;   // most channels of its backward
bool ln_grid_supported(const NormShape &s, int dtype, bool bwd);
cudaError_t launch_ln_grid_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd);
// writes dx and, unless partial is NULL, *nparts rows of [C][2] (dgamma, dbeta)
// partial sums
cudaError_t launch_ln_grid_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts);

// grid layout whose rows start anywhere (norm_odd.cu); dy given: backward, outputs as
// launch_ln_grid_bwd
bool ln_odd_supported(const NormShape &s, int dtype, bool bwd);
cudaError_t launch_ln_odd(const Launch &L, const NormShape &s, int dtype, const void *x,
                          const void *gamma, const void *beta, const void *dy, void *out,
                          float *mean_out, float *rstd_out, const float *mean_in,
                          const float *rstd_in, float *partial, int *nparts);

// rows (inner == 1), values held in registers (norm_rows.cu); outputs as above
bool ln_rows_supported(const NormShape &s, int dtype, bool bwd);
int ln_rows_parts(const NormShape &s, int dtype);   // most partial rows, on any device
cudaError_t launch_ln_rows_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd);
cudaError_t launch_ln_rows_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts);
// the grid layout as a TMA pipeline, at most 128 channels (norm_pipe.cu)
bool ln_pipe_supported(const NormShape &s, int dtype, bool bwd);
cudaError_t launch_ln_pipe_fwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const void *beta, void *y, float *mean,
                               float *rstd);
cudaError_t launch_ln_pipe_bwd(const Launch &L, const NormShape &s, int dtype, const void *x,
                               const void *gamma, const float *mean, const float *rstd,
                               const void *dy, void *dx, float *partial, int *nparts);

}  // namespace fno

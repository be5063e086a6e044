// layernorm.cu -- layer norm over rows, forward and backward.
//
// Forward, per row x of D elements:
//   mean = sum(x) / D,  var = sum((x - mean)^2) / D,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) * rstd * gamma + beta
// Backward, with xh = (x - mean) * rstd and g = gamma * dy:
//   dx     = rstd * (g - sum(g) / D - xh * sum(g * xh) / D)
//   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
// Arithmetic and every sum are fp32; y, dx, dgamma and dbeta are rounded once.
// Both passes are bound by HBM: 2 (forward) and 3 (backward) elements move per
// element of x, with about 8 and 14 flops each.  At 8192 x 4096 bf16 the forward
// runs 24.1 us (5.6 TB/s, 0.86 of a measured copy) and the backward 40.2 us with
// the reduction of dgamma and dbeta (5.0 TB/s, 0.78); fp32 46.1 and 68.6 us (0.90
// and 0.91).  16-bit elements cost twice the instructions a byte, so the work is
// in packed fp32 pairs on rows held in registers, few reductions, and copies
// that need no thread.
#include "layernorm.h"

#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "launch.h"

namespace mxn {
namespace {

// V consecutive elements of type T as fp32: 16 bytes (V * sizeof(T) == 16) in
// one access, or one element (V == 1).
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(uint32_t w, float* v) { v[0] = bf16lo(w); v[1] = bf16hi(w); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
};
template <> struct Elem<float> {
  static __device__ __forceinline__ float to_f(float x) { return x; }
  static __device__ __forceinline__ float from_f(float x) { return x; }
};

template <typename T, int V>
__device__ __forceinline__ void unpack16(uint4 u, float (&v)[V]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  } else {
    Elem<T>::unpack(u.x, v); Elem<T>::unpack(u.y, v + 2);
    Elem<T>::unpack(u.z, v + 4); Elem<T>::unpack(u.w, v + 6);
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_chunk(const T* p, float (&v)[V]) {
  // A plain load, not __ldg: for 16-bit types that is an inline-assembly load
  // the compiler may move above the bounds or null check that guards it.
  if constexpr (V == 1)
    v[0] = Elem<T>::to_f(*p);
  else
    unpack16<T, V>(ldg128_nc(p), v);
}

template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = Elem<T>::from_f(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    stg128_stream(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                __float_as_uint(v[3])));
  } else {
    stg128_stream(p, make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                                Elem<T>::pack(v[6], v[7])));
  }
}

// A 16-byte chunk as fp32 pairs, and back.
template <typename T>
__device__ __forceinline__ void unpack2(uint4 u, float2 (&v)[8 / sizeof(T)]) {
  float f[16 / sizeof(T)];
  unpack16<T, 16 / sizeof(T)>(u, f);
#pragma unroll
  for (int e = 0; e < 8 / (int)sizeof(T); ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const float2 (&v)[8 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  else
    return make_uint4(Elem<T>::pack(v[0].x, v[0].y), Elem<T>::pack(v[1].x, v[1].y), Elem<T>::pack(v[2].x, v[2].y),
                      Elem<T>::pack(v[3].x, v[3].y));
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}

// One element in shared memory, as fp32.
template <typename T>
__device__ __forceinline__ float lds_elem(uint32_t addr) {
  if constexpr (sizeof(T) == 4) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(addr));
    return f;
  } else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
    return Elem<T>::to_f(*reinterpret_cast<const T*>(&h));
  }
}

// A lane's J chunks of a row: element sums, centred squares and the result.
// Packed rows (V = 16 / sizeof(T) elements a chunk) stay as loaded.
template <typename T, int V, int J>
struct RowPart {
  uint4 u[J];
  // Loads the chunks c0, c0 + 32, .. below n and adds up their elements.
  template <bool ALL>
  __device__ __forceinline__ float load_sum(uint32_t row, int c0, int n) {
    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    // Past the row's end the last chunk is read and counts as zero: no branch a chunk.
#pragma unroll
    for (int j = 0; j < J; ++j) u[j] = lds128(row + 16u * (ALL ? c0 + 32 * j : min(c0 + 32 * j, n - 1)));
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!ALL && c0 + 32 * j >= n) u[j] = make_uint4(0, 0, 0, 0);
      float2 f[V / 2];
      unpack2<T>(u[j], f);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) acc[e & 1] = add2(acc[e & 1], f[e]);
    }
    return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
  }
  template <bool ALL>
  __device__ __forceinline__ float squares(float mean, int c0, int n) const {
    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float m = ALL || c0 + 32 * j < n ? -mean : 0.0f;
      const float2 m2 = make_float2(m, m);
      float2 f[V / 2];
      unpack2<T>(u[j], f);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        f[e] = add2(f[e], m2);
        acc[e & 1] = fma2(f[e], f[e], acc[e & 1]);
      }
    }
    return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
  }
  __device__ __forceinline__ void shift(float) {}                    // the row is as it came
  // (x - mean) * rstd * gamma + beta to y (this lane's first chunk).
  template <bool ALL>
  __device__ __forceinline__ void store(T* y, float mean, float rstd, uint32_t gamma, uint32_t beta, int c0, int n) const {
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = ALL ? c0 + 32 * j : min(c0 + 32 * j, n - 1);
      float2 f[V / 2], g[V / 2], b[V / 2];
      unpack2<T>(u[j], f);
      unpack2<T>(lds128(gamma + 16u * c), g);
      unpack2<T>(lds128(beta + 16u * c), b);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) f[e] = fma2(mul2(add2(f[e], m2), r2), g[e], b[e]);
      if (ALL || c0 + 32 * j < n) stg128_stream(y + (size_t)32 * j * V, pack2<T>(f));
    }
  }
};
// Single elements (rows off 16-byte boundaries), as fp32.
template <typename T, int J>
struct RowPart<T, 1, J> {
  float x[J];
  template <bool ALL>
  __device__ __forceinline__ float load_sum(uint32_t row, int c0, int n) {
    float a = 0.0f, b = 0.0f;
    row += (uint32_t)sizeof(T) * c0;
#pragma unroll
    for (int j = 0; j < J; ++j)
      x[j] = ALL || c0 + 32 * j < n ? lds_elem<T>(row + 32u * (uint32_t)sizeof(T) * j) : 0.0f;
#pragma unroll
    for (int j = 0; j < J; j += 2) {
      a += x[j];
      b += x[j + 1];
    }
    return a + b;
  }
  template <bool ALL>
  __device__ __forceinline__ float squares(float mean, int c0, int n) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j] -= mean;
      if (!ALL && c0 + 32 * j >= n) x[j] = 0.0f;
      if (j & 1) b = fmaf(x[j], x[j], b);
      else a = fmaf(x[j], x[j], a);
    }
    return a + b;
  }
  __device__ __forceinline__ void shift(float by) {
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] -= by;
  }
  template <bool ALL>
  __device__ __forceinline__ void store(T* y, float, float rstd, uint32_t gamma, uint32_t beta, int c0, int n) const {
    gamma += (uint32_t)sizeof(T) * c0;
    beta += (uint32_t)sizeof(T) * c0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!ALL && c0 + 32 * j >= n) continue;
      y[32 * j] = Elem<T>::from_f(fmaf(x[j] * rstd, lds_elem<T>(gamma + 32u * (uint32_t)sizeof(T) * j),
                                       lds_elem<T>(beta + 32u * (uint32_t)sizeof(T) * j)));
    }
  }
};

// Sum over a row group of nwarp warps, the same order in every thread.  `slots`:
// 32 floats of shared memory, zero beyond the group's warps; a second array is
// due for the next sum.
__device__ __forceinline__ float group_sum(float s, uint32_t slots, int nwarp, int barrier) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (nwarp == 1) return s;
  if ((threadIdx.x & 31) == 0) sts32(slots + 4u * ((threadIdx.x >> 5) % nwarp), __float_as_uint(s));
  named_barrier_sync(barrier, nwarp * 32);
  s = 0.0f;
  for (int w = 0; w < nwarp; w += 4) {
    const uint4 u = lds128(slots + 4u * w);
    s += (__uint_as_float(u.x) + __uint_as_float(u.y)) + (__uint_as_float(u.z) + __uint_as_float(u.w));
  }
  return s;
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// -------------------------------------------------------------------- forward

struct LnFwdArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  int64_t T, ld_x;
  int D, tpr;            // row length, threads per row (a multiple of 32)
  float eps;
};

// The sum's rounding leaves the mean a few ulp off, which counts where the mean is
// far above the deviation (a constant row of -12345.678 came out as 0.68 instead of
// 0).  Such rows add up what is left about the mean and move it by that: it is then
// right to its own rounding.  Far is beyond 16 deviations in fp32, where the first
// mean is good to 2e-6 of one, and beyond 64 in 16 bits, whose outputs are coarser.
template <typename T> constexpr float kLnFar = sizeof(T) == 4 ? 256.0f : 4096.0f;   // squared
template <typename T>
__device__ __forceinline__ bool far_mean(float mean, float var) { return mean * mean > kLnFar<T> * var; }

// f(column, element) for the columns of row x that thread tid of `threads` takes,
// eight loads ahead of their use.
template <typename T, typename F>
__device__ __forceinline__ void each_element(const T* x, int D, int tid, int threads, F f) {
#pragma unroll 1
  for (int c = tid; c < D; c += 8 * threads) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = Elem<T>::to_f(x[min(c + k * threads, D - 1)]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k * threads < D) f(c + k * threads, v[k]);
  }
}

// The same for rows on 16-byte boundaries, without the columns: four chunks of V
// elements ahead.
template <typename T, int V, typename F>
__device__ __forceinline__ void each_of(const T* x, int D, int tid, int threads, F f) {
  if constexpr (V == 1) {
    each_element(x, D, tid, threads, [&](int, float v) { f(v); });
  } else {
    const int n = D / V;
#pragma unroll 1
    for (int c = tid; c < n; c += 4 * threads) {
      uint4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = ldg128_nc(x + (int64_t)min(c + k * threads, n - 1) * V);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k * threads < n) {
          float v[V];
          unpack16<T, V>(u[k], v);
#pragma unroll
          for (int e = 0; e < V; ++e) f(v[e]);
        }
    }
  }
}

// The second mean and the variance about it, from the row in memory, so that the
// common path keeps no register for them.  With no row far 8000 x 5003 bf16 runs
// 49.9 us (48.3 without any of this, 54.3 with it from the registers' copy of the
// row, 51.8 not out of line) and 8192 x 4096 bf16 24.0 (23.9); with every row far
// 8192 x 4096 takes 57 us in bf16 and 104 in fp32.  sum(v, i): the row's sum of v,
// the i-th asked for.
template <typename T, int V, typename S>
__device__ __forceinline__ void refine(const T* x, int D, int tid, int threads, float inv_d, S sum, float* mean, float* var) {
  float m = *mean, s = 0.0f;
  each_of<T, V>(x, D, tid, threads, [&](float v) { s += v - m; });
  m += sum(s, 0) * inv_d;
  s = 0.0f;
  each_of<T, V>(x, D, tid, threads, [&](float v) { s = fmaf(v - m, v - m, s); });
  *var = sum(s, 1) * inv_d;
  *mean = m;
}

// A row lives in the registers of its tpr threads (chunk j of thread t holds
// columns V * (t + j * tpr) ..), so x is read once and the centred sum of
// squares is taken about the exact row mean: no cancellation when |mean| is
// far above the deviation.  One row a warp for tpr = 32, else one row a CTA.
template <typename T, int V, int J, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) ln_fwd_kernel(const LnFwdArgs A) {
  __shared__ float red[2][32];
  const int tid = A.tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int warp = threadIdx.x >> 5, nwarp = A.tpr >> 5;
  const int rows_per_cta = blockDim.x / A.tpr;
  const int nchunk = A.D / V;
  const float inv_d = 1.0f / (float)A.D;
  const T* gamma = static_cast<const T*>(A.gamma);
  const T* beta = static_cast<const T*>(A.beta);
  griddep_wait();
  griddep_launch_dependents();

  // Sum over the row's threads, the same order in every thread.
  auto row_sum = [&](float s, int slot) {
    s = warp_sum(s);
    if (nwarp > 1) {
      if ((threadIdx.x & 31) == 0) red[slot][warp] = s;
      __syncthreads();
      s = red[slot][0];
      for (int w = 1; w < nwarp; ++w) s += red[slot][w];
    }
    return s;
  };

  const int64_t step = (int64_t)gridDim.x * rows_per_cta;
  for (int64_t row = (int64_t)blockIdx.x * rows_per_cta + (nwarp == 1 ? warp : 0); row < A.T; row += step) {
    const T* x = static_cast<const T*>(A.x) + row * A.ld_x;
    float v[J][V];
    float s = 0.0f;
    // Chunks past the end read the last one and count as zero: loads without a
    // branch around each, so that they are all in flight together.
#pragma unroll
    for (int j = 0; j < J; ++j) load_chunk<T, V>(x + (int64_t)min(tid + j * A.tpr, nchunk - 1) * V, v[j]);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (tid + j * A.tpr >= nchunk) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] = 0.0f;
      }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[j][e];
    float mean = row_sum(s, 0) * inv_d;
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (tid + j * A.tpr < nchunk) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[j][e] -= mean;
          q = fmaf(v[j][e], v[j][e], q);
        }
      }
    float var = row_sum(q, 1) * inv_d;
    if (far_mean<T>(mean, var)) {
      const float first = mean;
      refine<T, V>(x, A.D, tid, A.tpr, inv_d, row_sum, &mean, &var);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] -= mean - first;
    }
    const float rstd = rsqrtf(var + A.eps);
    if (tid == 0) {
      if (A.mean) A.mean[row] = mean;
      if (A.rstd) A.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(A.y) + row * (int64_t)A.D;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) v[j][e] *= rstd;
    if (gamma) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float g[V];
        load_chunk<T, V>(gamma + min(tid + j * A.tpr, nchunk - 1) * V, g);
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] *= g[e];
      }
    }
    if (beta) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float b[V];
        load_chunk<T, V>(beta + min(tid + j * A.tpr, nchunk - 1) * V, b);
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] += b[e];
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (tid + j * A.tpr < nchunk) store_chunk<T, V>(y + (int64_t)(tid + j * A.tpr) * V, v[j]);
  }
}

// Rows of single elements too long for a ring: a CTA a row reads it three times,
// the second and third time from the caches, eight loads in flight a thread
// (2000 x 32767: bf16 212 us, fp32 231; held in registers they spilled, 647 and
// 678).
constexpr int kLnLongThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kLnLongThreads, 1) ln_fwd_long_kernel(const LnFwdArgs A) {
  __shared__ float red[2][32];
  const int D = A.D, tid = threadIdx.x;
  const float inv_d = 1.0f / (float)D;
  const T* gamma = static_cast<const T*>(A.gamma);
  const T* beta = static_cast<const T*>(A.beta);
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t row = blockIdx.x; row < A.T; row += gridDim.x) {
    const T* x = static_cast<const T*>(A.x) + row * A.ld_x;
    T* y = static_cast<T*>(A.y) + row * (int64_t)D;
    auto each = [&](auto f) { each_element(x, D, tid, kLnLongThreads, f); };
    auto row_sum = [&](float s, int slot) {
      s = warp_sum(s);
      if ((tid & 31) == 0) red[slot][tid >> 5] = s;
      __syncthreads();
      s = red[slot][0];
      for (int w = 1; w < kLnLongThreads / 32; ++w) s += red[slot][w];
      return s;
    };
    float s = 0.0f, q = 0.0f;
    each([&](int, float v) { s += v; });
    float mean = row_sum(s, 0) * inv_d;
    each([&](int, float v) { q = fmaf(v - mean, v - mean, q); });
    float var = row_sum(q, 1) * inv_d;
    if (far_mean<T>(mean, var)) refine<T, 1>(x, D, tid, kLnLongThreads, inv_d, row_sum, &mean, &var);
    const float rstd = rsqrtf(var + A.eps);
    if (tid == 0) {
      if (A.mean) A.mean[row] = mean;
      if (A.rstd) A.rstd[row] = rstd;
    }
    each([&](int c, float v) {
      v = (v - mean) * rstd;
      if (gamma) v *= Elem<T>::to_f(gamma[c]);
      if (beta) v += Elem<T>::to_f(beta[c]);
      y[c] = Elem<T>::from_f(v);
    });
  }
}

// The same for many rows: persistent CTAs whose row groups (whole warps) take
// their rows from a ring of shared-memory stages, filled by bulk copies that
// the group's first thread issues.  The row goes to registers at once and its
// stage is refilled behind the barrier of the first reduction, so a ring's
// worth of rows is in flight whatever phase the groups are in.  gamma and beta
// stay in shared memory, as stored.  A warp owns 32 * J consecutive chunks, so
// a lane's chunks are a constant apart.
//
// V elements a chunk: 16 bytes, kept packed (most elements a lane, so that one
// warp holds a row of up to 4096 16-bit elements: the two reductions are then
// five shuffles each and no barrier.  8192 x 4096 bf16 ran 23.6 us with one
// warp a row, 34.9 with four).  Rows that do not all start on 16-byte
// boundaries take V = 1: a copy covers the aligned window around the row, and
// a lane reads single elements, 32 apart.
struct LnFwdRing {
  LnFwdArgs A;
  unsigned* status;
  int ng, stages;                          // row groups per CTA, ring depth per group
  uint32_t slot_bytes;                     // of a stage
  uint32_t par_off, par_bytes;             // gamma, then beta
  uint32_t bar_off, red_off;               // shared-memory offsets (the rings at 0)
};

// The 16-byte window around elements [0, D) of `src`, a row of a tensor that
// ends at `end`: returns the bytes of it that a bulk copy may fetch from the
// window's start (src rounded down to 16).  Elements past the last 16 bytes
// that lie whole in the tensor are written to the slot here, ahead of the
// barrier arrival that publishes them.
template <typename T>
__device__ __forceinline__ uint32_t row_window(uint8_t* slot, const T* src, int D, const T* end) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15;
  uintptr_t b = (reinterpret_cast<uintptr_t>(src + D) + 15) & ~(uintptr_t)15;
  if (b > reinterpret_cast<uintptr_t>(end)) {
    b = reinterpret_cast<uintptr_t>(end) & ~(uintptr_t)15;
    for (const T* p = reinterpret_cast<const T*>(b); p < src + D; ++p)
      *reinterpret_cast<T*>(slot + (reinterpret_cast<uintptr_t>(p) - a)) = *p;
  }
  return (uint32_t)(b - a);
}

// The bulk copy of that window (none when no 16 bytes of it lie in the tensor).
template <typename T>
__device__ __forceinline__ void copy_window(uint8_t* slot, const T* src, uint32_t bytes, uint64_t* bar, uint64_t pol) {
  if (bytes)
    bulk_copy_g2s(slot, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15), bytes, bar, pol);
}

// After a wait gave up, leave no copy in flight: the thread that fetched `issued`
// rows (and fetches none once its wait gave up, since that stage's barrier is still
// armed) waits, bounded, for the last phase of every stage.
__device__ __forceinline__ void drain(uint64_t* full, int stages, int64_t issued, unsigned* status) {
  for (int64_t k = issued > stages ? issued - stages : 0; k < issued; ++k)
    mbar_wait_bounded(&full[k % stages], (uint32_t)(k / stages) & 1u, status);
}

// gamma or beta to shared memory as stored (16-byte aligned at both ends), by
// the whole CTA; a constant when there is none.
template <typename T>
__device__ __forceinline__ void stage_params(uint8_t* dst, const T* src, int D, float fill) {
  constexpr int V = 16 / sizeof(T);
  T* d = reinterpret_cast<T*>(dst);
  if (!src) {
    for (int c = threadIdx.x; c < D; c += blockDim.x) d[c] = Elem<T>::from_f(fill);
    return;
  }
  for (int c = threadIdx.x; c < D / V; c += 4 * blockDim.x) {          // four loads in flight
    uint4 t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = ldg128_nc(src + min(c + k * (int)blockDim.x, D / V - 1) * V);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k * (int)blockDim.x < D / V) sts128(smem_u32(d + (c + k * (int)blockDim.x) * V), t[k]);
  }
  for (int c = D / V * V + threadIdx.x; c < D; c += blockDim.x) d[c] = src[c];
}

// Threads of the ring kernel.  Registers are dealt by the warps of an SM's
// quarter: 255 a thread for up to 8 warps, which 14 and 16 chunks a lane need
// (8192 x 8192 bf16: 45.5 us, 49.6 with 12 warps), 168 for up to 12; shorter rows
// ran best at 14 warps (8192 x 2048: 14.1, 14.9 with 16), single elements at 20
// (8000 x 5003 bf16: 48.7, 53.6 with 16).
__host__ __device__ constexpr int ln_fwd_threads(int v, int j) {
  return v == 1 ? 640 : (j >= 14 ? 256 : j >= 10 ? 384 : 448);
}

// refine() over a row group of the ring kernel, out of line.
template <typename T, int V>
__device__ __noinline__ float2 refine_group(const T* x, int D, int tid, int threads, float mean, uint32_t red, int barrier) {
  float var;
  refine<T, V>(x, D, tid, threads, 1.0f / (float)D,
               [&](float v, int i) { return group_sum(v, red + 128u * i, threads >> 5, barrier); }, &mean, &var);
  return make_float2(mean, var);
}

template <typename T, int V, int J, bool FULL>
__global__ void __launch_bounds__(ln_fwd_threads(V, J), 1) ln_fwd_ring_kernel(const LnFwdRing R) {
  extern __shared__ __align__(128) uint8_t smem[];
  const LnFwdArgs& A = R.A;
  const int group = threadIdx.x / A.tpr;
  const int tid = threadIdx.x - group * A.tpr;
  const int nwarp = A.tpr >> 5;
  const int c0 = (tid >> 5) * 32 * J + (tid & 31);                   // this lane's first chunk
  const int nchunk = A.D / V;
  const bool all = FULL || (tid >> 5) * 32 * J + 32 * J <= nchunk;   // every chunk of this warp lies in the row
  const float inv_d = 1.0f / (float)A.D;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R.bar_off) + group * R.stages;
  const uint32_t red = smem_u32(smem) + R.red_off + (uint32_t)group * 256u;
  uint8_t* ring = smem + (size_t)(group * R.stages) * R.slot_bytes;
  const uint32_t params = smem_u32(smem) + R.par_off;

  if (tid == 0) {
    for (int s = 0; s < R.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  for (int k = tid; k < 64; k += A.tpr) reinterpret_cast<float*>(smem + R.red_off)[group * 64 + k] = 0.0f;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t g0 = (int64_t)group * gridDim.x + blockIdx.x, gstep = (int64_t)gridDim.x * R.ng;
  const int64_t n = g0 < A.T ? (A.T - g0 + gstep - 1) / gstep : 0;   // rows of this group
  const uint64_t pol = policy_evict_first();
  const T* x0 = static_cast<const T*>(A.x);
  const T* next = x0 + g0 * A.ld_x;                                  // next row to fetch
  int64_t left = n;                                                  // rows to fetch (first thread)
  auto refill = [&](int s) {
    uint8_t* slot = ring + (size_t)s * R.slot_bytes;
    if constexpr (V == 1) {
      const uint32_t bytes = row_window<T>(slot, next, A.D, x0 + (A.T - 1) * A.ld_x + A.D);
      mbar_arrive_expect_tx(&full[s], bytes);
      copy_window(slot, next, bytes, &full[s], pol);
    } else {
      mbar_arrive_expect_tx(&full[s], R.slot_bytes);
      bulk_copy_g2s(slot, next, R.slot_bytes, &full[s], pol);
    }
    next += gstep * A.ld_x;
    --left;
  };
  if (tid == 0)
    for (int s = 0; s < R.stages && left > 0; ++s) refill(s);
  stage_params<T>(smem + R.par_off, static_cast<const T*>(A.gamma), A.D, 1.0f);
  stage_params<T>(smem + R.par_off + R.par_bytes, static_cast<const T*>(A.beta), A.D, 0.0f);
  __syncthreads();

  bool ok = true;
  int s = 0;
  uint32_t ph = 0;
  T* y = static_cast<T*>(A.y) + g0 * (int64_t)A.D + (size_t)c0 * V;
  for (int64_t i = 0, row = g0; i < n; ++i, row += gstep) {
    if (ok) ok = mbar_wait_bounded(&full[s], ph, R.status);
    RowPart<T, V, J> v;
    // where element 0 of the row lies in its stage
    const uint32_t src = smem_u32(ring + (size_t)s * R.slot_bytes) +
                         (V == 1 ? (uint32_t)(reinterpret_cast<uintptr_t>(x0 + row * A.ld_x) & 15) : 0u);
    float sum = all ? v.template load_sum<true>(src, c0, nchunk) : v.template load_sum<false>(src, c0, nchunk);
    fence_proxy_async_smem();              // these reads before the refill's bulk copy
    float mean = group_sum(sum, red, nwarp, 1 + group) * inv_d;
    if (nwarp == 1) __syncwarp();
    if (tid == 0 && ok && left > 0) refill(s);
    if (++s == R.stages) { s = 0; ph ^= 1u; }
    sum = all ? v.template squares<true>(mean, c0, nchunk) : v.template squares<false>(mean, c0, nchunk);
    float var = group_sum(sum, red + 128u, nwarp, 1 + group) * inv_d;
    if (far_mean<T>(mean, var)) {
      const float first = mean;
      const float2 mv = refine_group<T, V>(x0 + row * A.ld_x, A.D, tid, A.tpr, mean, red, 1 + group);
      mean = mv.x;
      var = mv.y;
      v.shift(mean - first);
    }
    const float rstd = rsqrtf(var + A.eps);
    if (tid == 0) {
      if (A.mean) A.mean[row] = mean;
      if (A.rstd) A.rstd[row] = rstd;
    }
    if (all) v.template store<true>(y, mean, rstd, params, params + R.par_bytes, c0, nchunk);
    else v.template store<false>(y, mean, rstd, params, params + R.par_bytes, c0, nchunk);
    y += gstep * A.D;
  }
  if (tid == 0 && !ok) drain(full, R.stages, n - left, R.status);
}

// ------------------------------------------------------------------- backward

constexpr int kLnRedSlots = 32;          // warps per group, at most

struct LnBwdArgs {
  const void* x;
  const void* dy;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;        // fp32 [gridDim.x, 2, part_ld] (dgamma, dbeta sums of the CTA's rows), or null
  int64_t T, ld_x, ld_dy;
  unsigned* status;
  int D, part_ld;
  int tpr, ng, stages;   // threads per row group, row groups per CTA, ring depth per group
  uint32_t slot_bytes;   // of an x row, and of a dy row, in a stage
  uint32_t par_off, red_off, bar_off;               // shared-memory offsets (the rings at 0)
};

// Threads: 32 columns a thread cost 64 registers of sums.  With the row kept
// packed in 32 more, 384 threads (168 registers) fit; without, 512.
__host__ __device__ constexpr int ln_bwd_threads(bool keep) { return keep ? 384 : 512; }

// Row groups as in the forward's ring kernel; a stage holds a row of x and one
// of dy.  A thread keeps the dgamma and dbeta sums of its columns in registers
// over all the rows its group sees.  A row takes two passes: the sums of g and
// g * xh (and the column sums), then dx.  KEEP: the row stays in registers,
// packed, between the passes, and its stage is refilled behind the barrier of
// the reduction; otherwise the second pass reads the stage again and the
// barrier frees the row before (a ring of one stage has a barrier of its own).
// Measured at 8192 x 4096 bf16: 60.8 us with scalar arithmetic, 60.1 with a pass
// of row sums by warps and one of columns by all threads (32 instructions an
// element), 47.6 as here, 40.4 once the groups' column sums were folded side by
// side instead of in turn with conflicting banks.
// xh is the difference scaled, (x - mean) * rstd: as x * rstd - mean * rstd it takes
// an instruction less, but then the rounding of mean * rstd shifts the whole row, by
// 1e-5 where the mean is 1000 deviations away and 1e-3 at 100000.
// V = 16 / sizeof(T) elements a chunk, or 1 when rows do not all start on
// 16-byte boundaries.  gamma lies in shared memory as fp32, for V = 8 in two
// planes of four columns a chunk, so that lanes read 16 consecutive bytes.
template <typename T, int V, int J, bool KEEP>
__global__ void __launch_bounds__(ln_bwd_threads(KEEP), 1) ln_bwd_kernel(const LnBwdArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int W = V == 1 ? 1 : V / 2;
  const int group = threadIdx.x / A.tpr;
  const int tid = threadIdx.x - group * A.tpr;
  const int nwarp = A.tpr >> 5;
  const int c0 = (tid >> 5) * 32 * J + (tid & 31);                   // this lane's first chunk
  const int D = A.D, nchunk = D / V;
  const bool all = (tid >> 5) * 32 * J + 32 * J <= nchunk;           // every chunk of this warp lies in the row
  const float inv_d = 1.0f / (float)D;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + A.bar_off) + group * A.stages;
  uint8_t* ring = smem + (size_t)(group * A.stages) * 2 * A.slot_bytes;
  float2* red = reinterpret_cast<float2*>(smem + A.red_off) + group * 2 * kLnRedSlots;
  float* gs = reinterpret_cast<float*>(smem + A.par_off);
  const T* x0 = static_cast<const T*>(A.x);
  const T* y0 = static_cast<const T*>(A.dy);

  if (tid == 0) {
    for (int s = 0; s < A.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  const int64_t g0 = (int64_t)group * gridDim.x + blockIdx.x, gstep = (int64_t)gridDim.x * A.ng;
  const int64_t n = g0 < A.T ? (A.T - g0 + gstep - 1) / gstep : 0;   // rows of this group
  const uint64_t pol = policy_evict_first();
  int64_t next = g0;                                                 // next row to fetch (first thread)
  auto refill = [&](int s) {
    uint8_t* xs = ring + (size_t)s * 2 * A.slot_bytes;
    uint8_t* ys = xs + A.slot_bytes;
    const T* x = x0 + next * A.ld_x;
    const T* y = y0 + next * A.ld_dy;
    if constexpr (V == 1) {
      const uint32_t xb = row_window<T>(xs, x, D, x0 + (A.T - 1) * A.ld_x + D);
      const uint32_t yb = row_window<T>(ys, y, D, y0 + (A.T - 1) * A.ld_dy + D);
      mbar_arrive_expect_tx(&full[s], xb + yb);
      copy_window(xs, x, xb, &full[s], pol);
      copy_window(ys, y, yb, &full[s], pol);
    } else {
      mbar_arrive_expect_tx(&full[s], 2 * A.slot_bytes);
      bulk_copy_g2s(xs, x, A.slot_bytes, &full[s], pol);
      bulk_copy_g2s(ys, y, A.slot_bytes, &full[s], pol);
    }
    next += gstep;
  };
  if (tid == 0)
    for (int s = 0; s < A.stages && next < A.T; ++s) refill(s);
  {
    constexpr int VG = 16 / sizeof(T);
    const T* gamma = static_cast<const T*>(A.gamma);
    auto put = [&](int col, float v) { gs[V == 8 ? (col & 4) * (D / 8) + col / 8 * 4 + (col & 3) : col] = v; };
    const int whole = gamma ? D / VG : 0;
    for (int c = threadIdx.x; c < whole; c += 4 * blockDim.x) {        // four loads in flight
      uint4 t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = ldg128_nc(gamma + min(c + k * (int)blockDim.x, whole - 1) * VG);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int cc = c + k * (int)blockDim.x;
        float f[VG];
        unpack16<T, VG>(t[k], f);
        if (cc < whole) {
#pragma unroll
          for (int e = 0; e < VG; ++e) put(cc * VG + e, f[e]);
        }
      }
    }
    for (int c = whole * VG + threadIdx.x; c < D; c += blockDim.x) put(c, gamma ? Elem<T>::to_f(gamma[c]) : 1.0f);
  }
  float2 dgam[J][W], dbet[J][W];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < W; ++e) dgam[j][e] = dbet[j][e] = make_float2(0.0f, 0.0f);
  __syncthreads();

  const uint32_t params = smem_u32(gs);
  auto chunk_gamma = [&](int c, float2 (&g)[W]) {
    if constexpr (V == 1) {
      g[0].x = lds_elem<float>(params + 4u * c);
    } else {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const uint4 u = lds128(params + (uint32_t)k * 2u * D + 16u * c);
        g[2 * k] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        g[2 * k + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
      }
    }
  };

  bool ok = true;
  int s = 0;
  uint32_t ph = 0;
  float m_next = n > 0 ? A.mean[g0] : 0.0f, r_next = n > 0 ? A.rstd[g0] : 0.0f;
  T* dx = static_cast<T*>(A.dx) + g0 * (int64_t)D + (size_t)c0 * V;
  for (int64_t i = 0, row = g0; i < n; ++i, row += gstep) {
    const float a = r_next, b = -m_next;                             // xh = (x + b) a
    if (i + 1 < n) {
      m_next = A.mean[row + gstep];
      r_next = A.rstd[row + gstep];
    }
    if (ok) ok = mbar_wait_bounded(&full[s], ph, A.status);
    // element 0 of the row in its stage
    uint32_t xs = smem_u32(ring + (size_t)s * 2 * A.slot_bytes), ys = xs + A.slot_bytes;
    if constexpr (V == 1) {
      xs += (uint32_t)(reinterpret_cast<uintptr_t>(x0 + row * A.ld_x) & 15);
      ys += (uint32_t)(reinterpret_cast<uintptr_t>(y0 + row * A.ld_dy) & 15);
    }
    const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
    uint4 xk[KEEP ? J : 1], yk[KEEP ? J : 1];
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    auto pass1 = [&](auto whole) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = c0 + 32 * j;
      if (decltype(whole)::value || c < nchunk) {
        float2 xv[W], yv[W], gv[W];
        chunk_gamma(c, gv);
        if constexpr (V == 1) {
          const float xh = (lds_elem<T>(xs + (uint32_t)sizeof(T) * c) + b) * a;
          const float y = lds_elem<T>(ys + (uint32_t)sizeof(T) * c), g = y * gv[0].x;
          s1.x += g;
          s2.x = fmaf(g, xh, s2.x);
          dgam[j][0].x = fmaf(y, xh, dgam[j][0].x);
          dbet[j][0].x += y;
        } else {
          const uint4 xu = lds128(xs + 16u * c), yu = lds128(ys + 16u * c);
          if constexpr (KEEP) {
            xk[j] = xu;
            yk[j] = yu;
          }
          unpack2<T>(xu, xv);
          unpack2<T>(yu, yv);
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float2 xh = mul2(add2(xv[e], b2), a2), g = mul2(yv[e], gv[e]);
            s1 = add2(s1, g);
            s2 = fma2(g, xh, s2);
            dgam[j][e] = fma2(yv[e], xh, dgam[j][e]);
            dbet[j][e] = add2(dbet[j][e], yv[e]);
          }
        }
      }
    }
    };
    if (all) pass1(std::true_type{});
    else pass1(std::false_type{});
    if constexpr (KEEP) fence_proxy_async_smem();      // these reads before the refill's bulk copies
    float t1 = warp_sum(V == 1 ? s1.x : s1.x + s1.y), t2 = warp_sum(V == 1 ? s2.x : s2.x + s2.y);
    if (nwarp > 1) {
      float2* slot = red + (i & 1) * kLnRedSlots;
      if ((tid & 31) == 0) slot[tid >> 5] = make_float2(t1, t2);
      named_barrier_sync(1 + group, A.tpr);
      t1 = t2 = 0.0f;
      for (int w = 0; w < nwarp; ++w) {
        t1 += slot[w].x;
        t2 += slot[w].y;
      }
    } else {
      __syncwarp();
    }
    // dx = a (g - c1 - (x + b) a c2)
    const float n1 = -t1 * inv_d, n2 = -a * (t2 * inv_d);
    if (tid == 0 && ok && next < A.T) {
      if (KEEP) refill(s);
      else if (A.stages > 1 && i > 0) refill(s == 0 ? A.stages - 1 : s - 1);
    }
    const float2 n12 = make_float2(n1, n1), n22 = make_float2(n2, n2);
    auto pass2 = [&](auto whole) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = c0 + 32 * j;
      if (decltype(whole)::value || c < nchunk) {
        float2 xv[W], yv[W], gv[W];
        chunk_gamma(c, gv);
        if constexpr (V == 1) {
          const float xc = lds_elem<T>(xs + (uint32_t)sizeof(T) * c) + b;
          const float y = lds_elem<T>(ys + (uint32_t)sizeof(T) * c);
          dx[32 * j] = Elem<T>::from_f(fmaf(y, gv[0].x, fmaf(xc, n2, n1)) * a);
        } else {
          unpack2<T>(KEEP ? xk[KEEP ? j : 0] : lds128(xs + 16u * c), xv);
          unpack2<T>(KEEP ? yk[KEEP ? j : 0] : lds128(ys + 16u * c), yv);
#pragma unroll
          for (int e = 0; e < W; ++e)
            xv[e] = mul2(fma2(yv[e], gv[e], fma2(add2(xv[e], b2), n22, n12)), a2);
          stg128_stream(dx + (size_t)32 * j * V, pack2<T>(xv));
        }
      }
    }
    };
    if (all) pass2(std::true_type{});
    else pass2(std::false_type{});
    if constexpr (!KEEP) {
      fence_proxy_async_smem();
      if (A.stages == 1) {
        if (nwarp > 1) named_barrier_sync(1 + group, A.tpr);
        else __syncwarp();
        if (tid == 0 && ok && next < A.T) refill(0);
      }
    }
    dx += gstep * D;
    if (++s == A.stages) { s = 0; ph ^= 1u; }
  }

  if (tid == 0 && !ok) drain(full, A.stages, (next - g0) / gstep, A.status);

  if (!A.partial) return;
  // The CTA's sums: every group lays its own out in shared memory (each copy
  // has landed), then the columns are added up in group order and one row goes out.
  __syncthreads();
  float* acc = reinterpret_cast<float*>(smem);                       // [ng, 2, part_ld]
  const int ld = A.part_ld;
  float* mine = acc + (size_t)group * 2 * ld;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = c0 + 32 * j;
    if (c < nchunk) {
      if constexpr (V == 1) {
        mine[c] = dgam[j][0].x;
        mine[ld + c] = dbet[j][0].x;
      } else {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) {
          const float2 *g = &dgam[j][2 * k], *b = &dbet[j][2 * k];
          *reinterpret_cast<float4*>(mine + c * V + 4 * k) = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
          *reinterpret_cast<float4*>(mine + ld + c * V + 4 * k) = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
        }
      }
    }
  }
  __syncthreads();
  float* out = A.partial + (size_t)blockIdx.x * 2 * ld;
  for (int c = 4 * threadIdx.x; c < 2 * ld; c += 4 * blockDim.x) {
    float4 t = *reinterpret_cast<const float4*>(acc + c);
    for (int g = 1; g < A.ng; ++g) {
      const float4 u = *reinterpret_cast<const float4*>(acc + (size_t)g * 2 * ld + c);
      t.x += u.x;
      t.y += u.y;
      t.z += u.z;
      t.w += u.w;
    }
    *reinterpret_cast<float4*>(out + c) = t;
  }
}

// Adds the CTAs' partial rows [rows, 2, ld] in a fixed order: a block takes 32
// columns, four a lane, in 32 slices of rows, joined in slice order.
constexpr int kLnSlices = 32;
template <typename T>
__global__ void __launch_bounds__(8 * kLnSlices) ln_dgamma_kernel(const float* partial, int rows, int D, int ld,
                                                                  void* dgamma, void* dbeta) {
  __shared__ float4 part[kLnSlices][8];
  const int lane = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * lane;                        // of the 2 * ld: dgamma, then dbeta
  griddep_wait();
  griddep_launch_dependents();
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < 2 * ld) {
#pragma unroll 8
    for (int r = slice; r < rows; r += kLnSlices) {
      const float4 v = *reinterpret_cast<const float4*>(partial + (size_t)r * 2 * ld + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  part[slice][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int c = blockIdx.x * 32 + (int)threadIdx.x;                  // one column a thread from here on
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < kLnSlices; ++k) t += reinterpret_cast<const float*>(part[k])[threadIdx.x];
  T* out = static_cast<T*>(c < ld ? dgamma : dbeta);
  const int o = c < ld ? c : c - ld;
  if (out && o < D) out[o] = Elem<T>::from_f(t);
}

// ------------------------------------------------------------------- launches

int round32(int v) { return (v + 31) / 32 * 32; }

// Columns of a partial row: D up to a 16-byte multiple.
int part_ld(int D) { return (D + 3) / 4 * 4; }

// The kernel of rows that plan_fwd_ring leaves or fwd() keeps from it: up to 32
// elements a thread, a warp a row while that covers it.  16-bit packed
// rows come here with at most 32 chunks, single elements with at most 256 or
// rows too long for a ring.
template <typename T>
const void* fwd_kernel(bool vec, int chunks, int* tpr) {
  constexpr int V = 16 / sizeof(T);
  auto threads = [&](int j) { return round32((chunks + j - 1) / j); };
  *tpr = 32;
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      if (chunks > 64) {
        const int j = threads(4) <= 1024 ? 4 : 8;
        *tpr = threads(j);
        return j == 4 ? (const void*)ln_fwd_kernel<T, V, 4, 1024> : (const void*)ln_fwd_kernel<T, V, 8, 1024>;
      }
      if (chunks > 32) return (const void*)ln_fwd_kernel<T, V, 2, 1024>;
    }
    return (const void*)ln_fwd_kernel<T, V, 1, 1024>;
  }
  if (chunks <= 256) return (const void*)ln_fwd_kernel<T, 1, 8, 256>;
  *tpr = kLnLongThreads;
  return (const void*)ln_fwd_long_kernel<T>;
}

// Chunks a lane of the ring kernel holds, at most: a warp then covers 4096
// 16-bit or 1024 fp32 elements.
template <typename T> constexpr int kLnFwdMost = sizeof(T) == 4 ? 8 : 16;

// The ring kernel of j chunks a lane, j = 1, 2 or a greater even number.
template <typename T, int J = 1>
const void* fwd_ring_of(int j, bool full) {
  constexpr int V = 16 / sizeof(T), next = J == 1 ? 2 : J + 2;
  if constexpr (next <= kLnFwdMost<T>)
    if (j > J) return fwd_ring_of<T, next>(j, full);
  return full ? (const void*)ln_fwd_ring_kernel<T, V, J, true> : (const void*)ln_fwd_ring_kernel<T, V, J, false>;
}

template <typename T>
bool plan_fwd_ring(LnFwdRing& R, bool vec, int sms, const void** kernel, int* threads, int* grid, size_t* smem) {
  constexpr int V = 16 / sizeof(T);
  const int chunks = vec ? R.A.D / V : R.A.D;
  const size_t cap = 227 * 1024, row_bytes = sizeof(T) * (size_t)R.A.D;
  R.slot_bytes = (uint32_t)(vec ? row_bytes : (row_bytes + 15) / 16 * 16 + 16);
  R.par_bytes = (uint32_t)((row_bytes + 15) / 16 * 16);
  auto total = [&](int groups, int stages) {
    return 2 * (size_t)R.par_bytes + 144 + (size_t)groups * (stages * (R.slot_bytes + sizeof(uint64_t)) + 64 * sizeof(float));
  };
  const int64_t want = (R.A.T + sms - 1) / sms;    // few rows: spread them over the SMs
  auto warps_of = [&](int j) { return (chunks + j * 32 - 1) / (j * 32); };
  auto groups_of = [&](int j) {
    int n = ln_fwd_threads(vec ? V : 1, j) / (32 * warps_of(j));
    if (warps_of(j) > 1 && n > 15) n = 15;         // named barriers 1..15
    if (want < n) n = (int)want;
    // a deep ring before a fifth group (8192 x 4096 bf16: 26.3 us with 9 groups of 2 stages, 24.0 with 8 of 3)
    while (n > 1 && total(n, n > 4 ? 3 : 1) > cap) --n;
    return n;
  };
  // Chunks a lane, by the rounds of rows and the time of one, fitted to what was
  // measured: the SM takes 25 ns for each 32 chunks or empty places for them (21
  // with the registers of 14 and 16 a lane, which a ragged end slows down by
  // 0.9 us), a row alone 0.9 us and 0.055 for each of a lane's chunks; 0.2 us
  // more for the barriers of several warps.  8192 x 5120 bf16 runs 31.1 us with
  // 10 chunks a lane and ran 57.8 with 16, 8192 x 12288 67 with 16 and 75 with 12.
  int j = 32, ng = 0;                              // single elements: rows of more than 256
  if (vec) {
    double best = 0.0;
    for (int k = 1; k <= kLnFwdMost<T>; k += k == 1 ? 1 : 2) {
      const int n = groups_of(k);
      if (n < 1) continue;
      const int warps = warps_of(k);
      const double busy = (k >= 14 ? 0.0215 : 0.0245) * n * warps * k + 0.2, alone = 0.9 + 0.055 * k;
      const double t = (double)((want + n - 1) / n) * ((busy > alone ? busy : alone) + (warps > 1 ? 0.2 : 0.0) +
                                                       (k >= 14 && chunks % (32 * k) ? 0.9 : 0.0));
      if (ng == 0 || t < best) { best = t; j = k; ng = n; }
    }
  } else {
    ng = groups_of(j);
  }
  if (ng < 1) return false;
  *kernel = vec ? fwd_ring_of<T>(j, chunks % (32 * j) == 0) : (const void*)ln_fwd_ring_kernel<T, 1, 32, false>;
  R.A.tpr = 32 * warps_of(j);
  int stages = 4;
  while (stages > 1 && total(ng, stages) > cap) --stages;
  if (total(ng, stages) > cap) return false;
  R.ng = ng;
  R.stages = stages;
  R.par_off = (uint32_t)((size_t)ng * stages * R.slot_bytes);
  R.bar_off = (R.par_off + 2 * R.par_bytes + 127) / 128 * 128;
  R.red_off = R.bar_off + (uint32_t)((ng * stages * sizeof(uint64_t) + 15) / 16 * 16);
  *smem = R.red_off + (size_t)ng * 64 * sizeof(float);
  *threads = ng * R.A.tpr;
  const int64_t g = (R.A.T + ng - 1) / ng;
  *grid = (int)(g < sms ? g : sms);
  return true;
}

template <typename T>
int fwd(LnFwdArgs& A, int sms, unsigned* status, cudaStream_t stream, const char** why) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = A.D % V == 0 && A.ld_x % V == 0;
  // Rows over the ring or straight to registers.  Measured (us, ring / direct):
  // bf16 64 x 1024 2.6 / 2.9, 500 x 4096 3.7 / 4.0, 8192 x 4096 24.1 / 31.9,
  // 8192 x 8192 46.4 / 58, but 4000 x 256 3.5 / 2.2 (one chunk a lane: nothing
  // to overlap); fp32 500 x 4096 4.0 / 4.2, 1000 x 4096 8.3 / 7.2, 8192 x 4096
  // 45.9 / 49.1; single elements 3001 x 5003 fp32 26.5 / 66, 8000 x 1001 bf16
  // 11.3 / 24.0, 3001 x 251 4.4 / 4.0.
  if (vec ? A.D > 32 * V && (sizeof(T) == 2 || A.T >= 8 * (int64_t)sms) : A.D > 256) {
    LnFwdRing R{};
    R.A = A;
    R.status = status;
    const void* k;
    int threads, grid;
    size_t smem;
    if (plan_fwd_ring<T>(R, vec, sms, &k, &threads, &grid, &smem)) {
      void* argv[] = {&R};
      return launch_kernel(k, grid, threads, smem, argv, stream, "layernorm_fwd launch", why);
    }
  }
  const void* k = fwd_kernel<T>(vec, vec ? A.D / V : A.D, &A.tpr);
  int threads = A.tpr;
  if (A.tpr == 32) {                       // warps a CTA: up to 8, fewer while rows leave SMs idle
    int64_t rpc = A.T / sms;
    rpc = rpc < 1 ? 1 : (rpc > 8 ? 8 : rpc);
    threads = 32 * (int)rpc;
  }
  const int rpc = threads / A.tpr;
  int64_t grid = (A.T + rpc - 1) / rpc;
  if (grid > 0x7FFFFFFF) grid = 0x7FFFFFFF;
  void* argv[] = {&A};
  return launch_kernel(k, grid, threads, 0, argv, stream, "layernorm_fwd launch", why);
}

struct LnBwdPlan {
  const void* kernel;
  int threads, grid;
  size_t smem;
};

template <typename T>
bool plan_bwd(LnBwdArgs& A, int sms, LnBwdPlan* P) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = A.D % V == 0 && A.ld_x % V == 0 && A.ld_dy % V == 0;
  const int chunks = vec ? A.D / V : A.D;
  const bool keep = vec && sizeof(T) == 2 && A.D <= 32 * ln_bwd_threads(true);
  int j;                                           // chunks a thread, up to 32 columns
  if (vec) {
    constexpr int jmax = 32 / V;
    j = chunks <= 32 * jmax / 4 ? jmax / 4 : (chunks <= 32 * jmax / 2 ? jmax / 2 : jmax);
    constexpr bool half = sizeof(T) == 2;
    if (keep)
      P->kernel = j == jmax / 4 ? (const void*)ln_bwd_kernel<T, V, jmax / 4, half>
                : j == jmax / 2 ? (const void*)ln_bwd_kernel<T, V, jmax / 2, half>
                                : (const void*)ln_bwd_kernel<T, V, jmax, half>;
    else
      P->kernel = j == jmax / 4 ? (const void*)ln_bwd_kernel<T, V, jmax / 4, false>
                : j == jmax / 2 ? (const void*)ln_bwd_kernel<T, V, jmax / 2, false>
                                : (const void*)ln_bwd_kernel<T, V, jmax, false>;
  } else {
    j = chunks <= 256 ? 8 : 32;
    P->kernel = j == 8 ? (const void*)ln_bwd_kernel<T, 1, 8, false> : (const void*)ln_bwd_kernel<T, 1, 32, false>;
  }
  A.tpr = (chunks + j * 32 - 1) / (j * 32) * 32;
  int ng = ln_bwd_threads(keep) / A.tpr;
  if (A.tpr > 32 && ng > 15) ng = 15;              // named barriers 1..15
  const int64_t want = (A.T + sms - 1) / sms;      // few rows: spread them over the SMs
  if (want < ng) ng = (int)want;
  const size_t cap = 227 * 1024, row_bytes = sizeof(T) * (size_t)A.D;
  A.slot_bytes = (uint32_t)(vec ? row_bytes : (row_bytes + 15) / 16 * 16 + 16);
  const size_t par = ((size_t)A.D * 4 + 127) / 128 * 128;
  // The rings; at the end, every group's column sums in their place.
  auto ring = [&](int groups, int stages) {
    const size_t r = (size_t)groups * stages * 2 * A.slot_bytes, fold = (size_t)groups * 2 * sizeof(float) * A.part_ld;
    return ((r < fold ? fold : r) + 127) / 128 * 128;
  };
  auto total = [&](int groups, int stages) {
    return ring(groups, stages) + par + (size_t)groups * (2 * kLnRedSlots * sizeof(float2) + stages * sizeof(uint64_t));
  };
  while (ng > 1 && total(ng, 2) > cap) --ng;
  int stages = 4;
  while (stages > 1 && total(ng, stages) > cap) --stages;
  P->smem = total(ng, stages);
  if (P->smem > cap) return false;
  A.ng = ng;
  A.stages = stages;
  A.par_off = (uint32_t)ring(ng, stages);
  A.red_off = A.par_off + (uint32_t)par;
  A.bar_off = A.red_off + (uint32_t)(ng * 2 * kLnRedSlots * sizeof(float2));
  P->threads = ng * A.tpr;
  const int64_t grid = (A.T + ng - 1) / ng;
  P->grid = (int)(grid < sms ? grid : sms);
  return true;
}

template <typename T>
int bwd(LnBwdArgs& A, void* dgamma, void* dbeta, int sms, cudaStream_t stream, const char** why) {
  LnBwdPlan P;
  if (!plan_bwd<T>(A, sms, &P)) {
    *why = "row does not fit in shared memory";
    return (int)cudaErrorInvalidValue;
  }
  void* argv[] = {&A};
  int e = launch_kernel(P.kernel, P.grid, P.threads, P.smem, argv, stream, "layernorm_bwd launch", why);
  if (e || !A.partial) return e;
  int rows = P.grid;
  const float* partial = A.partial;
  void* argr[] = {&partial, &rows, &A.D, &A.part_ld, &dgamma, &dbeta};
  return launch_kernel((const void*)ln_dgamma_kernel<T>, (2 * A.part_ld + 31) / 32, 8 * kLnSlices, 0, argr, stream,
                "layernorm_bwd reduction launch", why);
}

}  // namespace

int layernorm_fwd_launch(const void* x, const void* gamma, const void* beta, void* y, float* mean, float* rstd,
                         int64_t T, int D, int64_t ld_x, float eps, int dtype, int sms, unsigned* status,
                         cudaStream_t stream,
                         const char** why) {
  LnFwdArgs A{x, gamma, beta, y, mean, rstd, T, ld_x, D, 0, eps};
  switch (dtype) {
    case kDtypeBF16: return fwd<__nv_bfloat16>(A, sms, status, stream, why);
    case kDtypeFP16: return fwd<__half>(A, sms, status, stream, why);
    default: return fwd<float>(A, sms, status, stream, why);
  }
}

size_t layernorm_bwd_workspace(int64_t T, int D, int, int sms) {
  // One partial row [2, D] per CTA, at most one CTA per SM and per row.
  return (size_t)(T < sms ? T : sms) * 2 * (size_t)part_ld(D) * sizeof(float);
}

int layernorm_bwd_launch(const void* x, const void* dy, const void* gamma, const float* mean, const float* rstd,
                         void* dx, void* dgamma, void* dbeta, int64_t T, int D, int64_t ld_x, int64_t ld_dy,
                         int dtype, void* workspace, int sms, unsigned* status, cudaStream_t stream,
                         const char** why) {
  LnBwdArgs A{};
  A.x = x; A.dy = dy; A.gamma = gamma; A.mean = mean; A.rstd = rstd; A.dx = dx;
  A.partial = (dgamma || dbeta) ? static_cast<float*>(workspace) : nullptr;
  A.T = T; A.D = D; A.part_ld = part_ld(D); A.ld_x = ld_x; A.ld_dy = ld_dy; A.status = status;
  switch (dtype) {
    case kDtypeBF16: return bwd<__nv_bfloat16>(A, dgamma, dbeta, sms, stream, why);
    case kDtypeFP16: return bwd<__half>(A, dgamma, dbeta, sms, stream, why);
    default: return bwd<float>(A, dgamma, dbeta, sms, stream, why);
  }
}

}  // namespace mxn

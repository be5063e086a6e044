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
// element of x, with about 8 and 14 flops each.
#include "layernorm.h"

#include <cuda_fp16.h>

#include "device_common.cuh"

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

// A row lives in the registers of its tpr threads (chunk j of thread t holds
// columns V * (t + j * tpr) ..), so x is read once and the centred sum of
// squares is taken about the exact row mean: no cancellation when |mean| is
// far above the deviation.  One row a warp for tpr = 32, else one row a CTA.
template <typename T, int V, int J>
__global__ void __launch_bounds__(1024, 1) ln_fwd_kernel(const LnFwdArgs A) {
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
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * A.tpr;
      if (c < nchunk) {
        load_chunk<T, V>(x + (int64_t)c * V, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[j][e];
    const float mean = row_sum(s, 0) * inv_d;
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
    const float rstd = 1.0f / sqrtf(row_sum(q, 1) * inv_d + A.eps);
    if (tid == 0) {
      if (A.mean) A.mean[row] = mean;
      if (A.rstd) A.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(A.y) + row * (int64_t)A.D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * A.tpr;
      if (c >= nchunk) continue;
      float g[V], b[V];
      if (gamma) load_chunk<T, V>(gamma + c * V, g);
      if (beta) load_chunk<T, V>(beta + c * V, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float o = v[j][e] * rstd;
        if (gamma) o *= g[e];
        if (beta) o += b[e];
        v[j][e] = o;
      }
      store_chunk<T, V>(y + (int64_t)c * V, v[j]);
    }
  }
}

// ------------------------------------------------------------------- backward

struct LnBwdArgs {
  const void* x;
  const void* dy;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;        // fp32 [gridDim.x, 2, D] (dgamma, dbeta sums of the CTA's rows), or null
  int64_t T, ld_x, ld_dy;
  unsigned* status;
  int D, tpr, ng;        // row length, threads per row group, row groups per CTA
  int stages;            // ring depth per group
  uint32_t row_bytes;    // of x, and of dy, in a stage
  uint32_t ring_off, bar_off, red_off;   // shared-memory offsets (gamma at 0)
};

constexpr int kLnRedSlots = 32;          // warps per group, at most

// Row groups of tpr threads, a row at a time each; a thread keeps the dgamma
// and dbeta sums of its columns (chunks t + j * tpr) in registers over all the
// rows its group sees.  RING: x and dy rows come through a ring of
// shared-memory stages per group, filled by bulk copies that the group's first
// thread issues (V elements = 16 bytes, rows 16-byte aligned).  Otherwise (odd
// row lengths or strides) V = 1 and the threads read global memory, twice.
// A row takes two passes: the sums (and dgamma, dbeta), then dx.  The barrier
// inside row i's reduction also says that every thread is done with row i - 1,
// whose stage is refilled then; a ring of one stage has a barrier of its own.
template <typename T, int V, int J, bool RING>
__global__ void __launch_bounds__(RING ? 512 : 1024, 1) ln_bwd_kernel(const LnBwdArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int group = threadIdx.x / A.tpr;
  const int tid = threadIdx.x - group * A.tpr;
  const int lane = threadIdx.x & 31, wig = tid >> 5, nwarp = A.tpr >> 5;
  const int D = A.D, nchunk = D / V;
  const float inv_d = 1.0f / (float)D;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + A.bar_off) + group * A.stages;
  float2* red = reinterpret_cast<float2*>(smem + A.red_off) + group * 2 * kLnRedSlots;
  const uint32_t ring = smem_u32(smem) + A.ring_off + (uint32_t)(group * A.stages) * 2u * A.row_bytes;
  const T* gamma = static_cast<const T*>(A.gamma);

  if (RING && tid == 0) {
    for (int s = 0; s < A.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();

  const int64_t g0 = (int64_t)blockIdx.x * A.ng + group, gstep = (int64_t)gridDim.x * A.ng;
  const int64_t n = g0 < A.T ? (A.T - g0 + gstep - 1) / gstep : 0;   // rows of this group
  const uint64_t pol = RING ? policy_evict_first() : 0;
  auto refill = [&](int64_t i) {                                     // group's first thread only
    const int s = (int)(i % A.stages);
    const int64_t row = g0 + i * gstep;
    uint8_t* dst = smem + A.ring_off + (size_t)(group * A.stages + s) * 2 * A.row_bytes;
    mbar_arrive_expect_tx(&full[s], 2 * A.row_bytes);
    bulk_copy_g2s(dst, static_cast<const T*>(A.x) + row * A.ld_x, A.row_bytes, &full[s], pol);
    bulk_copy_g2s(dst + A.row_bytes, static_cast<const T*>(A.dy) + row * A.ld_dy, A.row_bytes, &full[s], pol);
  };
  if (RING && tid == 0)
    for (int64_t i = 0; i < A.stages && i < n; ++i) refill(i);
  if (gamma) {
    T* gs = reinterpret_cast<T*>(smem);
    for (int c = threadIdx.x; c < D; c += blockDim.x) gs[c] = gamma[c];
  }
  __syncthreads();

  float dgam[J][V], dbet[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dgam[j][e] = dbet[j][e] = 0.0f;

  auto chunk_gamma = [&](int c, float (&v)[V]) {
    if (!gamma) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 1.0f;
    } else if constexpr (V == 1) {
      v[0] = Elem<T>::to_f(reinterpret_cast<const T*>(smem)[c]);
    } else {
      unpack16<T, V>(lds128(smem_u32(smem) + (uint32_t)c * 16u), v);
    }
  };

  bool ok = true;
  float mean = n > 0 ? A.mean[g0] : 0.0f, rstd = n > 0 ? A.rstd[g0] : 0.0f;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t row = g0 + i * gstep;
    const int s = (int)(i % A.stages);
    const uint32_t xs = ring + (uint32_t)s * 2u * A.row_bytes, ys = xs + A.row_bytes;
    const T* xg = static_cast<const T*>(A.x) + row * A.ld_x;
    const T* yg = static_cast<const T*>(A.dy) + row * A.ld_dy;
    auto chunk_x = [&](int c, float (&v)[V]) {
      if constexpr (RING) unpack16<T, V>(lds128(xs + (uint32_t)c * 16u), v);
      else load_chunk<T, V>(xg + c, v);
    };
    auto chunk_dy = [&](int c, float (&v)[V]) {
      if constexpr (RING) unpack16<T, V>(lds128(ys + (uint32_t)c * 16u), v);
      else load_chunk<T, V>(yg + c, v);
    };
    const float a = rstd, b = -mean * rstd;                          // xh = a x + b
    if (i + 1 < n) {
      mean = A.mean[row + gstep];
      rstd = A.rstd[row + gstep];
    }
    if (RING && ok) ok = mbar_wait_bounded(&full[s], (uint32_t)((i / A.stages) & 1), A.status);

    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * A.tpr;
      if (c < nchunk) {
        float xv[V], yv[V], gv[V];
        chunk_x(c, xv);
        chunk_dy(c, yv);
        chunk_gamma(c, gv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = fmaf(xv[e], a, b), g = yv[e] * gv[e];
          s1 += g;
          s2 = fmaf(g, xh, s2);
          dgam[j][e] = fmaf(yv[e], xh, dgam[j][e]);
          dbet[j][e] += yv[e];
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (nwarp > 1) {
      float2* slot = red + (i & 1) * kLnRedSlots;
      if (lane == 0) slot[wig] = make_float2(s1, s2);
      named_barrier_sync(1 + group, A.tpr);
      s1 = slot[0].x;
      s2 = slot[0].y;
      for (int w = 1; w < nwarp; ++w) {
        s1 += slot[w].x;
        s2 += slot[w].y;
      }
    } else {
      __syncwarp();
    }
    if (RING && A.stages > 1 && tid == 0 && i > 0 && i - 1 + A.stages < n) refill(i - 1 + A.stages);

    const float c1 = s1 * inv_d, c2 = s2 * inv_d;
    T* dx = static_cast<T*>(A.dx) + row * (int64_t)D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * A.tpr;
      if (c < nchunk) {
        float xv[V], yv[V], gv[V];
        chunk_x(c, xv);
        chunk_dy(c, yv);
        chunk_gamma(c, gv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = fmaf(xv[e], a, b);
          xv[e] = a * (fmaf(-xh, c2, yv[e] * gv[e]) - c1);
        }
        store_chunk<T, V>(dx + (int64_t)c * V, xv);
      }
    }
    if constexpr (RING) {
      fence_proxy_async_smem();            // these reads before the refill's bulk copy
      if (A.stages == 1) {
        if (nwarp > 1) named_barrier_sync(1 + group, A.tpr);
        else __syncwarp();
        if (tid == 0 && i + 1 < n) refill(i + 1);
      }
    }
  }

  if (!A.partial) return;
  // The CTA's sums: its groups add theirs in group order, then one row goes out.
  float* acc = reinterpret_cast<float*>(smem + A.ring_off);          // [2, D]; every copy has landed
  for (int gi = 0; gi < A.ng; ++gi) {
    __syncthreads();
    if (group != gi) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * A.tpr;
      if (c < nchunk) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int col = c * V + e;
          acc[col] = dgam[j][e] + (gi ? acc[col] : 0.0f);
          acc[D + col] = dbet[j][e] + (gi ? acc[D + col] : 0.0f);
        }
      }
    }
  }
  __syncthreads();
  float* out = A.partial + (size_t)blockIdx.x * 2 * D;
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) out[c] = acc[c];
}

// Adds the CTAs' partial rows [rows, 2, D] in a fixed order: 8 slices of rows
// a block, 32 columns each, joined in slice order.
template <typename T>
__global__ void __launch_bounds__(256) ln_dgamma_kernel(const float* partial, int rows, int D, void* dgamma,
                                                        void* dbeta) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  griddep_wait();
  griddep_launch_dependents();
  float s = 0.0f;
  if (col < 2 * D) {
#pragma unroll 8
    for (int r = slice; r < rows; r += 8) s += partial[(size_t)r * 2 * D + col];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice || col >= 2 * D) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += part[k][lane];
  T* out = static_cast<T*>(col < D ? dgamma : dbeta);
  if (out) out[col < D ? col : col - D] = Elem<T>::from_f(s);
}

// ------------------------------------------------------------------- launches

int launch(const void* kernel, int64_t grid, int threads, size_t smem, void** argv, cudaStream_t stream,
           const char* what, const char** why) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) { *why = what; return (int)e; }
  }
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, argv);
  if (e != cudaSuccess) { *why = what; return (int)e; }
  return 0;
}

int round32(int v) { return (v + 31) / 32 * 32; }

template <typename T>
const void* fwd_kernel(bool vec, int chunks, int* tpr) {
  constexpr int V = 16 / sizeof(T);
  // Up to 32 elements a thread; a warp a row while that covers it.
  auto pick = [&](int j) { *tpr = round32((chunks + j - 1) / j); return *tpr <= 1024; };
  if (vec) {
    if (chunks <= 32) { *tpr = 32; return (const void*)ln_fwd_kernel<T, V, 1>; }
    if (chunks <= 64) { *tpr = 32; return (const void*)ln_fwd_kernel<T, V, 2>; }
    if (pick(4)) return (const void*)ln_fwd_kernel<T, V, 4>;
    pick(8);
    if constexpr (sizeof(T) == 4) return (const void*)ln_fwd_kernel<T, V, 8>;
    else return nullptr;
  }
  if (chunks <= 128) { *tpr = 32; return (const void*)ln_fwd_kernel<T, 1, 4>; }
  if (chunks <= 8192) { pick(8); return (const void*)ln_fwd_kernel<T, 1, 8>; }
  pick(32);
  return (const void*)ln_fwd_kernel<T, 1, 32>;
}

template <typename T>
int fwd(LnFwdArgs& A, int sms, cudaStream_t stream, const char** why) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = A.D % V == 0 && A.ld_x % V == 0;
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
  return launch(k, grid, threads, 0, argv, stream, "layernorm_fwd launch", why);
}

struct LnBwdPlan {
  const void* kernel;
  int threads, grid;
  size_t smem;
};

template <typename T>
bool plan_bwd(LnBwdArgs& A, int sms, LnBwdPlan* P) {
  constexpr int V = 16 / sizeof(T);
  const bool ring = A.D % V == 0 && A.ld_x % V == 0 && A.ld_dy % V == 0;
  const int chunks = ring ? A.D / V : A.D;
  int j;
  if (ring) {
    const int jmax = 32 / V;               // 32 columns a thread
    j = chunks <= 32 * jmax / 4 ? jmax / 4 : (chunks <= 32 * jmax / 2 ? jmax / 2 : jmax);
    A.tpr = round32((chunks + j - 1) / j);
    if constexpr (sizeof(T) == 4)
      P->kernel = j == 2 ? (const void*)ln_bwd_kernel<T, V, 2, true>
                         : (j == 4 ? (const void*)ln_bwd_kernel<T, V, 4, true> : (const void*)ln_bwd_kernel<T, V, 8, true>);
    else
      P->kernel = j == 1 ? (const void*)ln_bwd_kernel<T, V, 1, true>
                         : (j == 2 ? (const void*)ln_bwd_kernel<T, V, 2, true> : (const void*)ln_bwd_kernel<T, V, 4, true>);
  } else {
    j = chunks <= 2048 ? 4 : 16;
    A.tpr = round32((chunks + j - 1) / j);
    P->kernel = j == 4 ? (const void*)ln_bwd_kernel<T, 1, 4, false> : (const void*)ln_bwd_kernel<T, 1, 16, false>;
  }
  const size_t cap = 227 * 1024;
  A.row_bytes = (uint32_t)(sizeof(T) * (size_t)A.D);
  const size_t gbytes = A.gamma ? (A.row_bytes + 127) / 128 * 128 : 0;
  const size_t stage = ring ? 2 * (size_t)A.row_bytes : 0;
  int ng = (ring ? 512 : 1024) / A.tpr;
  if (ng > 15) ng = A.tpr == 32 ? ng : 15;
  const int64_t want = (A.T + sms - 1) / sms;      // few rows: spread them over the SMs
  if (want < ng) ng = (int)want;
  auto fixed = [&](int groups, int stages) {
    return gbytes + 128 + (size_t)groups * (stages * sizeof(uint64_t) + 2 * kLnRedSlots * sizeof(float2));
  };
  int stages = 1;
  if (ring) {
    while (ng > 1 && fixed(ng, 2) + 2 * ng * stage > cap) --ng;
    stages = 4;
    while (stages > 1 && fixed(ng, stages) + (size_t)stages * ng * stage > cap) --stages;
  }
  size_t body = (size_t)stages * ng * stage;
  const size_t fold = 2 * sizeof(float) * (size_t)A.D;
  if (body < fold) body = fold;
  body = (body + 127) / 128 * 128;
  A.ng = ng;
  A.stages = stages;
  A.ring_off = (uint32_t)gbytes;
  A.bar_off = (uint32_t)(gbytes + body);
  A.red_off = A.bar_off + (uint32_t)((ng * stages * sizeof(uint64_t) + 15) / 16 * 16);
  P->smem = A.red_off + (size_t)ng * 2 * kLnRedSlots * sizeof(float2);
  if (P->smem > cap) return false;
  P->threads = ng * A.tpr;
  int64_t grid = (A.T + ng - 1) / ng;
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
  int e = launch(P.kernel, P.grid, P.threads, P.smem, argv, stream, "layernorm_bwd launch", why);
  if (e || !A.partial) return e;
  int rows = P.grid;
  const float* partial = A.partial;
  void* argr[] = {&partial, &rows, &A.D, &dgamma, &dbeta};
  return launch((const void*)ln_dgamma_kernel<T>, (2 * A.D + 31) / 32, 256, 0, argr, stream,
                "layernorm_bwd reduction launch", why);
}

}  // namespace

int layernorm_fwd_launch(const void* x, const void* gamma, const void* beta, void* y, float* mean, float* rstd,
                         int64_t T, int D, int64_t ld_x, float eps, int dtype, int sms, cudaStream_t stream,
                         const char** why) {
  LnFwdArgs A{x, gamma, beta, y, mean, rstd, T, ld_x, D, 0, eps};
  switch (dtype) {
    case kDtypeBF16: return fwd<__nv_bfloat16>(A, sms, stream, why);
    case kDtypeFP16: return fwd<__half>(A, sms, stream, why);
    default: return fwd<float>(A, sms, stream, why);
  }
}

size_t layernorm_bwd_workspace(int64_t T, int D, int, int sms) {
  // One partial row [2, D] per CTA, at most one CTA per SM and per row.
  return (size_t)(T < sms ? T : sms) * 2 * (size_t)D * sizeof(float);
}

int layernorm_bwd_launch(const void* x, const void* dy, const void* gamma, const float* mean, const float* rstd,
                         void* dx, void* dgamma, void* dbeta, int64_t T, int D, int64_t ld_x, int64_t ld_dy,
                         int dtype, void* workspace, int sms, unsigned* status, cudaStream_t stream,
                         const char** why) {
  LnBwdArgs A{};
  A.x = x; A.dy = dy; A.gamma = gamma; A.mean = mean; A.rstd = rstd; A.dx = dx;
  A.partial = (dgamma || dbeta) ? static_cast<float*>(workspace) : nullptr;
  A.T = T; A.D = D; A.ld_x = ld_x; A.ld_dy = ld_dy; A.status = status;
  switch (dtype) {
    case kDtypeBF16: return bwd<__nv_bfloat16>(A, dgamma, dbeta, sms, stream, why);
    case kDtypeFP16: return bwd<__half>(A, dgamma, dbeta, sms, stream, why);
    default: return bwd<float>(A, dgamma, dbeta, sms, stream, why);
  }
}

}  // namespace mxn

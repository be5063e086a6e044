// gated_mxfp8.cu -- gated feed-forward projection on MXFP8 operands.
//
//   gate = A Wg^T, up = A Wu^T, h = act(gate) * up
// A [T, K], Wg and Wu [F, K] in E4M3 with one E8M0 scale per 32 along K (the
// tcgen05 scale layout: what mxnorm_fwd and mxnorm_fold_weight write).  h is
// written as bf16, or quantised to MXFP8 in the epilogue -- E4M3 codes and E8M0
// scales, the operand of the next product -- so the fp32 result is rounded
// once either way and never makes a trip through memory in between.
//
// The kernel is the 128 x 256 tile of gemm_mxfp8.cu with the tile's 256
// columns made of 128 gate and the same 128 up features (each a whole 128-row
// scale atom).  A lane of the epilogue holds one row's gate and up values of
// the same 32 features, one MX block of h: activation, product, block maximum,
// scale and codes need no exchange between threads.
#include "gated_mxfp8.h"

#include "activations.cuh"
#include "gated_ffn.h"
#include "tcgen05.cuh"

namespace mxn {
namespace {

constexpr int kTileM = 128, kTileF = 128, kTileK = 128;
constexpr int kStages = 4;
constexpr int kEpiWarps = 8;                     // 4 lane quarters x 2 feature halves
constexpr int kThreads = 64 + 32 * kEpiWarps;    // producer warp, MMA warp, epilogue warps
constexpr uint32_t kABytes = kTileM * kTileK;
constexpr uint32_t kBBytes = 2 * kTileF * kTileK;
constexpr uint32_t kAtom = 512;                  // one 128 x 4 scale atom
constexpr uint32_t kStageTx = kABytes + kBBytes + 3 * kAtom;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol0 = 256;                // accumulator: columns 0..255; scales: 12 per stage
constexpr int kGroupM = 8;                       // tiles go m-first inside groups of 8 tile rows

struct Smem {
  uint8_t a[kStages][kABytes];                   // 1024-aligned (128B swizzle atoms)
  uint8_t b[kStages][kBBytes];                   // 128 gate rows, 128 up rows
  uint8_t sf[kStages][3 * kAtom];                // A, gate, up
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full, acc_empty, mma_done;
  uint32_t tmem_base;
  uint32_t failed;
};

struct Args {
  CUtensorMap a, g, u;
  const uint8_t *a_s, *g_s, *u_s;
  uint8_t *h, *h_s;
  unsigned* status;
  int T, F, K, m_tiles, n_tiles, act;
  int out;                                       // 0 bf16; 1 E4M3, scales row-major; 2 E4M3, scales in the tcgen05 layout
};

__device__ __forceinline__ bool failed_flag(const Smem& S) {
  return *reinterpret_cast<const volatile uint32_t*>(&S.failed) != 0;
}

// As in gemm_mxfp8.cu: E4M3 operands, E8M0 scales, M = 128, N = 256, K = 32.
__device__ __forceinline__ uint32_t instr_desc(uint32_t sf_id) {
  return (sf_id << 4) | ((uint32_t)(256 >> 3) << 17) | (1u << 23) | ((uint32_t)(kTileM >> 4) << 24) | (sf_id << 29);
}

__device__ __forceinline__ void tile_pos(const Args& A, int t, int* mt, int* nt) {
  const int m0 = t / (kGroupM * A.n_tiles) * kGroupM;
  const int gm = min(kGroupM, A.m_tiles - m0);
  t -= m0 * A.n_tiles;
  *mt = m0 + t % gm;
  *nt = t / gm;
}

template <int ACT>
__device__ __forceinline__ void gate_product(uint32_t (&g)[32], const uint32_t (&u)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    g[i] = __float_as_uint(act_f<ACT>(__uint_as_float(g[i])) * __uint_as_float(u[i]));
}

// 32 features of one row, from column col on (h: fp32 bits).
__device__ __forceinline__ void store_bf16(const Args& A, int row, int col, const uint32_t (&h)[32]) {
  uint8_t* p = A.h + ((int64_t)row * A.F + col) * 2;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (col + 8 * v >= A.F) break;               // F is a multiple of 8
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(h[8 * v + 2 * i]), __uint_as_float(h[8 * v + 2 * i + 1]));
      o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p + 16 * v) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void store_mxfp8(const Args& A, int row, int col, const uint32_t (&h)[32]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) m = max3_abs_nan(m, __uint_as_float(h[i]), __uint_as_float(h[i + 1]));
  const int e = e8m0_exponent_bits(__float_as_uint(m));
  const bool bad = e == 128;                     // NaN or infinity in the block
  const float inv = exp2_int(bad ? 0 : -e);
  uint8_t* p = A.h + (int64_t)row * A.F + col;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 16 * v + 4 * i;
      o[i] = cvt_e4m3x4_rn(__uint_as_float(h[j]) * inv, __uint_as_float(h[j + 1]) * inv,
                           __uint_as_float(h[j + 2]) * inv, __uint_as_float(h[j + 3]) * inv);
      if (bad) o[i] = 0x7F7F7F7Fu;
    }
    *reinterpret_cast<uint4*>(p + 16 * v) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  const int k = col / 32, K = A.F / 32;
  const int64_t at = A.out == 1 ? (int64_t)row * K + k
                                : ((int64_t)(row / 128) * ((K + 3) / 4) + k / 4) * 512 + (row % 32) * 16 +
                                      ((row % 128) / 32) * 4 + (k % 4);
  A.h_s[at] = (uint8_t)(bad ? 0xFF : e + 127);
}

__global__ void __launch_bounds__(kThreads, 1) gated_mxfp8_kernel(const __grid_constant__ Args A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = A.m_tiles * A.n_tiles;
  const int n_k = A.K / kTileK;                  // also the scale atoms of a 128-row tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, kEpiWarps);
    mbar_init(&S.mma_done, 1);
    S.failed = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  uint32_t n_issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t g = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        int mt, nt;
        tile_pos(A, t, &mt, &nt);
        for (int kb = 0; kb < n_k; ++kb, ++g) {
          const int s = (int)(g % kStages);
          if (!mbar_wait_bounded(&S.empty[s], ((g / kStages) & 1u) ^ 1u, A.status) || failed_flag(S)) {
            atomicOr(&S.failed, 1u);
            ok = false;
            break;
          }
          uint64_t* bar = &S.full[s];
          mbar_arrive_expect_tx(bar, kStageTx);
          tma_load_2d(S.a[s], &A.a, kb * kTileK, mt * kTileM, bar);
          tma_load_2d(S.b[s], &A.g, kb * kTileK, nt * kTileF, bar);
          tma_load_2d(S.b[s] + kBBytes / 2, &A.u, kb * kTileK, nt * kTileF, bar);
          bulk_g2s_plain(S.sf[s], A.a_s + ((size_t)mt * n_k + kb) * kAtom, kAtom, bar);
          bulk_g2s_plain(S.sf[s] + kAtom, A.g_s + ((size_t)nt * n_k + kb) * kAtom, kAtom, bar);
          bulk_g2s_plain(S.sf[s] + 2 * kAtom, A.u_s + ((size_t)nt * n_k + kb) * kAtom, kAtom, bar);
          n_issued = g + 1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------- MMA
      uint32_t g = 0, it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
        if (!mbar_wait_bounded(&S.acc_empty, (it & 1u) ^ 1u, A.status) || failed_flag(S)) {
          atomicOr(&S.failed, 1u);
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < n_k; ++kb, ++g) {
          const int s = (int)(g % kStages);
          if (!mbar_wait_bounded(&S.full[s], (g / kStages) & 1u, A.status) || failed_flag(S)) {
            atomicOr(&S.failed, 1u);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sfa = tmem + kSfCol0 + (uint32_t)s * 12u, sfb = sfa + 4u;
          for (int j = 0; j < 3; ++j)
            tmem_cp_sf(sfa + 4u * j, smem_desc(smem_u32(S.sf[s]) + kAtom * j, 0, 128, 0));
          const uint32_t a0 = smem_u32(S.a[s]), b0 = smem_u32(S.b[s]);
#pragma unroll
          for (int k = 0; k < kTileK / 32; ++k)
            mma_mxf8(tmem, smem_desc(a0 + 32u * k, 16, 1024, 2), smem_desc(b0 + 32u * k, 16, 1024, 2),
                     instr_desc((uint32_t)k), sfa | ((uint32_t)k << 30), sfb | ((uint32_t)k << 30),
                     (kb > 0 || k > 0) ? 1u : 0u);
          tc_commit(&S.empty[s]);
        }
        if (ok) tc_commit(&S.acc_full);
      }
      tc_commit(&S.mma_done);
      if (!ok) tc_commit(&S.acc_full);           // wake the epilogue; it sees the failure
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;            // features 64 * half .. of the tile
    uint32_t it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      int mt, nt;
      tile_pos(A, t, &mt, &nt);
      const bool got = mbar_wait_bounded(&S.acc_full, it & 1u, A.status);
      tc_fence_after();
      if (!got || failed_flag(S)) {
        if (lane == 0) atomicOr(&S.failed, 1u);
        break;
      }
      uint32_t r[2][32], u[2][32];
      const uint32_t ta = tmem + (uint32_t)(half * 64) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        tmem_ld32(ta + 32u * j, r[j]);
        tmem_ld32(ta + 128u + 32u * j, u[j]);
      }
      tmem_ld_fence(r[0], true);
      tmem_ld_fence(r[1], false);
      tmem_ld_fence(u[0], false);
      tmem_ld_fence(u[1], false);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.acc_empty);  // the MMA thread may overwrite the accumulator
      const int row = mt * kTileM + quarter * 32 + lane;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = nt * kTileF + half * 64 + 32 * j;
        if (A.act == kActSilu) gate_product<kActSilu>(r[j], u[j]);
        else if (A.act == kActGelu) gate_product<kActGelu>(r[j], u[j]);
        else gate_product<kActGeluTanh>(r[j], u[j]);
        if (row < A.T && col < A.F) {
          if (A.out == 0) store_bf16(A, row, col, r[j]);
          else store_mxfp8(A, row, col, r[j]);
        }
      }
      __syncwarp();                              // tcgen05.ld needs the warp converged
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && lane == 0) mbar_wait_bounded(&S.mma_done, 0, A.status);
  if (warp == 0 && lane == 0 && failed_flag(S))  // leave no copy in flight
    for (uint32_t j = (n_issued > (uint32_t)kStages ? n_issued - kStages : 0); j < n_issued; ++j)
      mbar_wait_bounded(&S.full[j % kStages], (j / kStages) & 1u, A.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// 2-D map over a row-major uint8 [rows, cols] matrix, boxes of 128 rows x 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, int rows, int cols) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols};
  const cuuint32_t box[2] = {(cuuint32_t)kTileK, 128};
  const cuuint32_t elem[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int gated_mxfp8_launch(const void* a_q, const void* a_s, const void* g_q, const void* g_s, const void* u_q,
                       const void* u_s, void* h, void* h_s, int T, int F, int K, int act, bool scale_mma, int sms,
                       unsigned* status, cudaStream_t stream, const char** why) {
  Args A{};
  if (!make_map(&A.a, a_q, T, K) || !make_map(&A.g, g_q, F, K) || !make_map(&A.u, u_q, F, K)) {
    *why = "cuTensorMapEncodeTiled failed";
    return -1;
  }
  A.a_s = static_cast<const uint8_t*>(a_s);
  A.g_s = static_cast<const uint8_t*>(g_s);
  A.u_s = static_cast<const uint8_t*>(u_s);
  A.h = static_cast<uint8_t*>(h);
  A.h_s = static_cast<uint8_t*>(h_s);
  A.status = status;
  A.T = T;
  A.F = F;
  A.K = K;
  A.m_tiles = (T + kTileM - 1) / kTileM;
  A.n_tiles = (F + kTileF - 1) / kTileF;
  A.act = act;
  A.out = !h_s ? 0 : (scale_mma ? 2 : 1);
  const int64_t tiles = (int64_t)A.m_tiles * A.n_tiles;
  if (tiles > 0x7FFFFFFF - sms) {
    *why = "too many tiles";
    return -1;
  }
  const size_t smem = sizeof(Smem);
  cudaError_t e = cudaFuncSetAttribute(gated_mxfp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) { *why = cudaGetErrorString(e); return (int)e; }
  void* argv[] = {&A};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles < sms ? (int)tiles : sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelExC(&cfg, (const void*)gated_mxfp8_kernel, argv);
  if (e != cudaSuccess) { *why = cudaGetErrorString(e); return (int)e; }
  return 0;
}

}  // namespace mxn

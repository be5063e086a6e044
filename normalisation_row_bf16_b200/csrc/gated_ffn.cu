// gated_ffn.cu -- gated feed-forward projections in bf16 on the tensor cores.
//
// Forward, x [T, D], Wg and Wu [F, D] (one output feature per row):
//   gate = x Wg^T, up = x Wu^T, h = act(gate) * up
// Backward, from dh and the kept gate and up:
//   dg = dh * up * act'(gate), du = dh * act(gate)       (bf16, workspace)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// Products accumulate in fp32 tensor memory; h, dx and the weight gradients are
// rounded once to bf16.  dg and du are rounded to bf16 because they are
// tensor-core operands (one rounding of 2^-9 each, as large as an output's).
//
// One kernel does the three products (Mode):
//   kGate  one tile holds the gate and the up columns of the same features, so
//          the activation and the product happen in its epilogue;
//   kDx    the contraction runs over dg, Wg and then du, Wu: one accumulator;
//   kDw    dWg and dWu tiles in one launch.
// All operands are read where they lie: a factor whose contraction index is not
// contiguous (Wg and Wu in kDx, dg, du and x in kDw) goes to the tensor cores
// as an MN-major operand, so nothing is transposed in memory.
#include "gated_ffn.h"

#include "activations.cuh"
#include "tcgen05.cuh"

namespace mxn {
namespace {

enum Mode { kGate, kDx, kDw };

constexpr int kTileM = 128;                      // output rows of a tile
constexpr int kTileK = 64;                       // contraction elements (128 bytes) per stage
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;                     // 4 lane quarters x 2 column halves
constexpr int kThreads = 64 + 32 * kEpiWarps;    // producer warp, MMA warp, epilogue warps
constexpr uint32_t kABytes = kTileM * kTileK * 2;
constexpr uint32_t kTmemCols = 512;              // two accumulators of up to 256 columns
constexpr int kGroupM = 8;                       // tiles go m-first inside groups of 8 tile rows: operand reuse in L2

struct Args {
  CUtensorMap a[2], b[2];
  uint16_t* out[3];      // kGate: h, gate, up (the last two may be null); kDx: dx; kDw: dWg, dWu
  unsigned* status;
  int64_t ld_out;
  int M, N;              // output rows and columns of one problem
  int m_tiles, n_tiles, tiles;   // tiles: of all problems
  int n_k, n_k0;         // K stages of a tile, and of its first segment (kDx)
  int tile_n;            // output columns of a tile (kGate: features, each with a gate and an up column)
  int acc_n;             // accumulator columns: 2 * tile_n (kGate) or tile_n
  int act;
  int stages;
  uint32_t stage_bytes;
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t failed;
};

__device__ __forceinline__ bool failed_flag(const Barriers& S) {
  return *reinterpret_cast<const volatile uint32_t*>(&S.failed) != 0;
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulator (bit 4), A and B bf16
// (bits 7, 10), MN-major A and B (bits 15, 16), N >> 3 in 17..22, M >> 4 in 24..28.
__device__ __forceinline__ uint32_t instr_desc(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Descriptors of K step k (16 elements) of an operand tile in 128-byte swizzle.
// K-major: rows of 128 bytes (64 contraction elements), 8-row atoms 1024 B apart.
// MN-major: blocks of 64 rows (M or N index, contiguous) x 64 contraction
// elements, 8 KiB each: 8-element contraction groups 1024 B apart (stride),
// the next 64 rows 8192 B on (leading).
__device__ __forceinline__ uint64_t op_desc(uint32_t base, int k, bool mn) {
  return mn ? smem_desc(base + 2048u * (uint32_t)k, 8192, 1024, 2) : smem_desc(base + 32u * (uint32_t)k, 16, 1024, 2);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// As tmem_ld_fence, for 16 registers.
__device__ __forceinline__ void tmem_ld16_fence(uint32_t (&r)[16], bool wait) {
#define MXN_R16 "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), \
                "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
  if (wait)
    asm volatile("tcgen05.wait::ld.sync.aligned;" : MXN_R16 :: "memory");
  else
    asm volatile("" : MXN_R16 :: "memory");
#undef MXN_R16
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Tile t of the launch -> problem, tile row, tile column.
struct TilePos {
  int p, mt, nt;
};
__device__ __forceinline__ TilePos tile_pos(const Args& A, int t) {
  TilePos q;
  const int per = A.m_tiles * A.n_tiles;
  q.p = t / per;
  t -= q.p * per;
  const int span = kGroupM * A.n_tiles;
  const int m0 = t / span * kGroupM;
  const int gm = min(kGroupM, A.m_tiles - m0);
  t -= m0 * A.n_tiles;
  q.mt = m0 + t % gm;
  q.nt = t / gm;
  return q;
}

// 16 output columns of one row, from col on: N is a multiple of 8.
__device__ __forceinline__ void store_cols16(uint16_t* row, int col, int n, const uint32_t (&o)[8]) {
  if (col < n) *reinterpret_cast<uint4*>(row + col) = make_uint4(o[0], o[1], o[2], o[3]);
  if (col + 8 < n) *reinterpret_cast<uint4*>(row + col + 8) = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int ACT>
__device__ __forceinline__ void gate_product(const uint32_t (&g)[16], const uint32_t (&u)[16], uint32_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = pack_bf16(act_f<ACT>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                     act_f<ACT>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
}

// Persistent CTAs, one per SM, walk the output tiles.  Warp 0 streams K stages
// of both operands into a shared-memory ring with TMA tensor copies (out of
// range rows and columns arrive as zeros); warp 1 issues tcgen05.mma into one
// of two accumulators; warps 2..9 drain the other.  Every wait is bounded, as
// in gemm_mxfp8.cu.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) gated_gemm_kernel(const __grid_constant__ Args A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Barriers& S = *reinterpret_cast<Barriers*>(smem_raw + (size_t)A.stages * A.stage_bytes);
  constexpr bool kAmn = MODE == kDw, kBmn = MODE != kGate;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.acc_full[b], 1);
      mbar_init(&S.acc_empty[b], kEpiWarps);
    }
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
      uint32_t s = 0, ph = 1;
      bool ok = true;
      for (int t = blockIdx.x; t < A.tiles && ok; t += gridDim.x) {
        const TilePos q = tile_pos(A, t);
        for (int kb = 0; kb < A.n_k; ++kb) {
          if (!mbar_wait_bounded(&S.empty[s], ph, A.status) || failed_flag(S)) {
            atomicOr(&S.failed, 1u);
            ok = false;
            break;
          }
          uint8_t* sa = smem_raw + (size_t)s * A.stage_bytes;
          uint8_t* sb = sa + kABytes;
          uint64_t* bar = &S.full[s];
          mbar_arrive_expect_tx(bar, A.stage_bytes);
          if constexpr (MODE == kGate) {
            tma_load_2d(sa, &A.a[0], kb * kTileK, q.mt * kTileM, bar);
            tma_load_2d(sb, &A.b[0], kb * kTileK, q.nt * A.tile_n, bar);
            tma_load_2d(sb + A.tile_n * 128, &A.b[1], kb * kTileK, q.nt * A.tile_n, bar);
          } else if constexpr (MODE == kDx) {
            const int seg = kb >= A.n_k0, k0 = (kb - seg * A.n_k0) * kTileK;
            tma_load_2d(sa, &A.a[seg], k0, q.mt * kTileM, bar);
            for (int c = 0; c < A.tile_n; c += 64) tma_load_2d(sb + c * 128, &A.b[seg], q.nt * A.tile_n + c, k0, bar);
          } else {
            for (int c = 0; c < kTileM; c += 64) tma_load_2d(sa + c * 128, &A.a[q.p], q.mt * kTileM + c, kb * kTileK, bar);
            for (int c = 0; c < A.tile_n; c += 64) tma_load_2d(sb + c * 128, &A.b[0], q.nt * A.tile_n + c, kb * kTileK, bar);
          }
          ++n_issued;
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------- MMA
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = true;
      const uint32_t idesc = instr_desc(kTileM, A.acc_n, kAmn, kBmn);
      for (int t = blockIdx.x; t < A.tiles && ok; t += gridDim.x, ++it) {
        const uint32_t buf = it & 1u;
        if (!mbar_wait_bounded(&S.acc_empty[buf], ((it >> 1) & 1u) ^ 1u, A.status) || failed_flag(S)) {
          atomicOr(&S.failed, 1u);
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < A.n_k; ++kb) {
          if (!mbar_wait_bounded(&S.full[s], ph, A.status) || failed_flag(S)) {
            atomicOr(&S.failed, 1u);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem_raw) + s * A.stage_bytes, b0 = a0 + kABytes;
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            mma_bf16(tmem + buf * 256u, op_desc(a0, k, kAmn), op_desc(b0, k, kBmn), idesc, (kb > 0 || k > 0) ? 1u : 0u);
          tc_commit(&S.empty[s]);
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
        }
        if (ok) tc_commit(&S.acc_full[buf]);
      }
      tc_commit(&S.mma_done);
      if (!ok) {                                 // wake the epilogue; it sees the failure
        tc_commit(&S.acc_full[0]);
        tc_commit(&S.acc_full[1]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;                // tcgen05.ld reaches lanes 32 * (warp % 4) ..
    const int half = (warp - 2) >> 2;            // 16-column chunks half, half + 2, ..
    uint32_t it = 0;
    for (int t = blockIdx.x; t < A.tiles; t += gridDim.x, ++it) {
      const TilePos q = tile_pos(A, t);
      const uint32_t buf = it & 1u;
      const bool got = mbar_wait_bounded(&S.acc_full[buf], (it >> 1) & 1u, A.status);
      tc_fence_after();
      if (!got || failed_flag(S)) {
        if (lane == 0) atomicOr(&S.failed, 1u);
        break;
      }
      const int row = q.mt * kTileM + quarter * 32 + lane;
      const bool live = row < A.M;
      const uint32_t ta = tmem + buf * 256u + ((uint32_t)(quarter * 32) << 16);
      for (int c = half * 16; c < A.tile_n; c += 32) {
        const int col = q.nt * A.tile_n + c;
        uint32_t r[16], o[8];
        tmem_ld16(ta + (uint32_t)c, r);
        if constexpr (MODE == kGate) {
          uint32_t u[16];
          tmem_ld16(ta + (uint32_t)(A.tile_n + c), u);
          tmem_ld16_fence(r, true);
          tmem_ld16_fence(u, false);
          if (A.act == kActSilu) gate_product<kActSilu>(r, u, o);
          else if (A.act == kActGelu) gate_product<kActGelu>(r, u, o);
          else gate_product<kActGeluTanh>(r, u, o);
          if (live) {
            store_cols16(A.out[0] + (int64_t)row * A.ld_out, col, A.N, o);
            if (A.out[1]) {
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
              store_cols16(A.out[1] + (int64_t)row * A.ld_out, col, A.N, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
              store_cols16(A.out[2] + (int64_t)row * A.ld_out, col, A.N, o);
            }
          }
        } else {
          tmem_ld16_fence(r, true);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
          if (live) store_cols16(A.out[MODE == kDw ? q.p : 0] + (int64_t)row * A.ld_out, col, A.N, o);
        }
        __syncwarp();                            // tcgen05.ld needs the warp converged
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.acc_empty[buf]);
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && lane == 0) mbar_wait_bounded(&S.mma_done, 0, A.status);
  // After a wait gave up, leave no copy in flight: the producer waits (bounded)
  // for the last issued phase of every stage.
  if (warp == 0 && lane == 0 && failed_flag(S))
    for (uint32_t j = (n_issued > (uint32_t)A.stages ? n_issued - A.stages : 0); j < n_issued; ++j)
      mbar_wait_bounded(&S.full[j % A.stages], (j / A.stages) & 1u, A.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// dg = dh * up * act'(gate), du = dh * act(gate): 8 elements a thread and step.
// Bound by HBM: 3 elements read and 2 written each.
template <int ACT>
__global__ void __launch_bounds__(256) gated_act_bwd_kernel(const uint16_t* dh, const uint16_t* gate,
                                                            const uint16_t* up, uint16_t* dg, uint16_t* du,
                                                            int64_t n8) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += (int64_t)gridDim.x * blockDim.x) {
    const uint4 h4 = ldg128_nc(dh + 8 * i), g4 = ldg128_nc(gate + 8 * i), u4 = ldg128_nc(up + 8 * i);
    const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w}, gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 h = bf16x2_to_f2(hw[k]), g = bf16x2_to_f2(gw[k]), u = bf16x2_to_f2(uw[k]);
      float a0, d0, a1, d1;
      act_grad_f<ACT>(g.x, &a0, &d0);
      act_grad_f<ACT>(g.y, &a1, &d1);
      og[k] = pack_bf16(h.x * u.x * d0, h.y * u.y * d1);
      ou[k] = pack_bf16(h.x * a0, h.y * a1);
    }
    *reinterpret_cast<uint4*>(dg + 8 * i) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(du + 8 * i) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// ------------------------------------------------------------------- launches

// 2-D map over a row-major bf16 [rows, cols] matrix of row stride ld, boxes of
// box_rows rows x 64 columns (128 bytes), 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int launch_pdl(const void* kernel, int grid, int threads, size_t smem, void** argv, cudaStream_t stream,
               const char* what, const char** why) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
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
    if (e != cudaSuccess) { *why = cudaGetErrorString(e); return (int)e; }
  }
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, argv);
  if (e != cudaSuccess) { *why = what; return (int)e; }
  return 0;
}

// Fills the tile and ring geometry of a launch.  Tile widths that divide the
// columns over the SMs in the fewest rounds of equal cost: with m_tiles tile
// rows, the candidate with the least (rounds x columns a tile).
// Returns false when the tiles outnumber an int.
bool plan_tiles(Args& A, int mode, int problems, int sms) {
  A.m_tiles = cdiv(A.M, kTileM);
  const int unit = mode == kGate ? 16 : 64, widest = mode == kGate ? 128 : 256;
  int64_t best = 0;
  for (int w = widest; w >= unit; w -= unit) {
    const int64_t tiles = (int64_t)A.m_tiles * cdiv(A.N, w) * problems;
    // A tile costs its columns, and its 128 rows of A once more.
    const int64_t cost = ((tiles + sms - 1) / sms) * ((mode == kGate ? 2 * w : w) + 64);
    if (best == 0 || cost < best) {
      best = cost;
      A.tile_n = w;
    }
  }
  A.n_tiles = cdiv(A.N, A.tile_n);
  const int64_t tiles = (int64_t)A.m_tiles * A.n_tiles * problems;
  if (tiles > 0x7FFFFFFF - sms) return false;
  A.tiles = (int)tiles;
  A.acc_n = mode == kGate ? 2 * A.tile_n : A.tile_n;
  A.stage_bytes = kABytes + (uint32_t)A.acc_n * 128u;
  const size_t cap = 227 * 1024 - sizeof(Barriers);
  A.stages = (int)(cap / A.stage_bytes);
  if (A.stages > kMaxStages) A.stages = kMaxStages;
  return true;
}

int launch_gemm(const void* kernel, Args& A, int sms, cudaStream_t stream, const char* what, const char** why) {
  void* argv[] = {&A};
  const size_t smem = (size_t)A.stages * A.stage_bytes + sizeof(Barriers);
  return launch_pdl(kernel, A.tiles < sms ? A.tiles : sms, kThreads, smem, argv, stream, what, why);
}

}  // namespace

int gated_ffn_fwd_launch(const void* x, const void* w_gate, const void* w_up, void* h, void* gate, void* up, int T,
                         int D, int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status,
                         cudaStream_t stream, const char** why) {
  Args A{};
  A.out[0] = static_cast<uint16_t*>(h);
  A.out[1] = static_cast<uint16_t*>(gate);
  A.out[2] = static_cast<uint16_t*>(up);
  A.status = status;
  A.ld_out = F;
  A.M = T;
  A.N = F;
  A.act = act;
  A.n_k = A.n_k0 = cdiv(D, kTileK);
  if (!plan_tiles(A, kGate, 1, sms)) { *why = "too many tiles"; return -1; }
  if (!make_map(&A.a[0], x, T, D, ld_x, kTileM) || !make_map(&A.b[0], w_gate, F, D, ld_w, A.tile_n) ||
      !make_map(&A.b[1], w_up, F, D, ld_w, A.tile_n)) {
    *why = "cuTensorMapEncodeTiled failed";
    return -1;
  }
  return launch_gemm((const void*)gated_gemm_kernel<kGate>, A, sms, stream, "gated_ffn_fwd launch", why);
}

int gated_ffn_bwd_launch(const void* dh, const void* x, const void* w_gate, const void* w_up, const void* gate,
                         const void* up, void* dx, void* dw_gate, void* dw_up, void* dg, void* du, int T, int D,
                         int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status, cudaStream_t stream,
                         const char** why) {
  const uint16_t *dhp = static_cast<const uint16_t*>(dh), *gp = static_cast<const uint16_t*>(gate),
                 *upp = static_cast<const uint16_t*>(up);
  uint16_t *dgp = static_cast<uint16_t*>(dg), *dup = static_cast<uint16_t*>(du);
  int64_t n8 = (int64_t)T * F / 8;
  void* argv[] = {&dhp, &gp, &upp, &dgp, &dup, &n8};
  const int64_t blocks = (n8 + 255) / 256, most = (int64_t)sms * 8;
  const void* k = act == kActSilu ? (const void*)gated_act_bwd_kernel<kActSilu>
                                  : (act == kActGelu ? (const void*)gated_act_bwd_kernel<kActGelu>
                                                     : (const void*)gated_act_bwd_kernel<kActGeluTanh>);
  int e = launch_pdl(k, (int)(blocks < most ? blocks : most), 256, 0, argv, stream, "gated_ffn_bwd activation launch", why);
  if (e) return e;
  if (dx) {
    Args A{};
    A.out[0] = static_cast<uint16_t*>(dx);
    A.status = status;
    A.ld_out = D;
    A.M = T;
    A.N = D;
    A.n_k0 = cdiv(F, kTileK);
    A.n_k = 2 * A.n_k0;
    if (!plan_tiles(A, kDx, 1, sms)) { *why = "too many tiles"; return -1; }
    if (!make_map(&A.a[0], dg, T, F, F, kTileM) || !make_map(&A.a[1], du, T, F, F, kTileM) ||
        !make_map(&A.b[0], w_gate, F, D, ld_w, kTileK) || !make_map(&A.b[1], w_up, F, D, ld_w, kTileK)) {
      *why = "cuTensorMapEncodeTiled failed";
      return -1;
    }
    e = launch_gemm((const void*)gated_gemm_kernel<kDx>, A, sms, stream, "gated_ffn_bwd dx launch", why);
    if (e) return e;
  }
  if (dw_gate) {
    Args A{};
    A.out[0] = static_cast<uint16_t*>(dw_gate);
    A.out[1] = static_cast<uint16_t*>(dw_up);
    A.status = status;
    A.ld_out = D;
    A.M = F;
    A.N = D;
    A.n_k = A.n_k0 = cdiv(T, kTileK);
    if (!plan_tiles(A, kDw, 2, sms)) { *why = "too many tiles"; return -1; }
    if (!make_map(&A.a[0], dg, T, F, F, kTileK) || !make_map(&A.a[1], du, T, F, F, kTileK) ||
        !make_map(&A.b[0], x, T, D, ld_x, kTileK)) {
      *why = "cuTensorMapEncodeTiled failed";
      return -1;
    }
    e = launch_gemm((const void*)gated_gemm_kernel<kDw>, A, sms, stream, "gated_ffn_bwd dw launch", why);
    if (e) return e;
  }
  return 0;
}

}  // namespace mxn

// gated_mxfp8.cu -- gated feed-forward projection on MXFP8 operands.
//
//   gate = A Wg^T, up = A Wu^T, h = act(gate) * up
// A [T, K], Wg and Wu [F, K] in E4M3 with one E8M0 scale per 32 along K (the
// tcgen05 scale layout: what mxnorm_fwd and mxnorm_fold_weight write).  h is
// written as bf16, or quantised to MXFP8 in the epilogue -- E4M3 codes and E8M0
// scales, the operand of the next product -- so the fp32 result is rounded
// once either way and never makes a trip through memory in between.  The tensor
// cores' sums are off by about 1e-6 of an entry at K = 4096, so a value that close
// to a rounding border takes the neighbouring code (a block's maximum, the
// neighbouring scale): against 64 bits, 162 to 197 codes by the activation and one
// scale of 1024 x 4096 x 14336's 14.7 million and 459 thousand.  The activation's
// own error has a share of 12 to 41 codes in that, as that of a plain fp32 form.
//
// Tiles hold 128 gate and the same 128 up features (each a whole 128-row scale
// atom) in 256 accumulator columns.  A lane of the epilogue holds one row's
// gate and up values of the same 32 features, one MX block of h: activation,
// product, block maximum, scale and codes need no exchange between threads.
#include "gated_mxfp8.h"

#include "activations.cuh"
#include "gated_ffn.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace mxn {
namespace {

constexpr int kTileF = 128, kTileK = 128;        // features of a tile; K elements (= bytes) per stage
constexpr int kMaxStages = 8;
constexpr int kEpiWarps = 8;                     // 4 lane quarters x 2 feature halves
constexpr int kThreads = 64 + 32 * kEpiWarps;    // producer warp, MMA warp, epilogue warps
constexpr uint32_t kRows128 = 128 * kTileK;      // 128 rows of an operand
constexpr uint32_t kAtom = 512;                  // one 128 x 4 scale atom
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol0 = 256;                // accumulator: columns 0..255; scales: 12 per stage
constexpr int kGroupM = 8;                       // tiles go m-first inside groups of 8 tile rows

struct Args {
  CUtensorMap a, w[2];                           // codes: A, gate and up
  CUtensorMap a_sf, w_sf[2];                     // pairs: their scale atoms as boxes of 4 rows of 128 bytes
  const uint8_t *a_s, *w_s[2];
  uint8_t *h, *h_s;
  unsigned* status;
  int T, F, K, m_tiles, n_tiles, act;
  int out;                                       // 0 bf16; 1 E4M3, scales row-major; 2 E4M3, scales in the tcgen05 layout
  int a_rows, stages;                            // rows of A a stage holds (single CTAs), ring depth
  uint32_t sf_off, stage_bytes;                  // of a stage: B after A's rows, scales at sf_off
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full, acc_empty, mma_done;
  uint32_t tmem_base;
  uint32_t failed;
};

__device__ __forceinline__ bool failed_flag(const Barriers& S) {
  return *reinterpret_cast<const volatile uint32_t*>(&S.failed) != 0;
}

// As in gemm_mxfp8.cu: E4M3 operands, E8M0 scales, M = m, N = 256, K = 32.
__device__ __forceinline__ uint32_t instr_desc(uint32_t m, uint32_t sf_id) {
  return (sf_id << 4) | ((uint32_t)(256 >> 3) << 17) | (1u << 23) | ((m >> 4) << 24) | (sf_id << 29);
}

// Tile t: 128-row (pairs: 256-row) block and feature block.
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

// Persistent CTAs as in gemm_mxfp8.cu.  PAIR: two CTAs (a cluster on two SMs)
// share 256 x 256 tiles; each loads 128 rows of A with their scale atom, one of
// the two weights' 128 rows (CTA 0 gate, CTA 1 up) and both weights' atoms, and
// CTA 0 issues tcgen05.mma.cta_group::2 for both: a third fewer operand bytes
// from L2 than 128 x 256 tiles.  At 8192 x 4096 x 14336 it runs 653 to 688 us
// (747 to 784 back to back, under the power limit).  K = 1024, 2048 and 4096 take
// 227, 362 and 688 us: 0.34 to 0.42 us a stage, where the MMAs alone take about
// 0.38 under the same clocks, and about 1.9 us a tile for its first stages and the
// change of accumulator, which 256 columns and the scales leave tensor memory no
// second copy of.
// The issuing threads are what this kernel was slow by: with one thread running
// each role's loop it took 807 us (882 with descriptors built every stage and a
// commit per CTA), because every operand of a TMA or tcgen05 instruction then
// moved from that thread's registers to uniform ones.  Built and measured before
// that, not kept: gate and up as two N = 128 MMAs over three rotating
// accumulators (1073 us), polling in place of sleeping waits (895 us).
// Single CTAs take the calls of few rows: a stage then holds only the rows of A
// there are (in eights), so that more stages of weights are in flight (16 rows:
// 34.4 -> 22.7 us); the MMA's 128-row window runs on into the bytes behind
// them, which only reach accumulator rows that are never stored.
template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gated_mxfp8_kernel(const __grid_constant__ Args A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if constexpr (PAIR) {
    // Without a two-CTA cluster the paired allocation would wait for a partner that does not exist.
    if (cluster_size() != 2) {
      if (threadIdx.x == 0) atomicOr(A.status, kStatusWaitTimeout);
      return;
    }
  }
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const int first = PAIR ? (int)cluster_id_x() : (int)blockIdx.x, step = PAIR ? (int)n_clusters_x() : (int)gridDim.x;
  Barriers& S = *reinterpret_cast<Barriers*>(smem_raw + (size_t)A.stages * A.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = A.m_tiles * A.n_tiles;
  const int n_k = A.K / kTileK;                  // also the scale atoms of a 128-row block
  const uint32_t b_off = PAIR ? kRows128 : (uint32_t)A.a_rows * kTileK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, PAIR ? 2 * kEpiWarps : kEpiWarps);
    mbar_init(&S.mma_done, 1);
    S.failed = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc<PAIR>(&S.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();        // both CTAs' barriers and allocation are in place
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  uint32_t n_issued = 0;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    uint32_t s = 0, ph = 1;
    bool ok = true;
    // bytes a CTA brings into a stage
    const uint32_t bytes = (PAIR ? 2 * kRows128 : b_off + 2 * kRows128) + 3 * kAtom;
    for (int t = first; t < tiles && ok; t += step) {
      if (__any_sync(0xFFFFFFFFu, failed_flag(S))) break;
      int mt, nt;
      tile_pos(A, t, &mt, &nt);
      const int mb = PAIR ? 2 * mt + (int)rank : mt;             // this CTA's 128-row block of A
      for (int kb = 0; kb < n_k; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&S.empty[s], ph, A.status));
        if (!ok) break;
        const uint32_t bar = PAIR ? cluster_addr(&S.full[s], 0) : smem_u32(&S.full[s]);
        if (leader) {
          uint8_t* sa = smem_raw + (size_t)s * A.stage_bytes;
          uint8_t* sf = sa + A.sf_off;
          if (rank == 0) mbar_arrive_expect_tx(&S.full[s], PAIR ? 2 * bytes : bytes);
          tma_load<PAIR>(sa, &A.a, kb * kTileK, mb * 128, bar);
          if constexpr (PAIR) {
            tma_load<PAIR>(sa + b_off, &A.w[rank], kb * kTileK, nt * kTileF, bar);
            // atom (block, kb) is rows 4 * (block * n_k + kb) .. + 3 of the 128-byte-row view; a block of A past the
            // last has no atom: it repeats the tile's first, for rows that are never stored
            const int ab = mb * 128 < A.T ? mb : 2 * mt;
            tma_load<PAIR>(sf, &A.a_sf, 0, 4 * (ab * n_k + kb), bar);
            tma_load<PAIR>(sf + kAtom, &A.w_sf[0], 0, 4 * (nt * n_k + kb), bar);
            tma_load<PAIR>(sf + 2 * kAtom, &A.w_sf[1], 0, 4 * (nt * n_k + kb), bar);
          } else {
            uint64_t* full = &S.full[s];
            tma_load<PAIR>(sa + b_off, &A.w[0], kb * kTileK, nt * kTileF, bar);
            tma_load<PAIR>(sa + b_off + kRows128, &A.w[1], kb * kTileK, nt * kTileF, bar);
            bulk_g2s_plain(sf, A.a_s + ((size_t)mb * n_k + kb) * kAtom, kAtom, full);
            bulk_g2s_plain(sf + kAtom, A.w_s[0] + ((size_t)nt * n_k + kb) * kAtom, kAtom, full);
            bulk_g2s_plain(sf + 2 * kAtom, A.w_s[1] + ((size_t)nt * n_k + kb) * kAtom, kAtom, full);
          }
        }
        __syncwarp();
        ++n_issued;
        if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
      }
    }
    if (!ok && leader) atomicOr(&S.failed, 1u);
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------ MMA (of a pair: CTA 0)
      const bool leader = elect_one();
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = true;
      auto commit = [&](uint64_t* bar) {         // to both CTAs of a pair
        if (leader) {
          if constexpr (PAIR) tc_commit_both(smem_u32(bar));
          else tc_commit(bar);
        }
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, A.status));
        tc_fence_after();
      };
      const uint32_t base = smem_u32(smem_raw), stage4 = A.stage_bytes >> 4;
      const uint64_t a_desc = smem_desc(base, 16, 1024, 2), b_desc = smem_desc(base + b_off, 16, 1024, 2),
                     sf_desc = smem_desc(base + A.sf_off, 0, 128, 0);
      for (int t = first; t < tiles && ok; t += step, ++it) {
        if (__any_sync(0xFFFFFFFFu, failed_flag(S))) ok = false;
        wait(&S.acc_empty, (it & 1u) ^ 1u);
        for (int kb = 0; kb < n_k && ok; ++kb) {
          wait(&S.full[s], ph);
          if (!ok) break;
          // descriptors: the start address (>> 4) is the low field
          const uint32_t at = s * stage4, sfa = tmem + kSfCol0 + s * 12u, sfb = sfa + 4u;
          if (leader) {
#pragma unroll
            for (int j = 0; j < 3; ++j) tmem_cp_sf<PAIR>(sfa + 4u * j, sf_desc + (at + j * (kAtom >> 4)));
#pragma unroll
            for (int k = 0; k < kTileK / 32; ++k)
              mma_mxf8<PAIR>(tmem, a_desc + (at + 2 * k), b_desc + (at + 2 * k), instr_desc(PAIR ? 256 : 128, (uint32_t)k),
                             sfa | ((uint32_t)k << 30), sfb | ((uint32_t)k << 30), (kb > 0 || k > 0) ? 1u : 0u);
          }
          commit(&S.empty[s]);
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
        }
        if (ok) commit(&S.acc_full);
      }
      if (leader) {
        if (!ok) atomicOr(&S.failed, 1u);
        if constexpr (PAIR) tc_commit_pair(smem_u32(&S.mma_done));
        else tc_commit(&S.mma_done);
      }
      __syncwarp();
      if (!ok) commit(&S.acc_full);              // wake the epilogues; they see the failure or time out
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;            // features 64 * half .. of the tile
    uint32_t it = 0;
    for (int t = first; t < tiles; t += step, ++it) {
      int mt, nt;
      tile_pos(A, t, &mt, &nt);
      // by vote: the tcgen05.ld of the next tile needs the whole warp, whichever lane's wait gave up
      const bool got = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&S.acc_full, it & 1u, A.status) && !failed_flag(S));
      tc_fence_after();
      if (!got) {
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
      if (lane == 0) {                           // the MMA thread may overwrite the accumulator
        if (rank == 0) mbar_arrive(&S.acc_empty);
        else mbar_arrive_remote(cluster_addr(&S.acc_empty, 0));
      }
      const int row = (PAIR ? 2 * mt + (int)rank : mt) * 128 + quarter * 32 + lane;
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
  if (warp == 1 && lane == 0 && rank == 0) mbar_wait_bounded(&S.mma_done, 0, A.status);
  if (warp == 0 && lane == 0 && rank == 0 && failed_flag(S))   // leave no copy in flight
    for (uint32_t j = (n_issued > (uint32_t)A.stages ? n_issued - A.stages : 0); j < n_issued; ++j)
      mbar_wait_bounded(&S.full[j % A.stages], (j / A.stages) & 1u, A.status);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();        // no MMA, copy or remote arrive into either CTA remains
  tc_fence_after();
  if (warp == 0) tmem_free<PAIR>(tmem, kTmemCols);
}

// 2-D map over a row-major uint8 [rows, cols] matrix, boxes of box_rows x 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows, bool swizzle = true) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols};
  const cuuint32_t box[2] = {(cuuint32_t)kTileK, (cuuint32_t)box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A scale array of a [rows, K] operand as rows of 128 bytes: an atom is a box of 4.
bool make_sf_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K) {
  return make_map(map, base, (rows + 127) / 128 * (K / kTileK) * 4, 128, 4, false);
}

// Ring of a CTA pair.
constexpr size_t kCap = 227 * 1024 - 512;
static_assert(sizeof(Barriers) <= 512, "barrier block");
constexpr uint32_t kPairStage = 2 * kRows128 + 2048;               // 1024-aligned
constexpr int kPairStages = (int)(kCap / kPairStage) < kMaxStages ? (int)(kCap / kPairStage) : kMaxStages;
constexpr size_t kPairSmem = (size_t)kPairStages * kPairStage + sizeof(Barriers);

}  // namespace

int gated_mxfp8_pairs_at_once(int sms) {
  const int pairs = cta_pair_capacity((const void*)gated_mxfp8_kernel<true>, kThreads, kPairSmem, 3);
  return pairs > sms / 2 ? sms / 2 : pairs;
}

// Pairs where their 256-row tiles take fewer rounds of tile time (twice the
// work of a 128-row tile on two SMs).
bool gated_mxfp8_pairs(int T, int F, int sms, int pairs, int64_t* units) {
  const int64_t n_tiles = (F + kTileF - 1) / kTileF;
  const int64_t t1 = (int64_t)((T + 127) / 128) * n_tiles, t2 = (int64_t)((T + 255) / 256) * n_tiles;
  const bool pair = T > 128 && pairs > 0 && (t2 + pairs - 1) / pairs <= (t1 + sms - 1) / sms;
  *units = pair ? t2 : t1;
  return pair;
}

int gated_mxfp8_launch(const void* a_q, const void* a_s, const void* g_q, const void* g_s, const void* u_q,
                       const void* u_s, void* h, void* h_s, int T, int F, int K, int act, bool scale_mma, int sms,
                       unsigned* status, cudaStream_t stream, const char** why) {
  Args A{};
  A.a_s = static_cast<const uint8_t*>(a_s);
  A.w_s[0] = static_cast<const uint8_t*>(g_s);
  A.w_s[1] = static_cast<const uint8_t*>(u_s);
  A.h = static_cast<uint8_t*>(h);
  A.h_s = static_cast<uint8_t*>(h_s);
  A.status = status;
  A.T = T;
  A.F = F;
  A.K = K;
  A.act = act;
  A.out = !h_s ? 0 : (scale_mma ? 2 : 1);
  A.n_tiles = (F + kTileF - 1) / kTileF;

  const void* kernel = (const void*)gated_mxfp8_kernel<true>;
  const int pairs = T > 128 ? gated_mxfp8_pairs_at_once(sms) : 0;
  int64_t tiles;
  const bool pair = gated_mxfp8_pairs(T, F, sms, pairs, &tiles);
  if (tiles > 0x7FFFFFFF - sms) {
    *why = "too many tiles";
    return -1;
  }
  A.m_tiles = pair ? (T + 255) / 256 : (T + 127) / 128;
  A.a_rows = pair || T >= 128 ? 128 : (T + 7) / 8 * 8;
  size_t smem;
  if (pair) {
    A.sf_off = 2 * kRows128;
    A.stage_bytes = kPairStage;
    A.stages = kPairStages;
    smem = kPairSmem;
  } else {
    kernel = (const void*)gated_mxfp8_kernel<false>;
    A.sf_off = (uint32_t)A.a_rows * kTileK + 2 * kRows128;
    A.stage_bytes = A.sf_off + 2048;
    A.stages = (int)(kCap / A.stage_bytes);
    if (A.stages > kMaxStages) A.stages = kMaxStages;
    smem = (size_t)A.stages * A.stage_bytes + sizeof(Barriers);    // B's 32 KiB cover the last stage's A window
  }
  if (!make_map(&A.a, a_q, T, K, A.a_rows) || !make_map(&A.w[0], g_q, F, K, 128) || !make_map(&A.w[1], u_q, F, K, 128) ||
      (pair && (!make_sf_map(&A.a_sf, a_s, T, K) || !make_sf_map(&A.w_sf[0], g_s, F, K) || !make_sf_map(&A.w_sf[1], u_s, F, K)))) {
    *why = "cuTensorMapEncodeTiled failed";
    return -1;
  }
  void* argv[] = {&A};
  const int units = pair ? pairs : sms;
  return launch_kernel(kernel, (tiles < units ? tiles : units) * (pair ? 2 : 1), kThreads, smem, argv, stream,
                       "mxfp8_gated_ffn launch", why, pair);
}

}  // namespace mxn

// gated_ffn.cu -- gated feed-forward projections in bf16 on the tensor cores.
//
// Forward, x [T, D], Wg and Wu [F, D] (one output feature per row):
//   gate = x Wg^T, up = x Wu^T, h = act(gate) * up
// Backward, from dh and the kept gate and up:
//   dg = dh * up * act'(gate), du = dh * act(gate)       (bf16, workspace)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// Products accumulate in fp32 tensor memory; h, dx and the weight gradients are
// rounded once to bf16.  dg and du are rounded to bf16 because they are
// tensor-core operands (one rounding of at most 2^-8 each, as large as an output's;
// the relative error of dx, dWg and dWu goes from 0.0017 to 0.0023 by it).
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

#include <mutex>

#include "activations.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace mxn {
namespace {

enum Mode { kGate, kDx, kDw };

constexpr int kTileK = 64;                       // contraction elements (128 bytes) of a k-block
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;                     // 4 lane quarters x 2 column halves
constexpr int kThreads = 64 + 32 * kEpiWarps;    // producer warp, MMA warp, epilogue warps
constexpr uint32_t kABytes = 128 * kTileK * 2;   // 128 rows of A
constexpr uint32_t kTmemCols = 512;              // two accumulators of up to 256 columns
constexpr uint32_t kBoxBytes = 32 * 128;         // store box of an epilogue warp (pairs): 32 rows x 64 columns
constexpr int kGroupM = 8;                       // tiles go m-first inside groups of 8 tile rows: operand reuse in L2

struct Args {
  CUtensorMap a[2], b[2], c[3];                  // c: outputs, of pairs
  uint16_t* out[3];      // kGate: h, gate, up (the last two may be null); kDx: dx; kDw: dWg, dWu
  float* partial;        // with splits > 1: fp32 [problems, M, N] in place of the outputs
  unsigned* status;
  int64_t ld_out;
  int problems;          // products of one shape: 1 (kDw 2: dWg and dWu) for each split
  int splits;            // parts that the contraction is dealt to; kDw's problem 2 s + i is part s of dW i
  int M, N;              // output rows and columns of one problem
  int m_tiles, n_tiles;  // tiles of one problem (pairs: whole 512-row tiles)
  int tiles, whole;      // work units of all problems; pairs: those that are whole 512-row tiles
  int m_halves;          // pairs: 256-row halves of one problem
  int n_k, n_k0;         // k-blocks of a tile, and of its first segment (kDx)
  int tile_n;            // output columns of a tile (kGate: features, each with a gate and an up column)
  int acc_n;             // accumulator columns: 2 * tile_n (kGate) or tile_n
  int act;
  int a_rows;            // rows of A that a stage of a single CTA holds
  int stages, group;     // ring depth, k-blocks (kTileK elements) a stage holds
  uint32_t stage_bytes, block_bytes;
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t failed;
};
static_assert(sizeof(Barriers) <= 512, "barrier block");
constexpr size_t kSmemCap = 227 * 1024 - 512;    // ring and store boxes

__device__ __forceinline__ bool failed_flag(const Barriers& S) {
  return *reinterpret_cast<const volatile uint32_t*>(&S.failed) != 0;
}

template <bool PAIR>
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
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

// Pairs: units of the last 256-row half when there is an odd number of them.
__host__ __device__ __forceinline__ int odd_halves(const Args& A) {
  return A.m_halves & 1 ? A.problems * A.n_tiles : 0;
}
// Work unit t of the launch: problem, first output row, tile column, and for
// pairs the 256-row halves it covers.
struct TilePos {
  int p, m0, nt, halves;
};
__device__ __forceinline__ TilePos tile_of(const Args& A, int t, int rows) {
  TilePos q;
  const int per = A.m_tiles * A.n_tiles;
  q.p = t / per;
  t -= q.p * per;
  const int span = kGroupM * A.n_tiles;
  const int g0 = t / span * kGroupM;
  const int gm = min(kGroupM, A.m_tiles - g0);
  t -= g0 * A.n_tiles;
  q.m0 = (g0 + t % gm) * rows;
  q.nt = t / gm;
  q.halves = 2;
  return q;
}
template <bool PAIR>
__device__ __forceinline__ TilePos tile_pos(const Args& A, int t) {
  if constexpr (!PAIR) return tile_of(A, t, 128);
  if (t < A.whole) return tile_of(A, t, 512);
  // The tiles past the last full round, as halves; then the odd half row.
  const int all = A.tiles == A.whole ? 0 : (A.tiles - A.whole - odd_halves(A)) / 2;
  t -= A.whole;
  TilePos q;
  if (t < 2 * all) {
    q = tile_of(A, A.whole + t / 2, 512);
    q.m0 += (t & 1) * 256;
  } else {
    t -= 2 * all;
    q.p = t / A.n_tiles;
    q.nt = t - q.p * A.n_tiles;
    q.m0 = (A.m_halves - 1) * 256;
  }
  q.halves = 1;
  return q;
}

// k-blocks [k_lo, k_hi) of problem p.
template <int MODE>
__device__ __forceinline__ int k_lo(const Args& A, int p) {
  return MODE == kGate ? 0 : (int)((int64_t)(MODE == kDw ? p >> 1 : p) * A.n_k / A.splits);
}
template <int MODE>
__device__ __forceinline__ int k_hi(const Args& A, int p) {
  return MODE == kGate ? A.n_k : (int)((int64_t)((MODE == kDw ? p >> 1 : p) + 1) * A.n_k / A.splits);
}

// 16 fp32 columns of one row of a partial product, those below n (a multiple of 8).
__device__ __forceinline__ void store_cols16_f32(float* row, int col, int n, const uint32_t (&r)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + 4 * i < n)
      *reinterpret_cast<uint4*>(row + col + 4 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}

// 16 output columns of one row, from col on, those below n (a multiple of 8).
__device__ __forceinline__ void store_cols16(uint16_t* row, int col, int n, const uint32_t (&o)[8]) {
  if (col < n) *reinterpret_cast<uint4*>(row + col) = make_uint4(o[0], o[1], o[2], o[3]);
  if (col + 8 < n) *reinterpret_cast<uint4*>(row + col + 8) = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void pack16(const uint32_t (&r)[16], uint32_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

template <int ACT>
__device__ __forceinline__ void gate_product_of(const uint32_t (&g)[16], const uint32_t (&u)[16], uint32_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = pack_bf16(act_f<ACT>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                     act_f<ACT>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
}
__device__ __forceinline__ void gate_product(int act, const uint32_t (&g)[16], const uint32_t (&u)[16], uint32_t (&o)[8]) {
  if (act == kActSilu) gate_product_of<kActSilu>(g, u, o);
  else if (act == kActGelu) gate_product_of<kActGelu>(g, u, o);
  else gate_product_of<kActGeluTanh>(g, u, o);
}

// 2-D tensor copy shared -> global of a store box (clipped at the tensor's
// edges), tracked by the issuing thread's bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
               "r"(smem_u32(src))
               : "memory");
}

// Persistent CTAs, one per SM, walk the output tiles.  Warp 0 streams K stages
// of both operands into a shared-memory ring with TMA tensor copies (out of
// range rows and columns arrive as zeros); warp 1 issues tcgen05.mma; warps
// 2..9 drain the accumulators.  Every wait is bounded, as in gemm_mxfp8.cu.
//
// Single CTAs: tiles of 128 rows x tile_n columns, two accumulators in turn,
// direct stores -- few rows, where many narrow tiles stream the weights.  Below
// 128 rows a stage holds only the rows of A there are (in eights), so that more
// stages of weights are in flight; the MMA's 128-row window runs on into the
// bytes behind them, which only reach accumulator rows that are never stored.
// PAIR: two CTAs (a cluster on two SMs) share tiles of 512 x 256, in two M = 256
// accumulators on one B.  Each CTA loads its 128 rows of either 256-row half of
// A and half of B's 256 -- in kGate CTA 0 the gate rows and CTA 1 the up rows of
// the tile's 128 features, so both accumulators hold both -- and CTA 0 issues
// tcgen05.mma.cta_group::2 for the pair.  What bounds this is the operand
// stream from L2: with 256 x 256 tiles and two accumulators in turn the tensor
// cores were busy 68% of 1456 us forward (8192 x 4096 x 14336, gate and up
// kept), 512 x 256 moves a quarter fewer operand bytes per product and runs
// 1257 us forward and 1237 and 1257 us for the two products of the backward, 93%
// busy; copies left out, the same MMAs take 1205.  Back to back, under the power
// limit: 1410 to 1450 us, and 3000 to 3120 with the backward's element-wise pass.
// Both accumulators fill at once, so a tile's epilogue is exposed, but for
// this: the next tile's first ring of stages goes to the first accumulator
// while the second still drains, and accumulators go back before the stores.
// Results leave through shared memory as 32 x 64 boxes by TMA (direct 16-byte
// stores cost 180 us of the forward).  Tiles past the last full round of pairs
// are dealt as 256-row halves.
// Copies of both CTAs of a pair complete on CTA 0's barriers, one
// tcgen05.commit frees a stage in both, and no copy is multicast.
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gated_gemm_kernel(const __grid_constant__ Args A) {
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
  uint8_t* store_box = smem_raw + (size_t)A.stages * A.stage_bytes;
  Barriers& S = *reinterpret_cast<Barriers*>(store_box + (PAIR ? (size_t)kEpiWarps * kBoxBytes : 0));
  constexpr bool kAmn = MODE == kDw, kBmn = MODE != kGate;
  const uint32_t b_off = PAIR ? 2 * kABytes : (uint32_t)A.a_rows * 128u;   // of a stage: A, then B
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.acc_full[b], 1);
      mbar_init(&S.acc_empty[b], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
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
  const int G = PAIR ? 1 : A.group;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    uint32_t s = 0, ph = 1;
    bool ok = true;
    for (int t = first; t < A.tiles && ok; t += step) {
      const TilePos q = tile_pos<PAIR>(A, t);
      // tiles of one half leave A's second block out
      const uint32_t block_bytes = PAIR && q.halves == 1 ? A.block_bytes - kABytes : A.block_bytes;
      const int k_end = k_hi<MODE>(A, q.p), blocks = PAIR ? q.halves : 1;
      if (__any_sync(0xFFFFFFFFu, failed_flag(S))) break;
      for (int kb0 = k_lo<MODE>(A, q.p); kb0 < k_end; kb0 += G) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&S.empty[s], ph, A.status));
        if (!ok) break;
        const int n = PAIR ? 1 : min(G, k_end - kb0);
        const uint32_t bar = PAIR ? cluster_addr(&S.full[s], 0) : smem_u32(&S.full[s]);
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&S.full[s], PAIR ? 2 * block_bytes : n * block_bytes);
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) { tma_load<PAIR>(dst, map, x, y, bar); };
          for (int g = 0; g < n; ++g) {
            const int kb = kb0 + g;
            uint8_t* sa = smem_raw + (size_t)s * A.stage_bytes + (size_t)g * A.block_bytes;
            uint8_t* sb = sa + b_off;
            if constexpr (MODE == kGate) {
              for (int h = 0; h < blocks; ++h) load(sa + h * kABytes, &A.a[0], kb * kTileK, q.m0 + h * 256 + (int)rank * 128);
              if constexpr (PAIR) {
                load(sb, &A.b[rank], kb * kTileK, q.nt * A.tile_n);
              } else {
                load(sb, &A.b[0], kb * kTileK, q.nt * A.tile_n);
                load(sb + A.tile_n * 128, &A.b[1], kb * kTileK, q.nt * A.tile_n);
              }
            } else {
              const int n0 = q.nt * A.tile_n + (PAIR ? (int)rank * 128 : 0), nb = PAIR ? 128 : A.tile_n;
              const int seg = MODE == kDx && kb >= A.n_k0, k0 = (kb - seg * A.n_k0) * kTileK;
              for (int h = 0; h < blocks; ++h) {
                const int m = q.m0 + h * 256 + (int)rank * 128;
                if constexpr (MODE == kDx) {
                  load(sa + h * kABytes, &A.a[seg], k0, m);
                } else {
                  load(sa + h * kABytes, &A.a[q.p & 1], m, k0);
                  load(sa + h * kABytes + kABytes / 2, &A.a[q.p & 1], m + 64, k0);
                }
              }
              for (int c = 0; c < nb; c += 64) load(sb + c * 128, &A.b[seg], n0 + c, k0);
            }
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
      uint32_t s = 0, ph = 0, it = 0, uses[2] = {0, 0};
      bool ok = true;
      const uint32_t idesc = instr_desc(PAIR ? 256 : 128, A.acc_n, kAmn, kBmn);
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
      // One k-block at `at` (bytes into the ring, >> 4) into accumulator `acc`, from the h-th block of A.
      const uint64_t a_desc = op_desc(smem_u32(smem_raw), 0, kAmn), b_desc = op_desc(smem_u32(smem_raw) + b_off, 0, kBmn);
      auto mma_block = [&](uint32_t at, int h, uint32_t acc, bool first_k) {
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            mma_bf16<PAIR>(tmem + acc * 256u, a_desc + (at + (uint32_t)h * (kABytes >> 4) + (kAmn ? 128u : 2u) * k),
                           b_desc + (at + (kBmn ? 128u : 2u) * k), idesc, (!first_k || k > 0) ? 1u : 0u);
        }
      };
      const uint32_t stage4 = A.stage_bytes >> 4, block4 = A.block_bytes >> 4;
      for (int t = first; t < A.tiles && ok; t += step, ++it) {
        const TilePos q = tile_pos<PAIR>(A, t);
        const int n_k = k_hi<MODE>(A, q.p) - k_lo<MODE>(A, q.p);
        if (__any_sync(0xFFFFFFFFu, failed_flag(S))) ok = false;
        if constexpr (!PAIR) {
          const uint32_t acc = it & 1u;
          wait(&S.acc_empty[acc], (uses[acc]++ & 1u) ^ 1u);
          for (int kb = 0; kb < n_k && ok; kb += G) {
            wait(&S.full[s], ph);
            if (!ok) break;
            const int n = min(G, n_k - kb);
            for (int g = 0; g < n; ++g) mma_block(s * stage4 + g * block4, 0, acc, kb + g == 0);
            commit(&S.empty[s]);
            if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
          }
          if (ok) commit(&S.acc_full[acc]);
        } else {
          const int halves = q.halves;
          const int lead = halves == 2 ? min(n_k, A.stages) : 0;   // stages that go to the first accumulator alone
          wait(&S.acc_empty[0], (uses[0]++ & 1u) ^ 1u);
          uint32_t s1 = s;
          for (int kb = 0; kb < lead && ok; ++kb) {
            wait(&S.full[s], ph);
            if (!ok) break;
            mma_block(s * stage4, 0, 0, kb == 0);
            if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
          }
          if (halves == 2) {
            wait(&S.acc_empty[1], (uses[1]++ & 1u) ^ 1u);
            for (int kb = 0; kb < lead && ok; ++kb) {
              mma_block(s1 * stage4, 1, 1, kb == 0);
              commit(&S.empty[s1]);
              if (++s1 == (uint32_t)A.stages) s1 = 0;
            }
          }
          for (int kb = lead; kb < n_k && ok; ++kb) {
            wait(&S.full[s], ph);
            if (!ok) break;
            mma_block(s * stage4, 0, 0, kb == 0);
            if (halves == 2) mma_block(s * stage4, 1, 1, kb == 0);
            commit(&S.empty[s]);
            if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1u; }
          }
          if (ok) commit(&S.acc_full[0]);
          if (ok && halves == 2) commit(&S.acc_full[1]);
        }
      }
      if (leader) {
        if (!ok) atomicOr(&S.failed, 1u);
        if constexpr (PAIR) tc_commit_pair(smem_u32(&S.mma_done));
        else tc_commit(&S.mma_done);
      }
      __syncwarp();
      if (!ok) {                                 // wake the epilogues; they see the failure or time out
        commit(&S.acc_full[0]);
        commit(&S.acc_full[1]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;                // tcgen05.ld reaches lanes 32 * (warp % 4) ..
    const int half = (warp - 2) >> 2;
    uint8_t* box = store_box + (size_t)(warp - 2) * kBoxBytes;
    // 16 columns (32 bytes) of this lane's row to the store box: 128-byte swizzle
    auto put2 = [&](int col8, const uint32_t (&o)[8]) {
      const uint32_t at = smem_u32(box) + 128u * lane;
      sts128(at + 16u * (col8 ^ (lane & 7)), make_uint4(o[0], o[1], o[2], o[3]));
      sts128(at + 16u * ((col8 + 1) ^ (lane & 7)), make_uint4(o[4], o[5], o[6], o[7]));
    };
    // The MMA thread may overwrite the accumulator.
    auto hand_back = [&](uint32_t acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&S.acc_empty[acc]);
        else mbar_arrive_remote(cluster_addr(&S.acc_empty[acc], 0));
      }
    };
    uint32_t it = 0, uses[2] = {0, 0};
    bool ok = true;
    auto wait_full = [&](uint32_t acc) {
      // by vote: the tcgen05.ld of the next tile needs the whole warp, whichever lane's wait gave up
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&S.acc_full[acc], uses[acc]++ & 1u, A.status) && !failed_flag(S));
      tc_fence_after();
      if (!ok && lane == 0) atomicOr(&S.failed, 1u);
      return ok;
    };
    for (int t = first; t < A.tiles && ok; t += step, ++it) {
      const TilePos q = tile_pos<PAIR>(A, t);
      const int row0 = q.m0 + (int)rank * 128 + quarter * 32;        // of the first accumulator; the second: 256 on
      const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
      if constexpr (!PAIR) {
        const uint32_t acc = it & 1u, ta = lanes + acc * 256u;
        if (!wait_full(acc)) break;
        const int row = row0 + lane;
        const bool live = row < A.M;
        const int end = min(A.N, (q.nt + 1) * A.tile_n);
        for (int c = half * 16; c < A.tile_n; c += 32) {
          const int col = q.nt * A.tile_n + c;
          uint32_t r[16], o[8];
          tmem_ld16(ta + (uint32_t)c, r);
          if constexpr (MODE == kGate) {
            uint32_t u[16];
            tmem_ld16(ta + (uint32_t)(A.tile_n + c), u);
            tmem_ld16_fence(r, true);
            tmem_ld16_fence(u, false);
            gate_product(A.act, r, u, o);
            if (live) {
              store_cols16(A.out[0] + (int64_t)row * A.ld_out, col, end, o);
              if (A.out[1]) {
                pack16(r, o);
                store_cols16(A.out[1] + (int64_t)row * A.ld_out, col, end, o);
                pack16(u, o);
                store_cols16(A.out[2] + (int64_t)row * A.ld_out, col, end, o);
              }
            }
          } else {
            tmem_ld16_fence(r, true);
            if (A.partial) {
              if (live) store_cols16_f32(A.partial + ((int64_t)q.p * A.M + row) * A.N, col, end, r);
            } else {
              pack16(r, o);
              if (live) store_cols16(A.out[MODE == kDw ? q.p & 1 : 0] + (int64_t)row * A.ld_out, col, end, o);
            }
          }
          __syncwarp();                          // tcgen05.ld needs the warp converged
        }
        hand_back(acc);
      } else if (MODE == kDx && A.partial) {     // of the products on pairs only dx is ever split
        for (int a = 0; a < q.halves; ++a) {
          if (!wait_full((uint32_t)a)) break;
          const int row = row0 + a * 256 + lane;
          for (int c = half * 128; c < half * 128 + 128; c += 16) {
            uint32_t r[16];
            tmem_ld16(lanes + (uint32_t)(a * 256 + c), r);
            tmem_ld16_fence(r, true);
            if (row < A.M)
              store_cols16_f32(A.partial + ((int64_t)q.p * A.M + row) * A.N, q.nt * A.tile_n + c, A.N, r);
            __syncwarp();
          }
          hand_back((uint32_t)a);
        }
      } else {
        // Boxes of 64 columns a warp: kGate h, gate and up of its 64 features, else two of its 128 columns.  An
        // accumulator goes to registers, packed, and back to the MMA thread before the stores; in the backward, whose
        // contractions can be short, both do (2048 rows: dw 398 -> 369 us; kGate has no registers for it).
        constexpr int kBoxes = MODE == kGate ? 3 : 2, kHeld = MODE == kGate ? 1 : 2;
        uint32_t o[kHeld][kBoxes][4][8];
        const int n_box = MODE == kGate ? (A.out[1] ? 3 : 1) : 2;
        auto drain = [&](int a) {
          const uint32_t ta = lanes + (uint32_t)(a * 256 + half * (MODE == kGate ? 64 : 128));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16], u[16];
            tmem_ld16(ta + 16u * c, r);
            tmem_ld16(ta + (MODE == kGate ? 128u : 64u) + 16u * c, u);
            tmem_ld16_fence(r, true);
            tmem_ld16_fence(u, false);
            if constexpr (MODE == kGate) {
              gate_product(A.act, r, u, o[a % kHeld][0][c]);
              pack16(r, o[a % kHeld][kBoxes - 2][c]);
              pack16(u, o[a % kHeld][kBoxes - 1][c]);
            } else {
              pack16(r, o[a % kHeld][0][c]);
              pack16(u, o[a % kHeld][1][c]);
            }
            __syncwarp();
          }
          hand_back((uint32_t)a);
        };
        auto store = [&](int a, int b) {
          const int row = row0 + a * 256;
          const int col = q.nt * A.tile_n + half * (MODE == kGate ? 64 : 128) + (MODE == kGate ? 0 : b * 64);
          if (lane == 0) bulk_wait_read_all();   // the box before has left
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 4; ++c) put2(2 * c, o[a % kHeld][b][c]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row < A.M && col < A.N) {
            tma_store_2d(&A.c[MODE == kGate ? b : (MODE == kDw ? q.p & 1 : 0)], box, col, row);
            bulk_commit();
          }
        };
        auto store_all = [&](int a) {
#pragma unroll
          for (int b = 0; b < kBoxes; ++b)
            if (b < n_box) store(a, b);
        };
        if (!wait_full(0)) break;
        drain(0);
        if constexpr (MODE == kGate) store_all(0);
        else store(0, 0);
        if (q.halves == 2) {
          if (!wait_full(1)) break;
          drain(1);
        }
        if constexpr (MODE != kGate) store(0, 1);
        if (q.halves == 2) store_all(1);
      }
    }
    if (PAIR && lane == 0) bulk_wait_read_all(); // before the CTA's shared memory goes
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && lane == 0 && rank == 0) mbar_wait_bounded(&S.mma_done, 0, A.status);
  // After a wait gave up, leave no copy in flight: the producer (of a pair, CTA
  // 0's, where both CTAs' copies complete) waits, bounded, for the last issued
  // phase of every stage.
  if (warp == 0 && lane == 0 && rank == 0 && failed_flag(S))
    for (uint32_t j = (n_issued > (uint32_t)A.stages ? n_issued - A.stages : 0); j < n_issued; ++j)
      mbar_wait_bounded(&S.full[j % A.stages], (j / A.stages) & 1u, A.status);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();        // no MMA, copy or remote arrive into either CTA remains
  tc_fence_after();
  if (warp == 0) tmem_free<PAIR>(tmem, kTmemCols);
}

// dg = dh * up * act'(gate), du = dh * act(gate): 8 elements a thread and step.
// Bound by HBM: 3 elements read and 2 written each, 188 us (6.2 TB/s) at 8192 x
// 14336.
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

// bf16 of the sum of the partial products [parts, n] in order, 8 elements a
// thread; those from n0 on go to out1.
__global__ void __launch_bounds__(256) gated_sum_kernel(const float* partial, int parts, int64_t n, int64_t n0, uint16_t* out0,
                                                        uint16_t* out1) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x); i < n; i += 8 * (int64_t)gridDim.x * blockDim.x) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float4 x = *reinterpret_cast<const float4*>(partial + p * n + i);
      const float4 y = *reinterpret_cast<const float4*>(partial + p * n + i + 4);
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
    *reinterpret_cast<uint4*>(i < n0 ? out0 + i : out1 + (i - n0)) =
        make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
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

struct Launch {
  const void* kernel;
  bool pair;
  int grid;
  size_t smem;
};

// Bytes of fp32 partial products of `problems` problems.
size_t partial_bytes(const Args& A, int problems) { return (size_t)problems * A.M * A.N * sizeof(float); }

template <int MODE>
const void* kernel_of(bool pair) {
  return pair ? (const void*)gated_gemm_kernel<MODE, true> : (const void*)gated_gemm_kernel<MODE, false>;
}
const void* kernel_of(int mode, bool pair) {
  return mode == kGate ? kernel_of<kGate>(pair) : mode == kDx ? kernel_of<kDx>(pair) : kernel_of<kDw>(pair);
}

// Ring of a CTA pair.
constexpr uint32_t kPairStage = 3 * kABytes;
constexpr int kPairStages = (int)((kSmemCap - kEpiWarps * kBoxBytes) / kPairStage);
constexpr size_t kPairSmem = (size_t)kPairStages * kPairStage + kEpiWarps * kBoxBytes + sizeof(Barriers);

// Pairs of CTAs that the current device runs at once.
int pairs_at_once(int mode, int sms) {
  const int pairs = cta_pair_capacity(kernel_of(mode, true), kThreads, kPairSmem, mode);
  return pairs > sms / 2 ? sms / 2 : pairs;
}

// Fills the tile and ring geometry of a launch from A's M, N and n_k, for `sms`
// SMs that run `pairs` CTA pairs at once (none are taken for at most 128 rows),
// with `room` bytes for partial products.  Returns false when the tiles
// outnumber an int.
//
// The shape with the least estimated time, from figures measured on B200: a
// single CTA's k-block takes as long as its bytes at 110 GB/s an SM (140 over
// one or two rounds of tiles, 60 where they come from HBM, 90 in kDw), 0.12 us at least; a
// pair's 0.40 us for a 256-row half and 0.66 for a whole tile; a tile 1 us more
// on single CTAs, whose epilogue overlaps (3 where the contraction is the short
// one, over the rows), and 4.5 on pairs, 6.5 with the activation; and all
// operands come from HBM once.  So pairs win
// where there are several rounds of tiles (4096 x 2048 x 5632 forward 130 us,
// 146 on single CTAs; 1000 x 1024 x 2816 19.1 and 15.9).  The
// backward's products may deal the contraction to up to 8 partial products,
// which another kernel adds up (3 us and their bytes at 6 TB/s): without it the
// dx of 333 x 1032 x 2744 took 25 us on 51 of 148 SMs, and the backward of 8192 x
// 512 x 1408 92 us (73 with its dW split, but on single CTAs alone: 768 x 2048
// split on pairs took 138 us, 121 whole).
bool plan_tiles(Args& A, int mode, int problems, int sms, int pairs, size_t room, Launch* L) {
  const int unit = mode == kGate ? 8 : 64, widest = mode == kGate ? 128 : 256;
  A.a_rows = mode == kDw || A.M >= 128 ? 128 : (A.M + 7) / 8 * 8;
  if (A.M <= 128) pairs = 0;
  const double hbm = 128.0 * A.n_k * (A.M + (double)A.N * (mode == kGate ? 2 : 1)) * (mode == kDw ? 2 : 1) / 6.5e6;
  double best = 0;
  auto better = [&](double us) {
    if (best != 0 && us > best) return false;      // equal: the narrower tile, on more SMs
    best = us;
    return true;
  };
  for (int split = 1; split <= (mode == kGate ? 1 : 8) && (split == 1 || A.n_k / split >= 4); ++split) {
    const int probs = problems * split;
    if (split > 1 && partial_bytes(A, probs) > room) break;
    const double nk = (double)A.n_k / split;
    const double sum = split > 1 ? 3.0 + 8.0 * probs * A.M * A.N / 6e6 : 0.0;
    for (int w = widest; w >= unit; w -= unit) {
      const int64_t tiles = (int64_t)cdiv(A.M, 128) * cdiv(A.N, w) * probs, rounds = (tiles + sms - 1) / sms;
      // the second operand streams from HBM where only one row of tiles reads it
      const bool cold = A.M <= 128;
      const double rate = mode == kDw ? 90e3 : rounds <= 2 ? 140e3 : 110e3;
      double kb = (A.a_rows / rate + (mode == kGate ? 2 * w : w) / (cold ? 60e3 : rate)) * 128;
      if (kb < 0.12) kb = 0.12;
      const double stream = rounds * nk * kb;
      if (better((stream > hbm ? stream : hbm) + 2.5 + rounds * (mode == kDw ? 3.0 * w / 256 : 1.0) + sum)) {
        L->pair = false;
        A.tile_n = w;
        A.problems = probs;
        A.splits = split;
      }
    }
    if (pairs > 0 && (split == 1 || mode == kDx)) {
      const int64_t n_tiles = (int64_t)cdiv(A.N, widest) * probs, halves = cdiv(A.M, 256);
      const int64_t whole = halves / 2 * n_tiles, odd = (halves & 1) * n_tiles, rest = whole % pairs;
      const double end = mode == kGate ? 6.5 : 4.5, t1 = nk * 0.40 + end, t2 = nk * 0.66 + end;
      const double us = 2 * rest + odd <= pairs
                            ? (double)(whole / pairs) * t2 + (rest || odd ? t1 : 0.0)
                            : (double)((whole + pairs - 1) / pairs) * t2 + (double)((odd + pairs - 1) / pairs) * t1;
      if (better((us > hbm ? us : hbm) + sum)) {
        L->pair = true;
        A.tile_n = widest;
        A.problems = probs;
        A.splits = split;
      }
    }
  }
  A.n_tiles = cdiv(A.N, A.tile_n);
  A.m_tiles = cdiv(A.M, L->pair ? 256 : 128);
  int64_t tiles = (int64_t)A.m_tiles * A.n_tiles * A.problems;
  if (tiles > 0x7FFFFFFF - sms) return false;
  if (L->pair) {
    A.m_halves = A.m_tiles;
    A.m_tiles = A.m_halves / 2;
    const int64_t whole = (int64_t)A.m_tiles * A.n_tiles * A.problems, odd = odd_halves(A);
    const int64_t rest = whole % pairs;          // past the last full round
    A.whole = (int)(2 * rest + odd <= pairs ? whole - rest : whole);
    tiles = A.whole + 2 * (whole - A.whole) + odd;
  }
  A.tiles = (int)tiles;
  A.acc_n = mode == kGate ? 2 * A.tile_n : A.tile_n;
  if (L->pair) {
    A.stage_bytes = A.block_bytes = kPairStage;
    A.group = 1;
    A.stages = kPairStages;
    L->smem = kPairSmem;
    L->grid = 2 * (A.tiles < pairs ? A.tiles : pairs);
  } else {
    // Small tiles put up to four k-blocks in a stage, 48 KiB in all: a stage's
    // waits and commit cost as much as those tiles' MMAs (7 x 2424 x 640: 13.9 ->
    // 8.6 us, 100 x 4096 x 4096 23.0 -> 17.8).
    A.block_bytes = (uint32_t)(A.a_rows + A.acc_n) * 128u;
    A.group = (int)(49152 / A.block_bytes);
    A.group = A.group < 1 ? 1 : (A.group > 4 ? 4 : A.group);
    A.stage_bytes = A.group * A.block_bytes;
    A.stages = (int)(kSmemCap / A.stage_bytes);
    if (A.stages > kMaxStages) A.stages = kMaxStages;
    // the last block's window of 128 rows of A lies in the shared memory too
    while ((size_t)A.stages * A.stage_bytes - A.block_bytes + kABytes > kSmemCap) --A.stages;
    L->smem = (size_t)A.stages * A.stage_bytes + sizeof(Barriers);
    const size_t window = (size_t)A.stages * A.stage_bytes - A.block_bytes + kABytes;
    if (L->smem < window) L->smem = window;
    L->grid = A.tiles < sms ? A.tiles : sms;
  }
  L->kernel = kernel_of(mode, L->pair);
  return true;
}

// The plans of gate and up [T, F] over D, of dx [T, D] = [dg du] [Wg; Wu] and of
// the two dW [F, D] over T.
bool plan_fwd(Args& A, int T, int D, int F, int sms, int pairs, Launch* L) {
  A.M = T;
  A.N = F;
  A.n_k = A.n_k0 = cdiv(D, kTileK);
  return plan_tiles(A, kGate, 1, sms, pairs, 0, L);
}

bool plan_dx(Args& A, int T, int D, int F, int sms, int pairs, size_t room, Launch* L) {
  A.M = T;
  A.N = D;
  A.n_k0 = cdiv(F, kTileK);
  A.n_k = 2 * A.n_k0;
  return plan_tiles(A, kDx, 1, sms, pairs, room, L);
}

bool plan_dw(Args& A, int T, int D, int F, int sms, int pairs, size_t room, Launch* L) {
  A.M = F;
  A.N = D;
  A.n_k = A.n_k0 = cdiv(T, kTileK);
  return plan_tiles(A, kDw, 2, sms, pairs, room, L);
}

// Bytes of dg and du, rounded up so that the partial products behind them stay aligned.
size_t grads_bytes(int T, int F) { return ((size_t)4 * T * F + 255) / 256 * 256; }

// The product, and the sum of its parts where it was split.
int launch_gemm(const Launch& L, Args& A, int sms, cudaStream_t stream, const char* what, const char** why) {
  void* argv[] = {&A};
  const int e = launch_kernel(L.kernel, L.grid, kThreads, L.smem, argv, stream, what, why, L.pair);
  if (e || !A.partial) return e;
  const float* partial = A.partial;
  int64_t n0 = (int64_t)A.M * A.N, n = n0 * (A.problems / A.splits);
  void* args[] = {&partial, &A.splits, &n, &n0, &A.out[0], &A.out[1]};
  const int64_t need = (n / 8 + 255) / 256, cap = (int64_t)sms * 8;
  return launch_kernel((const void*)gated_sum_kernel, (int)(need < cap ? need : cap), 256, 0, args, stream,
                    "gated_ffn_bwd sum launch", why);
}

// Maps of the outputs (bf16 [rows, cols] dense) for store boxes.
bool make_out_maps(Args& A) {
  for (int i = 0; i < 3; ++i)
    if (A.out[i] && !make_map(&A.c[i], A.out[i], A.M, A.N, A.ld_out, 32)) return false;
  return true;
}

}  // namespace

int cta_pair_capacity(const void* kernel, int threads, size_t smem, int slot) {
  static std::mutex mu;
  static int cached[64][4];                      // pairs + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || slot < 0 || slot >= 4) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev][slot]) return cached[dev][slot] - 1;
  int n = 0;
  if (allow_shared_memory(kernel) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  cached[dev][slot] = n + 1;
  return n;
}

bool gated_ffn_plan(int product, int T, int D, int F, int sms, int pairs, size_t room, FfnPlan* plan) {
  Args A{};
  Launch L;
  const bool ok = product == kPlanGate ? plan_fwd(A, T, D, F, sms, pairs, &L)
                  : product == kPlanDx ? plan_dx(A, T, D, F, sms, pairs, room, &L)
                                       : plan_dw(A, T, D, F, sms, pairs, room, &L);
  if (!ok) return false;
  const int odd = L.pair ? odd_halves(A) : 0;
  *plan = FfnPlan{L.pair, A.tile_n, A.splits, A.tiles, L.pair ? A.whole : 0, L.pair ? A.tiles - A.whole - odd : 0, odd,
                  L.grid};
  return true;
}

int gated_ffn_pairs(int product, int sms) { return pairs_at_once(product, sms); }

int gated_ffn_fwd_launch(const void* x, const void* w_gate, const void* w_up, void* h, void* gate, void* up, int T,
                         int D, int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status,
                         cudaStream_t stream, const char** why) {
  Args A{};
  A.out[0] = static_cast<uint16_t*>(h);
  A.out[1] = static_cast<uint16_t*>(gate);
  A.out[2] = static_cast<uint16_t*>(up);
  A.status = status;
  A.ld_out = F;
  A.act = act;
  Launch L;
  if (!plan_fwd(A, T, D, F, sms, T > 128 ? pairs_at_once(kGate, sms) : 0, &L)) { *why = "too many tiles"; return -1; }
  if (!make_map(&A.a[0], x, T, D, ld_x, A.a_rows) || !make_map(&A.b[0], w_gate, F, D, ld_w, A.tile_n) ||
      !make_map(&A.b[1], w_up, F, D, ld_w, A.tile_n) || (L.pair && !make_out_maps(A))) {
    *why = "cuTensorMapEncodeTiled failed";
    return -1;
  }
  return launch_gemm(L, A, sms, stream, "gated_ffn_fwd launch", why);
}

size_t gated_ffn_bwd_workspace(int T, int D, int F, int sms) {
  // dx is done with its parts before dW's are written
  Args X{}, W{};
  Launch L;
  if (!plan_dx(X, T, D, F, sms, T > 128 ? pairs_at_once(kDx, sms) : 0, SIZE_MAX, &L) ||
      !plan_dw(W, T, D, F, sms, F > 128 ? pairs_at_once(kDw, sms) : 0, SIZE_MAX, &L))
    return 0;
  const size_t x = X.splits > 1 ? partial_bytes(X, X.problems) : 0, w = W.splits > 1 ? partial_bytes(W, W.problems) : 0;
  return grads_bytes(T, F) + (x > w ? x : w);
}

int gated_ffn_bwd_launch(const void* dh, const void* x, const void* w_gate, const void* w_up, const void* gate,
                         const void* up, void* dx, void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes,
                         int T, int D, int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status, cudaStream_t stream,
                         const char** why) {
  uint16_t* dg = static_cast<uint16_t*>(workspace);
  uint16_t* du = dg + (int64_t)T * F;
  const uint16_t *dhp = static_cast<const uint16_t*>(dh), *gp = static_cast<const uint16_t*>(gate),
                 *upp = static_cast<const uint16_t*>(up);
  int64_t n8 = (int64_t)T * F / 8;
  void* argv[] = {&dhp, &gp, &upp, &dg, &du, &n8};
  const int64_t blocks = (n8 + 255) / 256, most = (int64_t)sms * 8;
  const void* k = act == kActSilu ? (const void*)gated_act_bwd_kernel<kActSilu>
                                  : (act == kActGelu ? (const void*)gated_act_bwd_kernel<kActGelu>
                                                     : (const void*)gated_act_bwd_kernel<kActGeluTanh>);
  int e = launch_kernel(k, (int)(blocks < most ? blocks : most), 256, 0, argv, stream, "gated_ffn_bwd activation launch", why);
  if (e) return e;
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + grads_bytes(T, F));
  const size_t room = workspace_bytes > grads_bytes(T, F) ? workspace_bytes - grads_bytes(T, F) : 0;
  if (dx) {
    Args A{};
    Launch L;
    A.out[0] = static_cast<uint16_t*>(dx);
    A.status = status;
    A.ld_out = D;
    if (!plan_dx(A, T, D, F, sms, T > 128 ? pairs_at_once(kDx, sms) : 0, room, &L)) { *why = "too many tiles"; return -1; }
    if (A.splits > 1) A.partial = partial;
    if (!make_map(&A.a[0], dg, T, F, F, A.a_rows) || !make_map(&A.a[1], du, T, F, F, A.a_rows) ||
        !make_map(&A.b[0], w_gate, F, D, ld_w, kTileK) || !make_map(&A.b[1], w_up, F, D, ld_w, kTileK) ||
        (L.pair && !make_out_maps(A))) {
      *why = "cuTensorMapEncodeTiled failed";
      return -1;
    }
    e = launch_gemm(L, A, sms, stream, "gated_ffn_bwd dx launch", why);
    if (e) return e;
  }
  if (dw_gate) {
    Args A{};
    A.out[0] = static_cast<uint16_t*>(dw_gate);
    A.out[1] = static_cast<uint16_t*>(dw_up);
    A.status = status;
    A.ld_out = D;
    Launch L;
    if (!plan_dw(A, T, D, F, sms, F > 128 ? pairs_at_once(kDw, sms) : 0, room, &L)) { *why = "too many tiles"; return -1; }
    if (A.splits > 1) A.partial = partial;
    if (!make_map(&A.a[0], dg, T, F, F, kTileK) || !make_map(&A.a[1], du, T, F, F, kTileK) ||
        !make_map(&A.b[0], x, T, D, ld_x, kTileK) || (L.pair && !make_out_maps(A))) {
      *why = "cuTensorMapEncodeTiled failed";
      return -1;
    }
    e = launch_gemm(L, A, sms, stream, "gated_ffn_bwd dw launch", why);
    if (e) return e;
  }
  return 0;
}

}  // namespace mxn

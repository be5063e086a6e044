// gated_ffn.h -- launchers of the bf16 gated feed-forward kernels (gated_ffn.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxn {

enum { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };

// Arguments are checked by the caller: T >= 1; D, F, ld_x, ld_w multiples of 8;
// pointers 16-byte aligned; sizes below 2^31.  Return 0, or non-zero with *why set.
int gated_ffn_fwd_launch(const void* x, const void* w_gate, const void* w_up, void* h, void* gate, void* up, int T,
                         int D, int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status,
                         cudaStream_t stream, const char** why);

// Scratch of the backward: dg and du, and the partial products of dx or of dW
// (one after the other in the same place) where few tiles split the contraction.
size_t gated_ffn_bwd_workspace(int T, int D, int F, int sms);

// dx, and the pair dw_gate, dw_up, may be null.  workspace_bytes: at least dg and
// du's (4 T F); contractions are split into the parts that the rest has room for.
int gated_ffn_bwd_launch(const void* dh, const void* x, const void* w_gate, const void* w_up, const void* gate,
                         const void* up, void* dx, void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes,
                         int T, int D, int F, int64_t ld_x, int64_t ld_w, int act, int sms, unsigned* status,
                         cudaStream_t stream, const char** why);

// How a product is dealt to `sms` SMs that run `pairs` CTA pairs at once, with `room` bytes for partial products: host
// arithmetic alone.
struct FfnPlan {
  int pair, tile_n, splits;          // CTA pairs; output columns of a tile; parts of the contraction
  int units, whole, dealt, odd;      // work units; of them, for pairs: 512-row tiles, halves of tiles that were dealt out, odd halves
  int grid;                          // CTAs
};
enum { kPlanGate = 0, kPlanDx = 1, kPlanDw = 2 };
bool gated_ffn_plan(int product, int T, int D, int F, int sms, int pairs, size_t room, FfnPlan* plan);
// The pairs that the current device runs at once.
int gated_ffn_pairs(int product, int sms);

}  // namespace mxn

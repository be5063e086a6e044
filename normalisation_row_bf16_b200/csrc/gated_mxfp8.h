// gated_mxfp8.h -- launcher of the MXFP8 gated feed-forward kernel (gated_mxfp8.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mxn {

// Arguments are checked by the caller: T >= 1; K % 128 == 0; F a multiple of 8
// (bf16 output) or 32 (E4M3 output); pointers 16-byte aligned; sizes below
// 2^31.  h_s is null for bf16 output.  scale_mma: layout of h_s.
// Returns 0, or non-zero with *why set.
int gated_mxfp8_launch(const void* a_q, const void* a_s, const void* g_q, const void* g_s, const void* u_q,
                       const void* u_s, void* h, void* h_s, int T, int F, int K, int act, bool scale_mma, int sms,
                       unsigned* status, cudaStream_t stream, const char** why);

// Whether the call takes CTA pairs, on `sms` SMs that run `pairs` of them at once, and its work units.
bool gated_mxfp8_pairs(int T, int F, int sms, int pairs, int64_t* units);
// The pairs that the current device runs at once.
int gated_mxfp8_pairs_at_once(int sms);

}  // namespace mxn

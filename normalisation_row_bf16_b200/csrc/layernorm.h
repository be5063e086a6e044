// layernorm.h -- launchers of the layer-norm kernels (layernorm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxn {

enum { kDtypeBF16 = 0, kDtypeFP16 = 1, kDtypeFP32 = 2 };

// Longest row of the backward: its per-column sums stay in registers.
constexpr int kLnMaxBwdD = 16384;

// Arguments are checked by the caller (T >= 1, D >= 1, bases 16-byte aligned,
// ld >= D).  Return 0 or a cudaError_t, with *why naming the failed step.
int layernorm_fwd_launch(const void* x, const void* gamma, const void* beta, void* y, float* mean, float* rstd,
                         int64_t T, int D, int64_t ld_x, float eps, int dtype, int sms, unsigned* status,
                         cudaStream_t stream, const char** why);

size_t layernorm_bwd_workspace(int64_t T, int D, int dtype, int sms);

int layernorm_bwd_launch(const void* x, const void* dy, const void* gamma, const float* mean, const float* rstd,
                         void* dx, void* dgamma, void* dbeta, int64_t T, int D, int64_t ld_x, int64_t ld_dy,
                         int dtype, void* workspace, int sms, unsigned* status, cudaStream_t stream,
                         const char** why);

}  // namespace mxn

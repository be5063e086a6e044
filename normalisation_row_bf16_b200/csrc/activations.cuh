// activations.cuh -- the gate activations of the feed-forward kernels and
// their derivatives, fp32.
#pragma once

#include <cuda_runtime.h>

namespace mxn {

// 1 / (1 + exp(-z)); 0 and 1 in the limits (exp overflows to infinity).
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// act(g): silu = g s(g); gelu = g Phi(g), the normal distribution function
// through erfc, which keeps its relative accuracy for negative g; gelu_tanh =
// g (1 + tanh z) / 2 = g s(2z) with z = sqrt(2/pi) (g + 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  if constexpr (ACT == 0) return g * sigmoid_f(g);
  else if constexpr (ACT == 1) return 0.5f * g * erfcf(g * -0.70710678118654752f);
  else return g * sigmoid_f(1.5957691216057308f * fmaf(0.044715f * g * g, g, g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void act_grad_f(float g, float* a, float* da) {
  if constexpr (ACT == 0) {
    const float s = sigmoid_f(g);
    *a = g * s;
    *da = s * fmaf(g, 1.0f - s, 1.0f);
  } else if constexpr (ACT == 1) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f);
    *a = g * phi;
    *da = fmaf(g, 0.39894228040143268f * __expf(-0.5f * g * g), phi);
  } else {
    const float s = sigmoid_f(1.5957691216057308f * fmaf(0.044715f * g * g, g, g));
    *a = g * s;
    *da = fmaf(g * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f * g, g, 1.0f), s);
  }
}

}  // namespace mxn

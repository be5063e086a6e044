// activations.cuh -- the gate activations of the feed-forward kernels and
// their derivatives, fp32.
#pragma once

#include <cuda_runtime.h>

namespace mxn {

// 1 / (1 + exp(-z)); 0 and 1 in the limits (exp overflows to infinity).
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// exp(-g^2 / 2) and the normal distribution function Phi(g).  With a = |g| and
// t = 1 / (1 + 0.35 a), Phi(-a) = exp(-a^2 / 2) t P(t): t P(t) is the scaled
// complementary error function erfcx(a / sqrt(2)) / 2, a smooth function of t,
// and P the polynomial of degree 8 that fits it with the least squared relative
// error on a in [0, 14.5] (2e-7 in fp32), so Phi keeps its relative accuracy in
// the lower tail.  A third of the instructions of erfcf, which took 55 of 153 us
// at 512 x 4096 x 14336.
__device__ __forceinline__ float normal_cdf(float g, float* e) {
  const float a = fabsf(g), t = __fdividef(1.0f, fmaf(0.35f, a, 1.0f));
  float p = -0.0295296554f;
  p = fmaf(p, t, 0.145783439f);
  p = fmaf(p, t, -0.259327978f);
  p = fmaf(p, t, 0.163135499f);
  p = fmaf(p, t, -0.0257086046f);
  p = fmaf(p, t, 0.106547907f);
  p = fmaf(p, t, 0.119586177f);
  p = fmaf(p, t, 0.139893457f);
  p = fmaf(p, t, 0.139619738f);
  *e = __expf(-0.5f * g * g);
  const float q = *e * (t * p);
  return g < 0.0f ? q : 1.0f - q;
}

// act(g): silu = g s(g); gelu = g Phi(g); gelu_tanh = g (1 + tanh z) / 2 =
// g s(2z) with z = sqrt(2/pi) (g + 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  if constexpr (ACT == 0) return g * sigmoid_f(g);
  else if constexpr (ACT == 1) { float e; return g * normal_cdf(g, &e); }
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
    float e;
    const float phi = normal_cdf(g, &e);
    *a = g * phi;
    *da = fmaf(g, 0.39894228040143268f * e, phi);
  } else {
    const float s = sigmoid_f(1.5957691216057308f * fmaf(0.044715f * g * g, g, g));
    *a = g * s;
    // s (1 - s) is 0 from |g| = 16 on; the square stops there, before it overflows and makes 0 * inf of the term
    const float b = fminf(fabsf(g), 16.0f);
    *da = fmaf(g * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f * b, b, 1.0f), s);
  }
}

}  // namespace mxn

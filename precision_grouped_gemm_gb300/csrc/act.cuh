// Activations of the products with biases (grouped_linear) and their derivatives, in fp32:
//
//   silu     z sigmoid(alpha z)
//   gelu     z Phi(z), Phi the normal distribution function (the exact form, by erfc: no
//            cancellation in the lower tail)
//   swiglu   g sigmoid(alpha g) (u + offset) of the halves [g | u] of z, with limit > 0 clamped
//            first: g <- min(g, limit), u <- clamp(u, -limit, limit)
//
// A NaN stays a NaN through the clamps (comparisons, not minimum and maximum).
#pragma once
#include <cuda_runtime.h>

namespace pgg {

enum Act : int { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

struct ActForm {
  float alpha, offset, limit;  // limit 0: no clamp
};

// 1 / (1 + e^-x).  FAST: the short exponential and quotient, whose error (some 2^-20 at |x| = 10) stays
// far inside the rounding to bf16; fp32 results take the full ones.
template <bool FAST = true>
__device__ __forceinline__ float sigmoid_f(float x) {
  return FAST ? __fdividef(1.0f, 1.0f + __expf(-x)) : 1.0f / (1.0f + expf(-x));
}
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

template <int ACT, bool FAST>
__device__ __forceinline__ float act_f(float z, const ActForm& f) {
  if (ACT == kActSilu) return z * sigmoid_f<FAST>(f.alpha * z);
  if (ACT == kActGelu) return z * normal_cdf(z);
  return z;
}
template <bool FAST>
__device__ __forceinline__ float swiglu_f(float g, float u, const ActForm& f) {
  if (f.limit > 0.0f) {
    g = g > f.limit ? f.limit : g;
    u = u > f.limit ? f.limit : u < -f.limit ? -f.limit : u;
  }
  return g * sigmoid_f<FAST>(f.alpha * g) * (u + f.offset);
}

// dy act'(z)
template <int ACT>
__device__ __forceinline__ float act_bwd_f(float dy, float z, const ActForm& f) {
  if (ACT == kActSilu) {
    const float s = sigmoid_f(f.alpha * z);
    return dy * (s * (1.0f + f.alpha * z * (1.0f - s)));
  }
  if (ACT == kActGelu) return dy * (normal_cdf(z) + z * 0.39894228040143268f * __expf(-0.5f * z * z));
  return dy;
}
// Gradients of g and u; none passes where a clamp is active.
__device__ __forceinline__ void swiglu_bwd_f(float dy, float g, float u, const ActForm& f, float& dg, float& du) {
  bool over_g = false, over_u = false;
  if (f.limit > 0.0f) {
    over_g = g > f.limit;
    over_u = u > f.limit || u < -f.limit;
    g = over_g ? f.limit : g;
    u = u > f.limit ? f.limit : u < -f.limit ? -f.limit : u;
  }
  const float s = sigmoid_f(f.alpha * g);
  dg = over_g ? 0.0f : dy * (u + f.offset) * (s * (1.0f + f.alpha * g * (1.0f - s)));
  du = over_u ? 0.0f : dy * g * s;
}

}  // namespace pgg

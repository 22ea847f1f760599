// Activations of the products with biases (grouped_linear) and their derivatives, in fp32:
//
//   silu     z sigmoid(alpha z)
//   gelu     z Phi(z), Phi the normal distribution function (the exact form; by e^(-z^2/2) times a fitted
//            polynomial, normal_cdf_f2: no cancellation in the lower tail)
//   swiglu   g sigmoid(alpha g) (u + offset) of the halves [g | u] of z, with limit > 0 clamped
//            first: g <- min(g, limit), u <- clamp(u, -limit, limit)
//
// A NaN stays a NaN through the clamps.
#pragma once
#include <cuda_runtime.h>

#include "packed.cuh"

namespace pgg {

enum Act : int { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

struct ActForm {
  float alpha, offset, limit;  // limit 0: no clamp
};

// e^x.  FAST: the short exponential, whose error (some 2^-20 at |x| = 10) stays far inside the rounding to
// bf16; fp32 Y takes the full one.  The gradient has the short one throughout, its fp32 sums too: a term is off by
// 2^-22 |dY| from it (e^-x is largest where its share of the sigmoid is smallest), no more than the sum's own additions.
template <bool FAST>
__device__ __forceinline__ float exp_f(float x) {
  return FAST ? __expf(x) : expf(x);
}
// 1 / (1 + e^-x), the quotient to two units of the last place.
template <bool FAST = true>
__device__ __forceinline__ float sigmoid_f(float x) {
  return __fdividef(1.0f, 1.0f + exp_f<FAST>(-x));
}

// The normal distribution function, two at a time, from e = exp(-z^2 / 2): Phi(-|z|) / e =
// erfcx(|z| / sqrt 2) / 2 is t P(t) with t = 1 / (1 + 0.3 |z|) and a polynomial P fitted to it over |z| <= 14.  The
// relative error of the fit is below 1.7e-7; in fp32 arithmetic 4.3e-7, and 8e-7 with a quotient that is off by its two
// units, in the tail too.
__device__ __forceinline__ f2 normal_cdf_f2(f2 z, f2 e) {
  float a, b, c, d;
  split2(z, a, b);
  split2(fma2(make2(fabsf(a), fabsf(b)), both(0.3f), both(1.0f)), c, d);
  const f2 t = make2(__fdividef(1.0f, c), __fdividef(1.0f, d));
  f2 p = fma2(both(0.035674799233675f), t, both(-0.15720318257808685f));
  p = fma2(p, t, both(0.20635367929935455f));
  p = fma2(p, t, both(-0.05368379130959511f));
  p = fma2(p, t, both(0.12856170535087585f));
  p = fma2(p, t, both(0.09991347044706345f));
  p = fma2(p, t, both(0.12075395882129669f));
  p = fma2(p, t, both(0.11962930113077164f));
  split2(mul2(mul2(p, t), e), c, d);
  return make2(a < 0.0f ? c : 1.0f - c, b < 0.0f ? d : 1.0f - d);
}
// exp(-z^2 / 2)
template <bool FAST = true>
__device__ __forceinline__ f2 gauss_f2(f2 z) {
  float a, b;
  split2(mul2(mul2(z, z), both(-0.5f)), a, b);
  return make2(exp_f<FAST>(a), exp_f<FAST>(b));
}

// Minimum and maximum that a NaN goes through.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_f(float z, const ActForm& f) {
  if (ACT == kActSilu) return z * sigmoid_f<FAST>(f.alpha * z);
  if (ACT == kActGelu) {
    const f2 v = both(z);
    float lo, hi;
    split2(mul2(v, normal_cdf_f2(v, gauss_f2<FAST>(v))), lo, hi);
    return lo;
  }
  return z;
}
template <bool FAST>
__device__ __forceinline__ float swiglu_f(float g, float u, const ActForm& f) {
  if (f.limit > 0.0f) {
    g = min_nan(g, f.limit);
    u = max_nan(min_nan(u, f.limit), -f.limit);
  }
  return g * sigmoid_f<FAST>(f.alpha * g) * (u + f.offset);
}

// Two at a time: dy act'(z), and the gradients of g and u, of which none passes where a clamp is active.
__device__ __forceinline__ f2 sigmoid_f2(f2 x) {
  float a, b;
  split2(x, a, b);
  split2(add2(make2(__expf(-a), __expf(-b)), both(1.0f)), a, b);
  return make2(__fdividef(1.0f, a), __fdividef(1.0f, b));
}
// The derivative of v s, s = sigmoid(alpha v), from s and p = v s: s + alpha (p (1 - s)).  In this order nothing that is
// not finite comes up where alpha v passes fp32's range, as 1 + alpha v (1 - s) and its product with s would there.
__device__ __forceinline__ f2 silu_slope_f2(f2 p, f2 s, float alpha) {
  return fma2(both(alpha), mul2(p, fma2(s, both(-1.0f), both(1.0f))), s);
}
template <int ACT>
__device__ __forceinline__ f2 act_bwd_f2(f2 dy, f2 z, const ActForm& f) {
  if (ACT == kActSilu) {
    const f2 s = sigmoid_f2(mul2(z, both(f.alpha)));
    return mul2(dy, silu_slope_f2(mul2(z, s), s, f.alpha));
  }
  const f2 e = gauss_f2(z);
  return mul2(dy, fma2(mul2(z, both(0.39894228040143268f)), e, normal_cdf_f2(z, e)));
}
__device__ __forceinline__ void swiglu_bwd_f2(f2 dy, f2 g, f2 u, const ActForm& f, f2& dg, f2& du) {
  float g0, g1, u0, u1, a, b;
  bool og0 = false, og1 = false, ou0 = false, ou1 = false;
  if (f.limit > 0.0f) {
    split2(g, g0, g1);
    split2(u, u0, u1);
    og0 = g0 > f.limit;
    og1 = g1 > f.limit;
    ou0 = fabsf(u0) > f.limit;
    ou1 = fabsf(u1) > f.limit;
    g = make2(min_nan(g0, f.limit), min_nan(g1, f.limit));
    u = make2(max_nan(min_nan(u0, f.limit), -f.limit), max_nan(min_nan(u1, f.limit), -f.limit));
  }
  const f2 s = sigmoid_f2(mul2(g, both(f.alpha))), p = mul2(g, s);
  dg = mul2(mul2(dy, add2(u, both(f.offset))), silu_slope_f2(p, s, f.alpha));
  du = mul2(dy, p);
  if (f.limit > 0.0f) {
    split2(dg, a, b);
    dg = make2(og0 ? 0.0f : a, og1 ? 0.0f : b);
    split2(du, a, b);
    du = make2(ou0 ? 0.0f : a, ou1 ? 0.0f : b);
  }
}

}  // namespace pgg

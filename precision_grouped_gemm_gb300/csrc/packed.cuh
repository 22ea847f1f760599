// Pairs of fp32 numbers in one 64-bit register: sm_100's packed arithmetic does two in one issue slot, each
// rounded as the scalar instruction rounds it.
#pragma once
#include "ptx.cuh"

namespace pgg {

struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 make2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 both(float x) { return make2(x, x); }
__device__ __forceinline__ void split2(f2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float sum2(f2 a) {
  float lo, hi;
  split2(a, lo, hi);
  return lo + hi;
}
// Eight bf16 numbers.
__device__ __forceinline__ void unpack2(const uint4& w, f2 (&f)[4]) {
  f[0] = make2(bf16_lo(w.x), bf16_hi(w.x));
  f[1] = make2(bf16_lo(w.y), bf16_hi(w.y));
  f[2] = make2(bf16_lo(w.z), bf16_hi(w.z));
  f[3] = make2(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ uint32_t round2(f2 a) {
  float lo, hi;
  split2(a, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 round8(const f2 (&f)[4]) {
  return make_uint4(round2(f[0]), round2(f[1]), round2(f[2]), round2(f[3]));
}

}  // namespace pgg

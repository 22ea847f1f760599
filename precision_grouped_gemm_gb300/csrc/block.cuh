// Shared by the kernels around the grouped GEMMs (norm, routing, few-token layer): argument
// checks, the MX scale rule on fp32 blocks, and small device helpers.
#pragma once
#include "internal.h"
#include "mx_codec.cuh"
#include "ptx.cuh"

namespace pgg {

inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Asynchronous 16-byte copy to shared memory, and its groups.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// block_scale (mx_codec.cuh) from the fp32 magnitude bits of a block's amax: an fp32 subnormal
// amax has exponent field 0 and clamps to E = -127 like zero.
template <int FMT>
__device__ __forceinline__ bool block_scale_f32(uint32_t amax_bits, uint32_t& code, float& mult) {
  if (amax_bits >= 0x7F800000u) {
    code = 0xFFu;
    mult = 0.0f;
    return false;
  }
  const int e = max((int)(amax_bits >> 23) - 127 - emax<FMT>(), -127);
  code = (uint32_t)(e + 127);
  mult = __uint_as_float((uint32_t)(127 - e) << 23);
  return true;
}

}  // namespace pgg

// The router of an expert layer: a token's k experts and their weights from the gate's logits,
// and the gradient of the logits.
//
//   key_e = logit_e + bias_e in fp32 (bias 0 without one); masked: key_e = -inf
//   S     = the k largest keys, ties to the lowest expert
//   a_e   = exp(logit_e - m) or sigmoid(logit_e); 0 for a masked expert (m: the largest logit of
//           those that Z sums)
//   w_j   = scale a_j / Z, Z = sum of a over all experts (softmax), over S (renormalised; for sigmoids that
//           are all small see kSmallSum), or 1
//
//   softmax over all   dlogit_e = p_e (D_e - sum_j D_j p_j), D_j = scale dw_j, 0 outside S
//   otherwise          dlogit_j = a_j / Z r_j (D_j - [renormalised] sum_i D_i a_i / Z), r_j = 1
//                      (softmax) or sigmoid(-logit_j), and 0 outside S
//
// One warp per token (four tokens for a large batch of bf16 logits), the row's keys in registers: lane l
// holds experts l, l + 32, ...  A key is ordered as an unsigned integer, so that one warp reduction finds
// the largest and a second one the lowest expert that has it.  Everything is fp32; sums run in a fixed
// order.
#include <algorithm>
#include <type_traits>

#include "block.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kRouteWarps = 4;  // tokens per block
constexpr unsigned kAll = 0xffffffffu;

// Order-preserving map of a float (not NaN) to unsigned: -inf maps to 0x007FFFFF, so 0 is below
// every key.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kOrderedNegInf = 0x007FFFFFu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
struct RouteArgs {
  const T* logits;
  const float* bias;  // or nullptr
  int64_t T_;
  int E, k;
  int softmax, renorm;
  float scale;
  int32_t* ids;
  float* w;
  const int32_t* ids_in;  // backward
  const float* dw;
  T* dlogits;
};

// A lane's logits and keys in fp32 of one token; past E: -inf.  (Every load before the first use: 33 x 256
// logits with a bias took 3.5 us with the loads one by one, 2.1 us so.)
template <typename T, int N>
__device__ __forceinline__ void load_row(const RouteArgs<T>& a, const T* row, int lane, float (&x)[N], float (&key)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = load_logit(row + min(lane + 32 * i, a.E - 1));
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = a.bias ? __ldg(a.bias + min(lane + 32 * i, a.E - 1)) : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < a.E ? x[i] + key[i] : -INFINITY;
}

// The logit of a key that has no bias in it.
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// The score of logit v: exp(v - m) or sigmoid(v), which is 0 below fp32's range.
__device__ __forceinline__ float score_of(int softmax, float v, float m) { return softmax ? expf(v - m) : sigmoid(v); }
// The softmax's m from the largest logit: over the choices for renormalised weights, which a bias may
// have chosen far below the others, over all experts otherwise.
__device__ __forceinline__ float shift_of(float top) {
  return top == -INFINITY ? 0.0f : top;  // -inf: every one is masked, all weights are 0
}

// Renormalised sigmoids whose sum is below kSmallSum are taken as exp(v - m) instead, as for a softmax: their
// ratios stay when they leave fp32's range themselves.  That is the same number, 1 + exp(v) being 1 in fp32
// for every one of them.  Below kNoScore, where a mask by the type's lowest value lies, they are 0.
constexpr float kSmallSum = 1e-8f, kNoScore = -700.0f;
constexpr float kSmallLogit = -18.0f;  // the same rule by the largest logit
__device__ __forceinline__ float small_score(bool on, float v, float m) {
  return on && v > kNoScore ? expf(v - m) : 0.0f;
}

// Weights of one token's choices from lane j's expert, its score's argument and whether it counts; m and
// Z: the shift and the sum of weights that are not renormalised.
template <typename T>
__device__ __forceinline__ void write_choice(const RouteArgs<T>& a, int64_t t, int lane, int mine, bool masked, float v,
                                             float m, float Z, bool bad) {
  const bool on = lane < a.k && !masked;
  if (a.softmax && a.renorm) m = shift_of(warp_max(on ? v : -INFINITY));
  float s = on ? score_of(a.softmax, v, m) : 0.0f;
  if (a.renorm) {
    Z = warp_sum(s);
    if (!a.softmax && Z < kSmallSum) {  // (the same in every lane)
      s = small_score(on, v, shift_of(warp_max(on ? v : -INFINITY)));
      Z = warp_sum(s);
    }
  }
  if (lane < a.k) {
    float w = s == 0.0f ? 0.0f : a.scale * s / Z;
    if (bad) w = __uint_as_float(0x7FC00000u);
    a.ids[t * a.k + lane] = mine;
    a.w[t * a.k + lane] = w;
  }
}

// Any logits and a bias: k rounds of the largest key left in the warp, then the lowest expert that
// holds it.  Bound by instructions for many tokens (16384 x 256 fp32, bias, sigmoid, k = 8: 16.2 us; the
// logits at the copy rate: 2.5), by latency for few (33 x 256: 2.1 us).
template <typename T, int N>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs<T> a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T_) return;
  const T* row = a.logits + t * a.E;
  float x[N], f[N];
  uint32_t key[N];
  load_row<T, N>(a, row, lane, x, f);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool nan = f[i] != f[i];  // ranked last
    bad |= nan;
    // -0 counts as +0, which compares equal to it
    key[i] = lane + 32 * i >= a.E ? 0u : nan ? kOrderedNegInf : ordered(f[i] == 0.0f ? 0.0f : f[i]);
    if (key[i] <= kOrderedNegInf) x[i] = -INFINITY;
  }
  bad = __any_sync(kAll, bad);
  float m = 0.0f, Z = 1.0f;
  if (a.softmax && !a.renorm) {
    m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;  // every expert is masked: all weights are 0
    Z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) Z += expf(x[i] - m);
    Z = warp_sum(Z);
  }
  int mine = 0;         // lane j: the expert of choice j
  uint32_t my_key = 0;  // and its key
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (key[i] == top) e = lane + 32 * i;
    e = __reduce_min_sync(kAll, e);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == (uint32_t)(lane + 32 * i)) key[i] = 0;
    if (lane == j) {
      mine = (int)e;
      my_key = top;
    }
  }
  // (with a bias the logit itself is not in the key)
  const float v = a.bias && lane < a.k ? load_logit(row + mine) : unordered(my_key);
  write_choice(a, t, lane, mine, my_key == kOrderedNegInf, v, m, Z, bad);
}

// Sorts a lane's N keys, largest first: the odd-even merge network, 19 exchanges for 8 keys.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(k[i + j], k[i + j + q]);
            k[i + j + q] = min(k[i + j], k[i + j + q]);
            k[i + j] = hi;
          }
}

// The ordered form of a bf16 logit from its key (a negative number's ends in ones).
__device__ __forceinline__ uint32_t ordered_bf16(uint32_t key) {
  return key & 0x80000000u ? key & 0xFFFF0000u : key | 0xFFFFu;
}

// bf16 logits without a bias, the gate of a bf16 model: a key is the 16 ordered bits with the expert,
// counted down, below them.  All keys differ, so one reduction gives both the largest key and the
// lowest expert that has it, and with every lane's keys sorted a round costs the winner's lane a
// shift: 16384 x 256 logits with k = 8 take 9.5 us (the kernel above: 17).
template <int N>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_bf16_kernel(const RouteArgs<__nv_bfloat16> a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T_) return;
  const unsigned short* row = reinterpret_cast<const unsigned short*>(a.logits) + t * a.E;
  uint32_t u[N], key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    u[i] = e < a.E ? (uint32_t)__ldg(row + e) << 16 : 0xFF800000u;  // -inf past the last expert
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    const bool nan = (u[i] & 0x7FFFFFFFu) > 0x7F800000u;
    bad |= nan;
    // the ordered form: -0 as +0, a NaN as -inf
    const uint32_t z = nan ? 0xFF800000u : u[i] == 0x80000000u ? 0u : u[i];
    const uint32_t o = z ^ ((uint32_t)((int32_t)z >> 31) | 0x80000000u);
    key[i] = e < a.E ? (o & 0xFFFF0000u) | (0xFFFFu - e) : 0u;
  }
  bad = __any_sync(kAll, bad);
  sort_keys<N>(key);
  uint32_t my_key = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(kAll, key[0]);
    if (lane == j) my_key = top;
    const bool won = key[0] == top;
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) key[i] = won ? key[i + 1] : key[i];
    key[N - 1] = won ? 0u : key[N - 1];
  }
  const int mine = (int)(0xFFFFu - (my_key & 0xFFFFu));
  const uint32_t o = ordered_bf16(my_key);
  const float v = unordered(o);
  const bool masked = o == kOrderedNegInf;
  float m = 0.0f, Z = 1.0f;
  if (a.softmax && !a.renorm) {
    m = __shfl_sync(kAll, v, 0);    // the first choice is the largest
    if (m == -INFINITY) m = 0.0f;  // every expert is masked: all weights are 0
    Z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) Z += expf(__uint_as_float(u[i]) - m);
    Z = warp_sum(Z);
  }
  write_choice(a, t, lane, mine, masked, v, m, Z, bad);
}

// The same for many tokens, where k <= 8 and rows are whole 16-byte chunks: eight lanes a token, so that a
// warp's work on the choices serves four tokens.  A lane takes eight experts at a time, in pairs of
// 16-bit halves up to their keys, sorts them, and merges them into the eight largest that it has seen:
// the larger of best[i] and key[7 - i] are the eight largest of both, in bitonic order.  Three such
// merges between lanes leave the token's choices in all of them.  Still bound by instructions: 16384 x
// 256, k = 8: 5.5 us (the kernel above: 9.5; the logits at the copy rate: 1.2); 2048 x 256: 2.4 (2.8).
// Up to kManyTokens its longer chain of steps loses: 256 x 256: 2.4 (2.15).  With 64-bit keys, for fp32
// logits or a bias, it gained nothing over the first kernel (17 us).
constexpr int kManyTokens = 1024;
__device__ __forceinline__ void merge_keys(uint32_t (&best)[8], const uint32_t (&key)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) best[i] = max(best[i], key[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const uint32_t hi = max(best[i], best[i + d]);
        best[i + d] = min(best[i], best[i + d]);
        best[i] = hi;
      }
}

__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_bf16_many_kernel(const RouteArgs<__nv_bfloat16> a) {
  constexpr int kAhead = 3;  // chunks in flight
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int64_t t0 = ((int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const int64_t t = t0 < a.T_ ? t0 : a.T_ - 1;  // (lanes past the last token do its work and store nothing)
  const uint4* row = reinterpret_cast<const uint4*>(a.logits + t * a.E);
  const int nvec = a.E >> 3;
  auto load = [&](int v) { return __ldg(row + min(v, nvec - 1)); };  // past the end: keys that are dropped
  uint4 next[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) next[i] = load(l + 8 * i);
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.0f), low = __float2bfloat162_rn(-INFINITY);
  __nv_bfloat162 any = low;  // the maximum of the logits, NaN if there is one
  uint32_t best[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
  for (int v = l; v - l < nvec; v += 8) {
    const uint32_t pair[4] = {next[0].x, next[0].y, next[0].z, next[0].w};
#pragma unroll
    for (int j = 0; j + 1 < kAhead; ++j) next[j] = next[j + 1];
    next[kAhead - 1] = load(v + 8 * kAhead);
    const uint32_t b = 0xFFFFu - 8 * v;
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&pair[i]);
      any = __hmax2_nan(any, x);
      x = __hmax2(__hadd2_rn(x, zero), low);  // -0 as +0, a NaN as -inf
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&x);
      uint32_t neg;  // the halves' signs, spread
      asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(neg) : "r"(u));
      const uint32_t o = u ^ (neg | 0x80008000u);
      key[2 * i] = (o << 16) | (b - 2 * i);
      key[2 * i + 1] = (o & 0xFFFF0000u) | (b - 2 * i - 1);
    }
    if (v >= nvec)
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = 0;
    sort_keys<8>(key);
    merge_keys(best, key);
  }
#pragma unroll 1
  for (int d = 1; d < 8; d <<= 1) {
    uint32_t other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, best[i], d);
    merge_keys(best, other);
  }
  const float2 top = __bfloat1622float2(any);
  const bool bad = (__ballot_sync(kAll, top.x != top.x || top.y != top.y) >> (lane & 24) & 0xFFu) != 0;
  uint32_t my_key = best[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) my_key = l == i ? best[i] : my_key;
  const uint32_t o = ordered_bf16(my_key);
  const bool on = l < a.k && o != kOrderedNegInf;
  const float v = unordered(o), m = shift_of(unordered(ordered_bf16(best[0])));  // the first choice is the largest
  auto sum8 = [](float x) {
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
    return x;
  };
  float Z = 1.0f;
  float s = on ? score_of(a.softmax, v, m) : 0.0f;
  if (a.renorm) {
    Z = sum8(s);
    const bool small = !a.softmax && Z < kSmallSum;
    if (__any_sync(kAll, small)) {  // of one of the four tokens
      const float e = small_score(on, v, m), sum = sum8(e);
      s = small ? e : s;
      Z = small ? sum : Z;
    }
  } else if (a.softmax) {
    Z = 0.0f;
#pragma unroll 1
    for (int i = l; i < nvec; i += 8) {
      float x[8];
      unpack8(__ldg(row + i), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) Z += expf(x[j] - m);
    }
    Z = sum8(Z);
  }
  if (l < a.k && t0 < a.T_) {
    float w = s == 0.0f ? 0.0f : a.scale * s / Z;
    if (bad) w = __uint_as_float(0x7FC00000u);
    a.ids[t * a.k + l] = (int)(0xFFFFu - (my_key & 0xFFFFu));
    a.w[t * a.k + l] = w;
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_bwd_kernel(const RouteArgs<T> a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T_) return;
  const T* row = a.logits + t * a.E;
  float x[N], key[N];
  load_row<T, N>(a, row, lane, x, key);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    bad |= key[i] != key[i];
    if (key[i] == -INFINITY) x[i] = -INFINITY;
  }
  bad = __any_sync(kAll, bad);
  // lane j: choice j (an id outside [0, E) has no part)
  int id = -1;
  float D = 0.0f, v = -INFINITY;
  if (lane < a.k) {
    id = __ldg(a.ids_in + t * a.k + lane);
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) {
      D = a.scale * __ldg(a.dw + t * a.k + lane);
      v = load_logit(row + id);
      if (a.bias && v + __ldg(a.bias + id) == -INFINITY) v = -INFINITY;
      if (v == -INFINITY) D = 0.0f;  // a masked choice has no part, whatever its dw
    }
  }
  const bool full = a.softmax && !a.renorm;
  float p = 0.0f;    // lane j: a_j / Z
  float c = 0.0f;    // lane j: its own term
  float dot = 0.0f;  // sum_j D_j p_j
  if (full) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    float Z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = expf(x[i] - m);
      Z += x[i];
    }
    Z = warp_sum(Z);
    const float inv = 1.0f / Z;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] == 0.0f ? 0.0f : x[i] * inv;
    p = expf(v - m);
    p = p == 0.0f ? 0.0f : p * inv;
    dot = warp_sum(D * p);
    c = D;
  } else {
    // (kSmallSum's rule without its branch, after which other code ran slower: 16384 x 64 softmax logits,
    // k = 6, 6.5 us with it, 6.3 so)
    const bool on = (lane < a.k) & (id >= 0) & (v != -INFINITY) & ((a.softmax != 0) | (v > kNoScore));
    float m = 0.0f;
    if (a.softmax || a.renorm) m = shift_of(warp_max(on ? v : -INFINITY));
    if (a.softmax) {
      p = on ? expf(v - m) : 0.0f;
    } else {
      const bool small = (a.renorm != 0) & (m < kSmallLogit);
      const float e = expf(small ? v - m : -v);
      p = on ? (small ? e : 1.0f / (1.0f + e)) : 0.0f;
    }
    if (a.renorm) {
      const float Z = warp_sum(p);
      p = p == 0.0f ? 0.0f : p / Z;
      dot = warp_sum(D * p);
    }
    c = p * (a.softmax ? 1.0f : sigmoid(-v)) * (D - dot);
  }
  // The row as if nothing were chosen, and then the choices over it.  (Comparing every expert with every
  // choice took 16.9 us for 16384 x 256 bf16 logits, softmax over all, k = 8, where this takes 9.6 us.)
  const float nan = __uint_as_float(0x7FC00000u);
  T* out = a.dlogits + t * a.E;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E) store_logit(out + e, bad ? nan : full ? -x[i] * dot : 0.0f);
  }
  float d = 0.0f;
  for (int j = 0; j < a.k; ++j) {  // choices in order: an expert named twice gets both terms
    const float cj = __shfl_sync(kAll, c, j);
    if (__shfl_sync(kAll, id, j) == id) d += cj;
  }
  __syncwarp();
  if (id >= 0 && !bad) store_logit(out + id, full ? p * (d - dot) : d);
}

template <typename T, bool BWD>
void launch_route(const RouteArgs<T>& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.T_ + kRouteWarps - 1) / kRouteWarps);
  const int n = (a.E + 31) / 32;
  auto go = [&](auto N) {
    if constexpr (BWD) moe_route_bwd_kernel<T, decltype(N)::value><<<grid, kRouteWarps * 32, 0, s>>>(a);
    else {
      if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        if (!a.bias) {
          if (a.k <= 8 && a.E % 8 == 0 && a.T_ > kManyTokens)
            moe_route_bf16_many_kernel<<<(grid + 3) / 4, kRouteWarps * 32, 0, s>>>(a);
          else
            moe_route_bf16_kernel<decltype(N)::value><<<grid, kRouteWarps * 32, 0, s>>>(a);
          return;
        }
      }
      moe_route_kernel<T, decltype(N)::value><<<grid, kRouteWarps * 32, 0, s>>>(a);
    }
  };
  if (n <= 1) go(std::integral_constant<int, 1>());
  else if (n <= 2) go(std::integral_constant<int, 2>());
  else if (n <= 4) go(std::integral_constant<int, 4>());
  else if (n <= 8) go(std::integral_constant<int, 8>());
  else if (n <= 16) go(std::integral_constant<int, 16>());
  else go(std::integral_constant<int, 32>());
}

int check_route(int dtype, int64_t T, int E, int k, int score, int renorm, float scale) {
  if (dtype != PGG_DTYPE_F32 && dtype != PGG_DTYPE_BF16) return PGG_ERR_INVALID_ARG;
  if (score != PGG_SCORE_SOFTMAX && score != PGG_SCORE_SIGMOID) return PGG_ERR_INVALID_ARG;
  if (renorm != 0 && renorm != 1) return PGG_ERR_INVALID_ARG;
  if (E < 1 || E > kMaxGroups || k < 1 || k > 32 || k > E) return PGG_ERR_INVALID_ARG;
  if (T < 0 || T >= ((int64_t)1 << 31) / 32) return PGG_ERR_INVALID_ARG;
  if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return PGG_ERR_INVALID_ARG;
  return PGG_OK;
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_moe_route(const void* logits, int dtype, const float* bias, int64_t T, int E, int k, int score,
                  int renormalize, float scale, int32_t* topk_ids, float* w, void* stream) {
  int st = check_route(dtype, T, E, k, score, renormalize, scale);
  if (st) return st;
  if (T == 0) return PGG_OK;
  if (!logits || !topk_ids || !w) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(logits, 16) || !aligned_to(bias, 4) || !aligned_to(topk_ids, 4) || !aligned_to(w, 4))
    return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto* p) {
    using T_ = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    launch_route<T_, false>(RouteArgs<T_>{p, bias, T, E, k, score == PGG_SCORE_SOFTMAX, renormalize, scale, topk_ids, w,
                                          nullptr, nullptr, nullptr}, s);
  };
  if (dtype == PGG_DTYPE_F32) go(static_cast<const float*>(logits));
  else go(static_cast<const __nv_bfloat16*>(logits));
  return cuda_status(cudaGetLastError());
}

int pgg_moe_route_bwd(const void* logits, int dtype, const float* bias, const int32_t* topk_ids, const float* dw,
                      int64_t T, int E, int k, int score, int renormalize, float scale, void* dlogits,
                      void* stream) {
  int st = check_route(dtype, T, E, k, score, renormalize, scale);
  if (st) return st;
  if (T == 0) return PGG_OK;
  if (!logits || !topk_ids || !dw || !dlogits) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(logits, 16) || !aligned_to(dlogits, 16) || !aligned_to(bias, 4) || !aligned_to(topk_ids, 4) ||
      !aligned_to(dw, 4))
    return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto* p, auto* d) {
    using T_ = std::remove_pointer_t<decltype(d)>;
    launch_route<T_, true>(RouteArgs<T_>{p, bias, T, E, k, score == PGG_SCORE_SOFTMAX, renormalize, scale, nullptr,
                                         nullptr, topk_ids, dw, d}, s);
  };
  if (dtype == PGG_DTYPE_F32) go(static_cast<const float*>(logits), static_cast<float*>(dlogits));
  else go(static_cast<const __nv_bfloat16*>(logits), static_cast<__nv_bfloat16*>(dlogits));
  return cuda_status(cudaGetLastError());
}

}  // extern "C"

// The router of an expert layer: a token's k experts and their weights from the gate's logits,
// and the gradient of the logits.
//
//   key_e = logit_e + bias_e in fp32 (bias 0 without one); masked: key_e = -inf
//   S     = the k largest keys, ties to the lowest expert
//   a_e   = exp(logit_e - max) or sigmoid(logit_e); 0 for a masked expert
//   w_j   = scale a_j / Z, Z = sum of a over all experts (softmax), over S (renormalised), or 1
//
//   softmax over all   dlogit_e = p_e (D_e - sum_j D_j p_j), D_j = scale dw_j, 0 outside S
//   otherwise          dlogit_j = a_j / Z r_j (D_j - [renormalised] sum_i D_i a_i / Z), r_j = 1
//                      (softmax) or sigmoid(-logit_j), and 0 outside S
//
// One warp per token, the row's keys in registers: lane l holds experts l, l + 32, ...  A key is
// ordered as an unsigned integer, so that one warp reduction finds the largest and a second one
// the lowest expert that has it.  Everything is fp32; sums run in a fixed order.
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

// A lane's logits (-inf where masked or past E) and keys of one token; returns whether the row
// holds a NaN key (in any lane).
template <typename T, int N>
__device__ __forceinline__ bool load_row(const RouteArgs<T>& a, const T* row, int lane, float (&x)[N],
                                         uint32_t (&key)[N]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    x[i] = -INFINITY;
    key[i] = 0;
    if (e < a.E) {
      const float v = load_logit(row + e);
      // + 0 turns -0 into +0, which compares equal to it
      const float kf = a.bias ? v + __ldg(a.bias + e) : v + 0.0f;
      const bool nan = kf != kf;
      bad |= nan;
      key[i] = nan ? kOrderedNegInf : ordered(kf == 0.0f ? 0.0f : kf);
      x[i] = key[i] == kOrderedNegInf ? -INFINITY : v;
    }
  }
  return __any_sync(kAll, bad);
}

// The logit of a key that has no bias in it.
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// Weights of one token's choices from lane j's expert, its score's argument and whether it counts.
template <typename T>
__device__ __forceinline__ void write_choice(const RouteArgs<T>& a, int64_t t, int lane, int mine, bool masked, float v,
                                             float m, float Z, bool bad) {
  float s = 0.0f;
  if (lane < a.k && !masked) s = a.softmax ? expf(v - m) : sigmoid(v);
  if (a.renorm) Z = warp_sum(s);
  if (lane < a.k) {
    float w = s == 0.0f ? 0.0f : a.scale * s / Z;
    if (bad) w = __uint_as_float(0x7FC00000u);
    a.ids[t * a.k + lane] = mine;
    a.w[t * a.k + lane] = w;
  }
}

// Any logits and a bias: k rounds of the largest key left in the warp, then the lowest expert that
// holds it.
template <typename T, int N>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs<T> a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T_) return;
  const T* row = a.logits + t * a.E;
  float x[N];
  uint32_t key[N];
  const bool bad = load_row<T, N>(a, row, lane, x, key);
  float m = 0.0f, Z = 1.0f;
  if (a.softmax) {
    m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;  // every expert is masked: all weights are 0
    if (!a.renorm) {
      Z = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) Z += expf(x[i] - m);
      Z = warp_sum(Z);
    }
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

// bf16 logits without a bias, the gate of a bf16 model: a key is the 16 ordered bits with the expert,
// counted down, below them.  All keys differ, so one reduction gives both the largest key and the
// lowest expert that has it, and with every lane's keys sorted a round costs the winner's lane a
// shift.  Bound by instructions: the kernel above took 17.1 us for 16384 x 256 logits with k = 8.
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
  // the logit back from its ordered form (a negative number's ends in ones)
  const uint32_t o = my_key & 0x80000000u ? my_key & 0xFFFF0000u : my_key | 0xFFFFu;
  const float v = unordered(o);
  const bool masked = o == kOrderedNegInf;
  float m = __shfl_sync(kAll, v, 0), Z = 1.0f;  // the first choice is the largest
  if (m == -INFINITY) m = 0.0f;                 // every expert is masked: all weights are 0
  if (a.softmax && !a.renorm) {
    Z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) Z += expf(__uint_as_float(u[i]) - m);
    Z = warp_sum(Z);
  }
  write_choice(a, t, lane, mine, masked, v, m, Z, bad);
}

template <typename T, int N>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_bwd_kernel(const RouteArgs<T> a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T_) return;
  const T* row = a.logits + t * a.E;
  float x[N];
  uint32_t key[N];
  const bool bad = load_row<T, N>(a, row, lane, x, key);
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
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] == 0.0f ? 0.0f : x[i] / Z;
    p = expf(v - m);
    p = p == 0.0f ? 0.0f : p / Z;
    dot = warp_sum(D * p);
    c = D;
  } else {
    if (a.softmax) {
      float m = warp_max(v);
      if (m == -INFINITY) m = 0.0f;
      p = expf(v - m);
    } else {
      p = lane < a.k && id >= 0 ? sigmoid(v) : 0.0f;
    }
    if (a.renorm) {
      const float Z = warp_sum(p);
      p = p == 0.0f ? 0.0f : p / Z;
      dot = warp_sum(D * p);
    }
    c = p * (a.softmax ? 1.0f : sigmoid(-v)) * (D - dot);
  }
  T* out = a.dlogits + t * a.E;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    float d = 0.0f;
    for (int j = 0; j < a.k; ++j) {  // choices in order: an expert named twice gets both terms
      const float cj = __shfl_sync(kAll, c, j);
      const int ij = __shfl_sync(kAll, id, j);
      if (ij == e) d += cj;
    }
    if (full) d = x[i] * (d - dot);
    if (bad) d = __uint_as_float(0x7FC00000u);
    if (e < a.E) store_logit(out + e, d);
  }
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

// Residual addition and RMS norm in front of an expert layer, with the MX operand of the
// next product, and the backward pass.
//
//   s = x + residual            h = bf16(s)
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y = s rstd gamma            stored as bf16 and / or as MX codes and scales
//
// s, the statistics and y are fp32; h, y and the codes are each rounded once, from fp32 (the
// codes are those of y itself, not of its bf16 rounding).
//
//   xh = h rstd, u = dy gamma   dx = dh + rstd (u - xh mean(u xh)),  dgamma = sum_rows dy xh
#include <algorithm>
#include <atomic>

#include "block.cuh"

namespace pgg {
namespace {

// Sum over the block, in a fixed order, in every thread.  `s` holds one float per warp; rows of
// a block alternate between two such buffers, so that one barrier a row is enough.
__device__ __forceinline__ float block_sum(float v, float* s, int nwarps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < nwarps ? s[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
  return t;
}

struct NormArgs {
  const uint4* x;
  const uint4* residual;  // or nullptr
  const uint4* gamma;
  int64_t R;
  int nvec;     // 8-element chunks of a row
  float inv_c;  // 1 / C
  float eps;
  uint4* h;         // outputs: each or nullptr
  uint4* y;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
};

// A block walks rows with a grid stride; thread t owns the row's chunks t, t + blockDim, ...
// (V of them), so a 32-element MX block is held by four neighbouring lanes.  The row stays in registers
// from its load to its outputs, so every byte moves once: memory bounds it.  16384 x 4096 with residual,
// y and e4m3 codes (606 MB): 92.7 us, 96% of the copy rate; 4 x 4096: 2.5 us.
template <int V, int FMT>
__global__ void __launch_bounds__(V == 1 ? 256 : 512) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float s_sum[2][32];
  const int nwarps = blockDim.x >> 5;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x, par ^= 1) {
    const int64_t base = row * a.nvec;
    float s[V][8];
    float sum = 0.0f;
    uint4 xv[V], rv[V];  // every load of the row before the first store (h may be x or residual)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v < a.nvec) {
        xv[j] = a.x[base + v];
        if (a.residual) rv[j] = a.residual[base + v];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v < a.nvec) {
        unpack8(xv[j], s[j]);
        if (a.residual) {
          float r[8];
          unpack8(rv[j], r);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[j][e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += s[j][e] * s[j][e];
        if (a.h) a.h[base + v] = pack8(s[j]);
      }
    }
    const float rstd = rsqrtf(block_sum(sum, s_sum[par], nwarps) * a.inv_c + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      // the four lanes of an MX block are in range together: nvec is a multiple of 4 with FMT
      const bool in = v < a.nvec;
      float y[8];
      if (in) {
        float g[8];
        unpack8(__ldg(a.gamma + v), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = s[j][e] * rstd * g[e];
        if (a.y) a.y[base + v] = pack8(y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.0f;
      }
      if (FMT) {
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = max(am, __float_as_uint(y[e]) & 0x7FFFFFFFu);
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        uint32_t sc;
        float mult;
        const bool fin = block_scale_f32<FMT>(am, sc, mult);
        if (in) {
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = fin ? y[e] * mult : 0.0f;
          if (FMT == kE4M3) {
            uint2 o;
            o.x = cvt_e4m3x2(q[0], q[1]) | (cvt_e4m3x2(q[2], q[3]) << 16);
            o.y = cvt_e4m3x2(q[4], q[5]) | (cvt_e4m3x2(q[6], q[7]) << 16);
            reinterpret_cast<uint2*>(a.codes)[base + v] = o;
          } else {
            reinterpret_cast<uint32_t*>(a.codes)[base + v] =
                cvt_e2m1x2(q[0], q[1]) | (cvt_e2m1x2(q[2], q[3]) << 8) | (cvt_e2m1x2(q[4], q[5]) << 16) |
                (cvt_e2m1x2(q[6], q[7]) << 24);
          }
          if ((v & 3) == 0) a.scales[(base + v) >> 2] = (uint8_t)sc;
        }
      }
    }
  }
}

struct NormBwdArgs {
  const uint4* dy;
  const uint4* dh;  // or nullptr
  const uint4* h;
  const uint4* gamma;
  const float* rstd;
  int64_t R;
  int nvec;
  float inv_c;
  uint4* dx;
  float* part;  // [gridDim.x, C] partial dgamma
};

// The same ownership: a thread's columns stay its own over all rows of the block, so dgamma's
// partial sums are registers, written once per block.  A thread copies its chunks of the next row
// into its own places of shared memory (no thread reads another's, so a wait for its own copies is
// enough): with the loads in registers instead, 8192 x 2880 took 40 us; with three rows ahead, and so
// fewer blocks, 36.5 us; as it is, 33.9 us with the reduction below (189 MB: 27.9 us at the copy
// rate).  Instructions come next: 68% of the issue slots.  With
// t = dy h: dgamma += rstd t, mean(u xh) = rstd mean(t gamma), dx = dh + rstd dy gamma - c h,
// c = rstd^2 mean(u xh): six operations an element besides the conversions.
constexpr int kNormBwdDepth = 2, kNormBwdThreads = 512;
template <int V>
__global__ void __launch_bounds__(V == 1 ? 384 : kNormBwdThreads) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kDepth = kNormBwdDepth;
  extern __shared__ uint4 s_row[];  // [kDepth][3][V][blockDim]
  __shared__ float s_sum[2][32];
  const int nwarps = blockDim.x >> 5;
  float dg[V][8];
  uint4 gam[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    gam[j] = v < a.nvec ? __ldg(a.gamma + v) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[j][e] = 0.0f;
  auto place = [&](int slot, int which, int j) {
    return s_row + ((slot * 3 + which) * V + j) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](int64_t row, int slot) {
    if (row < a.R) {
      const int64_t base = row * a.nvec;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < a.nvec) {
          cp_async_16(smem_u32(place(slot, 0, j)), a.h + base + v);
          cp_async_16(smem_u32(place(slot, 1, j)), a.dy + base + v);
          if (a.dh) cp_async_16(smem_u32(place(slot, 2, j)), a.dh + base + v);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
  int par = 0, slot = 0;
  float rstd_next = __ldg(a.rstd + blockIdx.x);
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x, par ^= 1) {
    const float rstd = rstd_next;
    if (row + gridDim.x < a.R) rstd_next = __ldg(a.rstd + row + gridDim.x);
    fetch(row + (int64_t)(kDepth - 1) * gridDim.x, slot == 0 ? kDepth - 1 : slot - 1);
    cp_async_wait<kDepth - 1>();
    uint4 h[V], y[V], d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[j] = *place(slot, 0, j);
      y[j] = *place(slot, 1, j);
      d[j] = *place(slot, 2, j);
    }
    if (++slot == kDepth) slot = 0;
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v < a.nvec) {
        float x[8], u[8], g[8];
        unpack8(h[j], x);
        unpack8(y[j], u);
        unpack8(gam[j], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = u[e] * x[e];
          dg[j][e] = fmaf(t, rstd, dg[j][e]);
          dot = fmaf(t, g[e], dot);
        }
      }
    }
    const float c = -rstd * rstd * (block_sum(dot, s_sum[par], nwarps) * rstd * a.inv_c);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v < a.nvec) {
        float x[8], u[8], g[8], o[8];
        unpack8(h[j], x);
        unpack8(y[j], u);
        unpack8(gam[j], g);
        if (a.dh) {
          unpack8(d[j], o);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(c, x[e], fmaf(u[e] * g[e], rstd, o[e]));
        a.dx[row * a.nvec + v] = pack8(o);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v < a.nvec) {
      float4* p = reinterpret_cast<float4*>(a.part + ((int64_t)blockIdx.x * a.nvec + v) * 8);
      p[0] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
      p[1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
    }
  }
}

// dgamma[c] = sum over the n partial rows, in a fixed order: a block has eight columns (a 32-byte
// sector of each row), thread (i, c) sums rows i, i + 64, ..., and the 64 sums of a column are
// joined by shuffles and one exchange.  Launched as the dependent of the kernel above (it waits for
// its rows).  456 rows of 2880 (5.3 MB): 6.6 us alone with cold
// caches.
constexpr int kReduceThreads = 512;
__global__ void __launch_bounds__(kReduceThreads) dgamma_reduce_kernel(const float* __restrict__ part, int n, int C,
                                                                       float* __restrict__ dgamma) {
  constexpr int kWarps = kReduceThreads / 32, kGroups = kReduceThreads / 8;
  __shared__ float s[kWarps][8];
  const int c = threadIdx.x & 7, i0 = threadIdx.x >> 3, w = threadIdx.x >> 5;
  const float* p = part + blockIdx.x * 8 + c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float t = 0.0f;
#pragma unroll 4
  for (int i = i0; i < n; i += kGroups) t += p[(int64_t)i * C];
  t += __shfl_xor_sync(0xffffffffu, t, 8);
  t += __shfl_xor_sync(0xffffffffu, t, 16);
  if ((threadIdx.x & 31) < 8) s[w][c] = t;
  __syncthreads();
  if (w == 0) {
    t = 0.0f;
    for (int k = threadIdx.x >> 3; k < kWarps; k += 4) t += s[k][c];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if (threadIdx.x < 8) dgamma[blockIdx.x * 8 + c] = t;
  }
}

// Threads of a block for rows of nvec chunks with V chunks a thread.
int norm_threads(int nvec, int V) { return std::max(32, ((nvec + V - 1) / V + 31) / 32 * 32); }
int norm_v(int nvec) { return nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4; }

// Blocks of the backward pass: a thread block's partial dgamma is one row of the workspace.
// At most as many as are resident at once (each walks its rows; a block of a second wave would start
// when the first ones end), which this bounds for the workspace.
int norm_bwd_v(int nvec) { return nvec <= 384 ? 1 : nvec <= 1024 ? 2 : 4; }
int norm_bwd_blocks(int64_t R, int64_t C) {
  const int V = norm_bwd_v((int)(C / 8)), threads = norm_threads((int)(C / 8), V);
  return (int)std::min<int64_t>(R, 160 * std::max(1, std::min(8, 1536 / threads) >> (V >> 1)));
}

template <int V>
void launch_norm(const NormArgs& a, int fmt, int grid, int threads, cudaStream_t s) {
  if (fmt == kE4M3) add_rmsnorm_kernel<V, kE4M3><<<grid, threads, 0, s>>>(a);
  else if (fmt == kE2M1) add_rmsnorm_kernel<V, kE2M1><<<grid, threads, 0, s>>>(a);
  else add_rmsnorm_kernel<V, 0><<<grid, threads, 0, s>>>(a);
}

}  // namespace

size_t add_rmsnorm_bwd_ws_bytes(int64_t R, int64_t C) {
  return (size_t)norm_bwd_blocks(R, C) * (size_t)C * sizeof(float);
}

int check_norm_dims(int64_t R, int64_t C, int mult) {
  if (R < 0 || R >= ((int64_t)1 << 31) || C < mult || C > PGG_NORM_MAX_COLS) return PGG_ERR_INVALID_ARG;
  return C % mult ? PGG_ERR_ALIGNMENT : PGG_OK;
}

}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_add_rmsnorm(const void* x, const void* residual, const void* gamma, int64_t R, int64_t C, float eps, int fmt,
                    void* h, void* y, uint8_t* codes, uint8_t* scales, float* rstd, void* stream) {
  if (fmt != 0 && fmt != PGG_FMT_E4M3 && fmt != PGG_FMT_E2M1) return PGG_ERR_INVALID_ARG;
  int st = check_norm_dims(R, C, fmt ? 32 : 8);
  if (st) return st;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return PGG_ERR_INVALID_ARG;
  if (R == 0) return PGG_OK;
  if ((fmt != 0) != (codes != nullptr) || (fmt != 0) != (scales != nullptr)) return PGG_ERR_INVALID_ARG;
  if (!x || !gamma || (!h && !y && !codes && !rstd)) return PGG_ERR_INVALID_ARG;
  for (const void* p : {x, residual, gamma, (const void*)h, (const void*)y, (const void*)codes})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(rstd, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  NormArgs a{static_cast<const uint4*>(x), static_cast<const uint4*>(residual), static_cast<const uint4*>(gamma),
             R, (int)(C / 8), 1.0f / (float)C, eps, static_cast<uint4*>(h), static_cast<uint4*>(y), codes, scales,
             rstd};
  const int V = norm_v(a.nvec), threads = norm_threads(a.nvec, V);
  const int grid = (int)std::min<int64_t>(R, (int64_t)dev.sms * std::max(1, 2048 / threads));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (V == 1) launch_norm<1>(a, fmt, grid, threads, s);
  else if (V == 2) launch_norm<2>(a, fmt, grid, threads, s);
  else launch_norm<4>(a, fmt, grid, threads, s);
  return cuda_status(cudaGetLastError());
}

int pgg_add_rmsnorm_bwd_workspace_size(int64_t R, int64_t C, size_t* bytes) {
  const int st = check_norm_dims(R, C, 8);
  if (st) return st;
  if (!bytes) return PGG_ERR_INVALID_ARG;
  *bytes = add_rmsnorm_bwd_ws_bytes(R, C);
  return PGG_OK;
}

int pgg_add_rmsnorm_bwd(const void* dy, const void* dh, const void* h, const void* gamma, const float* rstd,
                        int64_t R, int64_t C, void* dx, float* dgamma, void* ws, size_t ws_bytes, void* stream) {
  int st = check_norm_dims(R, C, 8);
  if (st) return st;
  if (!dgamma) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(dgamma, 16)) return PGG_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) return cuda_status(cudaMemsetAsync(dgamma, 0, (size_t)C * sizeof(float), s));
  if (!dy || !h || !gamma || !rstd || !dx || !ws) return PGG_ERR_INVALID_ARG;
  if (ws_bytes < add_rmsnorm_bwd_ws_bytes(R, C)) return PGG_ERR_INVALID_ARG;
  for (const void* p : {dy, dh, h, gamma, (const void*)dx, (const void*)ws})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(rstd, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  float* part = static_cast<float*>(ws);
  NormBwdArgs a{static_cast<const uint4*>(dy), static_cast<const uint4*>(dh), static_cast<const uint4*>(h),
                static_cast<const uint4*>(gamma), rstd, R, (int)(C / 8), 1.0f / (float)C, static_cast<uint4*>(dx),
                part};
  const int V = norm_bwd_v(a.nvec), threads = norm_threads(a.nvec, V);
  auto kern = V == 1 ? add_rmsnorm_bwd_kernel<1> : V == 2 ? add_rmsnorm_bwd_kernel<2> : add_rmsnorm_bwd_kernel<4>;
  const size_t smem = (size_t)kNormBwdDepth * 3 * V * threads * sizeof(uint4);
  cudaError_t e = cudaSuccess;
  // The most that the kernel is ever launched with, not this call's share: between this line and the launch
  // another thread may make a call of another width.  (V == 1 stays below the 48 KB that need no leave.)
  if (V > 1)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kNormBwdDepth * 3 * V * kNormBwdThreads * sizeof(uint4)));
  // Resident blocks of a configuration: the same on every device that the library runs on, and asked
  // for once (the query takes about a microsecond).
  static std::atomic<int> resident[5][17];
  std::atomic<int>& known = resident[V][threads / 32];
  int per_sm = known.load(std::memory_order_relaxed);
  if (e == cudaSuccess && per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    per_sm = std::max(1, per_sm);
    if (e == cudaSuccess) known.store(per_sm, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return cuda_status(e);
  const int grid = std::min(norm_bwd_blocks(R, C), dev.sms * per_sm);
  kern<<<grid, threads, smem, s>>>(a);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(C / 8));
  cfg.blockDim = dim3(kReduceThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, dgamma_reduce_kernel, (const float*)part, grid, (int)C, dgamma);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // extern "C"

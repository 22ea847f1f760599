// grouped_linear for few rows of X: a cluster of CTAs shares one tile (128 output columns by up to TN
// rows) and cuts its reduction, so that the weights of a small product are read by the whole GPU.  Each
// CTA multiplies its run of K, leaves its sums in its shared memory, and finishes a share of the rows:
// it reads the cluster's sums of them through distributed shared memory, in the order of K, and applies
// the epilogue.  Nothing goes through global memory, so the call needs no workspace.
#include "cluster.cuh"
#include "linear.cuh"

namespace pgg {
namespace {

constexpr int kMaxStages = 8;
constexpr int kRing = 104 * 1024;  // shared memory of the stages: two CTAs an SM
constexpr int kBarOff = kRing;
constexpr int kGroupOff = kBarOff + 256;
// Columns of tensor memory a CTA may take: two CTAs are resident on an SM, and one that waited for columns
// of another cluster's CTA, which waits for its own cluster, would wait for ever.
constexpr int kCols = 256;
size_t split_smem(int G) { return 1024 + (size_t)kGroupOff + 8 * ((size_t)G + 1); }

struct SplitArgs {
  LinArgs a;
  int tn, stages, stage_bytes, accs;  // accs: accumulators that the CTA's run of K is spread over
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
template <bool FAST>
__device__ __forceinline__ float act_any(float z, const LinArgs& a) {
  return a.act == kActSilu ? act_f<kActSilu, FAST>(z, a.form) : a.act == kActGelu ? act_f<kActGelu, FAST>(z, a.form) : z;
}

template <bool GATED, typename T>
__global__ void __launch_bounds__(kLinThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ SplitArgs sa) {
  constexpr int H = GATED ? 2 : 1;
  constexpr bool kFast = !std::is_same<T, float>::value;
  const LinArgs& a = sa.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(done + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + kGroupOff);
  int32_t* s_tile = s_off + (a.G + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), splits = (int)cluster_size();
  const int nct = (a.width + kBN - 1) / kBN, nkb = (a.K + kBK - 1) / kBK;
  const int cols = sa.accs * H * sa.tn;  // of tensor memory: a power of two from 32 on

  if (threadIdx.x == 0) {
    for (int s = 0; s < sa.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    s_ctl->abort = 0;
    s_ctl->limit_ns = a.wait_ns ? a.wait_ns : kWaitTimeoutNs;
    fence_mbar_init();
    fence_proxy_async_smem();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), cols < 32 ? 32 : cols);
    tmem_relinquish();
  }
  if (warp == 2) {
    const bool bad = lin_scan(a, sa.tn, nct, s_off, s_tile, lane);
    if (lane == 0) {
      *s_bad = bad ? 1 : 0;
      if (bad && blockIdx.x == 0) set_error(a.err, kErrBadGroupLens);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int t = (int)cluster_id();
  const bool live = !*s_bad && t < s_tile[a.G];  // (the same in all CTAs of a cluster)
  bool aborted = false;
  LinTile T_{0, 0, 0, 0};
  if (live) {
    GroupCursor cur;
    T_ = lin_tile<kBN, false>(t, a, sa.tn, nct, s_off, s_tile, cur);
  }
  const int k_begin = (int)((long long)nkb * rank / splits), k_end = (int)((long long)nkb * (rank + 1) / splits);
  const int run = live ? k_end - k_begin : 0;
  const int per = (run + sa.accs - 1) / max(1, sa.accs);  // k-blocks of one accumulator
  const int a_bytes = H * kBN * 128;
  const uint32_t ring = smem_u32(smem);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (int i = 0; i < run; ++i) {
      if (a.stall_at >= 0 && k_begin + i >= a.stall_at) break;
      if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
      if (lane == 0) {
        const uint32_t fb = smem_u32(&full[stage]), s = ring + stage * sa.stage_bytes;
        const int k = (k_begin + i) * kBK;
        mbar_arrive_expect_tx(fb, sa.stage_bytes);
        tma_load_3d(s, &tmW, fb, k, T_.col0, T_.g);
        if (GATED) tma_load_3d(s + kBN * 128, &tmW, fb, k, a.width + T_.col0, T_.g);
        tma_load_2d(s + a_bytes, &tmX, fb, k, T_.row0);
      }
      __syncwarp();
      ++issued;
      if (++stage == sa.stages) { stage = 0; phase ^= 1u; }
    }
    if (aborted && lane == 0) {
      int n = min(issued, sa.stages), s = stage;
      uint32_t p = phase;
      for (int i = 0; i < n; ++i) {
        if (--s < 0) { s = sa.stages - 1; p ^= 1u; }
        mbar_wait_drain(smem_u32(&full[s]), p);
      }
    }
  } else if (warp == 1 && run > 0) {
    // ------------------------------------------------------------ products
    const uint32_t idesc = idesc_bf16(kBN, (T_.rows + 15) & ~15, false, false);
    const uint64_t desc = smem_desc(ring, 16, 1024, kSwizzle128B);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < run; ++i) {
      if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      if (lane == 0) {
        const uint64_t da = desc + (uint64_t)(stage * sa.stage_bytes >> 4), db = da + (a_bytes >> 4);
        const uint32_t d = tmem + (i / per) * H * sa.tn;
#pragma unroll
        for (int ks = 0; ks < kBK / 16; ++ks) {
          const uint32_t more = i % per > 0 || ks > 0 ? 1u : 0u;
          mma_f16(d, da + 2 * ks, db + 2 * ks, idesc, more);
          if (GATED) mma_f16(d + sa.tn, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, more);
        }
        mma_commit(smem_u32(&empty[stage]));
      }
      __syncwarp();
      if (++stage == sa.stages) { stage = 0; phase ^= 1u; }
    }
    // every MMA is complete before the sums are read, or, after an abort, before the CTA goes
    if (lane == 0) mma_commit(smem_u32(done));
    __syncwarp();
    if (aborted && lane == 0) mbar_wait_drain(smem_u32(done), 0);
  } else if (warp >= 2 && run > 0) {
    // ------------------------------------------------------------ this CTA's sums: [half][row][128 columns]
    const int q = warp & 3;
    if (!warp_wait(smem_u32(done), 0, s_ctl) || s_ctl->abort) aborted = true;
    aborted = __any_sync(0xffffffffu, aborted);
    if (!aborted) {
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
      const int used = (run + per - 1) / per;
      float* part = reinterpret_cast<float*>(smem);  // (every stage has been read)
#pragma unroll 1
      for (int h = 0; h < H; ++h)
#pragma unroll 1
        for (int c = 0; c < T_.rows; c += 16) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0.0f;
#pragma unroll 1
          for (int i = 0; i < used; ++i) {
            uint32_t r[16];
            tmem_ld16(tb + (i * H + h) * sa.tn + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(h * sa.tn + c + j) * kBN + q * 32 + lane] = v[j];
        }
    }
  }
  __syncwarp();
  cluster_sync();
  // ------------------------------------------------------------ rows rank, rank + splits, ... of the tile
  if (warp >= 2 && run > 0 && !aborted) {
    const int col = T_.col0 + 4 * lane;  // a warp takes a row, a lane four columns
    if (col < a.width) {
      float4 bg = make_float4(0, 0, 0, 0), bu = bg;
      if (a.bias) {
        const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + col;
        bg = load4(b);
        if (GATED) bu = load4(b + a.width);
      }
      for (int r = rank + (warp - 2) * splits; r < T_.rows; r += 4 * splits) {
        const size_t row = (size_t)T_.row0 + r;
        float4 z = bg, u = bu, res = make_float4(0, 0, 0, 0);
        if (a.residual) res = load4(static_cast<const T*>(a.residual) + row * a.width + col);
#pragma unroll 1
        for (int s0 = 0; s0 < splits; s0 += 4) {
          float4 p[4], o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (s0 + i < splits) {
              const uint32_t at = map_rank(ring + (r * kBN + 4 * lane) * 4, s0 + i);
              p[i] = ld_cluster4(at);
              if (GATED) o[i] = ld_cluster4(at + sa.tn * kBN * 4);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (s0 + i < splits) {
              z.x += p[i].x; z.y += p[i].y; z.z += p[i].z; z.w += p[i].w;
              if (GATED) { u.x += o[i].x; u.y += o[i].y; u.z += o[i].z; u.w += o[i].w; }
            }
        }
        if (a.z) {
          store4(a.z + row * a.N + col, z);
          if (GATED) store4(a.z + row * a.N + a.width + col, u);
        }
        if (GATED) {
          z = make_float4(swiglu_f<kFast>(z.x, u.x, a.form), swiglu_f<kFast>(z.y, u.y, a.form), swiglu_f<kFast>(z.z, u.z, a.form),
                          swiglu_f<kFast>(z.w, u.w, a.form));
        } else if (a.act != kActNone) {
          z = make_float4(act_any<kFast>(z.x, a), act_any<kFast>(z.y, a), act_any<kFast>(z.z, a), act_any<kFast>(z.w, a));
        }
        z.x += res.x; z.y += res.y; z.z += res.z; z.w += res.w;
        store4(static_cast<T*>(a.y) + row * a.width + col, z);
      }
    }
  }
  if (aborted && lane == 0) set_error(a.err, kErrTimeout);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the other CTAs have read this one's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols < 32 ? 32 : cols);
  }
}

template <bool GATED, typename T>
int launch(const LinCall& c, int tn, int splits) {
  constexpr int H = GATED ? 2 : 1;
  auto kern = linear_split_kernel<GATED, T>;
  CUtensorMap tw, tx;
  int st = lin_maps(c, (uint32_t)tn, false, &tw, &tx);
  if (st) return st;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)split_smem(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  SplitArgs a{c.a, tn, 0, (H * kBN + tn) * 128, 1};
  a.stages = std::min(kMaxStages, kRing / a.stage_bytes);
  if (c.f32) {  // as many accumulators as there is room for: each takes fewer steps (see linear_kernel)
    const int most = (int)((c.a.K + kBK * splits - 1) / (kBK * splits));
    while (a.accs * 2 * H * tn <= kCols && a.accs < most) a.accs *= 2;
  }
  const int64_t nct = (c.a.width + kBN - 1) / kBN;
  const int64_t live = c.a.group_lens ? std::min<int64_t>(c.a.G, c.a.M) : 1;
  const int64_t tiles = ((c.a.M + tn - 1) / tn + (c.a.group_lens ? live - 1 : 0)) * nct;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * splits));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = split_smem(c.a.G);
  cfg.stream = c.stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

int launch_linear_split(const LinCall& c, const DeviceInfo&, int tn, int splits) {
  if (c.a.act == kActSwiglu)
    return c.f32 ? launch<true, float>(c, tn, splits) : launch<true, __nv_bfloat16>(c, tn, splits);
  return c.f32 ? launch<false, float>(c, tn, splits) : launch<false, __nv_bfloat16>(c, tn, splits);
}

}  // namespace pgg

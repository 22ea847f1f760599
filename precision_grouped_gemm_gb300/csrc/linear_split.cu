// grouped_linear for few rows of X: a cluster of CTAs shares one tile (128 output columns by up to TN
// rows) and cuts its reduction, so that the weights of a small product are read by the whole GPU.  Each
// CTA multiplies its run of K and sends its sums to the CTA that finishes the row, through distributed
// shared memory; that CTA adds them in the order of K and applies the epilogue.  Nothing goes through
// global memory, so the call needs no workspace.  Nobody reads another's memory, so that one barrier of the
// cluster is enough where the sums have a place of their own; many rows' sums take the place of the stages
// instead, when every CTA of the cluster has done with its own.
//
// Latency bounds it: 1 x 4096 x 4096 10.8 us on 5.0 of bytes, of which 2.5 are before the first load has landed
// and 2 behind the last one (sums out, the cluster's barrier, the rows); 37 x 256 x 4096 6.4 us.
#include <atomic>

#include "cluster.cuh"
#include "linear.cuh"

namespace pgg {
namespace {

constexpr int kMaxStages = 12;
// Shared memory: the ring of stages, the sums that this CTA receives (tn > 32: in the ring), barriers,
// group tables.  With more
// CTAs than SMs two share an SM, else one has it, so that its whole run of K can be in flight at once.
constexpr int kSmemTwo = 112 * 1024, kSmemOne = 216 * 1024, kSmemLeast = 80 * 1024;  // (at most two an SM)
// Columns of tensor memory a CTA may take: where two CTAs are resident on an SM, one that waited for columns
// of another cluster's CTA, which waits for its own cluster, would wait for ever.  (No other kernel here whose
// CTAs wait for one another fits beside kSmemLeast.)
constexpr int kColsTwo = 256;

struct SplitArgs {
  LinArgs a;
  int tn, stages, stage_bytes, accs;  // accs: accumulators that the CTA's run of K is spread over
  int own;                            // rows of the tile that a CTA finishes, at most
  int in_ring;                        // the sums are received in the place of the stages
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
__global__ void __launch_bounds__(kLinThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ SplitArgs sa) {
  constexpr int H = GATED ? 2 : 1;
  constexpr bool kFast = !std::is_same<T, float>::value;
  const LinArgs& a = sa.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int ring_bytes = sa.stages * sa.stage_bytes, recv_bytes = (int)cluster_size() * sa.own * H * kBN * 4;
  float* recv = reinterpret_cast<float*>(smem + (sa.in_ring ? 0 : ring_bytes));  // [splits][own][H][128]
  uint64_t* full =
      reinterpret_cast<uint64_t*>(smem + (sa.in_ring ? max(ring_bytes, recv_bytes) : ring_bytes + recv_bytes));
  uint64_t* empty = full + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(done + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(s_bad + 1);
  int32_t* s_tile = s_off + (a.G + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), splits = (int)cluster_size(), lg = 31 - __clz(splits);
  const int nct = (a.width + kBN - 1) / kBN, nkb = (a.K + kBK - 1) / kBK;
  const int cols = sa.accs * H * sa.tn;  // of tensor memory: a power of two from 32 on

  if (threadIdx.x == 0) {
    for (int s = 0; s < sa.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    s_ctl->abort = 0;
    s_ctl->limit_ns = a.wait_ns;
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
  if (!sa.in_ring) cluster_arrive();  // (waited for before the first access to another CTA's memory: it has to be there)
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int t = (int)cluster_id();
  const bool live = !*s_bad && t < s_tile[a.G];  // (the same in all CTAs of a cluster)
  bool aborted = false;
  LinTile T_{0, 0, 0, 0};
  if (live) {
    GroupCursor cur;
    T_ = lin_tile<kBN>(t, a, sa.tn, nct, s_off, s_tile, cur);
  }
  const int k_begin = (int)((long long)nkb * rank / splits), k_end = (int)((long long)nkb * (rank + 1) / splits);
  const int run = live ? k_end - k_begin : 0;
  const int per = (run + sa.accs - 1) / max(1, sa.accs);  // k-blocks of one accumulator
  const int a_bytes = H * kBN * 128;
  const uint32_t ring = smem_u32(smem);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int i = 0; i < run; ++i) {
        if (a.stall_at >= 0 && k_begin + i >= a.stall_at) break;
        if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        const uint32_t fb = smem_u32(&full[stage]), s = ring + stage * sa.stage_bytes;
        const int k = (k_begin + i) * kBK;
        mbar_arrive_expect_tx(fb, sa.stage_bytes);
        tma_load_3d(s, &tmW, fb, k, T_.col0, T_.g);
        if (GATED) tma_load_3d(s + kBN * 128, &tmW, fb, k, a.width + T_.col0, T_.g);
        tma_load_2d(s + a_bytes, &tmX, fb, k, T_.row0);
        ++issued;
        if (++stage == sa.stages) { stage = 0; phase ^= 1u; }
      }
      if (aborted) {
        for (int i = 0, n = min(issued, sa.stages); i < n; ++i) {
          if (--stage < 0) { stage = sa.stages - 1; phase ^= 1u; }
          mbar_wait_drain(smem_u32(&full[stage]), phase);
        }
      }
    }
  } else if (warp == 1 && run > 0) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16(kBN, (T_.rows + 15) & ~15, false, false);
      const uint64_t desc = smem_desc(ring, 16, 1024, kSwizzle128B);
      int stage = 0, left = per;  // k-blocks that the accumulator still takes
      uint32_t phase = 0, d = tmem;
      uint64_t da = desc;
      for (int i = 0; i < run; ++i) {
        if (!mbar_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint64_t db = da + (a_bytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kBK / 16; ++ks) {
          const uint32_t more = left < per || ks > 0 ? 1u : 0u;
          mma_f16(d, da + 2 * ks, db + 2 * ks, idesc, more);
          if (GATED) mma_f16(d + sa.tn, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, more);
        }
        mma_commit(smem_u32(&empty[stage]));
        da += sa.stage_bytes >> 4;
        if (++stage == sa.stages) { stage = 0; phase ^= 1u; da = desc; }
        if (--left == 0) { left = per; d += H * sa.tn; }
      }
      // every MMA is complete before the sums are read, or, after an abort, before the CTA goes
      mma_commit(smem_u32(done));
      if (aborted) mbar_wait_drain(smem_u32(done), 0);
    }
  } else if (warp >= 2 && run > 0) {
    // ------------------------------------------------------------ this CTA's sums: row r to CTA r % splits
    const int q = warp & 3;
    if (!warp_wait(smem_u32(done), 0, s_ctl) || s_ctl->abort) aborted = true;
    aborted = __any_sync(0xffffffffu, aborted);
    // (the stages, whose products are complete, before the sums that others write in their place)
    if (sa.in_ring) cluster_arrive_release();
    cluster_wait();
    if (!aborted) {
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
      const int used = (run + per - 1) / per;
#pragma unroll 1
      for (int h = 0; h < H; ++h)
#pragma unroll 1
        for (int c = 0; c < T_.rows; c += 16) {
          float v[16];
          uint32_t r[16];
          tmem_ld16(tb + h * sa.tn + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
#pragma unroll 1
          for (int i = 1; i < used; i += 2) {
            uint32_t r2[16];
            tmem_ld16(tb + (i * H + h) * sa.tn + c, r);
            if (i + 1 < used) tmem_ld16(tb + ((i + 1) * H + h) * sa.tn + c, r2);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[j] += __uint_as_float(r[j]);
              if (i + 1 < used) v[j] += __uint_as_float(r2[j]);
            }
          }
          const uint32_t at = smem_u32(recv + (rank * sa.own * H + h) * kBN + q * 32 + lane);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < T_.rows)  // (splits is a power of two)
              st_cluster(map_rank(at + ((c + j) >> lg) * (H * kBN * 4), (c + j) & (splits - 1)), v[j]);
        }
    }
  }
  __syncwarp();
  if (warp < 2 || run == 0) {
    if (sa.in_ring) cluster_arrive_release();
    cluster_wait();
  }
  // what the epilogue reads besides the sums: the bias, and the residual of this warp's first row
  const int col = T_.col0 + 4 * lane;  // a warp finishes a row, a lane four columns
  const bool mine = warp >= 2 && run > 0 && !aborted && col < a.width;
  float4 bg = make_float4(0, 0, 0, 0), bu = bg;
  if (mine && a.bias) {
    const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + col;
    bg = load4(b);
    if (GATED) bu = load4(b + a.width);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols < 32 ? 32 : cols);
  }
  if (mine) {
    for (int i = warp - 2; i * splits + rank < T_.rows; i += 4) {
      const size_t row = (size_t)T_.row0 + i * splits + rank;
      float4 z = bg, u = bu, res = make_float4(0, 0, 0, 0);
      if (a.residual) res = load4(static_cast<const T*>(a.residual) + row * a.width + col);
      const float4* from = reinterpret_cast<const float4*>(recv) + i * H * (kBN / 4) + lane;
#pragma unroll 4
      for (int s = 0; s < splits; ++s, from += sa.own * H * (kBN / 4)) {
        const float4 p = from[0];
        z.x += p.x; z.y += p.y; z.z += p.z; z.w += p.w;
        if (GATED) {
          const float4 o = from[kBN / 4];
          u.x += o.x; u.y += o.y; u.z += o.z; u.w += o.w;
        }
      }
      if (a.z) {
        store4(a.z + row * a.N + col, z);
        if (GATED) store4(a.z + row * a.N + a.width + col, u);
      }
      if (GATED) {
        z = make_float4(swiglu_f<kFast>(z.x, u.x, a.form), swiglu_f<kFast>(z.y, u.y, a.form),
                        swiglu_f<kFast>(z.z, u.z, a.form), swiglu_f<kFast>(z.w, u.w, a.form));
      } else if (a.act != kActNone) {
        z = make_float4(act_any<kFast>(z.x, a), act_any<kFast>(z.y, a), act_any<kFast>(z.z, a), act_any<kFast>(z.w, a));
      }
      z.x += res.x; z.y += res.y; z.z += res.z; z.w += res.w;
      store4(static_cast<T*>(a.y) + row * a.width + col, z);
    }
  }
  if (aborted) set_error(a.err, kErrTimeout);
}

cudaLaunchConfig_t config(unsigned grid, int splits, int smem, cudaStream_t stream, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = (unsigned)splits;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <bool GATED, typename T>
int launch(const LinCall& c, const DeviceInfo& dev, int tn, int splits) {
  constexpr int H = GATED ? 2 : 1;
  auto kern = linear_split_kernel<GATED, T>;
  CUtensorMap tw, tx;
  int st = lin_maps(c, (uint32_t)tn, false, &tw, &tx);
  if (st) return st;
  const int64_t nct = (c.a.width + kBN - 1) / kBN;
  const int64_t live = c.a.group_lens ? std::min<int64_t>(c.a.G, c.a.M) : 1;
  const int64_t tiles = ((c.a.M + tn - 1) / tn + (c.a.group_lens ? live - 1 : 0)) * nct;
  const bool one = tiles * splits <= dev.sms;
  const int recv = splits * ((tn + splits - 1) / splits) * H * kBN * 4;
  const bool in_ring = tn > 32;
  const int room = one ? kSmemOne : kSmemTwo;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
  if (e != cudaSuccess) return cuda_status(e);
  SplitArgs a{c.a, tn, 0, (H * kBN + tn) * 128, 1, (tn + splits - 1) / splits, in_ring};
  const int fixed = 1024 + (in_ring ? 0 : recv) + (2 * kMaxStages + 1) * 8 + 32 + 8 * (c.a.G + 1);
  const int nkb = (c.a.K + kBK - 1) / kBK;
  a.stages = std::min(std::min(kMaxStages, (nkb + splits - 1) / splits), (room - fixed) / a.stage_bytes);
  const int smem = std::max(fixed + std::max(a.stages * a.stage_bytes, in_ring ? recv : 0), kSmemLeast);
  if (c.f32)  // as many accumulators as there is room for: each takes fewer steps (see linear_kernel)
    while (a.accs * 2 * H * tn <= kColsTwo && a.accs * splits < nkb) a.accs *= 2;
  cudaLaunchAttribute at{};
  const cudaLaunchConfig_t cfg = config((unsigned)(tiles * splits), splits, smem, c.stream, &at);
  e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

// A cluster's CTAs are on the SMs of one GPC, so this is less than the SMs would hold.  The same on every
// device that the library runs on, and asked for once.
int linear_split_clusters(const DeviceInfo& dev, int splits, bool one, int* count) {
  static std::atomic<int> known[9][2];
  std::atomic<int>& slot = known[splits][one];
  *count = slot.load(std::memory_order_relaxed);
  if (*count > 0) return PGG_OK;
  auto kern = linear_split_kernel<false, __nv_bfloat16>;
  const int smem = one ? kSmemOne : kSmemTwo;
  cudaLaunchAttribute at{};
  const cudaLaunchConfig_t cfg = config((unsigned)(dev.sms * splits), splits, smem, nullptr, &at);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(count, kern, &cfg);
  if (e != cudaSuccess) {
    cudaGetLastError();  // (told by the status, not by the next launch too)
    return cuda_status(e);
  }
  slot.store(*count = std::max(1, *count), std::memory_order_relaxed);
  return PGG_OK;
}

int launch_linear_split(const LinCall& c, const DeviceInfo& dev, int tn, int splits) {
  if (c.a.act == kActSwiglu)
    return c.f32 ? launch<true, float>(c, dev, tn, splits) : launch<true, __nv_bfloat16>(c, dev, tn, splits);
  return c.f32 ? launch<false, float>(c, dev, tn, splits) : launch<false, __nv_bfloat16>(c, dev, tn, splits);
}

}  // namespace pgg

// grouped_linear on pairs of CTAs (cta_group::2), for long groups and bf16 results: one MMA multiplies
// 256 output columns by up to 256 rows of X over two SMs.  Each CTA of the pair stages its own 128
// columns of W and half of the tile's rows of X -- 32 KB a k-block instead of the 48 of a CTA on its
// own, which is what the loads from L2 bound there -- and has the accumulators of its own columns.
//
// Both CTAs' loads count their bytes on the leader's barrier, so no thread passes on that a stage has
// landed; the leader's MMAs free the stage in both CTAs by a multicast commit.  Only a tile's release of
// its accumulator takes arrivals from the other CTA.
#include "cluster.cuh"
#include "linear.cuh"

namespace pgg {
namespace {

template <bool GATED>
struct PairCfg {
  static constexpr int kTN = GATED ? 128 : 256;  // rows of X a tile; half of them in each CTA
  static constexpr int kStages = GATED ? 5 : 6;
  static constexpr int kABytes = (GATED ? 2 : 1) * kBN * kBK * 2;
  static constexpr int kBBytes = kTN / 2 * kBK * 2;
  static constexpr int kEpiOff = kStages * (kABytes + kBBytes);
  static constexpr int kBarOff = kEpiOff + 4 * 4096;
  static constexpr int kGroupOff = kBarOff + 256;
  static constexpr int kAcc = (GATED ? 2 : 1) * kTN;
  static __host__ __device__ constexpr size_t bytes(int G) { return 1024 + (size_t)kGroupOff + 8 * (size_t)(G + 1); }
};

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinArgs a) {
  using C = PairCfg<GATED>;
  constexpr int TN = C::kTN, STAGES = C::kStages, kCW = 2 * kBN;
  static_assert(2 * C::kAcc == 512, "two accumulators fill tensor memory");
  static_assert((2 * STAGES + 5) * 8 + 24 <= 256, "barrier area");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // (the leader's are used)
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // (the leader's are used)
  uint64_t* drain = tempty + 2;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + C::kGroupOff);
  int32_t* s_tile = s_off + (a.G + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int nct = (a.width + kCW - 1) / kCW, nkb = (a.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 8);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(drain), 1);
    s_ctl->abort = 0;
    s_ctl->limit_ns = a.wait_ns ? a.wait_ns : kWaitTimeoutNs;
    fence_mbar_init();
    fence_proxy_async_smem();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(s_tmem), 512);
    tmem_relinquish_pair();
  }
  if (warp == 2) {
    const bool bad = lin_scan(a, TN, nct, s_off, s_tile, lane);
    if (lane == 0) {
      *s_bad = bad ? 1 : 0;
      if (bad && blockIdx.x == 0) set_error(a.err, kErrBadGroupLens);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are set up
  tc_fence_after();

  const uint32_t tmem = *s_tmem;
  const int tiles = *s_bad ? 0 : s_tile[a.G];
  const int t0 = (int)cluster_id(), step = (int)cluster_count();
  const uint32_t smem_a = smem_u32(smem), smem_b = smem_a + STAGES * C::kABytes;
  bool aborted = false;
  GroupCursor cur;

  if (warp == 0) {
    // ------------------------------------------------------------ loads of this CTA's halves
    const uint32_t full0 = map_rank(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool stalled = false;
    for (int t = t0; t < tiles && !aborted && !stalled; t += step) {
      const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
      const int half = ((T_.rows + 15) & ~15) / 2;  // rows of X in each CTA
      const int boxes = (half + 63) / 64;
      const int col = T_.col0 + (int)rank * kBN, row = T_.row0 + (int)rank * half;
      for (int kb = 0; kb < nkb; ++kb) {
        if (issued == a.stall_at) { stalled = true; break; }
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        if (lane == 0) {
          const uint32_t fb = full0 + stage * 8;
          const uint32_t sa = smem_a + stage * C::kABytes, sb = smem_b + stage * C::kBBytes;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * (C::kABytes + boxes * 64 * 128));
          tma_load_3d_pair(sa, &tmW, fb, kb * kBK, col, T_.g);
          if (GATED) tma_load_3d_pair(sa + kBN * 128, &tmW, fb, kb * kBK, a.width + col, T_.g);
          for (int b = 0; b < boxes; ++b) tma_load_2d_pair(sb + b * 64 * 128, &tmX, fb, kb * kBK, row + b * 64);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // The last stages' commits arrive here before the CTA may go; after an abort the leader sees on its
    // barriers that the loads have landed.
    long long n = issued < STAGES ? issued : STAGES;
    for (long long i = 0; i < n; ++i) {
      if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
      if (aborted || stalled) {
        if (rank == 0 && lane == 0) mbar_wait_drain(smem_u32(&full[stage]), phase);
        __syncwarp();
      } else if (!warp_wait(smem_u32(&empty[stage]), phase, s_ctl)) {
        aborted = true;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products, issued by the leader
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      const uint64_t desc_a = smem_desc(smem_a, 16, 1024, kSwizzle128B);
      const uint64_t desc_b = smem_desc(smem_b, 16, 1024, kSwizzle128B);
      for (int t = t0; t < tiles && !aborted; t += step) {
        const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
        const uint32_t idesc = idesc_bf16(2 * kBN, (T_.rows + 15) & ~15, false, false);
        if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint32_t d = tmem + acc * C::kAcc;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t da = desc_a + (uint64_t)(stage * C::kABytes >> 4);
            const uint64_t db = desc_b + (uint64_t)(stage * C::kBBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
              const uint32_t more = kb > 0 || ks > 0 ? 1u : 0u;
              mma_f16_pair(d, da + 2 * ks, db + 2 * ks, idesc, more);
              if (GATED) mma_f16_pair(d + TN, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, more);
            }
            mma_commit_pair(smem_u32(&empty[stage]));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (aborted) break;
        if (lane == 0) mma_commit_pair(smem_u32(&tfull[acc]));
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (aborted && lane == 0) {
        mma_commit_pair(smem_u32(drain));
        mbar_wait_drain(smem_u32(drain), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue of this CTA's columns (warps 2..5)
    const int q = warp & 3;
    uint8_t* stg = smem + C::kEpiOff + (warp - 2) * 4096;
    const uint32_t tempty0 = map_rank(smem_u32(tempty), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = t0; t < tiles && !aborted; t += step) {
      const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
      const int col = T_.col0 + (int)rank * kBN + q * 32, n = col + lane;
      float bg = 0.0f, bu = 0.0f;
      if (a.bias && n < a.width) {
        const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + n;
        bg = __bfloat162float(b[0]);
        if (GATED) bu = __bfloat162float(b[a.width]);
      }
      if (!warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem + acc * C::kAcc + ((uint32_t)(q * 32) << 16);
      if (col < a.width) {
#pragma unroll 1
        for (int c = 0; c < T_.rows; c += 32) {
          float z[32], u[32];
          load_acc(tb + c, z, bg);
          if (GATED) load_acc(tb + TN + c, u, bu);
          finish_chunk<GATED, __nv_bfloat16>(a, z, u, (size_t)T_.row0 + c, col, min(32, T_.rows - c), stg, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + acc * 8);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  if (aborted && lane == 0) set_error(a.err, kErrTimeout);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA goes while the other's loads, commits or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool GATED>
int launch(const LinCall& c, const DeviceInfo& dev) {
  using C = PairCfg<GATED>;
  auto kern = linear_pair_kernel<GATED>;
  CUtensorMap tw, tx;
  const int st = lin_maps(c, 64, &tw, &tx);
  if (st) return st;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::bytes(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t nct = (c.a.width + 2 * kBN - 1) / (2 * kBN);
  const int64_t tiles = ((c.a.M + C::kTN - 1) / C::kTN + (c.a.group_lens ? c.a.G : 0)) * nct;
  const int grid = 2 * (int)std::max<int64_t>(1, std::min<int64_t>(dev.sms / 2, tiles));
  kern<<<grid, kLinThreads, C::bytes(c.a.G), c.stream>>>(tw, tx, c.a);
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_linear_pair(const LinCall& c, const DeviceInfo& dev) {
  return c.a.act == kActSwiglu ? launch<true>(c, dev) : launch<false>(c, dev);
}

}  // namespace pgg

// grouped_linear: the persistent kernel of one CTA per SM, the choice of a kernel, and the entry points.
#include "linear.cuh"

namespace pgg {
namespace {

constexpr int kChunk = 4;  // fp32 results: k-blocks that one accumulator takes

// Shared memory: the ring of stages (weights | rows of X), a 4 KB staging buffer per epilogue warp,
// the barriers, the group tables.
template <bool GATED, int TN, int STAGES>
struct LinSmem {
  static constexpr int kABytes = (GATED ? 2 : 1) * kBN * kBK * 2;
  static constexpr int kBBytes = TN * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kEpiOff = STAGES * kStageBytes;
  static constexpr int kBarOff = kEpiOff + 4 * 4096;
  static constexpr int kGroupOff = kBarOff + 256;
  static __host__ __device__ constexpr size_t bytes(int G) { return 1024 + (size_t)kGroupOff + 8 * (size_t)(G + 1); }
};

template <bool GATED, int TN, int STAGES, typename T>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinArgs a) {
  using L = LinSmem<GATED, TN, STAGES>;
  // fp32 results: the tensor core's own accumulation drops bits at each step (a sum over 4096 was off by
  // 3.4e-6 of its norm, a chain of fp32 additions by 1.5e-7), so the accumulators hold kChunk k-blocks and
  // the epilogue adds them up in registers
  constexpr bool kWide = std::is_same<T, float>::value;
  constexpr int kBufs = kWide ? 4 : 2;              // accumulators in turn
  constexpr int kAcc = (GATED ? 2 : 1) * TN;        // columns of an accumulator
  constexpr uint32_t kTmemCols = kBufs * kAcc;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert((2 * STAGES + 2 * kBufs + 1) * 8 + 24 <= 256, "barrier area");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + L::kGroupOff);
  int32_t* s_tile = s_off + (a.G + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nct = (a.width + kBN - 1) / kBN, nkb = (a.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 128);
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
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
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
  tc_fence_after();

  const uint32_t tmem = *s_tmem;
  const int tiles = *s_bad ? 0 : s_tile[a.G];
  const uint32_t smem_a = smem_u32(smem), smem_b = smem_a + STAGES * L::kABytes;
  bool aborted = false;
  GroupCursor cur;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool stalled = false;
    for (int t = blockIdx.x; t < tiles && !aborted && !stalled; t += gridDim.x) {
      const LinTile T_ = lin_tile<kBN, false>(t, a, TN, nct, s_off, s_tile, cur);
      for (int kb = 0; kb < nkb; ++kb) {
        if (issued == a.stall_at) { stalled = true; break; }
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        if (lane == 0) {
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t sa = smem_a + stage * L::kABytes, sb = smem_b + stage * L::kBBytes;
          mbar_arrive_expect_tx(fb, L::kStageBytes);
          tma_load_3d(sa, &tmW, fb, kb * kBK, T_.col0, T_.g);
          if (GATED) tma_load_3d(sa + kBN * 128, &tmW, fb, kb * kBK, a.width + T_.col0, T_.g);
          tma_load_2d(sb, &tmX, fb, kb * kBK, T_.row0);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (aborted && lane == 0) {
      // the loads still in flight land before the block's shared memory goes away
      long long n = issued < STAGES ? issued : STAGES;
      int s = stage;
      uint32_t p = phase;
      for (long long i = 0; i < n; ++i) {
        if (--s < 0) { s = STAGES - 1; p ^= 1u; }
        mbar_wait_drain(smem_u32(&full[s]), p);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    const uint64_t desc_a = smem_desc(smem_a, 16, 1024, kSwizzle128B);
    const uint64_t desc_b = smem_desc(smem_b, 16, 1024, kSwizzle128B);
    for (int t = blockIdx.x; t < tiles && !aborted; t += gridDim.x) {
      const LinTile T_ = lin_tile<kBN, false>(t, a, TN, nct, s_off, s_tile, cur);
      const uint32_t idesc = idesc_bf16(kBN, (T_.rows + 15) & ~15, false, false);
      for (int k0 = 0; k0 < nkb && !aborted; k0 += kWide ? kChunk : nkb) {
        const int k1 = kWide ? min(nkb, k0 + kChunk) : nkb;
        if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint32_t d = tmem + acc * kAcc;
        for (int kb = k0; kb < k1; ++kb) {
          if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t da = desc_a + (uint64_t)(stage * L::kABytes >> 4);
            const uint64_t db = desc_b + (uint64_t)(stage * L::kBBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
              const uint32_t more = kb > k0 || ks > 0 ? 1u : 0u;
              mma_f16(d, da + 2 * ks, db + 2 * ks, idesc, more);
              if (GATED) mma_f16(d + TN, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, more);
            }
            mma_commit(smem_u32(&empty[stage]));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (aborted) break;
        if (lane == 0) mma_commit(smem_u32(&tfull[acc]));
        __syncwarp();
        if (++acc == kBufs) { acc = 0; acc_phase ^= 1u; }
      }
    }
    if (aborted && lane == 0) {
      mma_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;  // the lane quarter of tensor memory that this warp may read
    uint8_t* stg = smem + L::kEpiOff + (warp - 2) * 4096;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < tiles && !aborted; t += gridDim.x) {
      const LinTile T_ = lin_tile<kBN, false>(t, a, TN, nct, s_off, s_tile, cur);
      const int col = T_.col0 + q * 32, n = col + lane;
      float bg = 0.0f, bu = 0.0f;
      if (a.bias && n < a.width) {
        const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + n;
        bg = __bfloat162float(b[0]);
        if (GATED) bu = __bfloat162float(b[a.width]);
      }
      if (kWide) {
        float z[TN / 32][32], u[GATED ? TN / 32 : 1][32];
#pragma unroll
        for (int i = 0; i < TN / 32; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            z[i][j] = bg;
            if (GATED) u[i][j] = bu;
          }
#pragma unroll 1
        for (int k0 = 0; k0 < nkb; k0 += kChunk) {
          if (!warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          const uint32_t tb = tmem + acc * kAcc + ((uint32_t)(q * 32) << 16);
#pragma unroll
          for (int i = 0; i < TN / 32; ++i) {
            if (i * 32 < T_.rows) {  // (the accumulator's columns past the rows hold nothing)
              add_acc(tb + i * 32, z[i]);
              if (GATED) add_acc(tb + TN + i * 32, u[GATED ? i : 0]);
            }
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&tempty[acc]));
          if (++acc == kBufs) { acc = 0; acc_phase ^= 1u; }
        }
        if (aborted) break;
        if (col < a.width) {
#pragma unroll
          for (int i = 0; i < TN / 32; ++i)
            if (i * 32 < T_.rows)
              finish_chunk<GATED, T>(a, z[i], u[GATED ? i : 0], (size_t)T_.row0 + i * 32, col, min(32, T_.rows - i * 32),
                                     stg, lane);
        }
        continue;
      }
      if (!warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem + acc * kAcc + ((uint32_t)(q * 32) << 16);
      if (col < a.width) {
#pragma unroll 1
        for (int c = 0; c < T_.rows; c += 32) {
          float z[32], u[32];
          load_acc(tb + c, z, bg);
          if (GATED) load_acc(tb + TN + c, u, bu);
          finish_chunk<GATED, T>(a, z, u, (size_t)T_.row0 + c, col, min(32, T_.rows - c), stg, lane);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == kBufs) { acc = 0; acc_phase ^= 1u; }
    }
  }

  if (aborted && lane == 0) set_error(a.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <bool GATED, int TN, int STAGES, typename T>
int launch(const LinCall& c, const DeviceInfo& dev) {
  using L = LinSmem<GATED, TN, STAGES>;
  auto kern = linear_kernel<GATED, TN, STAGES, T>;
  CUtensorMap tw, tx;
  const int st = lin_maps(c, TN, false, &tw, &tx);
  if (st) return st;
  // the most that the kernel is ever launched with: another thread may call with more groups meanwhile
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t tiles = ((c.a.M + TN - 1) / TN + (c.a.group_lens ? c.a.G : 0)) * ceil_div(c.a.width, kBN);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(dev.sms, tiles));
  kern<<<grid, kLinThreads, L::bytes(c.a.G), c.stream>>>(tw, tx, c.a);
  return cuda_status(cudaGetLastError());
}

// Which kernel: few rows of X in few tiles split the reduction over a cluster; bf16 results of long
// groups take CTA pairs; the rest the persistent kernel, with narrow row tiles where groups are short.
int dispatch(const LinCall& c, const DeviceInfo& dev) {
  const bool gated = c.a.act == kActSwiglu;
  const int nct = ceil_div(c.a.width, kBN), nkb = ceil_div(c.a.K, kBK);
  const int64_t live = c.a.group_lens ? std::min<int64_t>(c.a.G, c.a.M) : 1;  // groups that can have rows
  const int tn = c.a.M <= 16 ? 16 : 32;
  const int64_t tiles = ((c.a.M + tn - 1) / tn + (c.a.group_lens ? live - 1 : 0)) * nct;
  if (tiles * 2 <= dev.sms && nkb >= 4) {
    int splits = 2;
    while (splits < 8 && tiles * splits * 2 <= 2 * dev.sms && nkb >= splits * 4) splits *= 2;
    return launch_linear_split(c, dev, tn, splits);
  }
  const int64_t rows = c.a.M / live;  // of a group, on average
  if (c.f32) {
    if (gated) return rows <= 16 ? launch<true, 32, 5, float>(c, dev) : launch<true, 64, 5, float>(c, dev);
    return rows <= 16 ? launch<false, 32, 9, float>(c, dev) : launch<false, 128, 6, float>(c, dev);
  }
  if (rows >= 512) return launch_linear_pair(c, dev);
  if (gated) return rows <= 16 ? launch<true, 32, 5, __nv_bfloat16>(c, dev) : launch<true, 128, 4, __nv_bfloat16>(c, dev);
  return rows <= 16 ? launch<false, 32, 9, __nv_bfloat16>(c, dev) : launch<false, 128, 6, __nv_bfloat16>(c, dev);
}

int linear_impl(const void* X, const void* W, const int32_t* group_lens, const void* bias, const void* residual,
                void* Y, int dtype, void* Z, int64_t M, int64_t N, int64_t K, int G, int act, float alpha,
                float offset, float limit, unsigned long long wait_ns, long long stall_at, int32_t* err,
                void* stream) {
  if (G < 1 || G > kMaxGroups || (!group_lens && G != 1)) return PGG_ERR_INVALID_ARG;
  if (M < 0 || M >= ((int64_t)1 << 31)) return PGG_ERR_INVALID_ARG;
  if (act < PGG_ACT_NONE || act > PGG_ACT_SWIGLU) return PGG_ERR_INVALID_ARG;
  if (dtype != PGG_DTYPE_F32 && dtype != PGG_DTYPE_BF16) return PGG_ERR_INVALID_ARG;
  const int mult = act == PGG_ACT_SWIGLU ? 16 : 8;
  for (int64_t d : {N, K})
    if (d < 8 || d >= ((int64_t)1 << 30)) return PGG_ERR_INVALID_ARG;
  if (N % mult || K % 8) return PGG_ERR_ALIGNMENT;
  const float big = 3.0e38f;
  if (!(alpha >= -big && alpha <= big) || !(offset >= -big && offset <= big) || !(limit >= 0.0f && limit <= big))
    return PGG_ERR_INVALID_ARG;
  if (M == 0) return PGG_OK;
  if (!X || !W || !Y) return PGG_ERR_INVALID_ARG;
  for (const void* p : {X, W, bias, residual, (const void*)Y, (const void*)Z})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(group_lens, 4) || !aligned_to(err, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != PGG_OK) return st;
  LinCall c{X, W, {}, dtype == PGG_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)};
  c.a = {group_lens, G, M, (int)N, (int)K, (int)(act == PGG_ACT_SWIGLU ? N / 2 : N), act, {alpha, offset, limit},
         static_cast<const __nv_bfloat16*>(bias), residual, Y, static_cast<__nv_bfloat16*>(Z), err, wait_ns, stall_at};
  return dispatch(c, dev);
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_grouped_linear(const void* X, const void* W, const int32_t* group_lens, const void* bias, const void* residual,
                       void* Y, int dtype, void* Z, int64_t M, int64_t N, int64_t K, int G, int act, float alpha,
                       float offset, float limit, int32_t* err, void* stream) {
  return linear_impl(X, W, group_lens, bias, residual, Y, dtype, Z, M, N, K, G, act, alpha, offset, limit, 0, -1, err,
                     stream);
}

int pgg_test_stalled_linear(const void* X, const void* W, const int32_t* group_lens, void* Y, int64_t M, int64_t N,
                            int64_t K, int G, int act, int64_t stall_at, uint64_t wait_ns, int32_t* err, void* stream) {
  if (stall_at < 0 || wait_ns < 100000ull || wait_ns > 1000000000ull) return PGG_ERR_INVALID_ARG;
  return linear_impl(X, W, group_lens, nullptr, nullptr, Y, PGG_DTYPE_BF16, nullptr, M, N, K, G, act, 1.0f, 0.0f, 0.0f,
                     wait_ns, stall_at, err, stream);
}

}  // extern "C"

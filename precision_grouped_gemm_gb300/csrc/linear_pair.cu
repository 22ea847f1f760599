// grouped_linear on pairs of CTAs (cta_group::2), for long groups and bf16 results: one MMA multiplies
// 256 output columns by up to 256 rows of X over two SMs.  Each CTA of the pair stages its own 128
// columns of W and half of the tile's rows of X -- 32 KB a k-block instead of the 48 of a CTA on its
// own, which is what the loads from L2 bound there -- and has the accumulators of its own columns.
//
// With swiglu a CTA's 128 columns of W are 64 of the gate and the same 64 of the up half, so a tile moves
// no more bytes than without: the lanes of gate and up of one column are in different warps, which swap
// half of their rows through shared memory and finish 16 rows of 32 columns each.
//
// Both CTAs' loads count their bytes on the leader's barrier, so no thread passes on that a stage has
// landed; the leader's MMAs free the stage in both CTAs by a multicast commit.  Only a tile's release of
// its accumulator takes arrivals from the other CTA.
//
// The tensor cores bound it: 16384 x 4096 x 2048 with a residual 154 us, 1786 TFLOP/s, pipes 86% busy (13.5 waves
// of tiles in 14); 32 experts of 1092 rows, 5760 x 2880 with swiglu and Z 619 to 638 us by GPU, 1703 TFLOP/s, 91%.  Over
// seconds the power cap lowers the clock to 1.33 to 1.48 GHz: 179 and 732 to 758 us.
#include "cluster.cuh"
#include "linear.cuh"

namespace pgg {
namespace {

constexpr int kPairTN = 256;     // rows of X a tile; half of them in each CTA
constexpr int kPairStages = 6;
constexpr int kEpiWarps = 8;     // two for each lane quarter of tensor memory
constexpr int kPairThreads = 32 * (2 + kEpiWarps);
constexpr int kPairABytes = kBN * kBK * 2, kPairBBytes = kPairTN / 2 * kBK * 2;
constexpr int kStgBytes = 2048;  // of an epilogue warp: turn a chunk, or go to the partner
constexpr int kPairEpiOff = kPairStages * (kPairABytes + kPairBBytes);
constexpr int kPairBarOff = kPairEpiOff + kEpiWarps * kStgBytes;
constexpr int kPairGroupOff = kPairBarOff + 256;
size_t pair_smem(int G) { return 1024 + (size_t)kPairGroupOff + 8 * ((size_t)G + 1); }

// Barrier of the two warps that share 32 columns (64 threads); the form that tells each whether `ok` held in
// both makes them give up together, so that none is left at a later barrier.
__device__ __forceinline__ void partner_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool partner_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r != 0;
}

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinArgs a) {
  constexpr int TN = kPairTN, STAGES = kPairStages;
  constexpr int kCols = GATED ? kBN / 2 : kBN;  // output columns of a CTA
  constexpr int kCW = 2 * kCols;
  static_assert((2 * STAGES + 5) * 8 + 24 <= 256, "barrier area");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairBarOff);  // (the leader's are used)
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // (the leader's are used)
  uint64_t* drain = tempty + 2;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + kPairGroupOff);
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
      mbar_init(smem_u32(&tempty[i]), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(drain), 1);
    s_ctl->abort = 0;
    s_ctl->limit_ns = a.wait_ns;
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
  const uint32_t smem_a = smem_u32(smem), smem_b = smem_a + STAGES * kPairABytes;
  bool aborted = false;
  GroupCursor cur;

  // The first two roles are one thread each: their loops are short chains of waits and issues, which a
  // vote or a warp barrier a step would lengthen.
  if (warp == 0) {
    // ------------------------------------------------------------ loads of this CTA's halves
    if (elect_one()) {
      const uint32_t full0 = map_rank(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool stalled = false;
      for (int t = t0; t < tiles && !aborted && !stalled; t += step) {
        const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
        const int half = ((T_.rows + 15) & ~15) / 2;  // rows of X in each CTA
        const int col = T_.col0 + (int)rank * kCols, row = T_.row0 + (int)rank * half;
        for (int kb = 0; kb < nkb; ++kb) {
          if (issued == a.stall_at) { stalled = true; break; }
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          const uint32_t fb = full0 + stage * 8;
          const uint32_t sa = smem_a + stage * kPairABytes, sb = smem_b + stage * kPairBBytes;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * (kPairABytes + kPairBBytes));
          // one load an operand: each has a cost of its own (X in two of 64 rows and gate and up apart
          // took 5 and 15% longer)
          if (GATED) tma_load_4d_pair(sa, &tmW, fb, kb * kBK, col, 0, T_.g);
          else tma_load_3d_pair(sa, &tmW, fb, kb * kBK, col, T_.g);
          tma_load_2d_pair(sb, &tmX, fb, kb * kBK, row);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // The last stages' commits arrive here before the CTA may go; after an abort the leader sees on its
      // barriers that the loads have landed.
      const long long n = issued < STAGES ? issued : STAGES;
      for (long long i = 0; i < n; ++i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
        if (aborted || stalled) {
          if (rank == 0) mbar_wait_drain(smem_u32(&full[stage]), phase);
        } else if (!mbar_wait(smem_u32(&empty[stage]), phase, s_ctl)) {
          aborted = true;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products, issued by the leader
    if (rank == 0 && elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      const uint64_t desc_a = smem_desc(smem_a, 16, 1024, kSwizzle128B);
      const uint64_t desc_b = smem_desc(smem_b, 16, 1024, kSwizzle128B);
      uint64_t da = desc_a, db = desc_b;
      for (int t = t0; t < tiles && !aborted; t += step) {
        const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
        const uint32_t idesc = idesc_bf16(2 * kBN, (T_.rows + 15) & ~15, false, false);
        if (!mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint32_t d = tmem + acc * TN;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kBK / 16; ++ks) mma_f16_pair(d, da + 2 * ks, db + 2 * ks, idesc, kb > 0 || ks > 0 ? 1u : 0u);
          mma_commit_pair(smem_u32(&empty[stage]));
          da += kPairABytes >> 4;
          db += kPairBBytes >> 4;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; da = desc_a; db = desc_b; }
        }
        if (aborted) break;
        mma_commit_pair(smem_u32(&tfull[acc]));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (aborted) {
        mma_commit_pair_own(smem_u32(drain));  // (nobody waits in the other CTA, which may go before it arrived)
        mbar_wait_drain(smem_u32(drain), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue of this CTA's columns (warps 2..9)
    const int q = warp & 3, share = (warp - 2) >> 2;  // lane quarter; which chunks of 32 rows: share, share + 2, ...
    uint8_t* stg = smem + kPairEpiOff + (warp - 2) * kStgBytes;
    const uint32_t tempty0 = map_rank(smem_u32(tempty), 0);
    const bool up = GATED && q >= 2;  // this warp's lanes are columns of the up half
    const int pair_id = 1 + (q & 1) + 2 * share;
    const int lane_col = GATED ? (q & 1) * 32 : q * 32;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = t0; t < tiles && !aborted; t += step) {
      const LinTile T_ = lin_tile<kCW>(t, a, TN, nct, s_off, s_tile, cur);
      const int col = T_.col0 + (int)rank * kCols + lane_col, n = col + lane;
      const int ncols = min(32, a.width - col);
      float bias = 0.0f;
      if (a.bias && n < a.width) bias = __bfloat162float(a.bias[(size_t)T_.g * a.N + (up ? a.width : 0) + n]);
      uint4 res[4];
      if (!GATED && a.residual && ncols > 0 && 32 * share < T_.rows)
        fetch_chunk(res, static_cast<const __nv_bfloat16*>(a.residual) + ((size_t)T_.row0 + 32 * share) * a.width + col,
                    a.width, T_.rows - 32 * share, ncols, lane);
      bool ok = warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl);
      if (GATED) ok = partner_all(pair_id, ok);
      if (!ok) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem + acc * TN + ((uint32_t)(q * 32) << 16);
      if (ncols > 0) {
#pragma unroll 1
        for (int c = 32 * share; c < T_.rows; c += 64) {
          const size_t row = (size_t)T_.row0 + c;
          float z[32];
          load_acc(tb + c, z, bias);
          if constexpr (GATED) {
            // rows 0 .. 15 of the chunk are the gate warp's to finish, the others the up warp's
            float* mine = reinterpret_cast<float*>(stg);
            const float* theirs =
                reinterpret_cast<const float*>(smem + kPairEpiOff + (warp - 2 + (up ? 2 : -2)) * kStgBytes);
            float g[16], u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) mine[j * 32 + lane] = up ? z[j] : z[16 + j];
            partner_sync(pair_id);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float o = theirs[j * 32 + lane], k = up ? z[16 + j] : z[j];
              g[j] = up ? o : k;
              u[j] = up ? k : o;
            }
            partner_sync(pair_id);
            const int half = up ? 16 : 0, nrows = min(16, T_.rows - c - half);
            const size_t r0 = row + half;
            if (nrows > 0) {
              if (a.z) {
                put_rows16(stg, g, a.z + r0 * a.N + col, a.N, nrows, ncols, lane);
                put_rows16(stg + 1024, u, a.z + r0 * a.N + a.width + col, a.N, nrows, ncols, lane);
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) g[j] = swiglu_f<true>(g[j], u[j], a.form);
              if (a.residual) {
                const __nv_bfloat16* r =
                    static_cast<const __nv_bfloat16*>(a.residual) + r0 * a.width + min(n, a.width - 1);
#pragma unroll
                for (int j = 0; j < 16; ++j) u[j] = __bfloat162float(r[(size_t)min(j, nrows - 1) * a.width]);  // (see add_chunk)
#pragma unroll
                for (int j = 0; j < 16; ++j) g[j] += u[j];
                __syncwarp();  // (the residual may be Y: every row is read before it is written)
              }
              put_rows16(stg, g, static_cast<__nv_bfloat16*>(a.y) + r0 * a.width + col, a.width, nrows, ncols, lane);
            }
          } else {
            uint4 next[4];
            if (a.residual && c + 64 < T_.rows)
              fetch_chunk(next, static_cast<const __nv_bfloat16*>(a.residual) + (row + 64) * a.width + col, a.width,
                          T_.rows - c - 64, ncols, lane);
            finish_plain(a, z, res, row, col, min(32, T_.rows - c), ncols, stg, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) res[i] = next[i];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + acc * 8);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  if (aborted) set_error(a.err, kErrTimeout);
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
  auto kern = linear_pair_kernel<GATED>;
  CUtensorMap tw, tx;
  const int st = lin_maps(c, kPairTN / 2, GATED, &tw, &tx);
  if (st) return st;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)pair_smem(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  const int cw = GATED ? kBN : 2 * kBN;
  const int64_t nct = (c.a.width + cw - 1) / cw;
  const int64_t tiles = ((c.a.M + kPairTN - 1) / kPairTN + (c.a.group_lens ? c.a.G : 0)) * nct;
  const int grid = 2 * (int)std::max<int64_t>(1, std::min<int64_t>(dev.sms / 2, tiles));
  kern<<<grid, kPairThreads, pair_smem(c.a.G), c.stream>>>(tw, tx, c.a);
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_linear_pair(const LinCall& c, const DeviceInfo& dev) {
  return c.a.act == kActSwiglu ? launch<true>(c, dev) : launch<false>(c, dev);
}

}  // namespace pgg

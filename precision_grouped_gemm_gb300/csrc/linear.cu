// grouped_linear: the persistent kernel of one CTA per SM, the choice of a kernel, and the entry points.
#include <cmath>

#include "cluster.cuh"
#include "linear.cuh"

namespace pgg {
namespace {

// Shared memory: the ring of stages (weights | rows of X), a staging buffer per epilogue warp (4 KB, or 2 of
// eight warps), the barriers, the group tables.
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// One chunk of 32 rows of fp32 results, 16 rows at a time (registers, and half the staging of finish_chunk).
template <bool GATED>
__device__ __forceinline__ void finish_halves(const LinArgs& a, const float (&z)[32], const float (&u)[32], size_t row,
                                              int col, int nrows, uint8_t* stg, int lane) {
  const int ncols = min(32, a.width - col);
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    if (h >= nrows) break;
    const size_t r0 = row + h;
    float v[16], w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = z[h + j];
      w[j] = GATED ? u[h + j] : 0.0f;
    }
    if (a.z) {
      put_rows16(stg, v, a.z + r0 * a.N + col, a.N, nrows - h, ncols, lane);
      if (GATED) put_rows16(stg, w, a.z + r0 * a.N + a.width + col, a.N, nrows - h, ncols, lane);
    }
    if (GATED) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = swiglu_f<false>(v[j], w[j], a.form);
    } else if (a.act == kActSilu) {
      apply_act<kActSilu, false>(v, a.form);
    } else if (a.act == kActGelu) {
      apply_act<kActGelu, false>(v, a.form);
    }
    if (a.residual) {
      const float* r = static_cast<const float*>(a.residual) + r0 * a.width + col + min(lane, ncols - 1);
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = r[(size_t)min(j, nrows - h - 1) * a.width];  // (see add_chunk)
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += w[j];
    }
    __syncwarp();  // (the residual may be Y: every row is read before it is written)
    put_rows16(stg, v, static_cast<float*>(a.y) + r0 * a.width + col, a.width, nrows - h, ncols, lane);
  }
}

// One CTA per SM walks the tiles: one thread loads, one multiplies, four or eight warps finish, with two or
// four accumulators so that a tile's epilogue and the next one's products overlap.
//
// bf16 results of short groups, whose weights are read once for few rows: memory bounds it.  256 experts of 96
// rows, 4096 x 2048 (4.6 GB): 668 us, the plain copy rate; 128 rows over 32 experts, 5760 x 2880 with swiglu
// (985 MB): 145 us, the same.  fp32 results: the loads from L2 bound it, 8192 x 4096 x 4096 199 to 206 us by
// GPU, 1380 TFLOP/s; with swiglu, whose tiles are half as high, 270 to 288 us, 1019.
template <bool GATED, int TN, int STAGES, typename T, int SHARES>
__global__ void __launch_bounds__(64 + 128 * SHARES, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinArgs a) {
  using L = LinSmem<GATED, TN, STAGES>;
  // fp32 results: the tensor core's own accumulation drops bits at each step (a sum over 4096 was off by
  // 3.4e-6 of its norm, a chain of fp32 additions by 1.5e-7), so the accumulators hold kChunk k-blocks and
  // the epilogue adds them up in registers (64 sums a thread at most; the build fails where one is spilled).
  // SHARES 2: eight epilogue warps, which hide each other's latencies (16384 x 4096 x 1024 with silu 239 -> 145 us).
  constexpr bool kWide = std::is_same<T, float>::value;
  constexpr int kAcc = (GATED ? 2 : 1) * TN;        // columns of an accumulator
  constexpr int kBufs = kWide && kAcc <= 128 ? 4 : 2;  // accumulators in turn
  constexpr uint32_t kTmemCols = kBufs * kAcc;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert((2 * STAGES + 2 * kBufs + 1) * 8 + 24 <= 256, "barrier area");
  static_assert(kWide || SHARES == 1, "bf16 results: four epilogue warps");

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
      mbar_init(smem_u32(&tempty[i]), 128 * SHARES);
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
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool stalled = false;
      for (int t = blockIdx.x; t < tiles && !aborted && !stalled; t += gridDim.x) {
        const LinTile T_ = lin_tile<kBN>(t, a, TN, nct, s_off, s_tile, cur);
        for (int kb = 0; kb < nkb; ++kb) {
          if (issued == a.stall_at) { stalled = true; break; }
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t sa = smem_a + stage * L::kABytes, sb = smem_b + stage * L::kBBytes;
          mbar_arrive_expect_tx(fb, L::kStageBytes);
          tma_load_3d(sa, &tmW, fb, kb * kBK, T_.col0, T_.g);
          if (GATED) tma_load_3d(sa + kBN * 128, &tmW, fb, kb * kBK, a.width + T_.col0, T_.g);
          tma_load_2d(sb, &tmX, fb, kb * kBK, T_.row0);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (aborted) {
        // the loads still in flight land before the block's shared memory goes away
        for (long long i = 0, n = issued < STAGES ? issued : STAGES; i < n; ++i) {
          if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
          mbar_wait_drain(smem_u32(&full[stage]), phase);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      const uint64_t desc_a = smem_desc(smem_a, 16, 1024, kSwizzle128B);
      const uint64_t desc_b = smem_desc(smem_b, 16, 1024, kSwizzle128B);
      uint64_t da = desc_a, db = desc_b;
      for (int t = blockIdx.x; t < tiles && !aborted; t += gridDim.x) {
        const LinTile T_ = lin_tile<kBN>(t, a, TN, nct, s_off, s_tile, cur);
        const uint32_t idesc = idesc_bf16(kBN, (T_.rows + 15) & ~15, false, false);
        for (int k0 = 0; k0 < nkb && !aborted; k0 += kWide ? kChunk : nkb) {
          const int k1 = kWide ? min(nkb, k0 + kChunk) : nkb;
          if (!mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          const uint32_t d = tmem + acc * kAcc;
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
              const uint32_t more = kb > k0 || ks > 0 ? 1u : 0u;
              mma_f16(d, da + 2 * ks, db + 2 * ks, idesc, more);
              if (GATED) mma_f16(d + TN, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, more);
            }
            mma_commit(smem_u32(&empty[stage]));
            da += L::kABytes >> 4;
            db += L::kBBytes >> 4;
            if (++stage == STAGES) { stage = 0; phase ^= 1u; da = desc_a; db = desc_b; }
          }
          if (aborted) break;
          mma_commit(smem_u32(&tfull[acc]));
          if (++acc == kBufs) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (aborted) {
        mma_commit(smem_u32(drain));
        mbar_wait_drain(smem_u32(drain), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2 on)
    const int q = warp & 3;  // the lane quarter of tensor memory that this warp may read
    uint8_t* stg = smem + L::kEpiOff + (warp - 2) * (4096 / SHARES);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < tiles && !aborted; t += gridDim.x) {
      const LinTile T_ = lin_tile<kBN>(t, a, TN, nct, s_off, s_tile, cur);
      const int col = T_.col0 + q * 32, n = col + lane;
      float bg = 0.0f, bu = 0.0f;
      if (a.bias && n < a.width) {
        const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + n;
        bg = __bfloat162float(b[0]);
        if (GATED) bu = __bfloat162float(b[a.width]);
      }
      if constexpr (kWide) {
        // this warp's chunks of 32 rows: share, share + SHARES, ...
        constexpr int kStep = 32 * SHARES, kRuns = TN / kStep;
        const int r0 = 32 * ((warp - 2) >> 2);
        if (SHARES > 1 && a.residual && col < a.width) {
          // the residual's rows come to L2 meanwhile: registers to hold them are not left
#pragma unroll
          for (int i = 0; i < kRuns; ++i) {
            const int r = r0 + i * kStep + lane;
            if (r < T_.rows) {
              const float* row = static_cast<const float*>(a.residual) + ((size_t)T_.row0 + r) * a.width;
              prefetch_l2(row + col);
              prefetch_l2(row + min(col + 31, a.width - 1));
            }
          }
        }
        float z[kRuns][32], u[GATED ? kRuns : 1][32];
#pragma unroll
        for (int i = 0; i < kRuns; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            z[i][j] = bg;
            if (GATED) u[i][j] = bu;
          }
#pragma unroll 1
        for (int k0 = 0; k0 < nkb; k0 += kChunk) {
          if (!warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          const uint32_t tb = tmem + acc * kAcc + ((uint32_t)(q * 32) << 16) + r0;
#pragma unroll
          for (int i = 0; i < kRuns; ++i) {
            if (r0 + i * kStep < T_.rows) {  // (the accumulator's columns past the rows hold nothing)
              add_acc(tb + i * kStep, z[i]);
              if (GATED) add_acc(tb + TN + i * kStep, u[GATED ? i : 0]);
            }
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&tempty[acc]));
          if (++acc == kBufs) { acc = 0; acc_phase ^= 1u; }
        }
        if (aborted) break;
        if (col < a.width) {
#pragma unroll
          for (int i = 0; i < kRuns; ++i) {
            const int c = r0 + i * kStep;
            if (c < T_.rows) {
              if constexpr (SHARES == 1)
                finish_chunk<GATED, T>(a, z[i], u[GATED ? i : 0], (size_t)T_.row0 + c, col, T_.rows - c, stg, lane);
              else
                finish_halves<GATED>(a, z[i], u[GATED ? i : 0], (size_t)T_.row0 + c, col, T_.rows - c, stg, lane);
            }
          }
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

  if (aborted) set_error(a.err, kErrTimeout);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <bool GATED, int TN, int STAGES, typename T, int SHARES = 1>
int launch(const LinCall& c, const DeviceInfo& dev) {
  using L = LinSmem<GATED, TN, STAGES>;
  auto kern = linear_kernel<GATED, TN, STAGES, T, SHARES>;
  CUtensorMap tw, tx;
  const int st = lin_maps(c, TN, false, &tw, &tx);
  if (st) return st;
  // the most that the kernel is ever launched with: another thread may call with more groups meanwhile
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t tiles = ((c.a.M + TN - 1) / TN + (c.a.group_lens ? c.a.G : 0)) * ceil_div(c.a.width, kBN);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(dev.sms, tiles));
  kern<<<grid, 64 + 128 * SHARES, L::bytes(c.a.G), c.stream>>>(tw, tx, c.a);
  return cuda_status(cudaGetLastError());
}

// Which kernel, by an estimate of its time in microseconds.  The host knows the rows of all groups together, so
// the work is taken as that of groups whose lengths vary about their mean as a routed batch's do, and to a quarter
// of a batch with half of its rows in one group (64 groups of 2048 rows, 4096 x 2048, by Zipf's law: 168 us with 128
// rows a tile, 189 with 32).  The constants are what the kernels were measured to take: a k-block's stage, or its
// products at the tensor cores' rate, a start and an end.  (Times of split / one / pair: 1 x 4096 x 4096 10.1 / 12.9 /
// 24; 256 x 4096 x 4096 17.3 / 17.5 / 24.8; 512 x 4096 x 4096 - / 18.0 / 25.1; 1024 x 4096 x 4096 - / 29.6 / 26.0;
// 4000 rows of 16 groups, 2048 x 2048: - / 40 / 43; 32768 rows of 32, 5760 x 2880 with swiglu: - / 706 / 636.)
struct Plan {
  enum Kind { kSplit, kOne, kPair } kind;
  int tn, splits;
  double us;
};
// Rows of the high tiles of linear_kernel.
int one_rows(const LinCall& c) { return c.f32 && c.a.act == kActSwiglu ? 64 : 128; }
// CTAs of a split product's launch: a cluster for every tile that the lengths may make.
int64_t split_ctas(const LinCall& c, int tn, int splits) {
  const int64_t live = c.a.group_lens ? std::min<int64_t>(c.a.G, c.a.M) : 1;
  return ((c.a.M + tn - 1) / tn + live - 1) * ceil_div(c.a.width, kBN) * splits;
}
// Whether these tiles and cuts are a form of the split kernel for the sizes.
bool split_has(const LinCall& c, const DeviceInfo& dev, int tn, int splits) {
  const int H = c.a.act == kActSwiglu ? 2 : 1, nkb = ceil_div(c.a.K, kBK);
  const int64_t ctas = split_ctas(c, tn, splits);
  if ((H == 2 && tn > 64) || nkb < 2 * splits || ctas > 4 * (int64_t)dev.sms * splits) return false;
  if (tn > 32 && ctas > dev.sms) return false;  // (two CTAs an SM have not the room)
  const int run = ceil_div(nkb, splits), accs = std::min(run, 256 / (H * tn));
  return !c.f32 || run <= kChunk * accs;  // (sums in fp32: see linear_kernel)
}
int choose(const LinCall& c, const DeviceInfo& dev, Plan* plan) {
  const bool gated = c.a.act == kActSwiglu;
  const int H = gated ? 2 : 1, nkb = ceil_div(c.a.K, kBK);
  const double live = c.a.group_lens ? (double)std::min<int64_t>(c.a.G, c.a.M) : 1;  // groups that can have rows
  const double rows = (double)c.a.M / live;
  const double nct = ceil_div(c.a.width, kBN), sms = dev.sms;
  const double memory =
      (2.0 * live * c.a.N * c.a.K + (double)c.a.M * (2.0 * c.a.K + (c.f32 ? 4.0 : 2.0) * c.a.width)) / 6.7e6;
  auto row_tiles = [&](int tn) {
    const double even = live * std::ceil(rows / tn);
    if (live < 2) return even;
    const double half = 0.5 * (double)c.a.M, rest = live - 1;
    return 0.5 * (even + std::ceil(half / tn) + rest * std::ceil(half / rest / tn));
  };
  auto tiles = [&](int tn) { return row_tiles(tn) * nct; };
  auto block = [&](int tn) { return std::max((H * kBN + tn) * 128 / 150e3, H * std::min<double>(tn, rows) * 0.31 / 256); };
  // Waves of row tiles by `columns` column tiles over `at_once` places, times a mean tile's time a k-block, of
  // which `cost` is one with so many rows (shared out evenly: see lin_tile).
  auto walk = [&](int tn, double columns, double at_once, auto cost) {
    double n = 0, t = 0;
    auto add = [&](double groups, double len) {
      double each = std::ceil(len / tn);
      if (live > 1) {  // lengths vary by the root of their mean: past a whole number of tiles by chance
        const double k = std::floor(len / tn + 0.5);
        each = k < 1 ? 1 : k + 0.5 * std::erfc((k * tn - len) / std::sqrt(2 * len));
      }
      n += groups * each;
      t += groups * each * cost(std::min<double>(tn, len / each + (len > 16 ? 8 : 0)));
    };
    add(live < 2 ? 1 : 0.75 * live, rows);
    if (live > 1) {
      add(0.25, 0.5 * (double)c.a.M);
      add(0.25 * (live - 1), 0.5 * (double)c.a.M / (live - 1));
    }
    return std::max(1.0, std::ceil(n * columns / at_once - 0.02)) * t / n;
  };
  Plan best{Plan::kOne, 0, 1, 1e30};
  auto offer = [&](Plan p) {
    if (p.us < best.us) best = p;
  };
  auto both = [](double a, double b) { return std::max(a, b) + 0.2 * std::min(a, b); };  // they overlap, not wholly
  for (int tn : {32, one_rows(c)}) {
    if (tn == 32 && live > 1 && rows >= 32) continue;  // (as fast at best, and slow for a long group among them)
    const double load = tn < 128 || c.f32 ? (H * kBN + tn) * 128 / 150e3 : gated ? 0.36 : 0.21;
    const double t = walk(tn, nct, sms, [&](double r) { return std::max(load, H * r * 0.31 / 256); });
    offer({Plan::kOne, tn, 1, 4.5 + both(nkb * t, memory) + 0.003 * tn});
  }
  if (!c.f32) {
    const double t = walk(256, std::ceil(c.a.width / (gated ? 128.0 : 256.0)), dev.sms / 2,
                          [](double r) { return std::max(0.22, r * 0.31 / 256); });
    offer({Plan::kPair, 256, 1, 6 + both(nkb * t, memory)});
  }
  for (int tn : {16, 32, 64, 128}) {
    for (int splits : {2, 4, 8}) {
      if (!split_has(c, dev, tn, splits)) continue;
      const bool one = split_ctas(c, tn, splits) <= dev.sms;  // CTAs an SM
      int clusters;
      const int st = linear_split_clusters(dev, splits, one, &clusters);
      if (st) return st;
      if (tiles(tn) > clusters) continue;
      const int run = ceil_div(nkb, splits);
      offer({Plan::kSplit, tn, splits,
             (c.a.group_lens ? 6.5 : 5.0) + both(run * block(tn) * (one ? 1 : 2), memory) + 0.02 * tn});
    }
  }
  *plan = best;
  return PGG_OK;
}

// Whether a plan is one that `choose` can give for the sizes.
bool plan_has(const LinCall& c, const DeviceInfo& dev, const Plan& p) {
  if (p.kind == Plan::kPair) return !c.f32 && p.tn == 256 && p.splits == 1;
  if (p.kind == Plan::kOne) return (p.tn == 32 || p.tn == one_rows(c)) && p.splits == 1;
  return p.kind == Plan::kSplit && (p.tn == 16 || p.tn == 32 || p.tn == 64 || p.tn == 128) &&
         (p.splits == 2 || p.splits == 4 || p.splits == 8) && split_has(c, dev, p.tn, p.splits);
}

int run_plan(const LinCall& c, const DeviceInfo& dev, const Plan& p) {
  const bool gated = c.a.act == kActSwiglu;
  if (p.kind == Plan::kSplit) return launch_linear_split(c, dev, p.tn, p.splits);
  if (p.kind == Plan::kPair) return launch_linear_pair(c, dev);
  if (c.f32) {
    if (gated) return p.tn == 32 ? launch<true, 32, 5, float>(c, dev) : launch<true, 64, 5, float, 2>(c, dev);
    return p.tn == 32 ? launch<false, 32, 9, float>(c, dev) : launch<false, 128, 6, float, 2>(c, dev);
  }
  if (gated) return p.tn == 32 ? launch<true, 32, 5, __nv_bfloat16>(c, dev) : launch<true, 128, 4, __nv_bfloat16>(c, dev);
  return p.tn == 32 ? launch<false, 32, 9, __nv_bfloat16>(c, dev) : launch<false, 128, 6, __nv_bfloat16>(c, dev);
}

int check_sizes(int64_t M, int64_t N, int64_t K, int G, bool grouped, int act, int dtype) {
  if (G < 1 || G > kMaxGroups || (!grouped && G != 1)) return PGG_ERR_INVALID_ARG;
  if (M < 0 || M > INT32_MAX - 4096) return PGG_ERR_INVALID_ARG;
  if (act < PGG_ACT_NONE || act > PGG_ACT_SWIGLU) return PGG_ERR_INVALID_ARG;
  if (dtype != PGG_DTYPE_F32 && dtype != PGG_DTYPE_BF16) return PGG_ERR_INVALID_ARG;
  for (int64_t d : {N, K})
    if (d < 8 || d >= ((int64_t)1 << 30)) return PGG_ERR_INVALID_ARG;
  return N % (act == PGG_ACT_SWIGLU ? 16 : 8) || K % 8 ? PGG_ERR_ALIGNMENT : PGG_OK;
}

int linear_impl(const void* X, const void* W, const int32_t* group_lens, const void* bias, const void* residual,
                void* Y, int dtype, void* Z, int64_t M, int64_t N, int64_t K, int G, int act, float alpha,
                float offset, float limit, unsigned long long wait_ns, long long stall_at, int32_t* err,
                void* stream, const Plan* plan = nullptr) {
  int st = check_sizes(M, N, K, G, group_lens != nullptr, act, dtype);
  if (st) return st;
  const float big = 3.0e38f;
  if (!(alpha >= -big && alpha <= big) || !(offset >= -big && offset <= big) || !(limit >= 0.0f && limit <= big))
    return PGG_ERR_INVALID_ARG;
  if (M == 0) return PGG_OK;
  if (!X || !W || !Y) return PGG_ERR_INVALID_ARG;
  for (const void* p : {X, W, bias, residual, (const void*)Y, (const void*)Z})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(group_lens, 4) || !aligned_to(err, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  // (a tile's loads are waited for in one piece by its epilogue: the longest reductions need more than the default)
  if (wait_ns == 0) wait_ns = kWaitTimeoutNs + 2000ull * (unsigned long long)ceil_div(K, kBK);
  LinCall c{X, W, {}, dtype == PGG_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)};
  c.a = {group_lens, G, M, (int)N, (int)K, (int)(act == PGG_ACT_SWIGLU ? N / 2 : N), act, {alpha, offset, limit},
         static_cast<const __nv_bfloat16*>(bias), residual, Y, static_cast<__nv_bfloat16*>(Z), err, wait_ns, stall_at};
  if (plan) return plan_has(c, dev, *plan) ? run_plan(c, dev, *plan) : PGG_ERR_INVALID_ARG;
  Plan chosen;
  st = choose(c, dev, &chosen);
  return st ? st : run_plan(c, dev, chosen);
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

int pgg_test_linear_plan(int64_t M, int64_t N, int64_t K, int G, int grouped, int act, int dtype, int sms,
                         int32_t* plan) {
  int st = check_sizes(M, N, K, G, grouped != 0, act, dtype);
  if (st) return st;
  if (!plan || M < 1 || sms < 0) return PGG_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (sms) dev.sms = sms;
  else if ((st = current_device(&dev)) != PGG_OK) return st;
  LinCall c{nullptr, nullptr, {}, dtype == PGG_DTYPE_F32, nullptr};
  static const int32_t some = 0;  // (the choice asks whether there are lengths, not for them)
  c.a.group_lens = grouped ? &some : nullptr;
  c.a.G = G;
  c.a.M = M;
  c.a.N = (int)N;
  c.a.K = (int)K;
  c.a.width = (int)(act == PGG_ACT_SWIGLU ? N / 2 : N);
  c.a.act = act;
  Plan p;
  if ((st = choose(c, dev, &p))) return st;
  plan[0] = p.kind;
  plan[1] = p.tn;
  plan[2] = p.splits;
  plan[3] = p.kind == Plan::kSplit && split_ctas(c, p.tn, p.splits) > dev.sms ? 2 : 1;
  return PGG_OK;
}

int pgg_test_planned_linear(int kind, int tn, int splits, const void* X, const void* W, const int32_t* group_lens,
                            const void* bias, const void* residual, void* Y, int dtype, void* Z, int64_t M, int64_t N,
                            int64_t K, int G, int act, float alpha, float offset, float limit, int64_t stall_at,
                            uint64_t wait_ns, int32_t* err, void* stream) {
  if (kind < Plan::kSplit || kind > Plan::kPair || stall_at < -1) return PGG_ERR_INVALID_ARG;
  if (wait_ns != 0 && (wait_ns < 100000ull || wait_ns > 1000000000ull)) return PGG_ERR_INVALID_ARG;
  const Plan p{static_cast<Plan::Kind>(kind), tn, splits, 0.0};
  return linear_impl(X, W, group_lens, bias, residual, Y, dtype, Z, M, N, K, G, act, alpha, offset, limit, wait_ns,
                     stall_at, err, stream, &p);
}

}  // extern "C"

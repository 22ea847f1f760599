// Matrix products per group of rows with the bias, the activation and the residual's addition in
// the epilogue (tcgen05, kind::f16):
//
//   Z_g = X_g W_g^T + b_g        Y = act(Z) + R
//
// for ragged groups (experts) or one dense product.  Z stays fp32 up to Y; the copy of it that the
// backward pass reads is rounded once, from fp32.
//
// The weights are the MMA's A operand (128 output columns a tile), the rows of X its B operand: an
// accumulator row is an output column, an accumulator column a row of X.  So a tile takes as many
// MMA columns as the group has rows left, in steps of 16 -- a ragged tail costs what it holds -- a
// thread's bias is one number, and a few rows of X stream the weights through the same code.
#include <algorithm>

#include "act.cuh"
#include "block.cuh"
#include "epilogue.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kBN = 128;     // output columns of a tile (of each half with swiglu): TMEM lanes
constexpr int kBK = 64;      // one 128-byte swizzle atom of the reduction
constexpr int kThreads = 192;
constexpr int kBand = 16;    // row tiles that take their turns at one column tile

struct LinArgs {
  const int32_t* group_lens;  // or nullptr: one group of M rows
  int G;
  int64_t M;
  int N, K;    // rows and columns of a W_g
  int width;   // columns of Y: N, or N / 2 with swiglu
  int act;
  ActForm form;
  const __nv_bfloat16* bias;  // [G, N] or nullptr
  const void* residual;       // [M, width] of Y's type or nullptr
  void* y;
  __nv_bfloat16* z;           // [M, N] or nullptr
  int32_t* err;
  unsigned long long wait_ns;
  long long stall_at;         // test hook: the producer stops before this stage (-1: never)
};

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

struct LinTile {
  int g, row0, rows, col0;
};

template <int TN>
__device__ __forceinline__ LinTile lin_tile(int t, const LinArgs& a, int nct, const int32_t* s_off,
                                            const int32_t* s_tile, GroupCursor& cur) {
  cur.at(s_tile, s_off, nullptr, a.G, t);
  const int local = t - cur.t_lo, nmt = (cur.len + TN - 1) / TN;
  const int band = local / (kBand * nct), in = local - band * kBand * nct;
  const int bm = min(kBand, nmt - band * kBand);
  const int ct = in / bm, mt = band * kBand + in - ct * bm;
  return {cur.g, cur.off + mt * TN, min(TN, cur.len - mt * TN), ct * kBN};
}

// ---------------------------------------------------------------- epilogue
// A warp has 32 output columns (its lanes) and takes 32 rows of X (accumulator columns) at a time;
// a row of the chunk is 64 (bf16) or 128 (fp32) contiguous bytes of the output, so the chunk turns
// through shared memory and leaves in 16-byte pieces.

// Writes v (row j of the chunk, this lane's column) to dst, row stride ld: rows [0, nrows), columns
// [0, ncols) of the chunk exist (ncols a multiple of 8).
__device__ __forceinline__ void put_chunk(uint8_t* stg, const float (&v)[32], __nv_bfloat16* dst, size_t ld, int nrows,
                                          int ncols, int lane) {
  __nv_bfloat16* s = reinterpret_cast<__nv_bfloat16*>(stg);
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j * 32 + lane] = __float2bfloat16_rn(v[j]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = 8 * (lane & 3);
    const uint4 w = reinterpret_cast<const uint4*>(stg)[32 * i + lane];
    if (r < nrows && c < ncols) *reinterpret_cast<uint4*>(dst + (size_t)r * ld + c) = w;
  }
  __syncwarp();
}
__device__ __forceinline__ void put_chunk(uint8_t* stg, const float (&v)[32], float* dst, size_t ld, int nrows,
                                          int ncols, int lane) {
  float* s = reinterpret_cast<float*>(stg);
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j * 32 + lane] = v[j];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7);
    const uint4 w = reinterpret_cast<const uint4*>(stg)[32 * i + lane];
    if (r < nrows && c < ncols) *reinterpret_cast<uint4*>(dst + (size_t)r * ld + c) = w;
  }
  __syncwarp();
}
// v[j] += the residual's row j at this lane's column.
__device__ __forceinline__ void add_chunk(uint8_t* stg, float (&v)[32], const __nv_bfloat16* src, size_t ld, int nrows,
                                          int ncols, int lane) {
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = 8 * (lane & 3);
    w[i] = r < nrows && c < ncols ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * ld + c)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(stg)[32 * i + lane] = w[i];
  __syncwarp();
  const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(stg);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += __bfloat162float(s[j * 32 + lane]);
  __syncwarp();
}
__device__ __forceinline__ void add_chunk(uint8_t* stg, float (&v)[32], const float* src, size_t ld, int nrows,
                                          int ncols, int lane) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < nrows && lane < ncols) v[j] += __ldg(src + (size_t)j * ld + lane);
}

template <int ACT>
__device__ __forceinline__ void apply_act(float (&v)[32], const ActForm& f) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = act_f<ACT>(v[j], f);
}

// One chunk of 32 rows: z (and u, the other half) with the bias already in them -> Z, Y.
// row: the chunk's first output row; col: the warp's first column.
template <bool GATED, typename T>
__device__ __forceinline__ void finish_chunk(const LinArgs& a, float (&z)[32], float (&u)[32], size_t row, int col,
                                             int nrows, uint8_t* stg, int lane) {
  const int ncols = min(32, a.width - col);
  if (a.z) {
    put_chunk(stg, z, a.z + row * a.N + col, a.N, nrows, ncols, lane);
    if (GATED) put_chunk(stg, u, a.z + row * a.N + a.width + col, a.N, nrows, ncols, lane);
  }
  if (GATED) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = swiglu_f(z[j], u[j], a.form);
  } else if (a.act == kActSilu) {
    apply_act<kActSilu>(z, a.form);
  } else if (a.act == kActGelu) {
    apply_act<kActGelu>(z, a.form);
  }
  if (a.residual)
    add_chunk(stg, z, static_cast<const T*>(a.residual) + row * a.width + col, a.width, nrows, ncols, lane);
  put_chunk(stg, z, static_cast<T*>(a.y) + row * a.width + col, a.width, nrows, ncols, lane);
}

// The group tables: with no lengths given, one group of M rows.
template <int TN>
__device__ __forceinline__ bool lin_scan(const LinArgs& a, int nct, int32_t* s_off, int32_t* s_tile, int lane) {
  TileCount tc;
  tc.bm = TN;
  tc.per_row_tile = nct;
  if (a.group_lens) return scan_groups(a.group_lens, a.G, a.M, tc, s_off, s_tile, nullptr, 0, lane);
  if (lane == 0) {
    s_off[0] = s_tile[0] = 0;
    s_off[1] = (int32_t)a.M;
    s_tile[1] = tc((int)a.M);
  }
  return false;
}

template <bool GATED, int TN, int STAGES, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinArgs a) {
  using L = LinSmem<GATED, TN, STAGES>;
  constexpr int kBox = TN < 64 ? TN : 64;           // rows of X per load
  constexpr int kAcc = (GATED ? 2 : 1) * TN;        // columns of an accumulator
  constexpr uint32_t kTmemCols = 2 * kAcc;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert((2 * STAGES + 5) * 8 + 24 <= 256, "barrier area");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
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
    for (int i = 0; i < 2; ++i) {
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
    const bool bad = lin_scan<TN>(a, nct, s_off, s_tile, lane);
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
      const LinTile T_ = lin_tile<TN>(t, a, nct, s_off, s_tile, cur);
      const int boxes = (T_.rows + kBox - 1) / kBox;
      for (int kb = 0; kb < nkb; ++kb) {
        if (issued == a.stall_at) { stalled = true; break; }
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        if (lane == 0) {
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t sa = smem_a + stage * L::kABytes, sb = smem_b + stage * L::kBBytes;
          mbar_arrive_expect_tx(fb, L::kABytes + boxes * kBox * 128);
          tma_load_3d(sa, &tmW, fb, kb * kBK, T_.col0, T_.g);
          if (GATED) tma_load_3d(sa + kBN * 128, &tmW, fb, kb * kBK, a.width + T_.col0, T_.g);
          for (int b = 0; b < boxes; ++b) tma_load_2d(sb + b * kBox * 128, &tmX, fb, kb * kBK, T_.row0 + b * kBox);
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
      const LinTile T_ = lin_tile<TN>(t, a, nct, s_off, s_tile, cur);
      const uint32_t idesc = idesc_bf16(kBN, (T_.rows + 15) & ~15, false, false);
      if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      const uint32_t d = tmem + acc * kAcc;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t da = desc_a + (uint64_t)(stage * L::kABytes >> 4);
          const uint64_t db = desc_b + (uint64_t)(stage * L::kBBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < kBK / 16; ++ks) {
            mma_f16(d, da + 2 * ks, db + 2 * ks, idesc, (kb | ks) ? 1u : 0u);
            if (GATED) mma_f16(d + TN, da + (kBN * 128 >> 4) + 2 * ks, db + 2 * ks, idesc, (kb | ks) ? 1u : 0u);
          }
          mma_commit(smem_u32(&empty[stage]));
        }
        __syncwarp();
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (aborted) break;
      if (lane == 0) mma_commit(smem_u32(&tfull[acc]));
      __syncwarp();
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
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
      const LinTile T_ = lin_tile<TN>(t, a, nct, s_off, s_tile, cur);
      const int col = T_.col0 + q * 32, n = col + lane;
      float bg = 0.0f, bu = 0.0f;
      if (a.bias && n < a.width) {
        const __nv_bfloat16* b = a.bias + (size_t)T_.g * a.N + n;
        bg = __bfloat162float(b[0]);
        if (GATED) bu = __bfloat162float(b[a.width]);
      }
      if (!warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem + acc * kAcc + ((uint32_t)(q * 32) << 16);
      if (col < a.width) {
#pragma unroll 1
        for (int c = 0; c < T_.rows; c += 32) {
          uint32_t rg[32], ru[32];
          tmem_ld32(tb + c, rg);
          if (GATED) tmem_ld32(tb + TN + c, ru);
          tmem_ld_wait();
          float z[32], u[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            z[j] = __uint_as_float(rg[j]) + bg;
            u[j] = GATED ? __uint_as_float(ru[j]) + bu : 0.0f;
          }
          finish_chunk<GATED, T>(a, z, u, (size_t)T_.row0 + c, col, min(32, T_.rows - c), stg, lane);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
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

struct LinCall {
  const void *X, *W;
  LinArgs a;
  bool f32;
  cudaStream_t stream;
};

template <bool GATED, int TN, int STAGES, typename T>
int launch(const LinCall& c, const DeviceInfo& dev) {
  using L = LinSmem<GATED, TN, STAGES>;
  auto kern = linear_kernel<GATED, TN, STAGES, T>;
  CUtensorMap tw, tx;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t K = c.a.K, N = c.a.N;
  uint64_t dw[3] = {K, N, (uint64_t)c.a.G}, sw[2] = {K * 2, N * K * 2};
  uint32_t bw[3] = {kBK, kBN, 1};
  uint64_t dx[2] = {K, (uint64_t)c.a.M}, sx[1] = {K * 2};
  uint32_t bx[2] = {kBK, TN < 64 ? TN : 64};
  int st;
  if ((st = encode_tmap(&tw, bf, 3, c.W, dw, sw, bw, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  if ((st = encode_tmap(&tx, bf, 2, c.X, dx, sx, bx, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  // the most that the kernel is ever launched with: another thread may call with more groups meanwhile
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes(kMaxGroups));
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t tiles = ((c.a.M + TN - 1) / TN + (c.a.group_lens ? c.a.G : 0)) * ceil_div(c.a.width, kBN);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(dev.sms, tiles));
  kern<<<grid, kThreads, L::bytes(c.a.G), c.stream>>>(tw, tx, c.a);
  return cuda_status(cudaGetLastError());
}

template <typename T>
int dispatch(const LinCall& c, const DeviceInfo& dev) {
  const bool few = c.a.M <= 16 * (int64_t)c.a.G;  // rows of a group on average
  if (c.a.act == kActSwiglu) return few ? launch<true, 32, 5, T>(c, dev) : launch<true, 128, 4, T>(c, dev);
  return few ? launch<false, 32, 9, T>(c, dev) : launch<false, 256, 4, T>(c, dev);
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
  return c.f32 ? dispatch<float>(c, dev) : dispatch<__nv_bfloat16>(c, dev);
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

// The gradient before the activation of grouped_linear, and the biases' gradient:
//
//   dZ = dY act'(Z)          db_g = sum over the rows of group g of dZ, in fp32
//
// in one pass over dY and Z.  (The products' own gradients are the grouped dgrad and wgrad on dZ,
// the residual's is dY.)
//
// What bounds it is memory, so the work is cut by bytes and not by groups: a block has a slab of up
// to 256 columns and an equal run of rows, walks the groups that the run meets and sums each
// group's rows in registers.  A group that lies inside one run is finished there; of one that
// runs divide, every run leaves its sum in the workspace -- at most two a run, for the group that
// it begins in and the one that it ends in -- and a second kernel adds them in row order.
// 32768 x 5760 with swiglu, 32 groups (944 MB): 162 us, 86% of the copy rate (three streams in, two out).
#include <algorithm>

#include "act.cuh"
#include "block.cuh"
#include "packed.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kChunks = 32;      // 8-column pieces of a slab, one a lane
constexpr int kMinRows = 32;     // rows of a run
constexpr int kFewMean = 32;     // rows a group, below which they are few
constexpr int kFewRows = 8;      // of a group in a run that are one warp's
constexpr int kFewMinRows = 8;   // of one where the groups have few

struct LinBwdArgs {
  const uint4* dy;  // [M, width]
  const uint4* z;   // [M, N] or nullptr (no activation)
  uint4* dz;        // [M, N] or nullptr
  const int32_t* group_lens;
  int G;
  int64_t M;
  int nvec;         // 8-column pieces of `width`
  int per;          // of them in a slab
  int slabs, runs;
  int run_rows;
  ActForm form;
  float* db;        // [G, N]
  float* part;      // [runs][2][N]: sums of the group a run begins in, and of the one it ends in
  int32_t* offs;    // [G + 1] the groups' first rows, and [G + 1]: 1 if the lengths are bad
  int32_t* err;
};

// The group of a row: the last one that begins at or before it (empty ones before it begin there too).
__device__ __forceinline__ int group_of(const int32_t* s_off, int G, int64_t row) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_off[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Rows first, first + stride, ... of one group at piece v: dZ, added to their sums.  H: halves.
template <int ACT, int UNROLL, int H>
__device__ __forceinline__ void sum_rows(const LinBwdArgs& a, int v, int64_t first, int stride, int64_t end,
                                         f2 (&sum)[H][4]) {
  constexpr bool GATED = ACT == kActSwiglu;
  for (int64_t r = first; r < end; r += (int64_t)stride * UNROLL) {
    uint4 dy[UNROLL], z[UNROLL], u[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int64_t row = r + i * stride;
      if (row < end) {
        dy[i] = a.dy[row * a.nvec + v];
        if (ACT != kActNone) z[i] = a.z[row * H * a.nvec + v];
        if (GATED) u[i] = a.z[row * H * a.nvec + a.nvec + v];
      }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int64_t row = r + i * stride;
      if (row < end) {
        f2 d[4], zz[4], uu[4], o[4], o2[4];
        unpack2(dy[i], d);
        if (ACT != kActNone) unpack2(z[i], zz);
        if (GATED) unpack2(u[i], uu);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (GATED) swiglu_bwd_f2(d[e], zz[e], uu[e], a.form, o[e], o2[e]);
          else o[e] = ACT == kActNone ? d[e] : act_bwd_f2<ACT>(d[e], zz[e], a.form);
          sum[0][e] = add2(sum[0][e], o[e]);
          if (GATED) sum[H - 1][e] = add2(sum[H - 1][e], o2[e]);
        }
        if (ACT != kActNone && a.dz) {
          a.dz[row * H * a.nvec + v] = round8(o);
          if (GATED) a.dz[row * H * a.nvec + a.nvec + v] = round8(o2);
        }
      }
    }
  }
}

// (The scan and the sums' way out are written out here: with the functions that the kernel below has, swiglu took
// 166.6 us.)
template <int ACT, int UNROLL, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) linear_bwd_kernel(const LinBwdArgs a) {
  constexpr bool GATED = ACT == kActSwiglu;
  constexpr int H = GATED ? 2 : 1;
  extern __shared__ int32_t s_off[];  // [G + 1], and as many for the scan's tile counts
  __shared__ float s_sum[kWarps][H * 8][kChunks];
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    bool bad = false;
    if (a.group_lens) {
      TileCount tc{1, 0};
      bad = scan_groups(a.group_lens, a.G, a.M, tc, s_off, s_off + a.G + 1, nullptr, 0, lane);
    } else if (lane == 0) {
      s_off[0] = 0;
      s_off[1] = (int32_t)a.M;
    }
    if (lane == 0) {
      s_bad = bad;
      if (bad && blockIdx.x == 0) set_error(a.err, kErrBadGroupLens);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int g = threadIdx.x; g <= a.G; g += kThreads) a.offs[g] = s_off[g];
    if (threadIdx.x == 0) a.offs[a.G + 1] = s_bad;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (s_bad) return;

  const int slab = blockIdx.x % a.slabs, run = blockIdx.x / a.slabs;
  const int v = slab * a.per + lane;
  const bool in = lane < a.per && v < a.nvec;
  const int64_t r_begin = (int64_t)run * a.run_rows;
  const int64_t r_end = min(a.M, r_begin + a.run_rows);
  const int64_t N = (int64_t)H * a.nvec * 8;
  if (r_begin >= r_end) return;

  int g = group_of(s_off, a.G, r_begin);
  for (int64_t r0 = r_begin; r0 < r_end; ++g) {
    const int64_t r1 = min(r_end, (int64_t)s_off[g + 1]);
    if (r1 <= r0) continue;  // an empty group
    f2 sum[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[h][e] = both(0.0f);
    if (in) sum_rows<ACT, UNROLL, H>(a, v, r0 + warp, kWarps, r1, sum);
    // the warps' sums, in a fixed order
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(sum[h][e], s_sum[warp][h * 8 + 2 * e][lane], s_sum[warp][h * 8 + 2 * e + 1][lane]);
    __syncthreads();
    const bool first = s_off[g] < r_begin, last = s_off[g + 1] > r_end;  // divided before, behind this run
    float* dst = !first && !last ? a.db + (int64_t)g * N : a.part + (int64_t)(run * 2 + (first ? 0 : 1)) * N;
    for (int i = threadIdx.x; i < H * 8 * kChunks; i += kThreads) {
      const int h = i / (8 * kChunks), c = i % (8 * kChunks), vv = slab * a.per + c / 8;
      if (c / 8 < a.per && vv < a.nvec) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += s_sum[w][h * 8 + c % 8][c / 8];
        dst[(int64_t)h * a.nvec * 8 + vv * 8 + c % 8] = t;
      }
    }
    r0 = r1;
  }
}

// The groups' first rows into s_off, and by block 0 into the workspace; false if the lengths are bad.
__device__ __forceinline__ bool scan_block(const LinBwdArgs& a, int32_t* s_off, int* s_bad) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    bool bad = false;
    if (a.group_lens) {
      TileCount tc{1, 0};
      bad = scan_groups(a.group_lens, a.G, a.M, tc, s_off, s_off + a.G + 1, nullptr, 0, lane);
    } else if (lane == 0) {
      s_off[0] = 0;
      s_off[1] = (int32_t)a.M;
    }
    if (lane == 0) {
      *s_bad = bad;
      if (bad && blockIdx.x == 0) set_error(a.err, kErrBadGroupLens);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int g = threadIdx.x; g <= a.G; g += kThreads) a.offs[g] = s_off[g];
    if (threadIdx.x == 0) a.offs[a.G + 1] = *s_bad;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  return !*s_bad;
}

// Where the sums of group g's rows in a run go: first, last: the group is divided before, behind the run.
__device__ __forceinline__ float* sums_of(const LinBwdArgs& a, int run, bool first, bool last, int g, int64_t N) {
  return !first && !last ? a.db + (int64_t)g * N : a.part + (int64_t)(run * 2 + (first ? 0 : 1)) * N;
}

// Puts them there from all warps, in a fixed order.
template <int H>
__device__ __forceinline__ void put_block_sums(const LinBwdArgs& a, const f2 (&sum)[H][4], float (*s_sum)[H * 8][kChunks],
                                               int slab, int run, bool first, bool last, int g, int64_t N) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(sum[h][e], s_sum[warp][h * 8 + 2 * e][lane], s_sum[warp][h * 8 + 2 * e + 1][lane]);
  __syncthreads();
  float* dst = sums_of(a, run, first, last, g, N);
  for (int i = threadIdx.x; i < H * 8 * kChunks; i += kThreads) {
    const int h = i / (8 * kChunks), c = i % (8 * kChunks), vv = slab * a.per + c / 8;
    if (c / 8 < a.per && vv < a.nvec) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += s_sum[w][h * 8 + c % 8][c / 8];
      dst[(int64_t)h * a.nvec * 8 + vv * 8 + c % 8] = t;
    }
  }
}

// The gradient for groups of few rows (see `few_rows`): of the groups of a run, those with at most kFewRows there
// are the warps' in turn, so that their loads' latencies do not follow one another and no barrier joins them
// (62 rows of 199 groups, 2392 columns: 43 us without that, 9.6 with).
template <int ACT, int UNROLL>
__global__ void __launch_bounds__(kThreads) linear_bwd_few_kernel(const LinBwdArgs a) {
  constexpr int H = ACT == kActSwiglu ? 2 : 1;
  extern __shared__ int32_t s_off[];
  __shared__ float s_sum[kWarps][H * 8][kChunks];
  __shared__ int s_bad;
  if (!scan_block(a, s_off, &s_bad)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slab = blockIdx.x % a.slabs, run = blockIdx.x / a.slabs;
  const int v = slab * a.per + lane;
  const bool in = lane < a.per && v < a.nvec;
  const int64_t r_begin = (int64_t)run * a.run_rows;
  const int64_t r_end = min(a.M, r_begin + a.run_rows);
  const int64_t N = (int64_t)H * a.nvec * 8;
  if (r_begin >= r_end) return;

  int turn = 0;
  for (int at = group_of(s_off, a.G, r_begin); at < a.G && s_off[at] < r_end; at += 32) {
    // 32 groups at a time
    const int mine = at + lane;
    const int64_t rows = mine < a.G ? min(r_end, (int64_t)s_off[mine + 1]) - max(r_begin, (int64_t)s_off[mine]) : 0;
    const uint32_t many = __ballot_sync(0xffffffffu, rows > kFewRows);
    for (uint32_t m = __ballot_sync(0xffffffffu, rows > 0); m; m &= m - 1) {
      const int bit = __ffs(m) - 1, g = at + bit;
      const bool together = many >> bit & 1;
      if (!together && turn++ % kWarps != warp) continue;
      const bool first = s_off[g] < r_begin, last = s_off[g + 1] > r_end;
      const int64_t r0 = first ? r_begin : s_off[g], r1 = last ? r_end : s_off[g + 1];
      f2 sum[H][4];
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[h][e] = both(0.0f);
      if (in) sum_rows<ACT, UNROLL, H>(a, v, together ? r0 + warp : r0, together ? kWarps : 1, r1, sum);
      if (together) {
        put_block_sums<H>(a, sum, s_sum, slab, run, first, last, g, N);
      } else if (in) {
        float* dst = sums_of(a, run, first, last, g, N);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(sum[h][e], t[2 * e], t[2 * e + 1]);
          float4* to = reinterpret_cast<float4*>(dst + ((int64_t)h * a.nvec + v) * 8);
          to[0] = make_float4(t[0], t[1], t[2], t[3]);
          to[1] = make_float4(t[4], t[5], t[6], t[7]);
        }
      }
    }
  }
}

// db_g of the groups that runs divide, and zeros for the empty ones, launched while the kernel above runs.
// A warp has 32 columns; SHARE: the block's warps share out the runs of one group (few long groups), else each
// warp has groups of its own (32 groups of 1092 rows, 5760 columns: 4 us instead of 15.6).
constexpr int kRedWarps = 16;
template <bool SHARE>
__global__ void __launch_bounds__(32 * kRedWarps) bias_grad_reduce_kernel(const int32_t* __restrict__ offs,
                                                                          const float* __restrict__ part, int G,
                                                                          int run_rows, int64_t N,
                                                                          float* __restrict__ db) {
  __shared__ float s[SHARE ? kRedWarps : 1][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (offs[G + 1]) return;
  const int step = SHARE ? 1 : kRedWarps;
  for (int g = blockIdx.y * step + (SHARE ? 0 : warp); g < G; g += gridDim.y * step) {
    const int o0 = offs[g], o1 = offs[g + 1];
    const int p0 = o0 / run_rows, p1 = (o1 - 1) / run_rows;
    if (o0 != o1 && p0 == p1) continue;
    float t = 0.0f;
    if (c < N && o0 != o1) {
#pragma unroll 4
      for (int p = p0 + (SHARE ? warp : 0); p <= p1; p += SHARE ? kRedWarps : 1)
        t += part[(int64_t)(p * 2 + (o0 < p * run_rows ? 0 : 1)) * N + c];
    }
    if (SHARE) {
      s[warp][lane] = t;
      __syncthreads();
      t = 0.0f;
      if (warp == 0) {
#pragma unroll
        for (int w = 0; w < kRedWarps; ++w) t += s[SHARE ? w : 0][lane];
      }
      __syncthreads();
    }
    if ((!SHARE || warp == 0) && c < N) db[(int64_t)g * N + c] = t;
  }
}

// Groups of few rows, by the mean that the host knows: 4096 rows of 256 groups by Zipf's law, 4096 columns, silu:
// 52 us with the kernel for them, 86 without; 16384 rows of 256 equal groups, gelu: 104, 93.
bool few_rows(int64_t M, int G) { return M < (int64_t)kFewMean * G; }

// The cut: runs of equal rows, so many that all blocks together about fill the GPU (the count is
// fixed, not asked of the device, as it decides the workspace and the order of the sums).
struct Cut {
  int nvec, per, slabs, runs, run_rows;
};
// Resident blocks an SM, with the rows that a thread loads ahead (UNROLL): 32768 x 5760 with swiglu, 944 MB, 4
// blocks of one row 171 us when it was chosen (162 now), 3 of two 179, 5 of one (fewer registers than it needs) 208;
// 32768 x 4096 with gelu 4 of two 146, 3 of four 148, 5 of two 160; with silu 3 of four 127.5, 4 of two 128.
constexpr int per_sm(int act) { return act == kActNone ? 5 : act == kActSilu ? 3 : 4; }
Cut cut(int64_t M, int64_t N, int G, int act) {
  const int64_t width = act == kActSwiglu ? N / 2 : N;
  Cut c;
  c.nvec = (int)(width / 8);
  c.slabs = (c.nvec + kChunks - 1) / kChunks;
  c.per = (c.nvec + c.slabs - 1) / c.slabs;
  const int64_t most = std::max(1, 152 * per_sm(act) / c.slabs);
  const int64_t rows = std::max<int64_t>(few_rows(M, G) ? kFewMinRows : kMinRows, (M + most - 1) / most);
  c.run_rows = (int)((rows + kWarps - 1) / kWarps * kWarps);
  c.runs = (int)((M + c.run_rows - 1) / c.run_rows);
  return c;
}
size_t offs_bytes(int G) { return ((size_t)G + 2 + 3) / 4 * 16; }
size_t ws_need(const Cut& c, int G, int64_t N) { return offs_bytes(G) + (size_t)c.runs * 2 * (size_t)N * sizeof(float); }

int check_dims(int64_t M, int64_t N, int G, int act) {
  if (G < 1 || G > kMaxGroups || M < 0 || M > INT32_MAX - 4096) return PGG_ERR_INVALID_ARG;
  if (act < PGG_ACT_NONE || act > PGG_ACT_SWIGLU) return PGG_ERR_INVALID_ARG;
  if (N < 8 || N >= ((int64_t)1 << 30)) return PGG_ERR_INVALID_ARG;
  return N % (act == PGG_ACT_SWIGLU ? 16 : 8) ? PGG_ERR_ALIGNMENT : PGG_OK;
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_grouped_linear_bwd_workspace_size(int64_t M, int64_t N, int G, int act, size_t* bytes) {
  const int st = check_dims(M, N, G, act);
  if (st) return st;
  if (!bytes) return PGG_ERR_INVALID_ARG;
  *bytes = ws_need(cut(M, N, G, act), G, N);
  return PGG_OK;
}

int pgg_grouped_linear_bwd(const void* dY, const void* Z, const int32_t* group_lens, void* dZ, float* dbias, int64_t M,
                           int64_t N, int G, int act, float alpha, float offset, float limit, void* ws,
                           size_t ws_bytes, int32_t* err, void* stream) {
  int st = check_dims(M, N, G, act);
  if (st) return st;
  if (!group_lens && G != 1) return PGG_ERR_INVALID_ARG;
  const float big = 3.0e38f;
  if (!(alpha >= -big && alpha <= big) || !(offset >= -big && offset <= big) || !(limit >= 0.0f && limit <= big))
    return PGG_ERR_INVALID_ARG;
  if (!dbias) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(dbias, 16)) return PGG_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) return cuda_status(cudaMemsetAsync(dbias, 0, (size_t)G * N * sizeof(float), s));
  if (!dY || !ws || (act != PGG_ACT_NONE) != (Z != nullptr) || (dZ && act == PGG_ACT_NONE)) return PGG_ERR_INVALID_ARG;
  const Cut c = cut(M, N, G, act);
  if (ws_bytes < ws_need(c, G, N)) return PGG_ERR_INVALID_ARG;
  for (const void* p : {dY, Z, (const void*)dZ, (const void*)ws})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(group_lens, 4) || !aligned_to(err, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  int32_t* offs = static_cast<int32_t*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + offs_bytes(G));
  LinBwdArgs a{static_cast<const uint4*>(dY), static_cast<const uint4*>(Z), static_cast<uint4*>(dZ), group_lens, G, M,
               c.nvec, c.per, c.slabs, c.runs, c.run_rows, {alpha, offset, limit}, dbias, part, offs, err};
  const unsigned grid = (unsigned)(c.slabs * c.runs);
  const size_t smem = 2 * ((size_t)G + 1) * sizeof(int32_t);
  void (*kern)(const LinBwdArgs);
  if (few_rows(M, G))
    kern = act == PGG_ACT_NONE   ? linear_bwd_few_kernel<kActNone, 4>
           : act == PGG_ACT_SILU ? linear_bwd_few_kernel<kActSilu, 2>
           : act == PGG_ACT_GELU ? linear_bwd_few_kernel<kActGelu, 2>
                                 : linear_bwd_few_kernel<kActSwiglu, 1>;
  else
    kern = act == PGG_ACT_NONE   ? linear_bwd_kernel<kActNone, 4, per_sm(kActNone)>
           : act == PGG_ACT_SILU ? linear_bwd_kernel<kActSilu, 4, per_sm(kActSilu)>
           : act == PGG_ACT_GELU ? linear_bwd_kernel<kActGelu, 2, per_sm(kActGelu)>
                                 : linear_bwd_kernel<kActSwiglu, 1, per_sm(kActSwiglu)>;
  kern<<<grid, kThreads, smem, s>>>(a);
  if ((st = cuda_status(cudaGetLastError()))) return st;
  cudaLaunchConfig_t cfg{};
  const bool share = c.runs > 4 * G;
  cfg.gridDim = dim3((unsigned)((N + 31) / 32), (unsigned)(share ? std::min(G, 16) : (G + kRedWarps - 1) / kRedWarps));
  cfg.blockDim = dim3(32 * kRedWarps);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, share ? bias_grad_reduce_kernel<true> : bias_grad_reduce_kernel<false>,
                                           (const int32_t*)offs, (const float*)part, G,
                                           c.run_rows, N, dbias);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // extern "C"

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
//
// Three kernels: linear_pair.cu (long groups, bf16 results), linear.cu (one CTA per SM), linear_split.cu
// (few rows); linear.cu chooses.
#pragma once
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "block.cuh"
#include "epilogue.cuh"
#include "sched.cuh"

namespace pgg {

constexpr int kBN = 128;     // output columns of a tile (of each half with swiglu): TMEM lanes
constexpr int kBK = 64;      // one 128-byte swizzle atom of the reduction
constexpr int kLinThreads = 192;
constexpr int kChunk = 4;    // fp32 results: k-blocks that one accumulator takes
constexpr int kBand = 8;     // row tiles that take their turns at one column tile

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

struct LinTile {
  int g, row0, rows, col0;
};

// Tile t: up to TN rows by CW columns, nct column tiles.  Within a group, up to kBand row tiles take turns
// at one column tile, so that what runs at one time shares a band of X and a few column tiles of W in L2.
// A short group's rows are shared out evenly over its tiles (in steps of 16), so that its last tile is not a
// small one that costs the weights' loads of a full one; and CTAs take every 152nd tile, so that with two tiles a
// group one half of them would have all the small ones (64 groups of 300 rows, 4096 x 2048, on CTA pairs: 307 -> 259 us).
template <int CW>
__device__ __forceinline__ LinTile lin_tile(int t, const LinArgs& a, int TN, int nct, const int32_t* s_off,
                                            const int32_t* s_tile, GroupCursor& cur) {
  cur.at(s_tile, s_off, nullptr, a.G, t);
  const int local = t - cur.t_lo, nmt = (cur.len + TN - 1) / TN;
  const int band = local / (kBand * nct), in = local - band * kBand * nct;
  const int bm = min(kBand, nmt - band * kBand);
  const int ct = in / bm, mt = band * kBand + in - ct * bm;
  // (with at most 8 tiles of up to 256 rows the steps of 16 leave none without rows)
  const int per = nmt <= 8 ? ((cur.len + nmt - 1) / nmt + 15) & ~15 : TN;
  return {cur.g, cur.off + mt * per, min(per, cur.len - mt * per), ct * CW};
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
// 16 rows of 32 columns, as put_chunk.
__device__ __forceinline__ void put_rows16(uint8_t* stg, const float (&v)[16], __nv_bfloat16* dst, size_t ld, int nrows,
                                           int ncols, int lane) {
  __nv_bfloat16* s = reinterpret_cast<__nv_bfloat16*>(stg);
#pragma unroll
  for (int j = 0; j < 16; ++j) s[j * 32 + lane] = __float2bfloat16_rn(v[j]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 2), c = 8 * (lane & 3);
    const uint4 w = reinterpret_cast<const uint4*>(stg)[32 * i + lane];
    if (r < nrows && c < ncols) *reinterpret_cast<uint4*>(dst + (size_t)r * ld + c) = w;
  }
  __syncwarp();
}
__device__ __forceinline__ void put_rows16(uint8_t* stg, const float (&v)[16], float* dst, size_t ld, int nrows, int ncols,
                                           int lane) {
  float* s = reinterpret_cast<float*>(stg);
#pragma unroll
  for (int j = 0; j < 16; ++j) s[j * 32 + lane] = v[j];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7);
    const uint4 w = reinterpret_cast<const uint4*>(stg)[32 * i + lane];
    if (r < nrows && c < ncols) *reinterpret_cast<uint4*>(dst + (size_t)r * ld + c) = w;
  }
  __syncwarp();
}

// The chunk's residual in the order of its 16-byte pieces, zeros outside; and v[j] += its row j at this
// lane's column.
__device__ __forceinline__ void fetch_chunk(uint4 (&w)[4], const __nv_bfloat16* src, size_t ld, int nrows, int ncols,
                                            int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = 8 * (lane & 3);
    w[i] = r < nrows && c < ncols ? *reinterpret_cast<const uint4*>(src + (size_t)r * ld + c) : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void add_fetched(uint8_t* stg, float (&v)[32], const uint4 (&w)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(stg)[32 * i + lane] = w[i];
  __syncwarp();
  const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(stg);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += __bfloat162float(s[j * 32 + lane]);
  __syncwarp();
}
__device__ __forceinline__ void add_chunk(uint8_t* stg, float (&v)[32], const __nv_bfloat16* src, size_t ld, int nrows,
                                          int ncols, int lane) {
  uint4 w[4];
  fetch_chunk(w, src, ld, nrows, ncols, lane);
  add_fetched(stg, v, w, lane);
}
__device__ __forceinline__ void add_chunk(uint8_t* stg, float (&v)[32], const float* src, size_t ld, int nrows,
                                          int ncols, int lane) {
  // (places that are not there read the last that is: loads without a branch between them, whose latencies
  // would follow one another)
  const float* p = src + min(lane, ncols - 1);
  float w[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) w[j] = p[(size_t)min(j, nrows - 1) * ld];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += w[j];
  __syncwarp();  // (the residual may be Y: every row is read before it is written)
}

// 32 accumulator columns of this thread's lane, plus the bias; or added to what is there.
__device__ __forceinline__ void load_acc(uint32_t taddr, float (&v)[32], float bias) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) + bias;
}
__device__ __forceinline__ void add_acc(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
}

template <int ACT, bool FAST, int N>
__device__ __forceinline__ void apply_act(float (&v)[N], const ActForm& f) {
  if constexpr (ACT == kActGelu) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const f2 z = make2(v[j], v[j + 1]);
      split2(mul2(z, normal_cdf_f2(z, gauss_f2<FAST>(z))), v[j], v[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_f<ACT, FAST>(v[j], f);
  }
}

// One chunk of 32 rows: z (and u, the other half) with the bias already in them -> Z, Y.
// row: the chunk's first output row; col: the warp's first column.
template <bool GATED, typename T>
__device__ __forceinline__ void finish_chunk(const LinArgs& a, float (&z)[32], float (&u)[32], size_t row, int col,
                                             int nrows, uint8_t* stg, int lane) {
  constexpr bool kFast = !std::is_same<T, float>::value;
  const int ncols = min(32, a.width - col);
  if (a.z) {
    put_chunk(stg, z, a.z + row * a.N + col, a.N, nrows, ncols, lane);
    if (GATED) put_chunk(stg, u, a.z + row * a.N + a.width + col, a.N, nrows, ncols, lane);
  }
  if (GATED) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = swiglu_f<kFast>(z[j], u[j], a.form);
  } else if (a.act == kActSilu) {
    apply_act<kActSilu, kFast>(z, a.form);
  } else if (a.act == kActGelu) {
    apply_act<kActGelu, kFast>(z, a.form);
  }
  if (a.residual)
    add_chunk(stg, z, static_cast<const T*>(a.residual) + row * a.width + col, a.width, nrows, ncols, lane);
  put_chunk(stg, z, static_cast<T*>(a.y) + row * a.width + col, a.width, nrows, ncols, lane);
}

// The same for bf16 without halves, the residual's chunk fetched before.
__device__ __forceinline__ void finish_plain(const LinArgs& a, float (&z)[32], const uint4 (&res)[4], size_t row, int col,
                                             int nrows, int ncols, uint8_t* stg, int lane) {
  if (a.z) put_chunk(stg, z, a.z + row * a.N + col, a.N, nrows, ncols, lane);
  if (a.act == kActSilu) apply_act<kActSilu, true>(z, a.form);
  else if (a.act == kActGelu) apply_act<kActGelu, true>(z, a.form);
  if (a.residual) add_fetched(stg, z, res, lane);
  put_chunk(stg, z, static_cast<__nv_bfloat16*>(a.y) + row * a.width + col, a.width, nrows, ncols, lane);
}

// The group tables: with no lengths given, one group of M rows.
__device__ __forceinline__ bool lin_scan(const LinArgs& a, int TN, int nct, int32_t* s_off, int32_t* s_tile, int lane) {
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

struct LinCall {
  const void *X, *W;
  LinArgs a;
  bool f32;
  cudaStream_t stream;
};

// Tensor maps, one 128-byte swizzle atom of K wide: X as {K, M} in boxes of `xbox` rows; W as {K, N, G} in
// boxes of 128 rows or, with `halves`, as {K, N / 2, 2, G} in boxes of 64 rows of the gate and of the up half.
inline int lin_maps(const LinCall& c, uint32_t xbox, bool halves, CUtensorMap* tw, CUtensorMap* tx) {
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t K = c.a.K, N = c.a.N, G = c.a.G;
  const uint64_t d3[3] = {K, N, G}, s3[2] = {K * 2, N * K * 2};
  const uint32_t b3[3] = {kBK, kBN, 1};
  const uint64_t d4[4] = {K, N / 2, 2, G}, s4[3] = {K * 2, N * K, N * K * 2};
  const uint32_t b4[4] = {kBK, kBN / 2, 2, 1};
  const uint64_t dx[2] = {K, (uint64_t)c.a.M}, sx[1] = {K * 2};
  const uint32_t bx[2] = {kBK, xbox};
  const int st = halves ? encode_tmap(tw, bf, 4, c.W, d4, s4, b4, sw) : encode_tmap(tw, bf, 3, c.W, d3, s3, b3, sw);
  return st ? st : encode_tmap(tx, bf, 2, c.X, dx, sx, bx, sw);
}

// Launchers of the kernels (linear.cu, linear_pair.cu, linear_split.cu).
int launch_linear_pair(const LinCall& c, const DeviceInfo& dev);
int launch_linear_split(const LinCall& c, const DeviceInfo& dev, int tn, int splits);
// Clusters of `splits` CTAs that run at one time, with one CTA an SM or two, into *count.
int linear_split_clusters(const DeviceInfo& dev, int splits, bool one, int* count);

}  // namespace pgg

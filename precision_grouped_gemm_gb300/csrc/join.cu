// Between two blocks: the norm of a block's output, dropout, its gate, the scaled residual's
// addition, the next block's norm and the MX operand of its first product, in one pass:
//
//   t = x rstd1 gamma1 (or x)        rstd1 = 1 / sqrt(mean(x^2) + eps)
//   b = keep t / (1 - p)
//   s = ra residual + rb gate b      h = bf16(s)
//   y = s rstd2 gamma2               rstd2 = 1 / sqrt(mean(s^2) + eps)
//
// fp32 throughout, every output rounded once.  gate: a number per row, or per column.
//
// Backward, from x, h and the two rstd (xh = x rstd1, hh = h rstd2):
//
//   d = dh + rstd2 (u - hh mean(u hh)),  u = dy gamma2       dgamma2 = sum_rows dy hh
//   dresidual = ra d                                         dgate = rb sum d b (over columns, or rows)
//   dt = rb gate d keep / (1 - p)                            dgamma1 = sum_rows dt xh
//   dx = rstd1 (w - xh mean(w xh)),  w = dt gamma1 (or dx = dt)
//
// The mask is never stored: element i of the row-major tensor is kept where word i % 4 of block
// (i / 4, offset) of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as
// 1, 2, 3", 2011) under the key `seed` is at least floor(p 2^32); both passes compute it.
#include <algorithm>
#include <atomic>

#include "block.cuh"
#include "cluster.cuh"
#include "packed.cuh"

namespace pgg {
namespace {

// Sum over the block, in a fixed order, in every thread.  s: one of two buffers that successive sums
// alternate between, so that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float* s, int nwarps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  // (at most 16 warps)
  v = (threadIdx.x & 15) < nwarps ? s[threadIdx.x & 15] : 0.0f;
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The same for N = 4 or 8 sums at once: the first steps halve the sums that a lane carries, so that of N
// times five steps fewer than N + 4 are left.  CL > 1: over the CTAs of a cluster, which write each other's
// buffers; the buffers' turns keep a sum's writes behind the reads of the one before the last.
template <int N, int CL>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*s)[16 * CL], int nwarps) {
  constexpr int kSpan = 32 / N;  // lanes of one sum
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N, d = 16; n > 1; n >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? v[i] : v[i + n / 2], own = up ? v[i + n / 2] : v[i];
      v[i] = own + __shfl_xor_sync(0xffffffffu, give, d);
    }
  }
  float c = v[0];  // the sum number lane / kSpan
#pragma unroll
  for (int d = kSpan / 2; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
  const int i = lane / kSpan, k = lane % kSpan;
  if (CL == 1) {
    if (k == 0) s[i][threadIdx.x >> 5] = c;
    __syncthreads();
  } else {
    const uint32_t to = smem_u32(&s[i][16 * (blockIdx.x % CL) + (threadIdx.x >> 5)]);
    if (k < CL) st_cluster(map_rank(to, k), c);
    __syncwarp();
    cluster_sync();
  }
  // lane k of a sum's adds those of the warps k, k + kSpan, ...
  c = 0.0f;
#pragma unroll
  for (int r = 0; r < CL; ++r)
#pragma unroll
    for (int w = 0; w < 16; w += kSpan)
      if (w + k < nwarps) c += s[i][16 * r + w + k];
#pragma unroll
  for (int d = kSpan / 2; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = __shfl_sync(0xffffffffu, c, kSpan * j);
}

struct Drop {
  const int64_t* rng;  // {seed, offset}
  uint32_t below;      // words below it drop their element
  float inv;           // 1 / (1 - p); 1 without dropout
};

struct Key {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ Key load_key(const Drop& d) {
  const uint64_t seed = (uint64_t)__ldg(reinterpret_cast<const long long*>(d.rng));
  const uint64_t off = (uint64_t)__ldg(reinterpret_cast<const long long*>(d.rng) + 1);
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

__device__ __forceinline__ uint4 philox(uint64_t block, const Key& key) {
  uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = key.o0, x3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * x0, p1 = (uint64_t)0xCD9E8D57u * x2;
    x0 = (uint32_t)(p1 >> 32) ^ x1 ^ k0;
    x1 = (uint32_t)p1;
    x2 = (uint32_t)(p0 >> 32) ^ x3 ^ k1;
    x3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}
// Element e of the 8-element piece number `piece` of the tensor becomes 0 where it is dropped.
__device__ __forceinline__ void drop8(f2 (&t)[4], int64_t piece, const Drop& d, const Key& key) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = philox((uint64_t)piece * 2 + i, key);
    float a, b;
    split2(t[2 * i], a, b);
    t[2 * i] = make2(w.x >= d.below ? a : 0.0f, w.y >= d.below ? b : 0.0f);
    split2(t[2 * i + 1], a, b);
    t[2 * i + 1] = make2(w.z >= d.below ? a : 0.0f, w.w >= d.below ? b : 0.0f);
  }
}

// Bit e: element e of that piece is kept; and what is not kept made 0.
__device__ __forceinline__ uint32_t keep8(int64_t piece, const Drop& d, const Key& key) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = philox((uint64_t)piece * 2 + i, key);
    m |= ((w.x >= d.below ? 1u : 0u) | (w.y >= d.below ? 2u : 0u) | (w.z >= d.below ? 4u : 0u) |
          (w.w >= d.below ? 8u : 0u)) << (4 * i);
  }
  return m;
}
__device__ __forceinline__ void keep_only(f2 (&t)[4], uint32_t keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split2(t[i], a, b);
    t[i] = make2(keep & (1u << (2 * i)) ? a : 0.0f, keep & (2u << (2 * i)) ? b : 0.0f);
  }
}

// Piece v of a row of bf16 factors in fp32: ones where there are none, zeros past the row's end.
__device__ __forceinline__ void load_factors(const uint4* p, int v, int nvec, f2 (&f)[4]) {
  if (p && v < nvec) {
    unpack2(__ldg(p + v), f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = both(v < nvec ? 1.0f : 0.0f);
  }
}

struct JoinArgs {
  const uint4* x;
  const uint4* residual;  // or nullptr
  const uint4* gamma1;    // or nullptr
  const uint4* gamma2;    // or nullptr
  const float* gate_row;  // or nullptr
  const uint4* gate_col;  // or nullptr
  Drop drop;              // rng nullptr: none
  int64_t R;
  int nvec;
  float inv_c, eps, ra, rb;
  uint4* h;  // outputs: each or nullptr
  uint4* y;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd1;
  float* rstd2;
};

// A block walks rows with a grid stride; thread t owns the row's 8-element pieces t, t + blockDim, ...
// (V of them) in all of them, so gamma1 gate_col and gamma2 stay in registers, and each row from its
// load, one row ahead, to its outputs: every byte moves once.  16384 x 4096 with y and e4m3 codes (606 MB): 101 us,
// 88% of the copy rate; with dropout and without codes (537 MB) 107 us, 74%: instructions bound it then, 330 a
// piece of eight elements, of which the generator has 120.
template <int V, int FMT>
__global__ void __launch_bounds__(512) join_kernel(const JoinArgs a) {
  __shared__ float s_sum[2][32];
  const int nwarps = blockDim.x >> 5;
  Key key{};
  if (a.drop.rng) key = load_key(a.drop);
  f2 g1[V][4], g2[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    load_factors(a.gamma1, v, a.nvec, g1[j]);
    load_factors(a.gamma2, v, a.nvec, g2[j]);
    if (a.gate_col) {
      f2 c[4];
      load_factors(a.gate_col, v, a.nvec, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) g1[j][e] = mul2(g1[j][e], c[e]);
    }
  }
  const f2 ra = both(a.ra);
  uint4 xn[V], rn[V];  // the next row's pieces (zeros past the row's end)
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      xn[j] = rn[j] = make_uint4(0, 0, 0, 0);
      if (v < a.nvec && row < a.R) {
        xn[j] = a.x[row * a.nvec + v];
        if (a.residual) rn[j] = a.residual[row * a.nvec + v];
      }
    }
  };
  fetch(blockIdx.x);
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const int64_t base = row * a.nvec;
    uint4 xv[V], rv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      xv[j] = xn[j];
      rv[j] = rn[j];
    }
    float k = a.rb * a.drop.inv * (a.gate_row ? __ldg(a.gate_row + row) : 1.0f);
    fetch(row + gridDim.x);  // (h may be x or residual: other rows than the one that is written)
    if (a.gamma1) {
      f2 t = both(0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f2 f[4];
        unpack2(xv[j], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fma2(f[e], f[e], t);
      }
      const float q = block_sum(sum2(t), s_sum[par], nwarps);
      par ^= 1;
      const float rstd1 = rsqrtf(q * a.inv_c + a.eps);
      if (a.rstd1 && threadIdx.x == 0) a.rstd1[row] = rstd1;
      k *= rstd1;
    }
    f2 s[V][4], t2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      f2 t[4], r[4];
      unpack2(xv[j], t);
      unpack2(rv[j], r);
      // (before the mask: a row's NaN does not come into its dropped elements; nor past the row's end)
      const f2 kv = both(v < a.nvec ? k : 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = mul2(t[e], kv);
      if (a.drop.rng) drop8(t, base + v, a.drop, key);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = fma2(ra, r[e], mul2(t[e], g1[j][e]));
        t2 = fma2(s[j][e], s[j][e], t2);
      }
      if (a.h && v < a.nvec) a.h[base + v] = round8(s[j]);
    }
    if (!a.gamma2) continue;
    const float q2 = block_sum(sum2(t2), s_sum[par], nwarps);
    par ^= 1;
    const float rstd2 = rsqrtf(q2 * a.inv_c + a.eps);
    if (a.rstd2 && threadIdx.x == 0) a.rstd2[row] = rstd2;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      // the four lanes of an MX block are in range together: nvec is a multiple of 4 with FMT
      const bool in = v < a.nvec;
      f2 o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = mul2(mul2(s[j][e], both(rstd2)), g2[j][e]);
      if (a.y && in) a.y[base + v] = round8(o);
      if (FMT) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(o[e], y[2 * e], y[2 * e + 1]);
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = max(am, __float_as_uint(y[e]) & 0x7FFFFFFFu);
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        uint32_t sc;
        float mult;
        const bool fin = block_scale_f32<FMT>(am, sc, mult);
        if (in) {
          float c[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] = fin ? y[e] * mult : 0.0f;
          if (FMT == kE4M3) {
            uint2 o;
            o.x = cvt_e4m3x2(c[0], c[1]) | (cvt_e4m3x2(c[2], c[3]) << 16);
            o.y = cvt_e4m3x2(c[4], c[5]) | (cvt_e4m3x2(c[6], c[7]) << 16);
            reinterpret_cast<uint2*>(a.codes)[base + v] = o;
          } else {
            reinterpret_cast<uint32_t*>(a.codes)[base + v] =
                cvt_e2m1x2(c[0], c[1]) | (cvt_e2m1x2(c[2], c[3]) << 8) | (cvt_e2m1x2(c[4], c[5]) << 16) |
                (cvt_e2m1x2(c[6], c[7]) << 24);
          }
          if ((v & 3) == 0) a.scales[(base + v) >> 2] = (uint8_t)sc;
        }
      }
    }
  }
}

struct JoinBwdArgs {
  const uint4* dy;  // or nullptr (no gamma2)
  const uint4* dh;  // or nullptr
  const uint4* x;
  const uint4* h;
  const float* rstd1;
  const float* rstd2;
  const uint4* gamma1;
  const uint4* gamma2;
  const float* gate_row;
  const uint4* gate_col;
  Drop drop;
  int64_t R;
  int nvec;
  float inv_c, ra, rb;
  uint4* dx;
  uint4* dres;       // or nullptr
  float* dgate_row;  // or nullptr
  float* part;       // [3][gridDim.x][C]: the blocks' sums for dgamma1, dgamma2, dgate per column
};

// The same ownership: a thread's columns stay its own over all rows of the block, so the sums over
// rows are registers, written once per block.  A thread copies its pieces of coming rows into its own
// places of shared memory, a step ahead (no thread reads another's).  A step is ROWS rows, of which
// one's arithmetic fills the waits of another's sums.  The longest rows are shared out over CL CTAs.
//
// The chain of a row's steps bounds it before memory does (with dropout 56% of the issue slots taken), so the
// sums over a row are arranged to need one barrier.  With e = dh + rstd2 u, xk = x where it is kept, else 0, and
// gg = gamma1 gate_col (ones where there are none):
//   d = e + c h,  c = -rstd2^3 mean(u h)
//   q = sum gg xk d = sum gg xk e + c sum gg xk h
// and all the gradients of the branch come from q and, over the rows, S = sum gate_row rstd1 xk d.  With
// f = rb / (1 - p):
//   dgamma1 = f gate_col S    dgate_col = f gamma1 S    dgate_row = f rstd1 q
//   dx = f (gg g - x gate_row rstd1^3 q / C),  g = gate_row rstd1 d where it is kept, else 0
// 8192 x 2880 (283 MB, 41.8 us at the copy rate): 52 us, with dropout 67; 16384 x 4096 with
// dropout (805 MB) 150.
template <int V, int ROWS, int CL, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) join_bwd_kernel(const JoinBwdArgs a) {
  extern __shared__ uint4 s_row[];  // [DEPTH][ROWS][4][V][blockDim]
  __shared__ float s_sum[2][4 * ROWS][16 * CL];
  constexpr int DEPTH = 2;
  const int nwarps = blockDim.x >> 5;
  // the row's pieces that this CTA has: all of them, or its share
  const int own = CL == 1 ? a.nvec : (a.nvec + CL - 1) / CL, rank = blockIdx.x % CL, block = blockIdx.x / CL;
  const int v0 = rank * own, v1 = min(a.nvec, v0 + own);
  if (CL > 1) cluster_sync();  // (the other CTAs' shared memory is there)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Key key{};
  if (a.drop.rng) key = load_key(a.drop);
  f2 sum_b[V][4], sum_2[V][4], gg[V][4], g2[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = v0 + threadIdx.x + j * blockDim.x;
    load_factors(a.gamma1, v, v1, gg[j]);
    load_factors(a.gamma2, v, v1, g2[j]);
    if (a.gate_col) {
      f2 c[4];
      load_factors(a.gate_col, v, v1, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) gg[j][e] = mul2(gg[j][e], c[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum_b[j][e] = sum_2[j][e] = both(0.0f);
  }
  constexpr int kRow = 4 * V;
  uint4* mine = s_row + threadIdx.x;  // place i of a row: mine[i * blockDim.x]
  // places that no row is copied to read as zeros: those past the row's end, and of operands that are not given
#pragma unroll
  for (int i = 0; i < DEPTH * ROWS * kRow; ++i) {
    const int which = i % kRow / V, j = i % V;
    const bool given = which == 3 || (which == 2 ? a.dh != nullptr : a.gamma2 != nullptr);
    if (!given || v0 + (int)threadIdx.x + j * (int)blockDim.x >= v1) mine[i * blockDim.x] = make_uint4(0, 0, 0, 0);
  }
  const int64_t grid = gridDim.x / CL;
  auto fetch = [&](int64_t first, int slot) {
    const uint32_t step = blockDim.x * 16;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = first + k * grid;
      const uint32_t dst = smem_u32(mine) + (slot * ROWS + k) * kRow * step;
      if (row < a.R) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int v = v0 + threadIdx.x + j * blockDim.x;
          const int64_t at = row * a.nvec + v;
          if (v < v1) {
            if (a.gamma2) {
              cp_async_16(dst + j * step, a.h + at);
              cp_async_16(dst + (V + j) * step, a.dy + at);
            }
            if (a.dh) cp_async_16(dst + (2 * V + j) * step, a.dh + at);
            cp_async_16(dst + (3 * V + j) * step, a.x + at);
          }
        }
      } else if (k > 0) {  // a last row without its fellows: zeros, which change no sum
#pragma unroll
        for (int i = 0; i < kRow; ++i) mine[((slot * ROWS + k) * kRow + i) * blockDim.x] = make_uint4(0, 0, 0, 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) fetch(block + i * ROWS * grid, i);
  const float f = a.rb * a.drop.inv;
  int par = 0, slot = 0;
  // The rows' three numbers, of the block's next 32 rows one a lane: a load a row, with rows a grid apart,
  // took 7 of 62 us.
  const int lane = threadIdx.x & 31;
  float rstd1_of = 1.0f, rstd2_of = 0.0f, gate_of = 1.0f;
  int nth = 0;
  for (int64_t row = block; row < a.R; row += ROWS * grid, par ^= 1, nth += ROWS) {
    if ((nth & 31) == 0) {
      const int64_t of = row + lane * grid;
      const bool is = of < a.R;
      rstd1_of = is && a.gamma1 ? __ldg(a.rstd1 + of) : 1.0f;
      rstd2_of = is && a.gamma2 ? __ldg(a.rstd2 + of) : 0.0f;
      gate_of = is && a.gate_row ? __ldg(a.gate_row + of) : 1.0f;
    }
    fetch(row + (DEPTH - 1) * ROWS * grid, slot == 0 ? DEPTH - 1 : slot - 1);
    float rstd1[ROWS], rstd2[ROWS], scale[ROWS];
    uint32_t keep[ROWS][V];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      rstd1[k] = __shfl_sync(0xffffffffu, rstd1_of, (nth + k) & 31);
      rstd2[k] = __shfl_sync(0xffffffffu, rstd2_of, (nth + k) & 31);
      scale[k] = __shfl_sync(0xffffffffu, gate_of, (nth + k) & 31) * rstd1[k];
#pragma unroll
      for (int j = 0; j < V; ++j)
        keep[k][j] =
            a.drop.rng ? keep8((row + k * grid) * a.nvec + v0 + threadIdx.x + j * blockDim.x, a.drop, key) : 0xFFu;
    }
    cp_async_wait<DEPTH - 1>();
    const uint4* cur = mine + slot * ROWS * kRow * blockDim.x;  // row k's place i: cur[(k * kRow + i) * blockDim.x]
    f2 e[ROWS][V][4];
    float q[4 * ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      f2 t_uh = both(0.0f), t_xe = t_uh, t_xh = t_uh;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f2 hv[4], dy[4], x[4];
        unpack2(cur[(k * kRow + j) * blockDim.x], hv);
        unpack2(cur[(k * kRow + V + j) * blockDim.x], dy);
        unpack2(cur[(k * kRow + 2 * V + j) * blockDim.x], e[k][j]);
        unpack2(cur[(k * kRow + 3 * V + j) * blockDim.x], x);
        if (a.drop.rng) keep_only(x, keep[k][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 u = mul2(dy[i], g2[j][i]), gx = mul2(x[i], gg[j][i]);
          sum_2[j][i] = fma2(mul2(dy[i], hv[i]), both(rstd2[k]), sum_2[j][i]);
          e[k][j][i] = fma2(u, both(rstd2[k]), e[k][j][i]);
          t_uh = fma2(u, hv[i], t_uh);
          t_xe = fma2(gx, e[k][j][i], t_xe);
          t_xh = fma2(gx, hv[i], t_xh);
        }
      }
      q[k] = sum2(t_uh);
      q[ROWS + k] = sum2(t_xe);
      q[2 * ROWS + k] = sum2(t_xh);
      q[3 * ROWS + k] = 0.0f;
    }
    block_sums<4 * ROWS, CL>(q, s_sum[par], nwarps);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t base = (row + k * grid) * a.nvec + v0 + threadIdx.x;
      const bool is = k == 0 || row + k * grid < a.R;
      const float c = -rstd2[k] * rstd2[k] * (q[k] * rstd2[k] * a.inv_c);
      const float qx = fmaf(c, q[2 * ROWS + k], q[ROWS + k]);
      if (a.dgate_row && threadIdx.x == 0 && rank == 0 && is) a.dgate_row[row + k * grid] = f * rstd1[k] * qx;
      const float m = a.gamma1 ? -rstd1[k] * rstd1[k] * (qx * a.inv_c) * scale[k] : 0.0f;
      // x itself is masked where it is not normed, and of a row whose norm is not finite (rstd NaN or 0)
      const bool mask_x = a.drop.rng && !(a.gamma1 && rstd1[k] > 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = is && v0 + (int)threadIdx.x + j * (int)blockDim.x < v1;
        f2 hv[4], x[4], o[4];
        unpack2(cur[(k * kRow + j) * blockDim.x], hv);
        unpack2(cur[(k * kRow + 3 * V + j) * blockDim.x], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[k][j][i] = fma2(both(c), hv[i], e[k][j][i]);  // d
        if (a.dres && in) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(both(a.ra), e[k][j][i]);
          a.dres[base + j * blockDim.x] = round8(o);
        }
        // scale dk, masked behind the factor: a row's gate or norm does not come into its dropped places
#pragma unroll
        for (int i = 0; i < 4; ++i) e[k][j][i] = mul2(e[k][j][i], both(scale[k]));
        if (a.drop.rng) keep_only(e[k][j], keep[k][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mul2(gg[j][i], e[k][j][i]);
        if (a.gamma1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = fma2(x[i], both(m), o[i]);
        }
        if (mask_x) keep_only(x, keep[k][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum_b[j][i] = fma2(e[k][j][i], x[i], sum_b[j][i]);
          o[i] = mul2(both(f), o[i]);
        }
        if (in) a.dx[base + j * blockDim.x] = round8(o);
      }
    }
    if (++slot == DEPTH) slot = 0;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = v0 + threadIdx.x + j * blockDim.x;
    if (v < v1) {
      const int64_t plane = grid * a.nvec * 2;
      float4* p = reinterpret_cast<float4*>(a.part) + ((int64_t)block * a.nvec + v) * 2;
      auto put = [&](float4* dst, const f2 (&o)[4]) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(o[e], w[2 * e], w[2 * e + 1]);
        dst[0] = make_float4(w[0], w[1], w[2], w[3]);
        dst[1] = make_float4(w[4], w[5], w[6], w[7]);
      };
      f2 fac[4];
      if (a.gamma1) {
        load_factors(a.gate_col, v, v1, fac);
#pragma unroll
        for (int e = 0; e < 4; ++e) fac[e] = mul2(fac[e], mul2(both(f), sum_b[j][e]));
        put(p, fac);
      }
      if (a.gamma2) put(p + plane, sum_2[j]);
      if (a.gate_col) {
        load_factors(a.gamma1, v, v1, fac);
#pragma unroll
        for (int e = 0; e < 4; ++e) fac[e] = mul2(fac[e], mul2(both(f), sum_b[j][e]));
        put(p + 2 * plane, fac);
      }
    }
  }
}

// Columns of the three sums: n partial rows each, added in a fixed order; a block has 32 columns of one of
// them, each warp every 16th row.  It is launched while the kernel above runs and waits for its rows.
struct JoinReduce {
  const float* part;
  int n, C;
  float* out[3];  // of dgamma1, dgamma2, dgate; the first `count` of which[] are wanted
  int which[3];
};
constexpr int kReduceThreads = 512;
__global__ void __launch_bounds__(kReduceThreads) join_reduce_kernel(const JoinReduce a) {
  constexpr int kWarps = kReduceThreads / 32;
  __shared__ float s[kWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int which = a.which[blockIdx.y];
  const float* p = a.part + (int64_t)which * a.n * a.C + c;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float t = 0.0f;
  if (c < a.C) {
#pragma unroll 8
    for (int i = w; i < a.n; i += kWarps) t += p[(int64_t)i * a.C];
  }
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < a.C) {
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) t += s[k][lane];
    a.out[which][c] = t;
  }
}

int threads_of(int nvec, int V) { return std::max(32, ((nvec + V - 1) / V + 31) / 32 * 32); }
int join_v(int nvec) { return nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4; }
int bwd_v(int nvec) { return nvec <= 384 ? 1 : 2; }
// CTAs, a cluster, that share a row: four pieces a thread would not stay in registers (4096 x 16384 with dropout:
// 264 us, two CTAs 186, four 187; without 243, 171, 158; 4096 x 10240 with dropout 197, 141, 125).
int bwd_ctas(int nvec) { return nvec <= 1024 ? 1 : 4; }

// Blocks of the backward pass: at most as many as are resident at once, which this bounds for the
// workspace.
int bwd_blocks(int64_t R, int nvec) {
  const int threads = threads_of(nvec, bwd_v(nvec) * bwd_ctas(nvec));
  return (int)std::min<int64_t>(R, 160 / bwd_ctas(nvec) * std::max(1, std::min(8, 768 / threads)));
}

template <int V>
void launch_join(const JoinArgs& a, int fmt, int grid, int threads, cudaStream_t s) {
  if (fmt == kE4M3) join_kernel<V, kE4M3><<<grid, threads, 0, s>>>(a);
  else if (fmt == kE2M1) join_kernel<V, kE2M1><<<grid, threads, 0, s>>>(a);
  else join_kernel<V, 0><<<grid, threads, 0, s>>>(a);
}

int check(int64_t R, int64_t C, int mult, const void* gate, int gate_kind, const int64_t* rng, double p, float ra,
          float rb) {
  if (R < 0 || R >= ((int64_t)1 << 31) || C < mult || C > PGG_NORM_MAX_COLS) return PGG_ERR_INVALID_ARG;
  if (C % mult) return PGG_ERR_ALIGNMENT;
  if (gate_kind < PGG_GATE_NONE || gate_kind > PGG_GATE_CHANNEL) return PGG_ERR_INVALID_ARG;
  if (!(p >= 0.0 && p < 1.0)) return PGG_ERR_INVALID_ARG;
  const float big = 3.0e38f;
  if (!(ra >= -big && ra <= big) || !(rb >= -big && rb <= big)) return PGG_ERR_INVALID_ARG;
  if (R == 0) return PGG_OK;
  if ((gate_kind != PGG_GATE_NONE) != (gate != nullptr) || (p > 0.0 && !rng)) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(gate, gate_kind == PGG_GATE_TOKEN ? 4 : 16) || !aligned_to(rng, 8)) return PGG_ERR_ALIGNMENT;
  return PGG_OK;
}

Drop make_drop(const int64_t* rng, double p) {
  const uint32_t below = (uint32_t)(p * 4294967296.0);  // p < 1: below 2^32; toward zero
  return {p > 0.0 ? rng : nullptr, below, (float)(1.0 / (1.0 - p))};
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_block_join(const void* x, const void* residual, const void* gamma_post, const void* gamma, const void* gate,
                   int gate_kind, const int64_t* rng, int64_t R, int64_t C, double p, float residual_scale,
                   float branch_scale, float eps, int fmt, void* h, void* y, uint8_t* codes, uint8_t* scales,
                   float* rstd_post, float* rstd, void* stream) {
  if (fmt != 0 && fmt != PGG_FMT_E4M3 && fmt != PGG_FMT_E2M1) return PGG_ERR_INVALID_ARG;
  int st = check(R, C, fmt ? 32 : 8, gate, gate_kind, rng, p, residual_scale, branch_scale);
  if (st) return st;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return PGG_ERR_INVALID_ARG;
  if (R == 0) return PGG_OK;
  if ((fmt != 0) != (codes != nullptr) || (fmt != 0) != (scales != nullptr)) return PGG_ERR_INVALID_ARG;
  if (!x || (!gamma && (y || fmt || rstd)) || (!gamma_post && rstd_post)) return PGG_ERR_INVALID_ARG;
  if (!h && !y && !fmt && !rstd && !rstd_post) return PGG_ERR_INVALID_ARG;
  for (const void* q : {x, residual, gamma_post, gamma, (const void*)h, (const void*)y, (const void*)codes})
    if (!aligned_to(q, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(rstd_post, 4) || !aligned_to(rstd, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  JoinArgs a{static_cast<const uint4*>(x), static_cast<const uint4*>(residual), static_cast<const uint4*>(gamma_post),
             static_cast<const uint4*>(gamma),
             gate_kind == PGG_GATE_TOKEN ? static_cast<const float*>(gate) : nullptr,
             gate_kind == PGG_GATE_CHANNEL ? static_cast<const uint4*>(gate) : nullptr, make_drop(rng, p), R,
             (int)(C / 8), 1.0f / (float)C, eps, residual_scale, branch_scale, static_cast<uint4*>(h),
             static_cast<uint4*>(y), codes, scales, rstd_post, rstd};
  const int V = join_v(a.nvec), threads = threads_of(a.nvec, V);
  const int grid = (int)std::min<int64_t>(R, (int64_t)dev.sms * std::max(1, 2048 / threads));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (V == 1) launch_join<1>(a, fmt, grid, threads, s);
  else if (V == 2) launch_join<2>(a, fmt, grid, threads, s);
  else launch_join<4>(a, fmt, grid, threads, s);
  return cuda_status(cudaGetLastError());
}

int pgg_block_join_bwd_workspace_size(int64_t R, int64_t C, size_t* bytes) {
  const int st = check(R, C, 8, nullptr, 0, nullptr, 0.0, 1.0f, 1.0f);
  if (st) return st;
  if (!bytes) return PGG_ERR_INVALID_ARG;
  *bytes = (size_t)bwd_blocks(R, (int)(C / 8)) * 3 * (size_t)C * sizeof(float);
  return PGG_OK;
}

int pgg_block_join_bwd(const void* dy, const void* dh, const void* x, const void* h, const float* rstd_post,
                       const float* rstd, const void* gamma_post, const void* gamma, const void* gate, int gate_kind,
                       const int64_t* rng, int64_t R, int64_t C, double p, float residual_scale, float branch_scale,
                       void* dx, void* dresidual, float* dgamma_post, float* dgamma, float* dgate, void* ws,
                       size_t ws_bytes, void* stream) {
  int st = check(R, C, 8, gate, gate_kind, rng, p, residual_scale, branch_scale);
  if (st) return st;
  // R == 0 has no gamma to tell by: the sums that are asked for are zero
  if (R > 0 && ((gamma_post != nullptr) != (dgamma_post != nullptr) || (gamma != nullptr) != (dgamma != nullptr) ||
                (gate_kind != PGG_GATE_NONE) != (dgate != nullptr)))
    return PGG_ERR_INVALID_ARG;
  const bool col = gate_kind == PGG_GATE_CHANNEL;
  if (!aligned_to(dgamma_post, 4) || !aligned_to(dgamma, 4) || !aligned_to(dgate, 4)) return PGG_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) {
    for (float* q : {dgamma_post, dgamma, col ? dgate : nullptr})
      if (q && (st = cuda_status(cudaMemsetAsync(q, 0, (size_t)C * sizeof(float), s)))) return st;
    return PGG_OK;
  }
  if (!x || !dx || !ws || (gamma_post && !rstd_post) || (gamma && (!dy || !h || !rstd))) return PGG_ERR_INVALID_ARG;
  if (!gamma && dy) return PGG_ERR_INVALID_ARG;
  size_t need = 0;
  if ((st = pgg_block_join_bwd_workspace_size(R, C, &need))) return st;
  if (ws_bytes < need) return PGG_ERR_INVALID_ARG;
  for (const void* q : {dy, dh, x, h, gamma_post, gamma, (const void*)dx, (const void*)dresidual, (const void*)ws})
    if (!aligned_to(q, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(rstd_post, 4) || !aligned_to(rstd, 4)) return PGG_ERR_ALIGNMENT;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != PGG_OK) return st;
  const int nvec = (int)(C / 8), V = bwd_v(nvec), ctas = bwd_ctas(nvec);
  const int threads = threads_of((nvec + ctas - 1) / ctas, V);
  JoinBwdArgs a{static_cast<const uint4*>(dy), static_cast<const uint4*>(dh), static_cast<const uint4*>(x),
                static_cast<const uint4*>(h), rstd_post, rstd, static_cast<const uint4*>(gamma_post),
                static_cast<const uint4*>(gamma),
                gate_kind == PGG_GATE_TOKEN ? static_cast<const float*>(gate) : nullptr,
                col ? static_cast<const uint4*>(gate) : nullptr, make_drop(rng, p), R, nvec, 1.0f / (float)C,
                residual_scale, branch_scale, static_cast<uint4*>(dx), static_cast<uint4*>(dresidual),
                col ? nullptr : dgate, static_cast<float*>(ws)};
  // Up to 384 threads two rows at a time, on one block an SM of more registers (8192 x 2880, without dropout 52.1
  // us and with 65.8 when it was chosen, 52.3 and 66.9 now; one row 53.4 and 69, with two blocks an SM 54.5 and
  // 71.8; four rows 52.8 and 69.2).
  auto kern = V == 1      ? join_bwd_kernel<1, 2, 1, 384>
              : ctas == 1 ? join_bwd_kernel<2, 1, 1, 512>
                          : join_bwd_kernel<2, 1, 4, 512>;
  const size_t place = 16 * sizeof(uint4);  // a thread's shared memory: 16 pieces with each of the three
  const size_t smem = place * threads;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(place * 512));
  cudaLaunchConfig_t run{};
  run.blockDim = dim3((unsigned)threads);
  run.dynamicSmemBytes = smem;
  run.stream = s;
  cudaLaunchAttribute pair{};
  pair.id = cudaLaunchAttributeClusterDimension;
  pair.val.clusterDim.x = (unsigned)ctas;
  pair.val.clusterDim.y = pair.val.clusterDim.z = 1;
  run.attrs = &pair;
  run.numAttrs = ctas > 1 ? 1 : 0;
  // blocks, or clusters of them, that run at one time
  static std::atomic<int> resident[3][5][17];
  std::atomic<int>& known = resident[V][ctas][threads / 32];
  int most = known.load(std::memory_order_relaxed);
  if (e == cudaSuccess && most == 0) {
    run.gridDim = dim3((unsigned)(dev.sms * ctas));
    e = ctas == 1 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&most, kern, threads, smem)
                  : cudaOccupancyMaxActiveClusters(&most, kern, &run);
    most = std::max(1, ctas == 1 ? most * dev.sms : most);
    if (e == cudaSuccess) known.store(most, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return cuda_status(e);
  const int grid = std::min(bwd_blocks(R, nvec), most);
  run.gridDim = dim3((unsigned)(grid * ctas));
  e = cudaLaunchKernelEx(&run, kern, a);
  if ((st = cuda_status(e != cudaSuccess ? e : cudaGetLastError()))) return st;
  JoinReduce r{a.part, grid, (int)C, {dgamma_post, dgamma, col ? dgate : nullptr}, {0, 0, 0}};
  int sums = 0;
  for (int i = 0; i < 3; ++i)
    if (r.out[i]) r.which[sums++] = i;
  if (!sums) return PGG_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((C + 31) / 32), (unsigned)sums);
  cfg.blockDim = dim3(kReduceThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, join_reduce_kernel, r);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // extern "C"

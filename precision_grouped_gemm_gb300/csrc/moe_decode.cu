// A whole expert layer for a few tokens, in one kernel of two phases:
//
//   phase 1   A[r] = silu(g) u, [g; u] = W1_e x_t     every (expert, token) pair r of the batch
//   phase 2   out[t] = sum over t's experts e of w_te W2_e A[r]
//
// with W1 [E, 2I, H] (gate | up) and W2 [E, H, I] in bf16, or in MX codes with blocked scales
// (then x comes as MX codes and A is quantised to MX codes from fp32).
//
// With a few tokens per expert the weights of the experts that the batch names are read once and
// everything else is small: the kernels are weight streams.  Weights are the MMA's A operand
// (128 output rows a tile, loaded by TMA), the expert's tokens its B operand (N = tokens rounded
// up to 16), so a tile is multiplied as it lands in shared memory and no weight passes through a
// register.  The stages of all tiles of a phase form one sequence that is cut into equal runs,
// one per CTA, so every SM reads the same number of bytes whatever the routing; a tile that a cut
// divides is put together from fp32 partial sums in CTA order: in phase 1 by the CTA that begins it,
// in phase 2 by all of its CTAs, a share of the tokens each (a cooperative launch: every CTA is
// resident, and none waits before the sums that others wait for are out).
//
// Between the phases only the warps that fetch A wait for the other CTAs; the weight loads run on
// into phase 2 and keep the ring full.
//
// Every CTA builds the batch's expert list by itself from the ids: a bit per (expert, token), so
// an expert named twice by a token is computed once and its weights are added up.
//
// What bounds it: the weight stream where there is much of it.  The named experts' bytes at the plain
// copy rate, and the call's time: BF16, 32 tokens, 32 experts of 2880 x 2880: 219 us, 235 (93%);
// MXFP8, 8 tokens of 256 experts, 4096 x 2048: 172, 179 (96%; tensor pipe 4% busy); MXFP4, 64 skewed
// tokens: 255, 280 (91%: the CTAs with the hottest expert's activations are last).  Where there is
// little, the steps that are not streams: ~2 us to the first load, ~4 us from the last activation to
// the first product of phase 2 (partial sums, the count of CTAs, the fetch of A), ~1.5 us for the last
// sums.  One token, six BF16 experts: 44.6, 56; one token, eight MXFP4 experts: 15.8, 28.6.  At that
// size instruction fetch shows too: loops are not unrolled and the phases share their code.  (Comments on
// single steps give before and after on one machine each, some of them 2% faster.)
#include <algorithm>
#include <type_traits>

#include "block.cuh"
#include "epilogue.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kMaxT = PGG_MOE_DECODE_MAX_T;
constexpr int kMaxCtas = 160;   // CTAs of a launch (one per SM); sizes the workspace without a device
constexpr int kMaxStages = 8;
constexpr int kLoadWarps = 4;   // warps that fetch the token operand
constexpr int kBatch = 4;      // tokens that phase 2's epilogue works on at a time
constexpr int kFixedBytes = 768;  // barriers, plans
constexpr int kTileBytes = 128 * 128;  // 128 rows x one 128-byte swizzle atom of K

template <int FMT>
struct DecCfg {
  static constexpr int kBK = FMT == 0 ? 64 : FMT == kE4M3 ? 128 : 256;  // elements in 128 bytes
  static constexpr int kSub = FMT == 0 ? 0 : kBK / 128;                  // scale atoms of them
  static constexpr int kPerMma = kBK / 4;
  static constexpr int kCopier = FMT != 0;
  static constexpr int kThreads = 32 * (6 + kCopier + kLoadWarps);
};

// One matrix of a layer and what its phase reads.  Both matrices are seen as [E][halves][rows][red]
// (W1: gate and up halves; W2: one), so that the two phases run the same code.
struct DecodePhase {
  int rows;            // output rows of a half: I (phase 1), H (phase 2)
  int halves;          // 2 (phase 1), 1 (phase 2)
  int red;             // reduction length: H (phase 1), I (phase 2)
  int tiles, pieces;   // 128-row tiles of `rows`, 128-byte pieces of `red`
  FastDiv by_nk[2];    // by a tile's stages, with one and with two K pieces a stage
  const uint8_t* b;    // token operand, row-major: X (phase 1) or A (phase 2)
  int64_t b_ld;        // bytes of a row
  const uint8_t* sb;   // its scales, row-major, red / 32 bytes a row
  const uint8_t* sa;   // the weights' blocked scales
};

struct DecodeArgs {
  const int32_t* ids;  // [T, k]
  const float* w;      // [T, k] or nullptr
  int T, k, E, I;
  float limit;
  DecodePhase ph[2];
  uint8_t* act;         // A: bf16 (high part), or codes
  uint8_t* act_lo;      // bf16: what the rounding to the high part left over
  uint8_t* act_scales;  // MX: row-major scales
  __nv_bfloat16* out;   // [T, H]
  float* part[2];       // per phase and CTA: a tile of partial sums, zero between launches
  unsigned* done;       // CTAs that have finished phase 1; [1]: that have left.  Zero between launches.
                        // [2]: a launch gave up, so the sums in `part` are not to be trusted
  int ring_bytes;       // shared memory for the stages
  int slots_cap;        // most experts that the batch can name
  FastDiv by_grid;
  unsigned long long wait_ns;  // limit of every wait
  long long stall_at;          // test hook: the producer stops before this stage of its run (-1: never)
  int32_t* err;
};

// Four accumulator columns of this thread's row; the values are there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t (&r)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, float4 v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(__float_as_uint(v.x)),
               "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w))
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float as_float(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, uint32_t src_bytes) {  // 0 bytes: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t accum) {
  if (FMT == 0) mma_f16(d, ad, bd, idesc, accum);
  else if (FMT == kE4M3) mma_mxf8(d, ad, bd, idesc, sfa, sfb, accum);
  else mma_mxf4(d, ad, bd, idesc, sfa, sfb, accum);
}
// Warp 0 has laid out the work (`start_arrive`) and goes on to the first loads; the other roles wait
// for that (`start_wait`).  N: the block's threads.
template <int N>
__device__ __forceinline__ void start_arrive() { asm volatile("barrier.cta.arrive 3, %0;" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void start_wait() { asm volatile("barrier.cta.sync 3, %0;" ::"n"(N) : "memory"); }
// The other warps have read the list's scratch in the ring for the last time; warp 0 may load over it.
template <int N>
__device__ __forceinline__ void scratch_arrive() { asm volatile("barrier.cta.arrive 4, %0;" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void scratch_wait() { asm volatile("barrier.cta.sync 4, %0;" ::"n"(N) : "memory"); }

// Partial sums travel without flags or fences: a word that is not zero is a sum.  (A release under a
// full load of weight reads took 2 to 5 us on this path.)  A zero sum is sent as -0, which adds the
// same; the reader puts the zero back.
__device__ __forceinline__ float sent(float v) { return __float_as_uint(v) == 0u ? __uint_as_float(0x80000000u) : v; }
__device__ __forceinline__ float4 load_relaxed4(const float4* p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_relaxed4(float4* p, float4 v) {
  asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
// Barrier `ID` of 128 threads (the epilogue warps, the token-loading warps) that tells each whether
// `ok` held in all of them: they give up together, so that none is left at a later barrier.
template <int ID = 1>
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(ID)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// How a launch cuts up its work: computed by one warp of each CTA (the same in all of them).
struct Shape {  // what both phases share: the ring's stages and tensor memory
  int n_act;    // experts that the batch names
  int ncols;    // most tokens of one of them, rounded up to 16
  int ns;       // phase 2: K pieces per stage
  int stages, stage_bytes;
  int acc_cols, nacc, sf_col0, sf_per;
};
struct Plan {  // one phase
  int np;       // weight pieces of a stage: gate and up (phase 1), ns K pieces (phase 2)
  int nb;       // token pieces of a stage
  int nk;       // stages of one (expert, tile)
  int L;        // stages of one item: an (expert, tile) in phase 1, an output tile in phase 2
  int quot, rem;  // total stages = ctas quot + rem: the first rem CTAs get a stage more
  int b_off, b_piece, sf_off;  // layout of a stage: weights, token pieces, scale atoms
  int p, p1;    // this CTA's run of stages, and where it starts:
  int slot, tile, kb;
  // the CTA that stage p belongs to
  __device__ __forceinline__ int owner(int p) const {
    const int big = rem * (quot + 1);
    return p < big ? p / (quot + 1) : rem + (p - big) / quot;
  }
  // The stages of the run's next segment: those of one (expert, tile).
  __device__ __forceinline__ int length() const { return min(nk - kb, p1 - p); }
  __device__ __forceinline__ void step(int n_act) {
    p += length();
    kb = 0;
    if (++slot == n_act) {
      slot = 0;
      ++tile;
    }
  }
};

// Columns (rows of the token operand) of n tokens in phase 2: bf16 keeps the high and the low parts
// of A next to each other, each rounded up to the 8 rows of a swizzle atom.
template <int FMT>
__device__ __forceinline__ int cols2(int n) {
  return FMT == 0 ? (2 * ((n + 7) & ~7) + 15) & ~15 : (n + 15) & ~15;
}

// a / b for 0 <= a < 2^20, b > 0: (a + 1/2) / b is at least 2^-21 of itself away from a whole number,
// the fast division within 2^-22 of the quotient.
__device__ __forceinline__ int div_small(int a, int b) { return (int)__fdividef((float)a + 0.5f, (float)b); }

template <int FMT>
__device__ __forceinline__ void make_plan(const DecodeArgs& a, int n_act, int max_n, int ph, Shape& S, Plan& P) {
  using C = DecCfg<FMT>;
  S.n_act = n_act;
  S.ncols = (max_n + 15) & ~15;
  const int b1 = S.ncols * 128, b2 = cols2<FMT>(max_n) * 128;
  const int s1 = 2 * kTileBytes + b1 + C::kSub * 3 * 512;
  const int two = 2 * (kTileBytes + b2 + C::kSub * 1024), one = kTileBytes + b2 + C::kSub * 1024;
  // phase 2: two K pieces a stage, or one where many tokens would leave fewer than three stages
  const int st1 = (max(s1, one) + 1023) >> 10, st2 = (max(s1, two) + 1023) >> 10;
  const int n1 = div_small(a.ring_bytes >> 10, st1), n2 = div_small(a.ring_bytes >> 10, st2);
  S.ns = n2 >= min(3, n1) ? 2 : 1;
  S.stage_bytes = (S.ns == 2 ? st2 : st1) << 10;
  S.stages = min(kMaxStages, S.ns == 2 ? n2 : n1);
  S.acc_cols = max(2 * S.ncols, b2 / 128);
  S.sf_per = C::kSub * max(12, S.ns * 8);
  S.nacc = 2 * S.acc_cols + S.stages * S.sf_per <= 512 ? 2 : 1;
  S.sf_col0 = S.nacc * S.acc_cols;

  const int pieces = a.ph[ph].pieces, tiles = a.ph[ph].tiles;
  P.np = ph == 0 ? 2 : S.ns;
  P.nb = ph == 0 ? 1 : S.ns;
  P.nk = P.nb == 2 ? (pieces + 1) >> 1 : pieces;
  P.b_off = P.np * kTileBytes;
  P.b_piece = ph == 0 ? b1 : b2;
  P.sf_off = P.b_off + P.nb * P.b_piece;
  P.L = ph == 0 ? P.nk : n_act * P.nk;
  const int total = n_act * tiles * P.nk, grid = gridDim.x, cta = blockIdx.x;
  const int ctas = min(grid, total);  // CTAs that get any
  P.quot = total < grid ? 1 : (int)a.by_grid.div(total);
  P.rem = total < grid ? 0 : total - grid * P.quot;
  P.p = cta < ctas ? cta * P.quot + min(cta, P.rem) : 0;
  P.p1 = cta < ctas ? P.p + P.quot + (cta < P.rem) : 0;
  const int unit = (int)a.ph[ph].by_nk[P.nb - 1].div(P.p);  // (expert, tile) number
  P.kb = P.p - unit * P.nk;
  // Experts change from one (expert, tile) to the next, so that the tiles of an expert with many tokens,
  // which take longer, are spread over the CTAs.  (Expert after expert in phase 1: 64 skewed tokens,
  // MXFP8 78.8 us instead of 77.1, MXFP4 276.6 instead of 275.4; BF16 32 tokens 230.1 instead of 228.8.)
  P.tile = div_small(unit, max(n_act, 1));
  P.slot = unit - P.tile * n_act;
}

template <int FMT>
__global__ void __launch_bounds__(DecCfg<FMT>::kThreads, 1)
    moe_decode_kernel(const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmW2,
                      const __grid_constant__ DecodeArgs a) {
  using C = DecCfg<FMT>;
  constexpr int kNT = C::kThreads;
  constexpr int kLoadWarp0 = 6 + C::kCopier;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.ring_bytes);
  uint64_t* full = bars;
  uint64_t* empty = full + kMaxStages;
  uint64_t* sfull = empty + kMaxStages;  // a stage's scales are in tensor memory
  uint64_t* tfull = sfull + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* cdrain = drain + 1;
  volatile WaitCtl* s_ctl = reinterpret_cast<volatile WaitCtl*>(cdrain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<WaitCtl*>(s_ctl) + 1);
  int* s_last_tile = reinterpret_cast<int*>(s_tmem + 1);  // the last output tile of this CTA's run
  int* s_scan = s_last_tile + 1;  // [2 * 16]
  Shape* s_shape = reinterpret_cast<Shape*>(s_scan + 32);
  Plan* s_plan = reinterpret_cast<Plan*>(s_shape + 1);  // [2]
  float* s_acc = reinterpret_cast<float*>(smem + a.ring_bytes + kFixedBytes);  // phase 2: [T][128]
  float* s_w = s_acc + a.T * 128;                                       // [T k]
  uint16_t* s_off = reinterpret_cast<uint16_t*>(s_w + a.T * a.k);       // [slots + 1]: an expert's first entry
  uint16_t* s_exp = s_off + a.slots_cap + 1;                            // [slots]
  uint8_t* s_tok = reinterpret_cast<uint8_t*>(s_exp + a.slots_cap);     // [T k]: the entries' tokens

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the batch's experts and their tokens.  Scratch: the place of phase 2's sums; where that is too
  // small (many experts, few tokens), the ring, before the first stage lands.
  const int W = (a.T + 31) / 32;  // mask words per expert
  const bool in_ring = a.E * (4 * W + 2) + a.T * a.k * 6 > a.T * 512;
  uint32_t* s_mask = in_ring ? reinterpret_cast<uint32_t*>(smem) : reinterpret_cast<uint32_t*>(s_acc);  // [E][W]
  float* s_wid = reinterpret_cast<float*>(s_mask + a.E * W);          // [T k]: the weights as given
  int16_t* s_id = reinterpret_cast<int16_t*>(s_wid + a.T * a.k);      // [T k]: the ids, -1 out of range
  uint16_t* s_eoff = reinterpret_cast<uint16_t*>(s_id + a.T * a.k);   // [E]: first entry
  const int n_ids = a.T * a.k;
  // Up to 32 ids: warp 0 works the list out in registers (lane i has id i), with the slots in the order
  // of first mention, and starts loading weights while the other warps are still coming up.
  const bool few = n_ids <= 32;
  int id = -1;
  float wid = 0.0f;
  if (few && warp == 0 && lane < n_ids) {  // (their latency passes while the barriers are set up)
    id = __ldg(a.ids + lane);
    wid = a.w ? __ldg(a.w + lane) : 1.0f;
  }
  if (!few) {
#pragma unroll 1
    for (int i = threadIdx.x; i < n_ids; i += kNT) {
      const int e = __ldg(a.ids + i);
      const bool ok = e >= 0 && e < a.E;
      if (!ok && blockIdx.x == 0) set_error(a.err, kErrBadExpert);
      s_id[i] = (int16_t)(ok ? e : -1);
      s_wid[i] = a.w ? __ldg(a.w + i) : 1.0f;
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < a.E * W; i += kNT) s_mask[i] = 0;
  }
  if (warp == 0) {
    if (lane < kMaxStages) {
      mbar_init(smem_u32(&full[lane]), 1 + 32 * kLoadWarps);
      mbar_init(smem_u32(&empty[lane]), 1);
      mbar_init(smem_u32(&sfull[lane]), 1);
    } else if (lane < kMaxStages + 2) {
      mbar_init(smem_u32(&tfull[lane - kMaxStages]), 1);
      mbar_init(smem_u32(&tempty[lane - kMaxStages]), 128);
    } else if (lane == kMaxStages + 2) {
      mbar_init(smem_u32(drain), 1);
      mbar_init(smem_u32(cdrain), 1);
      s_ctl->abort = 0;
      s_ctl->limit_ns = a.wait_ns;
      prefetch_tmap(&tmW1);
      prefetch_tmap(&tmW2);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  int n_act = 0, max_n = 0;
  if (few && warp == 0) {
    const int tok = lane < n_ids ? div_small(lane, a.k) : 0;
    if (lane < n_ids && (id < 0 || id >= a.E)) {
      if (blockIdx.x == 0) set_error(a.err, kErrBadExpert);
      id = -1;
    }
    const unsigned all = 0xffffffffu, below = (1u << lane) - 1u;
    const unsigned same = __match_any_sync(all, id), pair = __match_any_sync(all, id * kMaxT + tok);
    const bool entry = id >= 0 && (pair & below) == 0;  // the token's first choice of this expert
    const unsigned entries = __ballot_sync(all, entry), slots = __ballot_sync(all, id >= 0 && (same & below) == 0);
    n_act = __popc(slots);
    const int head = __ffs(same) - 1;  // the lane that mentions the expert first
    const int n = id >= 0 ? __popc(same & entries) : 0;
    max_n = __reduce_max_sync(all, n);
    const int mine = id >= 0 && lane == head ? n : 0;  // counted once, at the first mention
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(all, inc, d);
      if (lane >= d) inc += o;
    }
    if (mine) {
      const int slot = __popc(slots & below);
      s_exp[slot] = (uint16_t)id;
      s_off[slot + 1] = (uint16_t)inc;
    }
    if (lane == 0) s_off[0] = 0;
    const int first = __shfl_sync(all, inc - mine, head);
    float wt = 0.0f;  // the weights of all of the token's choices of this expert
#pragma unroll 1
    for (int i = 0; i < n_ids; ++i) {
      const float o = __shfl_sync(all, wid, i);
      if (pair >> i & 1) wt += o;
    }
    if (entry) {
      const int r = first + __popc(same & entries & below);
      s_tok[r] = (uint8_t)tok;
      s_w[r] = wt;
    }
  } else if (!few) {
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < n_ids; i += kNT) {
      const int t = i / a.k;
      if (s_id[i] >= 0) atomicOr(&s_mask[s_id[i] * W + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    {
      const int per = (a.E + kNT - 1) / kNT;
      const int lo = min((int)threadIdx.x * per, a.E), hi = min(lo + per, a.E);
      int v = 0, mx = 0;  // experts << 16 | tokens
#pragma unroll 1
      for (int e = lo; e < hi; ++e) {
        int n = 0;
#pragma unroll 1
        for (int q = 0; q < W; ++q) n += __popc(s_mask[e * W + q]);
        if (n) v += (1 << 16) + n;
        mx = max(mx, n);
      }
      int inc = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 31) {
        s_scan[warp] = inc;
        s_scan[16 + warp] = mx;
      }
      __syncthreads();
      int run = inc - v, all = 0;
      max_n = 0;
#pragma unroll 1
      for (int q = 0; q < kNT / 32; ++q) {
        if (q < warp) run += s_scan[q];
        all += s_scan[q];
        max_n = max(max_n, s_scan[16 + q]);
      }
      n_act = all >> 16;
      if (threadIdx.x == 0) s_off[n_act] = (uint16_t)(all & 0xFFFF);
#pragma unroll 1
      for (int e = lo; e < hi; ++e) {
        int n = 0;
#pragma unroll 1
        for (int q = 0; q < W; ++q) n += __popc(s_mask[e * W + q]);
        if (!n) continue;
        s_exp[run >> 16] = (uint16_t)e;
        s_off[run >> 16] = s_eoff[e] = (uint16_t)(run & 0xFFFF);
        run += (1 << 16) + n;
      }
    }
    __syncthreads();
  }
  // Warp 0 knows enough for the first weights; the others write the experts' entries meanwhile.
  if (warp == 0) {
    if (lane < 2) {
      Shape S;
      Plan P{};
      make_plan<FMT>(a, n_act, max_n, lane, S, P);
      s_plan[lane] = P;
      if (lane == 0) *s_shape = S;
    }
    __syncwarp();
    if (!few && in_ring) {
      scratch_wait<kNT>();
      fence_proxy_async_smem();
    }
  } else if (!few) {
#pragma unroll 1
    for (int i = threadIdx.x - 32; i < n_ids; i += kNT - 32) {
      const int e = s_id[i];
      if (e < 0) continue;
      const int t = i / a.k, i0 = t * a.k;
      bool first = true;  // the token's first choice of this expert writes the entry
#pragma unroll 1
      for (int j = i0; j < i; ++j) first &= s_id[j] != e;
      if (!first) continue;
      int r = s_eoff[e];
#pragma unroll 1
      for (int q = 0; q < (t >> 5); ++q) r += __popc(s_mask[e * W + q]);
      r += __popc(s_mask[e * W + (t >> 5)] & ((1u << (t & 31)) - 1u));
      s_tok[r] = (uint8_t)t;
      float wt = 0.0f;
#pragma unroll 1
      for (int j = i; j < i0 + a.k; ++j)
        if (s_id[j] == e) wt += s_wid[j];
      s_w[r] = wt;
    }
    if (in_ring) {
      fence_proxy_async_smem();
      scratch_arrive<kNT>();
    }
  }

  const int cta = blockIdx.x;
  const uint32_t smem0 = smem_u32(smem);
  bool aborted = false;
  int stage = 0;
  uint32_t phase = 0;

  tc_fence_before();
  if (warp == 0) start_arrive<kNT>();
  else start_wait<kNT>();
  tc_fence_after();
  const Shape H = *s_shape;
  const uint32_t tmem_base = *s_tmem;
  auto advance = [&]() {
    if (++stage == H.stages) { stage = 0; phase ^= 1u; }
  };
  if (H.n_act == 0)  // no expert is named: the layer's output is zero
    for (int64_t i = (int64_t)cta * kNT + threadIdx.x; i < (int64_t)a.T * a.ph[1].rows; i += (int64_t)gridDim.x * kNT)
      a.out[i] = __float2bfloat16_rn(0.0f);

  // Wait for another CTA's sums: repeats `load`, which says whether all of its words are there, and
  // raises the abort flag when that takes too long.
  auto until = [&](auto load) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; !load(); ++i) {
      if (i & 63u) continue;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (s_ctl->abort || t - t0 > s_ctl->limit_ns) {
        s_ctl->abort = 1;
        break;
      }
    }
    __syncwarp();
  };
  auto there = [](const float4& v) {
    return __float_as_uint(v.x) != 0u && __float_as_uint(v.y) != 0u && __float_as_uint(v.z) != 0u &&
           __float_as_uint(v.w) != 0u;
  };
  const float4 zero4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

  // This CTA's sums of output tile `tile`, of which its run has reached the end or its own: stored, or
  // sent.  Warp w of n takes a token at a time, a lane four rows of it.
  auto flush = [&](int tile, int w, int n) {
    const Plan& Q = s_plan[1];
    const int item0 = tile * Q.L, r4 = tile * 128 + 4 * lane, rows = a.ph[1].rows;
    const bool begins = Q.p <= item0, whole = begins && Q.p1 >= item0 + Q.L;
    float4* part = reinterpret_cast<float4*>(a.part[1]) + (int64_t)(cta * 2 + begins) * kMaxT * 32 + lane;
    for (int t = w; t < a.T; t += n) {
      const float4 v = reinterpret_cast<float4*>(s_acc)[t * 32 + lane];
      if (!whole)
        store_relaxed4(part + t * 32, make_float4(sent(v.x), sent(v.y), sent(v.z), sent(v.w)));
      else if (r4 < rows)  // rows is a multiple of 8
        *reinterpret_cast<uint2*>(a.out + (int64_t)t * rows + r4) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ weights: TMA tiles, bulk scale atoms
    // The producer runs into phase 2 without waiting: its weights do not depend on phase 1.
    long long issued = 0;
    bool stalled = false;
#pragma unroll 1
    for (int ph = 0; ph < 2 && !stalled; ++ph) {
      const DecodePhase& F = a.ph[ph];
      const CUtensorMap* map = ph == 0 ? &tmW1 : &tmW2;
      const int natom = F.red >> 7;  // MX: scale atoms of a 128-row block along K
      for (Plan P = s_plan[ph]; P.p < P.p1 && !aborted && !stalled; P.step(H.n_act)) {
        const int e = s_exp[P.slot], row0 = P.tile * 128;
        for (int kb = P.kb, end = P.kb + P.length(); kb < end; ++kb) {
          if (issued == a.stall_at) { stalled = true; break; }
          if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          if (lane == 0) {
            const uint32_t fb = smem_u32(&full[stage]);
            const uint32_t st = smem0 + stage * H.stage_bytes;
            const int kk0 = kb * P.nb;
            // K pieces that exist, and (MX) their scale atoms
            const int n = P.nb == 2 && kk0 + 1 < F.pieces ? 2 : 1, nt = ph == 0 ? 2 : n;
            const int nat = C::kSub ? min(C::kSub * n, natom - kk0 * C::kSub) * F.halves : 0;
            mbar_arrive_expect_tx(fb, nt * kTileBytes + 512 * nat);
#pragma unroll 1
            for (int s = 0; s < nt; ++s) {
              const int half = ph == 0 ? s : 0, kk = ph == 0 ? kk0 : kk0 + s;
              tma_load_4d(st + s * kTileBytes, map, fb, kk * (FMT == 0 ? 64 : 128), row0, half, e);
              if (C::kSub) {
                const int64_t rb = (((int64_t)e * F.halves + half) * F.rows + row0) >> 7;
                bulk_load(st + P.sf_off + s * C::kSub * 512, F.sa + (rb * natom + kk * C::kSub) * 512,
                          512 * min(C::kSub, natom - kk * C::kSub), fb);
              }
            }
          }
          __syncwarp();
          ++issued;
          advance();
        }
      }
    }
    if (aborted && lane == 0) {
      // drain: the copies in flight land before the CTA's shared memory goes away.  Their full
      // barriers may lack the token loaders' arrivals, so this may run to its own limit.
      const long long n = issued < H.stages ? issued : H.stages;
      for (long long i = 0; i < n; ++i) {
        if (--stage < 0) { stage = H.stages - 1; phase ^= 1u; }
        mbar_wait_drain(smem_u32(&full[stage]), phase);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int acc = 0;
    uint32_t acc_phase = 0;
#pragma unroll 1
    for (int ph = 0; ph < 2; ++ph) {
      const int red = a.ph[ph].red;
      Plan P = s_plan[ph];
      // descriptors of stage 0's tiles; an address d bytes further on adds d / 16
      const uint64_t desc_a = smem_desc(smem0, 16, 1024, kSwizzle128B);
      const uint64_t desc_b = smem_desc(smem0 + P.b_off, 16, 1024, kSwizzle128B);
      // from a stage's first piece to its second: phase 1 has the up half's accumulator and the same
      // tokens, phase 2 the same accumulator and the next K piece's tokens
      const uint32_t d_step = ph == 0 ? H.ncols : 0, b_step = ph == 0 ? 0 : P.b_piece >> 4;
      const uint32_t sfb0 = P.np * C::kSub * 4, sfb_step = ph == 0 ? 0 : C::kSub * 4;
      while (P.p < P.p1 && !aborted) {
        const int n = s_off[P.slot + 1] - s_off[P.slot];
        const uint32_t N = ph == 0 ? (n + 15) & ~15 : cols2<FMT>(n);
        const uint32_t idesc = FMT == 0 ? idesc_bf16(128, N, false, false) : idesc_mx(FMT == kE4M3 ? 0 : 1, 128, N);
        if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * H.acc_cols;
        const int end = P.kb + P.length();
        for (int kb = P.kb; kb < end; ++kb) {
          if (!warp_wait(smem_u32(C::kCopier ? &sfull[stage] : &full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          if (!C::kCopier) fence_proxy_async_smem();  // the token operand's cp.async writes
          if (lane == 0) {
            const uint64_t so = (uint64_t)(stage * H.stage_bytes) >> 4;
            uint64_t ad = desc_a + so, bd = desc_b + so;
            uint32_t dd = d, sfa = tmem_base + H.sf_col0 + stage * H.sf_per, sfb = sfa + sfb0;
            // reduction elements left from this piece on: MMAs past them (an e2m1 K may end inside a
            // piece) and pieces past them are skipped; the zero-filled end of a bf16 K adds nothing
            int left = red - kb * P.nb * C::kBK;
            uint32_t accum = kb > P.kb;
#pragma unroll 1
            for (int s = 0; s < P.np; ++s) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j * C::kPerMma >= left) break;
                // the scale bytes of an MMA's K range: e4m3 block j of its atom, e2m1 a pair of blocks
                const uint32_t id = FMT == kE4M3 ? j : 2 * (j & 1), at = FMT == kE2M1 ? 4 * (j >> 1) : 0;
                mma<FMT>(dd, ad + 2 * j, bd + 2 * j, FMT == 0 ? idesc : idesc | idesc_sf_ids(id, id), sfa + at,
                         sfb + at, j == 0 ? accum : 1u);
              }
              ad += kTileBytes >> 4;
              bd += b_step;
              dd += d_step;
              sfa += C::kSub * 4;
              sfb += sfb_step;
              if (ph != 0) {
                left -= C::kBK;
                accum = 1;
              }
            }
            mma_commit(smem_u32(&empty[stage]));
          }
          __syncwarp();
          advance();
        }
        if (aborted) break;
        if (lane == 0) mma_commit(smem_u32(&tfull[acc]));
        __syncwarp();
        if (++acc == H.nacc) { acc = 0; acc_phase ^= 1u; }
        P.step(H.n_act);
      }
    }
    if (aborted && lane == 0) {
      mma_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
  } else if (C::kCopier && warp == 6) {
    // ------------------------------------------------------------ scale copier: a stage's atoms -> tensor memory
#pragma unroll 1
    for (int ph = 0; ph < 2; ++ph) {
      const int natom = a.ph[ph].red >> 7;
      Plan P = s_plan[ph];
      const uint64_t ds0 = smem_desc(smem0 + P.sf_off, 0, 128, kSwizzleNone);
      while (P.p < P.p1 && !aborted) {
        const int end = P.kb + P.length();
        for (int kb = P.kb; kb < end; ++kb) {
          if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          fence_proxy_async_smem();  // the token operand's and its scales' cp.async writes
          if (lane == 0) {
            uint64_t ds = ds0 + ((uint64_t)(stage * H.stage_bytes) >> 4);
            uint32_t sf = tmem_base + H.sf_col0 + stage * H.sf_per;
            // the weight pieces' atoms, then the token pieces'; those past the end of K are skipped
            const int at0 = kb * P.nb * C::kSub;
#pragma unroll 1
            for (int s = 0; s < P.np + P.nb; ++s) {
              const int at = at0 + (ph == 0 ? 0 : (s & (P.nb - 1)) * C::kSub);
#pragma unroll
              for (int i = 0; i < C::kSub; ++i)
                if (at + i < natom) tmem_cp_32x128b_x4(sf + 4 * i, ds + (i * 512 >> 4));
              ds += C::kSub * 512 >> 4;
              sf += C::kSub * 4;
            }
            mma_commit(smem_u32(&sfull[stage]));
          }
          __syncwarp();
          advance();
        }
        if (aborted) break;
        P.step(H.n_act);
      }
    }
    if (aborted && lane == 0) {
      mma_commit(smem_u32(cdrain));
      mbar_wait_drain(smem_u32(cdrain), 0);
    }
  } else if (warp >= kLoadWarp0) {
    // ------------------------------------------------------------ the token operand
    // Thread (r0, j) fetches 16-byte chunk j of rows r0, r0 + 16, ...: chunk j of row r goes to chunk
    // j ^ (r % 8) of its 128 bytes (the 128-byte swizzle), so its places are kStep bytes apart.
    // Rows past n hold leftovers, which only reach accumulator columns that nobody reads.
    // Scales are fetched by the threads counted from the other end: with few tokens a warp has
    // either kind.
    constexpr int kRows = 4 * kLoadWarps, kStep = kRows * 128, kHeld = 4;
    const int tid = threadIdx.x - kLoadWarp0 * 32, sid = 32 * kLoadWarps - 1 - tid;
    const int j = tid & 7, r0 = tid >> 3;
    const uint32_t place = r0 * 128 + ((j ^ (r0 & 7)) << 4);
    const uint32_t splace = (sid & 31) * 16 + (sid >> 5) * 4;  // row r's scales: word 4 (r % 32) + r / 32
    const int64_t lo_off = FMT == 0 ? a.act_lo - a.act : 0;
#pragma unroll 1
    for (int ph = 0; ph < 2; ++ph) {
      const DecodePhase& F = a.ph[ph];
      const int natom = F.red >> 7;
      const int64_t sb_ld = F.red >> 5;
      Plan P = s_plan[ph];
      if (ph == 1) {
        // A is complete when every CTA has finished phase 1 (all are resident: a cooperative launch)
        static_assert(kLoadWarps == 4, "epi_all's 128 threads");
        if (warp == kLoadWarp0 && !aborted && P.p < P.p1) {
          const uint64_t t0 = globaltimer();
          while (!aborted && load_acquire(a.done) != gridDim.x) {
            aborted = s_ctl->abort || globaltimer() - t0 > s_ctl->limit_ns;
            if (aborted) s_ctl->abort = 1;
          }
        }
        aborted = !epi_all<2>(!aborted);
      }
      for (; P.p < P.p1 && !aborted; P.step(H.n_act)) {
        const int off = s_off[P.slot], n = s_off[P.slot + 1] - off;
        const uint32_t lo_place = (uint32_t)((n + 7) & ~7) * 128;
        auto row_of = [&](int r) -> int64_t { return ph == 0 ? (int64_t)s_tok[off + r] : (int64_t)(off + r); };
        // the first rows' sources stay in registers over the segment
        const uint8_t* src[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          src[i] = F.b + (r0 + i * kRows < n ? row_of(r0 + i * kRows) : 0) * F.b_ld + j * 16;
        const uint8_t* ssrc = C::kSub ? F.sb + (sid < n ? row_of(sid) : 0) * sb_ld : nullptr;
        for (int kb = P.kb, end = P.kb + P.length(); kb < end; ++kb) {
          if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          const uint32_t st = smem0 + stage * H.stage_bytes;
#pragma unroll 1
          for (int s = 0; s < P.nb; ++s) {
            const int kk = kb * P.nb + s;
            if (kk >= F.pieces) break;
            const int kbyte = kk * 128;
            const uint32_t size = kbyte + j * 16 < F.b_ld ? 16u : 0u;  // past the end of K: zeros
            const int go = size ? kbyte : -j * 16;
            const uint32_t dst = st + P.b_off + s * P.b_piece + place;
            auto fetch = [&](const uint8_t* from, uint32_t to) {
              cp_async_16z(to, from + go, size);
              if (FMT == 0 && ph == 1) cp_async_16z(to + lo_place, from + lo_off + go, size);
            };
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
              if (r0 + i * kRows >= n) break;
              fetch(src[i], dst + i * kStep);
            }
            for (int i = kHeld; r0 + i * kRows < n; ++i)
              fetch(F.b + row_of(r0 + i * kRows) * F.b_ld + j * 16, dst + i * kStep);
            if (C::kSub && sid < n) {
              const uint32_t ssf = st + P.sf_off + (P.np + s) * C::kSub * 512 + splace;
#pragma unroll
              for (int sub = 0; sub < C::kSub; ++sub) {
                const int at = kk * C::kSub + sub;
                if (at < natom) cp_async_4(ssf + sub * 512, ssrc + at * 4, 4u);
              }
            }
          }
          cp_async_arrive_noinc(smem_u32(&full[stage]));
          __syncwarp();
          advance();
        }
      }
    }
    cp_async_wait_all();  // nothing of this warp's lands after the block exits
  } else {
    // ------------------------------------------------------------ epilogue (warps 2 .. 5)
    // An item that a cut divides begins at the end of one CTA's run.  That CTA finishes it; the others
    // send it their fp32 sums, which all but a whole-run CTA do at the start of their run.
    const int q = warp & 3, row = q * 32 + lane;  // accumulator row of this thread
    // (read while this warp would wait for the first product, so it costs no time)
    if (cta == 0 && threadIdx.x == 64 && load_acquire(a.done + 2) != 0u) set_error(a.err, kErrTimeout);
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&]() {  // the accumulator has been read
      tc_fence_before();
      mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == H.nacc) { acc = 0; acc_phase ^= 1u; }
    };
    auto activation = [&](float gate, float up) {
      if (a.limit > 0.0f) {  // NaN stays NaN
        gate = gate > a.limit ? a.limit : gate;
        up = up > a.limit ? a.limit : (up < -a.limit ? -a.limit : up);
      }
      return silu_f(gate) * up;
    };

    for (Plan P = s_plan[0]; P.p < P.p1; P.step(H.n_act)) {
      const int off = s_off[P.slot], n = s_off[P.slot + 1] - off;
      const int out_row = P.tile * 128 + row;
      const bool head = P.kb != 0, divided = !head && P.length() != P.nk;
      const int c_last = divided ? P.owner(P.p + P.L - 1) : cta;
      if (!epi_all(warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl))) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem_base + acc * H.acc_cols + ((uint32_t)(q * 32) << 16);
      // The other CTAs' sums lie in float4s of four tokens: [token / 4][gate, up][row].  All of `per`
      // tokens' loads are in flight; with few tokens the shorter code counts for more (one token, eight
      // MXFP4 experts: 28.65 us with 8, 28.85 with 16; 64 skewed tokens: 282 and 280).
      auto join = [&](auto per) {
        constexpr int kQuads = decltype(per)::value / 4;
        for (int x = cta + 1; x <= c_last; ++x) {
          for (int c0 = 0; c0 < n; c0 += 4 * kQuads) {
            const int m = n - c0;
            float4* o = reinterpret_cast<float4*>(a.part[0]) + ((int64_t)x * (kMaxT / 4) + c0 / 4) * 256 + row;
            float4 v[2 * kQuads];
            until([&]() {
              bool all = true;
#pragma unroll
              for (int i = 0; i < kQuads; ++i) {
                v[2 * i] = 4 * i < m ? load_relaxed4(o + i * 256) : zero4;
                v[2 * i + 1] = 4 * i < m ? load_relaxed4(o + i * 256 + 128) : zero4;
              }
#pragma unroll
              for (int i = 0; i < kQuads; ++i) all &= 4 * i >= m || (there(v[2 * i]) && there(v[2 * i + 1]));
              return all;
            });
            uint32_t own[2 * kQuads][4];
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
              if (4 * i < m) {
                store_relaxed4(o + i * 256, zero4);  // ready for the next launch
                store_relaxed4(o + i * 256 + 128, zero4);
                tmem_ld4(tb + c0 + 4 * i, own[2 * i]);
                tmem_ld4(tb + H.ncols + c0 + 4 * i, own[2 * i + 1]);
              }
            }
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 2 * kQuads; ++i)
              if (4 * (i >> 1) < m)
                tmem_st4(tb + (i & 1) * H.ncols + c0 + 4 * (i >> 1),
                         make_float4(as_float(own[i][0]) + v[i].x, as_float(own[i][1]) + v[i].y,
                                     as_float(own[i][2]) + v[i].z, as_float(own[i][3]) + v[i].w));
          }
          tmem_st_wait();  // the next CTA's sums are added to what has been stored here
        }
      };
      if (n <= 8) join(std::integral_constant<int, 8>());
      else join(std::integral_constant<int, 16>());
      if (head) {  // columns past n hold something as well, and the reader skips them
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += 4) {
          uint32_t g[4], u[4];
          tmem_ld4(tb + c0, g);
          tmem_ld4(tb + H.ncols + c0, u);
          tmem_ld_wait();
          float4* o = reinterpret_cast<float4*>(a.part[0]) + ((int64_t)cta * (kMaxT / 4) + c0 / 4) * 256 + row;
          store_relaxed4(o, make_float4(sent(as_float(g[0])), sent(as_float(g[1])), sent(as_float(g[2])), sent(as_float(g[3]))));
          store_relaxed4(o + 128, make_float4(sent(as_float(u[0])), sent(as_float(u[1])), sent(as_float(u[2])), sent(as_float(u[3]))));
        }
      } else {
        // Two tokens at a time: the even lanes store the first one's, the odd lanes the second one's, two
        // rows each, so that both take one conversion and one store.  Two such pairs overlap.
        const int odd = lane & 1;
        int64_t at = (int64_t)(off + odd) * a.I + (out_row & ~1);
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += 4) {
          uint32_t g[4], u[4];
          tmem_ld4(tb + c0, g);
          tmem_ld4(tb + H.ncols + c0, u);
          tmem_ld_wait();
          float v[4], x[2], y[2];
          uint32_t am[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = activation(as_float(g[c]), as_float(u[c]));
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (FMT != 0) am[c] = __reduce_max_sync(0xffffffffu, __float_as_uint(v[c]) & 0x7FFFFFFFu);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
            x[i] = odd ? other : v[2 * i];
            y[i] = odd ? v[2 * i + 1] : other;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i, at += 2 * (int64_t)a.I) {
            const bool on = c0 + 2 * i + odd < n;
            if (FMT == 0) {
              // A as the sum of two bf16 numbers (16 mantissa bits): both are multiplied
              const __nv_bfloat162 hi = __floats2bfloat162_rn(x[i], y[i]);
              const float lx = x[i] - __low2float(hi), ly = y[i] - __high2float(hi);
              if (on && out_row < a.I) {
                *reinterpret_cast<__nv_bfloat162*>(a.act + 2 * at) = hi;
                *reinterpret_cast<uint32_t*>(a.act_lo + 2 * at) =
                    pack_bf16x2(fabsf(lx) < INFINITY ? lx : 0.0f, fabsf(ly) < INFINITY ? ly : 0.0f);
              }
            } else {
              // the warp's 32 rows are one MX block of each token
              uint32_t sc;
              float mult;
              const bool fin = block_scale_f32<FMT == 0 ? kE4M3 : FMT>(odd ? am[2 * i + 1] : am[2 * i], sc, mult);
              x[i] = fin ? x[i] * mult : 0.0f;
              y[i] = fin ? y[i] * mult : 0.0f;
              if (on) {
                if (FMT == kE4M3) *reinterpret_cast<uint16_t*>(a.act + at) = (uint16_t)cvt_e4m3x2(x[i], y[i]);
                else a.act[at >> 1] = (uint8_t)cvt_e2m1x2(x[i], y[i]);
                if (lane < 2) a.act_scales[at >> 5] = (uint8_t)sc;
              }
            }
          }
        }
      }
      release();
    }
    // this CTA's part of A is written (or it has given up, which the others must not wait for)
    epi_sync();
    if (threadIdx.x == 64) add_release(a.done, 1u);

    Plan P = s_plan[1];
    int last_tile = P.tile;  // of this run
    for (const int p0 = P.p; P.p < P.p1 && !aborted; P.step(H.n_act)) {
      const int off = s_off[P.slot], n = s_off[P.slot + 1] - off;
      const int p_end = P.p + P.length();
      const int item0 = P.tile * P.L, item1 = item0 + P.L;
      last_tile = P.tile;
      if (P.p == p0 || P.p == item0)
        for (int t = 0; t < a.T; ++t) s_acc[t * 128 + row] = 0.0f;
      if (!epi_all(warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl))) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem_base + acc * H.acc_cols + ((uint32_t)(q * 32) << 16);
      const int lo = (n + 7) & ~7;  // bf16: the column of the first low part
      for (int c0 = 0; c0 < n; c0 += kBatch) {
        uint32_t vr[kBatch], left[kBatch];
        tmem_ld4(tb + c0, vr);
        if (FMT == 0) tmem_ld4(tb + lo + c0, left);
        tmem_ld_wait();
        float v[kBatch];
#pragma unroll
        for (int c = 0; c < kBatch; ++c) v[c] = FMT == 0 ? as_float(vr[c]) + as_float(left[c]) : as_float(vr[c]);
        float* at[kBatch];  // an expert's tokens differ, so a batch's sums are apart
        float sum[kBatch];
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const int r = off + min(c0 + c, n - 1);
          at[c] = s_acc + s_tok[r] * 128 + row;
          sum[c] = *at[c] + s_w[r] * v[c];
        }
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
          if (c0 + c < n) *at[c] = sum[c];
      }
      release();
      if (p_end == item1 && p_end != P.p1) {  // an output tile ends inside the run (the last one: below)
        epi_sync();
        flush(P.tile, warp - 2, 4);
        epi_sync();  // s_acc has been read by other threads than its writers
      }
    }
    if (threadIdx.x == 64) *s_last_tile = last_tile;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // The divided tiles of this CTA's run, its first and its last: each of a tile's CTAs adds up an
  // equal share of the tokens, by all of its warps and in CTA order.  All have sent everything before
  // they wait here.  (Left to one CTA, the sums of 42 tokens from 50 CTAs took 60 us.)
  const Plan Q = s_plan[1];
  const int last_tile = *s_last_tile;
  if (Q.p < Q.p1 && !__any_sync(0xffffffffu, s_ctl->abort)) flush(last_tile, warp, kNT / 32);
  // (the whole warp goes by one reading of the flag)
  for (int tile = Q.tile; Q.p < Q.p1 && !__any_sync(0xffffffffu, s_ctl->abort); tile = last_tile) {
    const int item0 = tile * Q.L, item1 = item0 + Q.L;
    if (Q.p > item0 || Q.p1 < item1) {
      const int c_first = Q.owner(item0), m = Q.owner(item1 - 1) - c_first + 1;
      const int r4 = tile * 128 + 4 * lane, rows = a.ph[1].rows;
      for (int t = cta - c_first + warp * m; t < a.T; t += kNT / 32 * m) {
        // the first CTA's sums are those of an item that begins in its run, the others' are not
        float4* part = reinterpret_cast<float4*>(a.part[1]) + ((int64_t)c_first * 2 * kMaxT + t) * 32 + lane;
        auto from = [&](int i) { return part + (int64_t)(2 * i + (i == 0)) * kMaxT * 32; };
        float4 sum = zero4;
        for (int i0 = 0; i0 < m; i0 += 4) {
          float4 v[4];
          until([&]() {  // four loads in flight (eight or sixteen were slower: more code to fetch)
            bool all = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i0 + i < m ? load_relaxed4(from(i0 + i)) : zero4;
#pragma unroll
            for (int i = 0; i < 4; ++i) all &= i0 + i >= m || there(v[i]);
            return all;
          });
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i0 + i < m) store_relaxed4(from(i0 + i), zero4);  // ready for the next launch
            sum.x += v[i].x; sum.y += v[i].y; sum.z += v[i].z; sum.w += v[i].w;
          }
        }
        if (r4 < rows)
          *reinterpret_cast<uint2*>(a.out + (int64_t)t * rows + r4) =
              make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      }
    }
    if (tile == last_tile) break;
  }
  if (s_ctl->abort && lane == 0) {  // a role gave up (whichever did has raised the flag), or sums never came
    set_error(a.err, kErrTimeout);
    atomicExch(a.done + 2, 1u);  // what other CTAs have sent to this one is left behind
  }
  // the last CTA to leave clears the count that the others have waited on
  if (threadIdx.x == 0 && atomicInc(a.done + 1, gridDim.x - 1) == gridDim.x - 1) atomicExch(a.done, 0u);
}

// ---------------------------------------------------------------- workspace
// [CTAs done and left, given up][partial sums of both phases][A: bf16 high and low parts, or codes and
// scales].  The first two are zero between calls, so they have the same place whatever the sizes.
constexpr size_t kPartBytes = (size_t)kMaxCtas * kMaxT * (256 + 2 * 128) * sizeof(float);
struct DecodeWs {
  size_t part, act, act_lo, act_scales, bytes;
};
DecodeWs decode_ws(int fmt, int64_t T, int k, int64_t I) {
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  const size_t rows = (size_t)T * k;
  const size_t row = fmt == 0 ? (size_t)I * 2 : fmt == PGG_FMT_E4M3 ? (size_t)I : (size_t)I / 2;
  DecodeWs w;
  w.part = 1024;
  w.act = w.part + kPartBytes;
  w.act_lo = w.act + up(rows * row);
  w.act_scales = w.act_lo;
  w.bytes = w.act_lo + (fmt == 0 ? up(rows * row) : up(rows * (size_t)I / 32));
  return w;
}

int check_decode_dims(int fmt, int64_t T, int k, int64_t H, int64_t I, int E) {
  if (fmt != 0 && fmt != PGG_FMT_E4M3 && fmt != PGG_FMT_E2M1) return PGG_ERR_INVALID_ARG;
  if (T < 0 || k < 1 || k > 32 || E < 1 || E > kMaxGroups) return PGG_ERR_INVALID_ARG;
  const int mult = fmt == 0 ? 8 : 128;
  if (H < mult || I < mult || H > 65536 || I > 65536) return PGG_ERR_INVALID_ARG;
  if (H % mult || I % mult) return PGG_ERR_ALIGNMENT;
  if (T > kMaxT) return PGG_ERR_TOO_LARGE;
  return PGG_OK;
}

constexpr unsigned long long kWaitLimit = kWaitTimeoutNs;
template <int FMT>
int run_decode(const uint8_t* X, const uint8_t* xs, const int32_t* ids, const float* w, const void* W1,
               const uint8_t* w1s, const void* W2, const uint8_t* w2s, void* out, int64_t T, int k, int64_t H,
               int64_t I, int E, float limit, uint8_t* ws, int32_t* err, cudaStream_t s,
               unsigned long long wait_ns = kWaitLimit, long long stall_at = -1) {
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != PGG_OK) return st;
  const DecodeWs L = decode_ws(FMT, T, k, I);
  const auto dt = FMT == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint32_t bx = FMT == 0 ? 64 : 128;  // elements of the map in 128 bytes
  auto elems = [&](int64_t n) { return (uint64_t)(FMT == kE2M1 ? n / 2 : n); };
  auto bytes = [&](int64_t n) { return elems(n) * (FMT == 0 ? 2 : 1); };
  CUtensorMap t1, t2;
  {
    uint64_t d[4] = {elems(H), (uint64_t)I, 2, (uint64_t)E};
    uint64_t sb[3] = {bytes(H), bytes(H) * (uint64_t)I, bytes(H) * (uint64_t)I * 2};
    uint32_t b[4] = {bx, 128, 1, 1};
    if ((st = encode_tmap(&t1, dt, 4, W1, d, sb, b, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  }
  {
    uint64_t d[4] = {elems(I), (uint64_t)H, 1, (uint64_t)E};
    uint64_t sb[3] = {bytes(I), bytes(I) * (uint64_t)H, bytes(I) * (uint64_t)H};
    uint32_t b[4] = {bx, 128, 1, 1};
    if ((st = encode_tmap(&t2, dt, 4, W2, d, sb, b, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  }
  DecodeArgs a{};
  a.ids = ids;
  a.w = w;
  a.T = (int)T;
  a.k = k;
  a.E = E;
  a.I = (int)I;
  a.limit = limit;
  auto cdiv = [](int64_t x, int64_t y) { return (int)((x + y - 1) / y); };
  constexpr int kBK = DecCfg<FMT>::kBK;
  auto phase = [&](int64_t rows, int halves, int64_t red, const uint8_t* b, const uint8_t* sb, const uint8_t* sa) {
    const int tiles = cdiv(rows, 128), pieces = cdiv(red, kBK);
    return DecodePhase{(int)rows, halves, (int)red, tiles, pieces,
                       {FastDiv((uint32_t)pieces), FastDiv((uint32_t)(pieces + 1) / 2)}, b, (int64_t)bytes(red), sb, sa};
  };
  a.ph[0] = phase(I, 2, H, X, xs, w1s);
  a.ph[1] = phase(H, 1, I, ws + L.act, ws + L.act_scales, w2s);
  const int grid = std::min(dev.sms, kMaxCtas);
  a.by_grid = FastDiv((uint32_t)grid);
  a.act = ws + L.act;
  a.act_lo = ws + L.act_lo;
  a.act_scales = ws + L.act_scales;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.part[0] = reinterpret_cast<float*>(ws + L.part);
  a.part[1] = a.part[0] + (size_t)kMaxCtas * kMaxT * 256;
  a.done = reinterpret_cast<unsigned*>(ws);
  a.err = err;
  a.wait_ns = wait_ns;
  a.stall_at = stall_at;
  a.slots_cap = std::min(E, a.T * k);
  const size_t lists = kFixedBytes + (size_t)a.T * 512 + (size_t)a.T * k * 4 + 2 * (2 * (size_t)a.slots_cap + 1) +
                       (size_t)a.T * k;
  // the whole of an SM's shared memory, so that a CTA has its SM and the tensor memory to itself
  const size_t smem = dev.smem_optin;
  a.ring_bytes = (int)((smem - 1024 - lists) / 1024 * 1024);
  auto kern = moe_decode_kernel<FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(DecCfg<FMT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeCooperative;  // CTAs wait for one another between the phases
  at.val.cooperative = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, t1, t2, a);
  return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

int check_decode(int fmt, const void* X, const int32_t* ids, const float* w, const void* W1, const void* W2, void* out,
                 int64_t T, int k, int64_t H, int64_t I, int E, float limit, void* ws, size_t ws_bytes,
                 const int32_t* err) {
  const int st = check_decode_dims(fmt, T, k, H, I, E);
  if (st) return st;
  if (!(limit >= 0.0f) || limit > 3.0e38f) return PGG_ERR_INVALID_ARG;
  if (T == 0) return PGG_OK;
  if (!X || !ids || !W1 || !W2 || !out || !ws) return PGG_ERR_INVALID_ARG;
  if (ws_bytes < decode_ws(fmt, T, k, I).bytes) return PGG_ERR_INVALID_ARG;
  for (const void* p : {X, W1, W2, (const void*)out, (const void*)ws})
    if (!aligned_to(p, 16)) return PGG_ERR_ALIGNMENT;
  if (!aligned_to(ids, 4) || !aligned_to(w, 4) || !aligned_to(err, 4)) return PGG_ERR_ALIGNMENT;
  return PGG_OK;
}

}  // namespace
}  // namespace pgg

using namespace pgg;

extern "C" {

int pgg_moe_decode_workspace_size(int fmt, int64_t T, int k, int64_t H, int64_t I, int E, size_t* bytes) {
  const int st = check_decode_dims(fmt, T, k, H, I, E);
  if (st) return st;
  if (!bytes) return PGG_ERR_INVALID_ARG;
  *bytes = decode_ws(fmt, T, k, I).bytes;
  return PGG_OK;
}

int pgg_moe_decode(const void* X, const int32_t* topk_ids, const float* w, const void* W1, const void* W2, void* out,
                   int64_t T, int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes,
                   int32_t* err, void* stream) {
  const int st = check_decode(0, X, topk_ids, w, W1, W2, out, T, k, H, I, E, swiglu_limit, ws, ws_bytes, err);
  if (st || T == 0) return st;
  return run_decode<0>(static_cast<const uint8_t*>(X), nullptr, topk_ids, w, W1, nullptr, W2, nullptr, out, T, k, H, I,
                       E, swiglu_limit, static_cast<uint8_t*>(ws), err, reinterpret_cast<cudaStream_t>(stream));
}

static int mx_decode(int fmt, const uint8_t* X, const uint8_t* SX, const int32_t* topk_ids, const float* w,
                     const uint8_t* W1, const uint8_t* SW1, const uint8_t* W2, const uint8_t* SW2, void* out, int64_t T,
                     int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes, int32_t* err,
                     void* stream, unsigned long long wait_ns, long long stall_at) {
  if (fmt != PGG_FMT_E4M3 && fmt != PGG_FMT_E2M1) return PGG_ERR_INVALID_ARG;
  const int st = check_decode(fmt, X, topk_ids, w, W1, W2, out, T, k, H, I, E, swiglu_limit, ws, ws_bytes, err);
  if (st || T == 0) return st;
  if (!SX || !SW1 || !SW2) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(SX, 4) || !aligned_to(SW1, 16) || !aligned_to(SW2, 16)) return PGG_ERR_ALIGNMENT;
  auto go = fmt == PGG_FMT_E4M3 ? run_decode<kE4M3> : run_decode<kE2M1>;
  return go(X, SX, topk_ids, w, W1, SW1, W2, SW2, out, T, k, H, I, E, swiglu_limit, static_cast<uint8_t*>(ws), err,
            reinterpret_cast<cudaStream_t>(stream), wait_ns, stall_at);
}

int pgg_mx_moe_decode(int fmt, const uint8_t* X, const uint8_t* SX, const int32_t* topk_ids, const float* w,
                      const uint8_t* W1, const uint8_t* SW1, const uint8_t* W2, const uint8_t* SW2, void* out,
                      int64_t T, int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes,
                      int32_t* err, void* stream) {
  return mx_decode(fmt, X, SX, topk_ids, w, W1, SW1, W2, SW2, out, T, k, H, I, E, swiglu_limit, ws, ws_bytes, err,
                   stream, kWaitLimit, -1);
}

int pgg_test_stalled_moe_decode(int fmt, const void* X, const uint8_t* SX, const int32_t* topk_ids, const void* W1,
                                const uint8_t* SW1, const void* W2, const uint8_t* SW2, void* out, int64_t T, int k,
                                int64_t H, int64_t I, int E, int64_t stall_at, uint64_t wait_ns, void* ws,
                                size_t ws_bytes, int32_t* err, void* stream) {
  if (stall_at < 0 || wait_ns < 100000ull || wait_ns > 1000000000ull) return PGG_ERR_INVALID_ARG;
  if (fmt != 0)
    return mx_decode(fmt, static_cast<const uint8_t*>(X), SX, topk_ids, nullptr, static_cast<const uint8_t*>(W1), SW1,
                     static_cast<const uint8_t*>(W2), SW2, out, T, k, H, I, E, 0.0f, ws, ws_bytes, err, stream, wait_ns,
                     stall_at);
  const int st = check_decode(0, X, topk_ids, nullptr, W1, W2, out, T, k, H, I, E, 0.0f, ws, ws_bytes, err);
  if (st || T == 0) return st;
  return run_decode<0>(static_cast<const uint8_t*>(X), nullptr, topk_ids, nullptr, W1, nullptr, W2, nullptr, out, T, k,
                       H, I, E, 0.0f, static_cast<uint8_t*>(ws), err, reinterpret_cast<cudaStream_t>(stream), wait_ns,
                       stall_at);
}

}  // extern "C"

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
// divides is put together from fp32 partial sums by the last of its CTAs to arrive, in CTA order
// (the result does not depend on which one that is).
//
// Between the phases only the warps that fetch A wait for the other CTAs (a cooperative launch
// makes all of them resident); the weight loads run on into phase 2 and keep the ring full.
//
// Every CTA builds the batch's expert list by itself from the ids: a bit per (expert, token), so
// an expert named twice by a token is computed once and its weights are added up.
#include <algorithm>
#include <type_traits>

#include "block.cuh"
#include "epilogue.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kMaxT = PGG_MOE_DECODE_MAX_T;
constexpr int kMaxCtas = 192;   // CTAs of a launch (one per SM); sizes the workspace without a device
constexpr int kMaxStages = 8;
constexpr int kLoadWarps = 4;   // warps that fetch the token operand
constexpr int kBatch = 4;      // tokens that the epilogue works on at a time
constexpr int kTileBytes = 128 * 128;  // 128 rows x one 128-byte swizzle atom of K

template <int FMT>
struct DecCfg {
  static constexpr int kBK = FMT == 0 ? 64 : FMT == kE4M3 ? 128 : 256;  // elements in 128 bytes
  static constexpr int kSub = FMT == 0 ? 0 : kBK / 128;                  // scale atoms of them
  static constexpr int kPerMma = kBK / 4;
  static constexpr int kCopier = FMT != 0;
  static constexpr int kThreads = 32 * (6 + kCopier + kLoadWarps);
};

// One matrix of a layer and what the MMAs of its phase read and write.
struct DecodePhase {
  int rows;            // output rows per expert: I (phase 1), H (phase 2)
  int red;             // reduction length: H (phase 1), I (phase 2)
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
  float* part;          // partial sums: 2 tiles per CTA
  unsigned* cnt;        // arrivals at a divided tile by its first CTA, for each phase
  unsigned* done;       // CTAs that have finished phase 1; [1]: that have left.  All zero between launches
  int ring_bytes;       // shared memory for the stages
  int slots_cap;        // most experts that the batch can name
  int32_t* err;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&f)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// The MMAs of one lane (`go`), issued by a whole converged warp: with the branch on the lane inside
// the instruction's own predicate, descriptors stay warp-uniform values.
template <int FMT>
__device__ __forceinline__ void mma_if(uint32_t go, uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accum) {
  if (FMT == 0)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accum), "r"(go)
        : "memory");
  else if (FMT == kE4M3)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(go)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(go)
        : "memory");
}
// Barrier of the four epilogue warps that tells each whether `ok` held in all of them: they give
// up together, so that none is left at a later barrier.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// What both phases share of a launch's cut: the shape of a ring stage and of tensor memory.
struct Shape {
  int n_act;    // experts that the batch names
  int ncols;    // most tokens of one of them, rounded up to 16
  int ns;       // phase 2: 128-byte K pieces per stage
  int stages, stage_bytes;
  int acc_cols, nacc, sf_col0, sf_per;  // tensor memory
};
// One phase's stages, cut into equal runs; every CTA computes the same.
struct Plan {
  int tiles;      // 128-row output tiles per expert
  int nk;         // stages of one (expert, tile)
  int L;          // stages of one item: an (expert, tile) in phase 1, an output tile in phase 2
  int total;      // stages of the phase
  int quot, rem;  // total = ctas quot + rem: the first rem CTAs get a stage more
  int b_off, b_piece, sf_off;  // layout of a stage: weights, token pieces, scale atoms
  int p0, p1;     // this CTA's run
  __device__ __forceinline__ int start(int c) const { return c * quot + min(c, rem); }
  // the CTA that stage p belongs to
  __device__ __forceinline__ int owner(int p) const {
    const int big = rem * (quot + 1);
    return p < big ? p / (quot + 1) : rem + (p - big) / quot;
  }
};

// Columns (rows of the token operand) of n tokens in phase 2: bf16 keeps the high and the low parts
// of A next to each other, each rounded up to the 8 rows of a swizzle atom.
template <int FMT>
__device__ __forceinline__ int cols2(int n) {
  return FMT == 0 ? (2 * ((n + 7) & ~7) + 15) & ~15 : (n + 15) & ~15;
}

template <int FMT>
__device__ __forceinline__ Shape make_shape(const DecodeArgs& a, int n_act, int max_n) {
  using C = DecCfg<FMT>;
  Shape S;
  S.n_act = n_act;
  S.ncols = (max_n + 15) & ~15;
  const int b1 = S.ncols * 128, b2 = cols2<FMT>(max_n) * 128;
  const int s1 = 2 * kTileBytes + b1 + C::kSub * 3 * 512;
  const int two = 2 * (kTileBytes + b2 + C::kSub * 1024), one = kTileBytes + b2 + C::kSub * 1024;
  // phase 2: two K pieces a stage, or one where many tokens would leave fewer than three stages
  const int st1 = (max(s1, one) + 1023) & ~1023, st2 = (max(s1, two) + 1023) & ~1023;
  S.ns = a.ring_bytes / st2 >= min(3, a.ring_bytes / st1) ? 2 : 1;
  S.stage_bytes = S.ns == 2 ? st2 : st1;
  S.stages = min(kMaxStages, a.ring_bytes / S.stage_bytes);
  S.acc_cols = max(2 * S.ncols, b2 / 128);
  S.sf_per = C::kSub * max(12, S.ns * 8);
  S.nacc = 2 * S.acc_cols + S.stages * S.sf_per <= 512 ? 2 : 1;
  S.sf_col0 = S.nacc * S.acc_cols;
  return S;
}

template <int FMT, int PHASE>
__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, const Shape& S, int max_n) {
  using C = DecCfg<FMT>;
  Plan P;
  const int kb = (a.ph[PHASE - 1].red + C::kBK - 1) / C::kBK;
  P.tiles = (a.ph[PHASE - 1].rows + 127) / 128;
  if (PHASE == 1) {
    P.nk = kb;
    P.b_off = 2 * kTileBytes;
    P.b_piece = S.ncols * 128;
    P.sf_off = P.b_off + P.b_piece;
  } else {
    P.nk = S.ns == 2 ? (kb + 1) >> 1 : kb;
    P.b_off = S.ns * kTileBytes;
    P.b_piece = cols2<FMT>(max_n) * 128;
    P.sf_off = P.b_off + S.ns * P.b_piece;
  }
  P.L = PHASE == 1 ? P.nk : S.n_act * P.nk;
  P.total = S.n_act * P.tiles * P.nk;
  const int ctas = max(1, min((int)gridDim.x, P.total)), cta = blockIdx.x;
  P.quot = P.total / ctas;
  P.rem = P.total - ctas * P.quot;
  P.p0 = cta < ctas ? P.start(cta) : 0;
  P.p1 = cta < ctas ? P.start(cta + 1) : 0;
  return P;
}

// A run of stages [kb0, kb1) of one (expert slot, tile); `item` is what partial sums are joined by.
struct Seg {
  int slot, tile, item, kb0, kb1;
};

template <int PHASE>
__device__ __forceinline__ Seg seg_at(const Plan& P, int p) {
  Seg s;
  s.item = p / P.L;
  const int q = p - s.item * P.L;
  if (PHASE == 1) {
    s.slot = s.item / P.tiles;
    s.tile = s.item - s.slot * P.tiles;
    s.kb0 = q;
  } else {
    s.tile = s.item;
    s.slot = q / P.nk;
    s.kb0 = q - s.slot * P.nk;
  }
  s.kb1 = min(P.nk, s.kb0 + (P.p1 - p));
  return s;
}

using Phase1 = std::integral_constant<int, 1>;
using Phase2 = std::integral_constant<int, 2>;

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
  int* s_last = reinterpret_cast<int*>(s_tmem + 1);
  int* s_scan = s_last + 1;  // [2 * 16]
  float* s_acc = reinterpret_cast<float*>(smem + a.ring_bytes + 512);  // phase 2: [T][128]
  float* s_w = s_acc + a.T * 128;                                       // [T k]
  uint16_t* s_off = reinterpret_cast<uint16_t*>(s_w + a.T * a.k);       // [slots + 1]: an expert's first entry
  uint16_t* s_exp = s_off + a.slots_cap + 1;                            // [slots]
  uint8_t* s_tok = reinterpret_cast<uint8_t*>(s_exp + a.slots_cap);     // [T k]: the entries' tokens

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the batch's experts and their tokens (scratch: the ring, before the first stage lands)
  const int W = (a.T + 31) / 32;  // mask words per expert
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem);               // [E][W]
  float* s_wid = reinterpret_cast<float*>(s_mask + a.E * W);          // [T k]: the weights as given
  int16_t* s_id = reinterpret_cast<int16_t*>(s_wid + a.T * a.k);      // [T k]: the ids, -1 out of range
  uint16_t* s_eoff = reinterpret_cast<uint16_t*>(s_id + a.T * a.k);   // [E]: first entry
  const int n_ids = a.T * a.k;
  // Up to 32 ids: every warp works the list out in registers (lane i has id i) and all of them write
  // the same; the slots are in the order of first mention.  Saves three block barriers and the scan
  // over the experts (a third of the time before the first load, which a one-token call feels).
  const bool few = n_ids <= 32;
  int id = -1, tok = 0;
  float wid = 0.0f;
  if (few) {
    if (lane < n_ids) {
      id = __ldg(a.ids + lane);
      wid = a.w ? __ldg(a.w + lane) : 1.0f;
      tok = lane / a.k;
      if (id < 0 || id >= a.E) {
        if (blockIdx.x == 0) set_error(a.err, kErrBadExpert);
        id = -1;
      }
    }
  } else {
    for (int i = threadIdx.x; i < n_ids; i += kNT) {
      const int e = __ldg(a.ids + i);
      const bool ok = e >= 0 && e < a.E;
      if (!ok && blockIdx.x == 0) set_error(a.err, kErrBadExpert);
      s_id[i] = (int16_t)(ok ? e : -1);
      s_wid[i] = a.w ? __ldg(a.w + i) : 1.0f;
    }
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
      s_ctl->limit_ns = kWaitTimeoutNs;
      prefetch_tmap(&tmW1);
      prefetch_tmap(&tmW2);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  int n_act, max_n;
  if (few) {
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
    for (int i = 0; i < n_ids; ++i) {
      const float o = __shfl_sync(all, wid, i);
      if (pair >> i & 1) wt += o;
    }
    if (entry) {
      const int r = first + __popc(same & entries & below);
      s_tok[r] = (uint8_t)tok;
      s_w[r] = wt;
    }
  } else {
    __syncthreads();
    for (int i = threadIdx.x; i < n_ids; i += kNT) {
      const int t = i / a.k;
      if (s_id[i] >= 0) atomicOr(&s_mask[s_id[i] * W + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    {
      const int per = (a.E + kNT - 1) / kNT;
      const int lo = min((int)threadIdx.x * per, a.E), hi = min(lo + per, a.E);
      int v = 0, mx = 0;  // experts << 16 | tokens
      for (int e = lo; e < hi; ++e) {
        int n = 0;
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
      for (int e = lo; e < hi; ++e) {
        int n = 0;
        for (int q = 0; q < W; ++q) n += __popc(s_mask[e * W + q]);
        if (!n) continue;
        s_exp[run >> 16] = (uint16_t)e;
        s_off[run >> 16] = s_eoff[e] = (uint16_t)(run & 0xFFFF);
        run += (1 << 16) + n;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_ids; i += kNT) {
      const int e = s_id[i];
      if (e < 0) continue;
      const int t = i / a.k, i0 = t * a.k;
      bool first = true;  // the token's first choice of this expert writes the entry
      for (int j = i0; j < i; ++j) first &= s_id[j] != e;
      if (!first) continue;
      int r = s_eoff[e];
      for (int q = 0; q < (t >> 5); ++q) r += __popc(s_mask[e * W + q]);
      r += __popc(s_mask[e * W + (t >> 5)] & ((1u << (t & 31)) - 1u));
      s_tok[r] = (uint8_t)t;
      float wt = 0.0f;
      for (int j = i; j < i0 + a.k; ++j)
        if (s_id[j] == e) wt += s_wid[j];
      s_w[r] = wt;
    }
  }
  fence_proxy_async_smem();  // the ring's scratch use, before its first bulk copies
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const Shape H = make_shape<FMT>(a, n_act, max_n);
  const Plan plan1 = make_plan<FMT, 1>(a, H, max_n), plan2 = make_plan<FMT, 2>(a, H, max_n);
  const int cta = blockIdx.x;
  const uint32_t tmem_base = *s_tmem;
  const uint32_t smem0 = smem_u32(smem);
  bool aborted = false;
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++stage == H.stages) { stage = 0; phase ^= 1u; }
  };

  if (n_act == 0) {  // no expert is named: the layer's output is zero
    for (int64_t i = (int64_t)cta * kNT + threadIdx.x; i < (int64_t)a.T * a.ph[1].rows; i += (int64_t)gridDim.x * kNT)
      a.out[i] = __float2bfloat16_rn(0.0f);
  }

  if (warp == 0) {
    // ------------------------------------------------------------ weights: TMA tiles, bulk scale atoms
    // The producer runs into phase 2 without waiting: its weights do not depend on phase 1.
    long long issued = 0;
    auto produce = [&](auto ph, const Plan& P) {
      constexpr int PHASE = decltype(ph)::value;
      const DecodePhase& F = a.ph[PHASE - 1];
      const int natom = F.red >> 7;  // MX: scale atoms of a 128-row block along K
      for (int p = P.p0; p < P.p1 && !aborted;) {
        const Seg S = seg_at<PHASE>(P, p);
        const int e = s_exp[S.slot], row0 = S.tile * 128;
        for (int kb = S.kb0; kb < S.kb1; ++kb) {
          if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          if (lane == 0) {
            const uint32_t fb = smem_u32(&full[stage]);
            const uint32_t st = smem0 + stage * H.stage_bytes;
            if (PHASE == 1) {
              const int at0 = kb * C::kSub, nat = C::kSub ? min(C::kSub, natom - at0) : 0;
              mbar_arrive_expect_tx(fb, 2 * kTileBytes + 2 * 512 * nat);
              const int x = kb * (FMT == 0 ? 64 : 128);
              tma_load_4d(st, &tmW1, fb, x, row0, 0, e);
              tma_load_4d(st + kTileBytes, &tmW1, fb, x, row0, 1, e);
              if (C::kSub) {
                const int64_t rg = ((int64_t)e * 2 * a.I + row0) >> 7, ru = ((int64_t)e * 2 * a.I + a.I + row0) >> 7;
                bulk_load(st + P.sf_off, F.sa + (rg * natom + at0) * 512, 512 * nat, fb);
                bulk_load(st + P.sf_off + C::kSub * 512, F.sa + (ru * natom + at0) * 512, 512 * nat, fb);
              }
            } else {
              const int kk0 = kb * H.ns, at0 = kk0 * C::kSub, nat = C::kSub ? min(H.ns * C::kSub, natom - at0) : 0;
              const bool second = H.ns == 2 && (kk0 + 1) * C::kBK < F.red;
              mbar_arrive_expect_tx(fb, (second ? 2 : 1) * kTileBytes + 512 * nat);
              const int x = kk0 * (FMT == 0 ? 64 : 128);
              tma_load_3d(st, &tmW2, fb, x, row0, e);
              if (second) tma_load_3d(st + kTileBytes, &tmW2, fb, x + (FMT == 0 ? 64 : 128), row0, e);
              if (C::kSub)
                bulk_load(st + P.sf_off, F.sa + ((((int64_t)e * F.rows + row0) >> 7) * natom + at0) * 512, 512 * nat,
                          fb);
            }
          }
          __syncwarp();
          ++issued;
          advance();
        }
        p += S.kb1 - S.kb0;
      }
    };
    produce(Phase1(), plan1);
    produce(Phase2(), plan2);
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
    auto multiply = [&](auto ph, const Plan& P) {
      constexpr int PHASE = decltype(ph)::value;
      const int red = a.ph[PHASE - 1].red;
      const uint32_t one = lane == 0;
      // descriptors of stage 0's tiles; an address d bytes further on adds d / 16
      const uint64_t desc_a = smem_desc(smem0, 16, 1024, kSwizzle128B);
      const uint64_t desc_b = smem_desc(smem0 + P.b_off, 16, 1024, kSwizzle128B);
      for (int p = P.p0; p < P.p1 && !aborted;) {
        const Seg S = seg_at<PHASE>(P, p);
        const int n = s_off[S.slot + 1] - s_off[S.slot];
        const uint32_t N = PHASE == 1 ? (n + 15) & ~15 : cols2<FMT>(n);
        const uint32_t idesc = FMT == 0 ? idesc_bf16(128, N, false, false) : idesc_mx(FMT == kE4M3 ? 0 : 1, 128, N);
        if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * H.acc_cols;
        for (int kb = S.kb0; kb < S.kb1; ++kb) {
          if (!warp_wait(smem_u32(C::kCopier ? &sfull[stage] : &full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          if (!C::kCopier) fence_proxy_async_smem();  // the token operand's cp.async writes
          const uint64_t so = (uint64_t)(stage * H.stage_bytes) >> 4;
          const uint32_t sf = tmem_base + H.sf_col0 + stage * H.sf_per;
#pragma unroll
          for (int s = 0; s < 2; ++s) {  // phase 1: gate and up; phase 2: K pieces
            if (PHASE == 2 && s == H.ns) break;
            const int kk = PHASE == 1 ? kb : kb * H.ns + s;
            // MMAs of this piece that hold data (an e2m1 K may end inside it; the zero-filled end
            // of a bf16 K adds nothing)
            const int left = red - kk * C::kBK;
            const uint64_t ad = desc_a + so + s * (kTileBytes >> 4);
            const uint64_t bd = desc_b + so + (PHASE == 1 ? 0 : s * (P.b_piece >> 4));
            const uint32_t dd = PHASE == 1 ? d + s * H.ncols : d;
            const uint32_t sfa = sf + s * C::kSub * 4;
            const uint32_t sfb = sf + (PHASE == 1 ? C::kSub * 8 : (H.ns + s) * C::kSub * 4);
            const bool fresh = kb == S.kb0 && (PHASE == 1 || s == 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j * C::kPerMma >= left) break;
              // the scale bytes of an MMA's K range: e4m3 block j of its atom, e2m1 a pair of blocks
              const uint32_t id = FMT == kE4M3 ? j : 2 * (j & 1), at = FMT == kE2M1 ? 4 * (j >> 1) : 0;
              mma_if<FMT>(one, dd, ad + 2 * j, bd + 2 * j, FMT == 0 ? idesc : idesc | idesc_sf_ids(id, id), sfa + at,
                          sfb + at, !(fresh && j == 0));
            }
          }
          if (one) mma_commit(smem_u32(&empty[stage]));
          __syncwarp();
          advance();
        }
        if (aborted) break;
        if (lane == 0) mma_commit(smem_u32(&tfull[acc]));
        __syncwarp();
        if (++acc == H.nacc) { acc = 0; acc_phase ^= 1u; }
        p += S.kb1 - S.kb0;
      }
    };
    multiply(Phase1(), plan1);
    multiply(Phase2(), plan2);
    if (aborted && lane == 0) {
      mma_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
  } else if (C::kCopier && warp == 6) {
    // ------------------------------------------------------------ scale copier: a stage's atoms -> tensor memory
    auto copy = [&](auto ph, const Plan& P) {
      constexpr int PHASE = decltype(ph)::value;
      const int natom = a.ph[PHASE - 1].red >> 7;
      // groups of atoms: phase 1 gate, up, tokens; phase 2 weights, tokens
      const int per = PHASE == 1 ? C::kSub : H.ns * C::kSub;
      const uint64_t ds0 = smem_desc(smem0 + P.sf_off, 0, 128, kSwizzleNone);
      for (int p = P.p0; p < P.p1 && !aborted;) {
        const Seg S = seg_at<PHASE>(P, p);
        for (int kb = S.kb0; kb < S.kb1; ++kb) {
          if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
          tc_fence_after();
          if (lane == 0) {
            fence_proxy_async_smem();  // the token operand's and its scales' cp.async writes
            const uint64_t ds = ds0 + ((uint64_t)(stage * H.stage_bytes) >> 4);
            const uint32_t sf = tmem_base + H.sf_col0 + stage * H.sf_per;
            const int nat = min(per, natom - kb * per);
            for (int g = 0; g < (PHASE == 1 ? 3 : 2); ++g)
              for (int i = 0; i < nat; ++i) tmem_cp_32x128b_x4(sf + 4 * (g * per + i), ds + (((g * per + i) * 512) >> 4));
            mma_commit(smem_u32(&sfull[stage]));
          }
          __syncwarp();
          advance();
        }
        p += S.kb1 - S.kb0;
      }
    };
    copy(Phase1(), plan1);
    copy(Phase2(), plan2);
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
    const int64_t lo_off = FMT == 0 ? a.act_lo - a.act : 0;
    auto load = [&](auto ph, const Plan& P) {
      constexpr int PHASE = decltype(ph)::value;
      const DecodePhase& F = a.ph[PHASE - 1];
      const int natom = F.red >> 7;
      const int64_t sb_ld = F.red >> 5;
      for (int p = P.p0; p < P.p1 && !aborted;) {
        const Seg S = seg_at<PHASE>(P, p);
        const int off = s_off[S.slot], n = s_off[S.slot + 1] - off;
        const uint32_t lo_place = (uint32_t)((n + 7) & ~7) * 128;
        auto row_of = [&](int r) -> int64_t { return PHASE == 1 ? (int64_t)s_tok[off + r] : (int64_t)(off + r); };
        // the first rows' sources stay in registers over the segment
        const uint8_t* src[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          src[i] = F.b + (r0 + i * kRows < n ? row_of(r0 + i * kRows) : 0) * F.b_ld + j * 16;
        const uint8_t* ssrc = C::kSub ? F.sb + (sid < n ? row_of(sid) : 0) * sb_ld : nullptr;
        const uint32_t splace = (sid & 31) * 16 + (sid >> 5) * 4;  // row r's scales: word 4 (r % 32) + r / 32
        for (int kb = S.kb0; kb < S.kb1; ++kb) {
          if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
          const uint32_t st = smem0 + stage * H.stage_bytes;
#pragma unroll
          for (int s = 0; s < PHASE; ++s) {
            const int kk = PHASE == 1 ? kb : kb * H.ns + s;
            if (PHASE == 2 && (s == H.ns || kk * C::kBK >= F.red)) break;
            const int kbyte = kk * 128;
            const uint32_t size = kbyte + j * 16 < F.b_ld ? 16u : 0u;  // past the end of K: zeros
            const int go = size ? kbyte : -j * 16;
            const uint32_t dst = st + P.b_off + s * P.b_piece + place;
            auto fetch = [&](const uint8_t* from, uint32_t to) {
              cp_async_16(to, from + go, size);
              if (PHASE == 2 && FMT == 0) cp_async_16(to + lo_place, from + lo_off + go, size);
            };
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
              if (r0 + i * kRows >= n) break;
              fetch(src[i], dst + i * kStep);
            }
            for (int i = kHeld; r0 + i * kRows < n; ++i)
              fetch(F.b + row_of(r0 + i * kRows) * F.b_ld + j * 16, dst + i * kStep);
            if (C::kSub && sid < n) {
              const uint32_t ssf = st + P.sf_off + (PHASE == 1 ? 2 * C::kSub : (H.ns + s) * C::kSub) * 512 + splace;
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
        p += S.kb1 - S.kb0;
      }
    };
    load(Phase1(), plan1);
    // A is complete when every CTA has finished phase 1 (all are resident: a cooperative launch)
    if (!aborted && plan2.p0 < plan2.p1) {
      const uint64_t t0 = globaltimer();
      while (load_acquire(a.done) != gridDim.x && !aborted) {
        if (s_ctl->abort) aborted = true;
        else if (globaltimer() - t0 > s_ctl->limit_ns) s_ctl->abort = 1;
      }
      aborted = __any_sync(0xffffffffu, aborted);
    }
    load(Phase2(), plan2);
    cp_async_wait_all();  // nothing of this warp's lands after the block exits
  } else {
    // ------------------------------------------------------------ epilogue (warps 2 .. 5)
    const int q = warp & 3, row = q * 32 + lane;  // accumulator row of this thread
    int acc = 0;
    uint32_t acc_phase = 0;

    // Arrive at a divided item after writing this CTA's partial sums; true in the last CTA.
    // (The barriers order the warps' writes and reads around one thread's fences.)
    auto join = [&](unsigned* cnt, int c_first, int c_last) {
      epi_sync();
      if (threadIdx.x == 64) {
        const unsigned last = (unsigned)(c_last - c_first);
        __threadfence();
        *s_last = atomicInc(cnt + c_first, last) == last;  // wraps to 0: ready for the next launch
        __threadfence();
      }
      epi_sync();
      return *s_last != 0;
    };
    // Partial sums of an item: CTA c keeps those of an item that begins in its run (`begins`: it is the
    // first of the CTAs) apart from those of the item that its run enters in the middle.
    const int t16 = (a.T + 15) & ~15;
    auto part_of = [&](int c, bool begins, int rows) { return a.part + (int64_t)(c * 2 + begins) * rows * t16; };
    auto release = [&]() {  // the accumulator has been read
      tc_fence_before();
      mbar_arrive(smem_u32(&tempty[acc]));
      if (++acc == H.nacc) { acc = 0; acc_phase ^= 1u; }
    };
    // The accumulator of the next segment, or false when the pipeline has given up.
    auto next = [&]() {
      if (!epi_all(warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl))) {
        aborted = true;
        return false;
      }
      tc_fence_after();
      return true;
    };

    // The activations of this thread's row for kBatch entries from r on, of which m exist: a batch is
    // computed whole, so that its exponentials, maxima and conversions overlap.
    auto finish = [&](int r, int m, int out_row, const float* g, const float* u) {
      float v[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        float gate = g[c], up = u[c];
        if (a.limit > 0.0f) {  // NaN stays NaN
          gate = gate > a.limit ? a.limit : gate;
          up = up > a.limit ? a.limit : (up < -a.limit ? -a.limit : up);
        }
        v[c] = silu_f(gate) * up;
      }
      const int64_t at = (int64_t)r * a.I + out_row;
      if (FMT == 0) {
        if (out_row >= a.I) return;
        __nv_bfloat16* act = reinterpret_cast<__nv_bfloat16*>(a.act) + at;
        __nv_bfloat16* act_lo = reinterpret_cast<__nv_bfloat16*>(a.act_lo) + at;
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          // A as the sum of two bf16 numbers (16 mantissa bits): both are multiplied
          const __nv_bfloat16 hi = __float2bfloat16_rn(v[c]);
          const float left = v[c] - __bfloat162float(hi);
          if (c < m) {
            act[(int64_t)c * a.I] = hi;
            act_lo[(int64_t)c * a.I] = __float2bfloat16_rn(fabsf(left) < INFINITY ? left : 0.0f);
          }
        }
      } else {
        // the warp's 32 rows are one MX block of each entry
        uint32_t sc[kBatch];
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(v[c]) & 0x7FFFFFFFu);
          float mult;
          const bool fin = block_scale_f32<FMT == 0 ? kE4M3 : FMT>(am, sc[c], mult);
          v[c] = fin ? v[c] * mult : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const int64_t e = at + (int64_t)c * a.I;
          if (FMT == kE4M3) {
            if (c < m) a.act[e] = (uint8_t)cvt_e4m3x2(v[c], 0.0f);
          } else {
            const float y = __shfl_down_sync(0xffffffffu, v[c], 1);
            if (c < m && (lane & 1) == 0) a.act[e >> 1] = (uint8_t)cvt_e2m1x2(v[c], y);
          }
          if (c < m && lane == 0) a.act_scales[e >> 5] = (uint8_t)sc[c];
        }
      }
    };

    for (int p = plan1.p0; p < plan1.p1;) {
      const Seg S = seg_at<1>(plan1, p);
      const int off = s_off[S.slot], n = s_off[S.slot + 1] - off;
      const int out_row = S.tile * 128 + row;
      if (!next()) break;
      const uint32_t tb = tmem_base + acc * H.acc_cols + ((uint32_t)(q * 32) << 16);
      const bool whole = S.kb0 == 0 && S.kb1 == plan1.nk;
      bool write = whole;
      int c_first = cta, c_last = cta;
      if (!whole) {
        float* mine = part_of(cta, S.kb0 == 0, 256);
        for (int c0 = 0; c0 < n; c0 += 16) {
          float g[16], u[16];
          tmem_ld16(tb + c0, g);
          tmem_ld16(tb + H.ncols + c0, u);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c < n) {
              mine[(c0 + c) * 256 + row] = g[c];
              mine[(c0 + c) * 256 + 128 + row] = u[c];
            }
          }
        }
        release();
        c_first = plan1.owner(S.item * plan1.L);
        c_last = plan1.owner(S.item * plan1.L + plan1.L - 1);
        write = join(a.cnt, c_first, c_last);
      }
      if (write) {
        for (int c0 = 0; c0 < n; c0 += 16) {
          float g[16], u[16];
          if (whole) {
            tmem_ld16(tb + c0, g);
            tmem_ld16(tb + H.ncols + c0, u);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) g[c] = u[c] = 0.0f;
            for (int x = c_first; x <= c_last; ++x) {
              const float* o = part_of(x, x == c_first, 256) + c0 * 256 + row;
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                if (c0 + c < n) {
                  g[c] += __ldcg(o + c * 256);
                  u[c] += __ldcg(o + c * 256 + 128);
                }
              }
            }
          }
#pragma unroll
          for (int b = 0; b < 16; b += kBatch) {
            if (c0 + b >= n) break;
            finish(off + c0 + b, min(kBatch, n - c0 - b), out_row, &g[b], &u[b]);
          }
        }
      }
      if (whole) release();
      p += S.kb1 - S.kb0;
    }
    // this CTA's part of A is written (or it has given up, which the others must not wait for)
    epi_sync();
    if (threadIdx.x == 64) {
      __threadfence();
      atomicAdd(a.done, 1u);
    }

    for (int p = plan2.p0; p < plan2.p1 && !aborted;) {
      const Seg S = seg_at<2>(plan2, p);
      const int off = s_off[S.slot], n = s_off[S.slot + 1] - off;
      const int p_end = p + S.kb1 - S.kb0;
      const int item0 = S.item * plan2.L, item1 = item0 + plan2.L;
      if (p == plan2.p0 || p == item0)
        for (int t = 0; t < a.T; ++t) s_acc[t * 128 + row] = 0.0f;
      if (!next()) break;
      const uint32_t tb = tmem_base + acc * H.acc_cols + ((uint32_t)(q * 32) << 16);
      const int lo = (n + 7) & ~7;  // bf16: the column of the first low part
      for (int c0 = 0; c0 < n; c0 += 16) {
        float v[16];
        tmem_ld16(tb + c0, v);
        if (FMT == 0) {
          float left[16];
          tmem_ld16(tb + lo + c0, left);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += left[c];
        }
#pragma unroll
        for (int b = 0; b < 16; b += kBatch) {
          if (c0 + b >= n) break;
          float* at[kBatch];  // an expert's tokens differ, so a batch's sums are apart
          float sum[kBatch];
#pragma unroll
          for (int c = 0; c < kBatch; ++c) {
            const int r = off + min(c0 + b + c, n - 1);
            at[c] = s_acc + s_tok[r] * 128 + row;
            sum[c] = *at[c] + s_w[r] * v[b + c];
          }
#pragma unroll
          for (int c = 0; c < kBatch; ++c)
            if (c0 + b + c < n) *at[c] = sum[c];
        }
      }
      release();
      if (p_end == plan2.p1 || p_end == item1) {  // this CTA's part of the output tile is complete
        const int out_row = S.tile * 128 + row, rows = a.ph[1].rows;
        if (plan2.p0 <= item0 && p_end == item1) {
          if (out_row < rows)
            for (int t = 0; t < a.T; ++t)
              a.out[(int64_t)t * rows + out_row] = __float2bfloat16_rn(s_acc[t * 128 + row]);
        } else {
          const int c_first = plan2.owner(item0), c_last = plan2.owner(item1 - 1);
          float* mine = part_of(cta, plan2.p0 <= item0, 128);
          for (int t = 0; t < a.T; ++t) mine[t * 128 + row] = s_acc[t * 128 + row];
          if (join(a.cnt + kMaxCtas, c_first, c_last)) {
            // a warp takes four tokens at a time, a lane four rows of each; eight loads in flight
            const float4* first = reinterpret_cast<const float4*>(part_of(c_first, true, 128)) + lane;
            const float4* rest = reinterpret_cast<const float4*>(part_of(0, false, 128)) + lane;
            const int step = 2 * 128 / 4 * t16;  // float4s from a CTA's partial sums to the next CTA's
            for (int t0 = (warp - 2) * 4; t0 < a.T; t0 += 16) {
              float4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = t0 + i < a.T ? __ldcg(first + (t0 + i) * 32) : make_float4(0, 0, 0, 0);
#pragma unroll 2
              for (int x = c_first + 1; x <= c_last; ++x) {
                const float4* o = rest + (int64_t)x * step;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (t0 + i >= a.T) break;
                  const float4 w4 = __ldcg(o + (t0 + i) * 32);
                  v[i].x += w4.x; v[i].y += w4.y; v[i].z += w4.z; v[i].w += w4.w;
                }
              }
              const int r4 = S.tile * 128 + 4 * lane;
              if (r4 < rows)  // rows is a multiple of 8
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (t0 + i < a.T)
                    *reinterpret_cast<uint2*>(a.out + (int64_t)(t0 + i) * rows + r4) =
                        make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
            }
          }
        }
      }
      p = p_end;
    }
  }

  if (aborted && lane == 0) set_error(a.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // the last CTA to leave clears the count that the others have waited on
  if (threadIdx.x == 0 && atomicInc(a.done + 1, gridDim.x - 1) == gridDim.x - 1) atomicExch(a.done, 0u);
}

// ---------------------------------------------------------------- workspace
// [counters of both phases, CTAs done and left][partial sums][A: bf16 high and low parts, or codes and scales]
struct DecodeWs {
  size_t part, act, act_lo, act_scales, bytes;
};
DecodeWs decode_ws(int fmt, int64_t T, int k, int64_t I) {
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  const size_t rows = (size_t)T * k;
  const size_t row = fmt == 0 ? (size_t)I * 2 : fmt == PGG_FMT_E4M3 ? (size_t)I : (size_t)I / 2;
  DecodeWs w;
  w.part = up((2 * kMaxCtas + 2) * sizeof(unsigned));
  w.act = w.part + up((size_t)kMaxCtas * 2 * 256 * ((T + 15) / 16 * 16) * sizeof(float));
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

template <int FMT>
int run_decode(const uint8_t* X, const uint8_t* xs, const int32_t* ids, const float* w, const void* W1,
               const uint8_t* w1s, const void* W2, const uint8_t* w2s, void* out, int64_t T, int k, int64_t H,
               int64_t I, int E, float limit, uint8_t* ws, int32_t* err, cudaStream_t s) {
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
    uint64_t d[3] = {elems(I), (uint64_t)H, (uint64_t)E};
    uint64_t sb[2] = {bytes(I), bytes(I) * (uint64_t)H};
    uint32_t b[3] = {bx, 128, 1};
    if ((st = encode_tmap(&t2, dt, 3, W2, d, sb, b, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  }
  DecodeArgs a{};
  a.ids = ids;
  a.w = w;
  a.T = (int)T;
  a.k = k;
  a.E = E;
  a.I = (int)I;
  a.limit = limit;
  a.ph[0] = {(int)I, (int)H, X, (int64_t)bytes(H), xs, w1s};
  a.ph[1] = {(int)H, (int)I, ws + L.act, (int64_t)bytes(I), ws + L.act_scales, w2s};
  a.act = ws + L.act;
  a.act_lo = ws + L.act_lo;
  a.act_scales = ws + L.act_scales;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.done = a.cnt + 2 * kMaxCtas;
  a.err = err;
  a.slots_cap = std::min(E, a.T * k);
  const size_t lists = 512 + (size_t)a.T * 512 + (size_t)a.T * k * 4 + 2 * (2 * (size_t)a.slots_cap + 1) +
                       (size_t)a.T * k;
  // the whole of an SM's shared memory, so that a CTA has its SM and the tensor memory to itself
  const size_t smem = dev.smem_optin;
  a.ring_bytes = (int)((smem - 1024 - lists) / 1024 * 1024);
  auto kern = moe_decode_kernel<FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min(dev.sms, kMaxCtas));
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

int pgg_mx_moe_decode(int fmt, const uint8_t* X, const uint8_t* SX, const int32_t* topk_ids, const float* w,
                      const uint8_t* W1, const uint8_t* SW1, const uint8_t* W2, const uint8_t* SW2, void* out,
                      int64_t T, int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes,
                      int32_t* err, void* stream) {
  if (fmt != PGG_FMT_E4M3 && fmt != PGG_FMT_E2M1) return PGG_ERR_INVALID_ARG;
  const int st = check_decode(fmt, X, topk_ids, w, W1, W2, out, T, k, H, I, E, swiglu_limit, ws, ws_bytes, err);
  if (st || T == 0) return st;
  if (!SX || !SW1 || !SW2) return PGG_ERR_INVALID_ARG;
  if (!aligned_to(SX, 4) || !aligned_to(SW1, 16) || !aligned_to(SW2, 16)) return PGG_ERR_ALIGNMENT;
  auto go = fmt == PGG_FMT_E4M3 ? run_decode<kE4M3> : run_decode<kE2M1>;
  return go(X, SX, topk_ids, w, W1, SW1, W2, SW2, out, T, k, H, I, E, swiglu_limit, static_cast<uint8_t*>(ws), err,
            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// A whole expert layer for a few tokens, in two kernels:
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
// register.  The stages of all tiles of the batch form one sequence that is cut into equal runs,
// one per CTA, so every SM reads the same number of bytes whatever the routing; a tile that a cut
// divides is put together from fp32 partial sums by the last of its CTAs to arrive, in CTA order
// (the result does not depend on which one that is).
//
// Every CTA builds the batch's expert list by itself from the ids: a bit per (expert, token), so
// an expert named twice by a token is computed once and its weights are added up.
#include <algorithm>

#include "block.cuh"
#include "epilogue.cuh"
#include "sched.cuh"

namespace pgg {
namespace {

constexpr int kMaxT = PGG_MOE_DECODE_MAX_T;
constexpr int kMaxCtas = 192;   // CTAs of a launch (one per SM); sizes the workspace without a device
constexpr int kMaxStages = 8;
constexpr int kLoadWarps = 2;   // warps that fetch the token operand
constexpr int kTileBytes = 128 * 128;  // 128 rows x one 128-byte swizzle atom of K

template <int FMT>
struct DecCfg {
  static constexpr int kBK = FMT == 0 ? 64 : FMT == kE4M3 ? 128 : 256;  // elements in 128 bytes
  static constexpr int kSub = FMT == 0 ? 0 : kBK / 128;                  // scale atoms of them
  static constexpr int kPerMma = kBK / 4;
  static constexpr int kCopier = FMT != 0;
  static constexpr int kThreads = 32 * (6 + kCopier + kLoadWarps);
};

struct DecodeArgs {
  const int32_t* ids;  // [T, k]
  const float* w;      // [T, k] or nullptr
  int T, k, E;
  int rows;            // output rows per expert: I (phase 1), H (phase 2)
  int red;             // reduction length: H (phase 1), I (phase 2)
  int I;
  float limit;
  const uint8_t* b;     // token operand: X (phase 1) or A (phase 2), row-major
  const uint8_t* b_lo;  // phase 2, bf16: the part of A that its bf16 rounding left over
  int64_t b_ld;         // bytes of a row
  const uint8_t* sb;    // its scales, row-major, sb_ld bytes a row
  int64_t sb_ld;
  const uint8_t* sa;    // the weights' blocked scales
  uint8_t* act;         // phase 1 output (and act_lo / act_scales)
  uint8_t* act_lo;
  uint8_t* act_scales;
  __nv_bfloat16* out;   // phase 2 output [T, H]
  float* part;          // partial sums: 2 tiles per CTA
  unsigned* cnt;        // arrivals at a divided tile, by its first CTA; zero between launches
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
// Wait until the kernels that this launch depends on have completed and their writes are visible
// (returns at once when it was not launched as their dependent).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// How a launch cuts up its work; every CTA computes the same.
struct Plan {
  int n_act;    // experts that the batch names
  int ncols;    // most tokens of one of them, rounded up to 16
  int ns;       // phase 2: 128-byte K pieces per stage
  int nk;       // stages of one (expert, tile)
  int L;        // stages of one item: an (expert, tile) in phase 1, an output tile in phase 2
  int total;    // stages of the launch
  int ctas;     // CTAs that get any
  int quot, rem;  // total = ctas quot + rem: the first rem CTAs get a stage more
  int stages;   // ring depth
  int stage_bytes, b_off, b_piece, sf_off;  // layout of a stage
  int acc_cols, nacc, sf_col0, sf_per;  // tensor memory
  __device__ __forceinline__ int start(int c) const { return c * quot + min(c, rem); }
  // the CTA that stage p belongs to
  __device__ __forceinline__ int owner(int p) const {
    const int big = rem * (quot + 1);
    return p < big ? p / (quot + 1) : rem + (p - big) / quot;
  }
};

template <int FMT, int PHASE>
__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, int n_act, int max_n) {
  using C = DecCfg<FMT>;
  Plan P;
  P.n_act = n_act;
  P.ncols = (max_n + 15) & ~15;
  const int tiles = (a.rows + 127) / 128;
  const int kb = (a.red + C::kBK - 1) / C::kBK;
  const int bsub = P.ncols * 128 * (PHASE == 2 && FMT == 0 ? 2 : 1);
  P.b_piece = bsub;
  if (PHASE == 1) {
    P.ns = 1;
    P.nk = kb;
    P.b_off = 2 * kTileBytes;
    P.sf_off = P.b_off + bsub;
    P.stage_bytes = (P.sf_off + C::kSub * 3 * 512 + 1023) & ~1023;
    P.sf_per = C::kSub * 12;
    P.acc_cols = 2 * P.ncols;
  } else {
    // two K pieces a stage, or one where many tokens would leave fewer than three stages
    const int two = (2 * (kTileBytes + bsub + C::kSub * 1024) + 1023) & ~1023;
    P.ns = a.ring_bytes / two >= 3 ? 2 : 1;
    P.nk = (kb + P.ns - 1) / P.ns;
    P.b_off = P.ns * kTileBytes;
    P.sf_off = P.b_off + P.ns * bsub;
    P.stage_bytes = (P.sf_off + P.ns * C::kSub * 1024 + 1023) & ~1023;
    P.sf_per = P.ns * C::kSub * 8;
    P.acc_cols = P.ncols * (FMT == 0 ? 2 : 1);
  }
  P.stages = min(kMaxStages, a.ring_bytes / max(P.stage_bytes, 1));
  P.nacc = 2 * P.acc_cols + P.stages * P.sf_per <= 512 ? 2 : 1;
  P.sf_col0 = P.nacc * P.acc_cols;
  P.L = PHASE == 1 ? P.nk : n_act * P.nk;
  P.total = n_act * tiles * P.nk;
  P.ctas = max(1, min((int)gridDim.x, P.total));
  P.quot = P.total / P.ctas;
  P.rem = P.total - P.ctas * P.quot;
  return P;
}

// A run of stages [kb0, kb1) of one (expert slot, tile); `item` is what partial sums are joined by.
struct Seg {
  int slot, tile, item, kb0, kb1;
};

template <int PHASE>
__device__ __forceinline__ Seg seg_at(const Plan& P, int tiles, int p, int p1) {
  Seg s;
  s.item = p / P.L;
  const int q = p - s.item * P.L;
  if (PHASE == 1) {
    s.slot = s.item / tiles;
    s.tile = s.item - s.slot * tiles;
    s.kb0 = q;
  } else {
    s.tile = s.item;
    s.slot = q / P.nk;
    s.kb0 = q - s.slot * P.nk;
  }
  s.kb1 = min(P.nk, s.kb0 + (p1 - p));
  return s;
}

template <int FMT, int PHASE>
__global__ void __launch_bounds__(DecCfg<FMT>::kThreads, 1)
    moe_decode_kernel(const __grid_constant__ CUtensorMap tmW, const DecodeArgs a) {
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
  float* s_w = s_acc + (PHASE == 2 ? a.T * 128 : 0);                    // phase 2: [T k]
  uint16_t* s_off = reinterpret_cast<uint16_t*>(s_w + (PHASE == 2 ? a.T * a.k : 0));  // [slots + 1]
  uint16_t* s_exp = s_off + a.slots_cap + 1;                                         // [slots]
  uint8_t* s_tok = reinterpret_cast<uint8_t*>(s_exp + a.slots_cap);                  // [T k]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (PHASE == 1) grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1 + 32 * kLoadWarps);
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&sfull[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&tfull[s]), 1);
      mbar_init(smem_u32(&tempty[s]), 128);
    }
    mbar_init(smem_u32(drain), 1);
    mbar_init(smem_u32(cdrain), 1);
    s_ctl->abort = 0;
    s_ctl->limit_ns = kWaitTimeoutNs;
    fence_mbar_init();
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }

  // ---- the batch's experts and their tokens (scratch: the ring, before the first stage lands)
  const int W = (a.T + 31) / 32;  // mask words per expert
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem);                  // [E][W]
  uint16_t* s_eoff = reinterpret_cast<uint16_t*>(s_mask + a.E * W);      // [E]: first entry
  const int n_ids = a.T * a.k;
  for (int i = threadIdx.x; i < a.E * W; i += kNT) s_mask[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n_ids; i += kNT) {
    const int e = __ldg(a.ids + i), t = i / a.k;
    if (e < 0 || e >= a.E) {
      if (blockIdx.x == 0) set_error(a.err, kErrBadExpert);
    } else {
      atomicOr(&s_mask[e * W + (t >> 5)], 1u << (t & 31));
    }
  }
  __syncthreads();
  int n_act, max_n;
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
    const int e = __ldg(a.ids + i);
    if (e < 0 || e >= a.E) continue;
    const int t = i / a.k, i0 = t * a.k;
    bool first = true;  // the token's first choice of this expert writes the entry
    for (int j = i0; j < i; ++j) first &= __ldg(a.ids + j) != e;
    if (!first) continue;
    int r = s_eoff[e];
    for (int q = 0; q < (t >> 5); ++q) r += __popc(s_mask[e * W + q]);
    r += __popc(s_mask[e * W + (t >> 5)] & ((1u << (t & 31)) - 1u));
    s_tok[r] = (uint8_t)t;
    if (PHASE == 2) {
      float wt = 0.0f;
      for (int j = i; j < i0 + a.k; ++j)
        if (__ldg(a.ids + j) == e) wt += a.w ? __ldg(a.w + j) : 1.0f;
      s_w[r] = wt;
    }
  }
  fence_proxy_async_smem();  // the ring's scratch use, before its first bulk copies
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const Plan P = make_plan<FMT, PHASE>(a, n_act, max_n);
  const int tiles = (a.rows + 127) / 128;
  const int cta = blockIdx.x;
  const int p0 = cta < P.ctas && P.total ? P.start(cta) : 0;
  const int p1 = cta < P.ctas && P.total ? P.start(cta + 1) : 0;
  const uint32_t tmem_base = *s_tmem;
  const uint32_t smem0 = smem_u32(smem);
  bool aborted = false;
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++stage == P.stages) { stage = 0; phase ^= 1u; }
  };

  if (PHASE == 2 && P.total == 0) {  // no expert is named: the layer's output is zero
    for (int64_t i = (int64_t)cta * kNT + threadIdx.x; i < (int64_t)a.T * a.rows; i += (int64_t)gridDim.x * kNT)
      a.out[i] = __float2bfloat16_rn(0.0f);
  }

  if (warp == 0) {
    // ------------------------------------------------------------ weights: TMA tiles, bulk scale atoms
    long long issued = 0;
    for (int p = p0; p < p1 && !aborted;) {
      const Seg S = seg_at<PHASE>(P, tiles, p, p1);
      const int e = s_exp[S.slot], row0 = S.tile * 128;
      for (int kb = S.kb0; kb < S.kb1; ++kb) {
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        if (lane == 0) {
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t st = smem0 + stage * P.stage_bytes;
          const int natom = a.red >> 7;  // MX: scale atoms of a 128-row block along K
          if (PHASE == 1) {
            const int at0 = kb * C::kSub, nat = C::kSub ? min(C::kSub, natom - at0) : 0;
            mbar_arrive_expect_tx(fb, 2 * kTileBytes + 2 * 512 * nat);
            const int x = kb * (FMT == 0 ? 64 : 128);
            tma_load_4d(st, &tmW, fb, x, row0, 0, e);
            tma_load_4d(st + kTileBytes, &tmW, fb, x, row0, 1, e);
            if (C::kSub) {
              const int64_t rg = ((int64_t)e * 2 * a.I + row0) >> 7, ru = ((int64_t)e * 2 * a.I + a.I + row0) >> 7;
              bulk_load(st + P.sf_off, a.sa + (rg * natom + at0) * 512, 512 * nat, fb);
              bulk_load(st + P.sf_off + C::kSub * 512, a.sa + (ru * natom + at0) * 512, 512 * nat, fb);
            }
          } else {
            const int at0 = kb * P.ns * C::kSub, nat = C::kSub ? min(P.ns * C::kSub, natom - at0) : 0;
            const int kk0 = kb * P.ns, nsub = min(P.ns, (a.red - kk0 * C::kBK + C::kBK - 1) / C::kBK);
            mbar_arrive_expect_tx(fb, nsub * kTileBytes + 512 * nat);
            for (int s = 0; s < nsub; ++s)
              tma_load_3d(st + s * kTileBytes, &tmW, fb, (kk0 + s) * (FMT == 0 ? 64 : 128), row0, e);
            if (C::kSub)
              bulk_load(st + P.sf_off, a.sa + ((((int64_t)e * a.rows + row0) >> 7) * natom + at0) * 512, 512 * nat, fb);
          }
        }
        __syncwarp();
        ++issued;
        advance();
      }
      p += S.kb1 - S.kb0;
    }
    if (aborted && lane == 0) {
      // drain: the copies in flight land before the CTA's shared memory goes away.  Their full
      // barriers may lack the token loaders' arrivals, so this may run to its own limit.
      long long n = issued < P.stages ? issued : P.stages;
      for (long long i = 0; i < n; ++i) {
        if (--stage < 0) { stage = P.stages - 1; phase ^= 1u; }
        mbar_wait_drain(smem_u32(&full[stage]), phase);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int acc = 0;
    uint32_t acc_phase = 0;
    // descriptors of stage 0's tiles; an address d bytes further on adds d / 16
    const uint64_t desc_a = smem_desc(smem0, 16, 1024, kSwizzle128B);
    const uint64_t desc_b = smem_desc(smem0 + P.b_off, 16, 1024, kSwizzle128B);
    for (int p = p0; p < p1 && !aborted;) {
      const Seg S = seg_at<PHASE>(P, tiles, p, p1);
      const uint32_t n16 = (uint32_t)((s_off[S.slot + 1] - s_off[S.slot] + 15) & ~15);
      const uint32_t N = PHASE == 2 && FMT == 0 ? 2 * n16 : n16;
      const uint32_t idesc = FMT == 0 ? idesc_bf16(128, N, false, false) : idesc_mx(FMT == kE4M3 ? 0 : 1, 128, N);
      if (!warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, s_ctl)) { aborted = true; break; }
      tc_fence_after();
      const uint32_t d = tmem_base + acc * P.acc_cols;
      for (int kb = S.kb0; kb < S.kb1; ++kb) {
        if (!warp_wait(smem_u32(C::kCopier ? &sfull[stage] : &full[stage]), phase, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        if (lane == 0) {
          if (!C::kCopier) fence_proxy_async_smem();  // the token operand's cp.async writes
          const uint64_t so = (uint64_t)(stage * P.stage_bytes) >> 4;
          const uint32_t sf = tmem_base + P.sf_col0 + stage * P.sf_per;
#pragma unroll
          for (int s = 0; s < 2; ++s) {  // phase 1: gate and up; phase 2: K pieces
            if (PHASE == 2 && s == P.ns) break;
            const int kk = PHASE == 1 ? kb : kb * P.ns + s;
            // MMAs of this piece that hold data (an e2m1 K may end inside it; the zero-filled end
            // of a bf16 K adds nothing)
            const int left = a.red - kk * C::kBK;
            const uint64_t ad = desc_a + so + s * (kTileBytes >> 4);
            const uint64_t bd = desc_b + so + (PHASE == 1 ? 0 : s * (P.b_piece >> 4));
            const uint32_t dd = PHASE == 1 ? d + s * P.ncols : d;
            const uint32_t sfa = sf + s * C::kSub * 4;
            const uint32_t sfb = sf + (PHASE == 1 ? C::kSub * 8 : (P.ns + s) * C::kSub * 4);
            const bool fresh = kb == S.kb0 && (PHASE == 1 || s == 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j * C::kPerMma >= left) break;
              const uint32_t accum = !(fresh && j == 0);
              if (FMT == 0) {
                mma_f16(dd, ad + 2 * j, bd + 2 * j, idesc, accum);
              } else if (FMT == kE4M3) {
                mma_mxf8(dd, ad + 2 * j, bd + 2 * j, idesc | idesc_sf_ids(j, j), sfa, sfb, accum);
              } else {
                const uint32_t id = 2 * (j & 1);
                mma_mxf4(dd, ad + 2 * j, bd + 2 * j, idesc | idesc_sf_ids(id, id), sfa + 4 * (j >> 1),
                         sfb + 4 * (j >> 1), accum);
              }
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
      if (++acc == P.nacc) { acc = 0; acc_phase ^= 1u; }
      p += S.kb1 - S.kb0;
    }
    if (aborted && lane == 0) {
      mma_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
  } else if (C::kCopier && warp == 6) {
    // ------------------------------------------------------------ scale copier: a stage's atoms -> tensor memory
    for (int p = p0; p < p1 && !aborted;) {
      const Seg S = seg_at<PHASE>(P, tiles, p, p1);
      for (int kb = S.kb0; kb < S.kb1; ++kb) {
        if (!warp_wait(smem_u32(&full[stage]), phase, s_ctl)) { aborted = true; break; }
        tc_fence_after();
        if (lane == 0) {
          fence_proxy_async_smem();  // the token operand's and its scales' cp.async writes
          const uint64_t ds = smem_desc(smem0 + stage * P.stage_bytes + P.sf_off, 0, 128, kSwizzleNone);
          const uint32_t sf = tmem_base + P.sf_col0 + stage * P.sf_per;
          // groups of atoms: phase 1 gate, up, tokens; phase 2 weights, tokens
          const int per = PHASE == 1 ? C::kSub : P.ns * C::kSub;
          const int nat = min(per, (a.red >> 7) - kb * per);
          for (int g = 0; g < (PHASE == 1 ? 3 : 2); ++g)
            for (int i = 0; i < nat; ++i) tmem_cp_32x128b_x4(sf + 4 * (g * per + i), ds + (((g * per + i) * 512) >> 4));
          mma_commit(smem_u32(&sfull[stage]));
        }
        __syncwarp();
        advance();
      }
      p += S.kb1 - S.kb0;
    }
    if (aborted && lane == 0) {
      mma_commit(smem_u32(cdrain));
      mbar_wait_drain(smem_u32(cdrain), 0);
    }
  } else if (warp >= kLoadWarp0) {
    // ------------------------------------------------------------ the token operand
    if (PHASE == 2) grid_wait();  // A is phase 1's
    // Thread (r0, j) fetches 16-byte chunk j of rows r0, r0 + 8, ...: chunk j of row r goes to chunk
    // j ^ (r % 8) of its 128 bytes (the 128-byte swizzle), so its places are 1024 bytes apart.
    // Rows past n hold leftovers, which only reach accumulator columns that nobody reads.
    const int tid = threadIdx.x - kLoadWarp0 * 32;
    const int j = tid & 7, r0 = tid >> 3;
    const uint32_t place = r0 * 128 + ((j ^ r0) << 4);
    const int natom = a.red >> 7;
    const int64_t lo_off = PHASE == 2 && FMT == 0 ? a.b_lo - a.b : 0;
    for (int p = p0; p < p1 && !aborted;) {
      const Seg S = seg_at<PHASE>(P, tiles, p, p1);
      const int off = s_off[S.slot], n = s_off[S.slot + 1] - off;
      const uint32_t lo_place = (uint32_t)((n + 15) & ~15) * 128;
      auto row_of = [&](int r) -> int64_t { return PHASE == 1 ? (int64_t)s_tok[off + r] : (int64_t)(off + r); };
      // the first rows' sources stay in registers over the segment
      const uint8_t* src0 = a.b + (r0 < n ? row_of(r0) : 0) * a.b_ld + j * 16;
      const uint8_t* src1 = a.b + (r0 + 8 < n ? row_of(r0 + 8) : 0) * a.b_ld + j * 16;
      const uint8_t* ssrc = C::kSub ? a.sb + (tid < n ? row_of(tid) : 0) * a.sb_ld : nullptr;
      for (int kb = S.kb0; kb < S.kb1; ++kb) {
        if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, s_ctl)) { aborted = true; break; }
        const uint32_t st = smem0 + stage * P.stage_bytes;
#pragma unroll
        for (int s = 0; s < PHASE; ++s) {
          const int kk = kb * P.ns + s;
          if (PHASE == 2 && (s == P.ns || kk * C::kBK >= a.red)) break;
          const int kbyte = kk * 128;
          const uint32_t size = kbyte + j * 16 < a.b_ld ? 16u : 0u;  // past the end of K: zeros
          const int go = size ? kbyte : -j * 16;
          const uint32_t dst = st + P.b_off + s * P.b_piece + place;
          auto fetch = [&](const uint8_t* from, uint32_t to) {
            cp_async_16(to, from + go, size);
            if (PHASE == 2 && FMT == 0) cp_async_16(to + lo_place, from + lo_off + go, size);
          };
          if (r0 < n) fetch(src0, dst);
          if (r0 + 8 < n) fetch(src1, dst + 1024);
          for (int r = r0 + 16; r < n; r += 8) fetch(a.b + row_of(r) * a.b_ld + j * 16, dst + (r - r0) * 128);
          if (C::kSub) {
            // row r's 4 scales of a 128-element atom: word 4 (r % 32) + r / 32
            const uint32_t ssf = st + P.sf_off + (PHASE == 1 ? 2 * C::kSub : (P.ns + s) * C::kSub) * 512;
#pragma unroll
            for (int sub = 0; sub < C::kSub; ++sub) {
              const int at = kk * C::kSub + sub;
              if (at >= natom) break;
              if (tid < n) cp_async_4(ssf + sub * 512 + (tid & 31) * 16 + (tid >> 5) * 4, ssrc + at * 4, 4u);
              for (int r = tid + 32 * kLoadWarps; r < n; r += 32 * kLoadWarps)
                cp_async_4(ssf + sub * 512 + (r & 31) * 16 + (r >> 5) * 4, a.sb + row_of(r) * a.sb_ld + at * 4, 4u);
            }
          }
        }
        cp_async_arrive_noinc(smem_u32(&full[stage]));
        __syncwarp();
        advance();
      }
      p += S.kb1 - S.kb0;
    }
    cp_async_wait_all();  // nothing of this warp's lands after the block exits
  } else if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = q * 32 + lane;  // accumulator row of this thread
    int acc = 0;
    uint32_t acc_phase = 0;
    if (PHASE == 2) grid_wait();  // the partial sums' space and the counters are phase 1's too

    // Arrive at a divided item after writing this CTA's partial sums; true in the last CTA.
    auto join = [&](int item, int c_first, int c_last) {
      __threadfence();
      epi_sync();
      if (threadIdx.x == 64) {
        const unsigned last = (unsigned)(c_last - c_first);
        *s_last = atomicInc(a.cnt + c_first, last) == last;  // wraps to 0: ready for the next launch
        __threadfence();
      }
      epi_sync();
      const bool mine = *s_last != 0;
      epi_sync();
      if (mine) __threadfence();
      return mine;
    };
    // Partial sums of an item: CTA c keeps those of an item that begins in its run (`begins`: it is the
    // first of the CTAs) apart from those of the item that its run enters in the middle.
    const int part_sz = (PHASE == 1 ? 256 : 128) * ((a.T + 15) & ~15);
    auto part_of = [&](int c, bool begins) { return a.part + (int64_t)(c * 2 + begins) * part_sz; };

    for (int p = p0; p < p1 && !aborted;) {
      const Seg S = seg_at<PHASE>(P, tiles, p, p1);
      const int off = s_off[S.slot], n = s_off[S.slot + 1] - off;
      const int p_end = p + S.kb1 - S.kb0;
      const int item0 = S.item * P.L, item1 = item0 + P.L;
      const int out_row = S.tile * 128 + row;
      if (PHASE == 2 && (p == p0 || p == item0))
        for (int t = 0; t < a.T; ++t) s_acc[t * 128 + row] = 0.0f;
      if (!epi_all(warp_wait(smem_u32(&tfull[acc]), acc_phase, s_ctl))) { aborted = true; break; }
      tc_fence_after();
      const uint32_t tb = tmem_base + acc * P.acc_cols + ((uint32_t)(q * 32) << 16);

      if (PHASE == 1) {
        // 16 entries' activations of this thread's row from its gate and up sums
        auto finish = [&](int c0, const float (&g)[16], const float (&u)[16]) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c >= n) break;
            float gate = g[c], up = u[c];
            if (a.limit > 0.0f) {  // NaN stays NaN
              gate = gate > a.limit ? a.limit : gate;
              up = up > a.limit ? a.limit : (up < -a.limit ? -a.limit : up);
            }
            const float v = silu_f(gate) * up;
            const int64_t r = off + c0 + c;
            if (FMT == 0) {
              if (out_row < a.I) {
                // A as the sum of two bf16 numbers (16 mantissa bits): both are multiplied
                const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                const float left = v - __bfloat162float(hi);
                reinterpret_cast<__nv_bfloat16*>(a.act)[r * a.I + out_row] = hi;
                reinterpret_cast<__nv_bfloat16*>(a.act_lo)[r * a.I + out_row] =
                    __float2bfloat16_rn(fabsf(left) < INFINITY ? left : 0.0f);
              }
            } else {
              // the warp's 32 rows are one MX block of this entry
              const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
              uint32_t sc;
              float mult;
              const bool fin = block_scale_f32<FMT == 0 ? kE4M3 : FMT>(am, sc, mult);
              const float x = fin ? v * mult : 0.0f;
              if (FMT == kE4M3) {
                a.act[r * a.I + out_row] = (uint8_t)cvt_e4m3x2(x, 0.0f);
              } else {
                const float y = __shfl_down_sync(0xffffffffu, x, 1);
                if ((lane & 1) == 0) a.act[(r * a.I + out_row) >> 1] = (uint8_t)cvt_e2m1x2(x, y);
              }
              if (lane == 0) a.act_scales[(r * a.I + out_row) >> 5] = (uint8_t)sc;
            }
          }
        };
        const bool whole = S.kb0 == 0 && S.kb1 == P.nk;
        float* mine = part_of(cta, S.kb0 == 0);
        for (int c0 = 0; c0 < n; c0 += 16) {
          float g[16], u[16];
          tmem_ld16(tb + c0, g);
          tmem_ld16(tb + P.ncols + c0, u);
          if (whole) {
            finish(c0, g, u);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (c0 + c >= n) break;
              mine[(c0 + c) * 256 + row] = g[c];
              mine[(c0 + c) * 256 + 128 + row] = u[c];
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&tempty[acc]));
        if (!whole) {
          const int c_first = P.owner(item0), c_last = P.owner(item1 - 1);
          if (join(S.item, c_first, c_last)) {
            for (int c0 = 0; c0 < n; c0 += 16) {
              float g[16], u[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) g[c] = u[c] = 0.0f;
              for (int x = c_first; x <= c_last; ++x) {
                const float* o = part_of(x, x == c_first) + c0 * 256 + row;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  if (c0 + c >= n) break;
                  g[c] += __ldcg(o + c * 256);
                  u[c] += __ldcg(o + c * 256 + 128);
                }
              }
              finish(c0, g, u);
            }
          }
        }
      } else {
        const int n16 = (n + 15) & ~15;
        for (int c0 = 0; c0 < n; c0 += 16) {
          float v[16];
          tmem_ld16(tb + c0, v);
          if (FMT == 0) {
            float lo[16];
            tmem_ld16(tb + n16 + c0, lo);
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] += lo[c];
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c >= n) break;
            s_acc[s_tok[off + c0 + c] * 128 + row] += s_w[off + c0 + c] * v[c];
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&tempty[acc]));
        if (p_end == p1 || p_end == item1) {  // this CTA's part of the output tile is complete
          if (p0 <= item0 && p_end == item1) {
            if (out_row < a.rows)
              for (int t = 0; t < a.T; ++t)
                a.out[(int64_t)t * a.rows + out_row] = __float2bfloat16_rn(s_acc[t * 128 + row]);
          } else {
            const int c_first = P.owner(item0), c_last = P.owner(item1 - 1);
            float* mine = part_of(cta, p0 <= item0);
            for (int t = 0; t < a.T; ++t) mine[t * 128 + row] = s_acc[t * 128 + row];
            if (join(S.item, c_first, c_last)) {
              // a warp takes four tokens at a time, a lane four rows of each; eight loads in flight
              const float4* first = reinterpret_cast<const float4*>(part_of(c_first, true)) + lane;
              const float4* rest = reinterpret_cast<const float4*>(part_of(0, false)) + lane;
              const int step = part_sz / 2;  // float4s from a CTA's partial sums to the next CTA's
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
                if (r4 < a.rows)  // rows is a multiple of 8
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (t0 + i < a.T)
                      *reinterpret_cast<uint2*>(a.out + (int64_t)(t0 + i) * a.rows + r4) =
                          make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
              }
            }
          }
        }
      }
      if (++acc == P.nacc) { acc = 0; acc_phase ^= 1u; }
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
}

// ---------------------------------------------------------------- workspace
// [counters of both phases][partial sums][A: bf16 high and low parts, or codes and scales]
struct DecodeWs {
  size_t cnt, part, act, act_lo, act_scales, bytes;
};
DecodeWs decode_ws(int fmt, int64_t T, int k, int64_t I) {
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  const size_t rows = (size_t)T * k;
  const size_t row = fmt == 0 ? (size_t)I * 2 : fmt == PGG_FMT_E4M3 ? (size_t)I : (size_t)I / 2;
  DecodeWs w;
  w.cnt = 0;
  w.part = up(2 * kMaxCtas * sizeof(unsigned));
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

template <int FMT, int PHASE>
int run_phase(const CUtensorMap& tm, DecodeArgs a, const DeviceInfo& dev, cudaStream_t s) {
  a.slots_cap = std::min(a.E, a.T * a.k);
  const size_t lists = 512 + (PHASE == 2 ? (size_t)a.T * 512 + (size_t)a.T * a.k * 4 : 0) +
                       2 * (2 * (size_t)a.slots_cap + 1) + (size_t)a.T * a.k;
  // the whole of an SM's shared memory, so that a CTA has its SM and the tensor memory to itself
  const size_t smem = dev.smem_optin;
  a.ring_bytes = (int)((smem - 1024 - lists) / 1024 * 1024);
  auto kern = moe_decode_kernel<FMT, PHASE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_status(e);
  kern<<<std::min(dev.sms, kMaxCtas), DecCfg<FMT>::kThreads, smem, s>>>(tm, a);
  return cuda_status(cudaGetLastError());
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
  a.err = err;
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.cnt = reinterpret_cast<unsigned*>(ws + L.cnt);
  DecodeArgs a1 = a;
  a1.rows = (int)I;
  a1.red = (int)H;
  a1.b = X;
  a1.b_ld = (int64_t)bytes(H);
  a1.sb = xs;
  a1.sb_ld = H / 32;
  a1.sa = w1s;
  a1.act = ws + L.act;
  a1.act_lo = ws + L.act_lo;
  a1.act_scales = ws + L.act_scales;
  if ((st = run_phase<FMT, 1>(t1, a1, dev, s))) return st;
  DecodeArgs a2 = a;
  a2.rows = (int)H;
  a2.red = (int)I;
  a2.b = ws + L.act;
  a2.b_lo = ws + L.act_lo;
  a2.b_ld = (int64_t)bytes(I);
  a2.sb = ws + L.act_scales;
  a2.sb_ld = I / 32;
  a2.sa = w2s;
  a2.out = static_cast<__nv_bfloat16*>(out);
  a2.cnt += kMaxCtas;
  return run_phase<FMT, 2>(t2, a2, dev, s);
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

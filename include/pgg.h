/*
 * pgg.h -- C ABI of the GB300 (sm_103a) MoE expert grouped GEMM library.
 *
 * The operation (from "Enabling DeepSeek-V4-Flash Training on AMD Instinct
 * MI355X GPUs with Primus", section "Expert parallelism: DeepEP and the grouped
 * GEMM"): tokens are already sorted by expert; each local expert multiplies its
 * own, different number of tokens by its own weights, and one kernel runs all
 * of the experts' GEMMs over the ragged batch instead of a per-expert loop.
 * The per-expert token counts ("m_splits" in "[Megatron-LM] feat: add grouped
 * gemm fp4 support ... Pull Request #891", review comments) are produced by
 * routing and bounded by the token count; here they are `group_lens`.
 *
 * Notation: G groups (experts), M = sum(group_lens) rows; group g owns rows
 * [off_g, off_g + len_g) with off_0 = 0 and off_{g+1} = off_g + len_g.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers, row-major, densely packed, and
 *    16-byte aligned; "bf16" means IEEE bfloat16 (2 bytes).
 *  - group_lens is a device int32[G]; it is scanned on the device (no host
 *    synchronisation).  1 <= G <= 1024.
 *  - The caller owns and allocates every buffer; the library allocates
 *    nothing and keeps no state beyond pgg_init's device properties.
 *  - Calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL is
 *    the legacy default stream).
 *  - Host-detectable problems (null pointer, bad size, misalignment, an
 *    unsupported format or device) return a non-zero pgg_status and launch
 *    nothing.
 *  - Device-detectable problems (a negative group length, sum(group_lens) !=
 *    M, a bounded wait that expired) write a code to *err (a device int32,
 *    first error wins; may be NULL) and the kernel still terminates, writing
 *    no output for bad group_lens.  Clear *err to 0 before the call.
 *  - Results are deterministic: no floating-point atomics in any reduction.
 */
#ifndef PGG_H_
#define PGG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PGG_OK = 0,
  PGG_ERR_INVALID_ARG = 1,   /* null pointer, non-positive or too large size, bad enum */
  PGG_ERR_UNSUPPORTED = 2,   /* device is not sm_103, or a shape the kernels do not cover */
  PGG_ERR_ALIGNMENT = 3,     /* pointer not 16-byte aligned, or a dimension off its multiple */
  PGG_ERR_NOT_INITIALIZED = 4,
  PGG_ERR_CUDA = 5,          /* a CUDA runtime call failed */
  PGG_ERR_TOO_LARGE = 6,     /* the problem does not fit a no-alloc entry point's fixed scratch */
  /* codes written to the device error word */
  PGG_ERR_BAD_GROUP_LENS = 16, /* some len < 0, or sum(len) != M */
  PGG_ERR_TIMEOUT = 17,        /* a bounded pipeline wait expired; output incomplete */
  PGG_ERR_PAD_OVERFLOW = 18,   /* column-wise MX: sum(round_up(len, 128)) > M_pad */
  PGG_ERR_BAD_EXPERT = 19      /* MoE permute: an expert id outside [0, E) */
} pgg_status;

typedef enum { PGG_FMT_E4M3 = 1, PGG_FMT_E2M1 = 2 } pgg_mx_fmt;
typedef enum { PGG_MODE_FWD = 0, PGG_MODE_DGRAD = 1, PGG_MODE_WGRAD = 2 } pgg_mode;
typedef enum { PGG_EPI_NONE = 0, PGG_EPI_SWIGLU = 1 } pgg_epilogue;

/* Padding granule of the column-wise MX layout (rows per group are rounded up to it). */
#define PGG_MX_PAD 128

/* Library ABI version (major*100 + minor). */
int pgg_version(void);

/* Select `device` and check that it is an sm_103 GPU (compute capability
 * 10.3), caching its SM count.  Called implicitly by every entry point on the
 * current device; calling it first surfaces PGG_ERR_UNSUPPORTED early.  The
 * pages' counterpart is the hardware capability check made when the MXFP4
 * recipe is entered (Pull Request #891, review comments). */
int pgg_init(int device);

/* Static string for a status code. */
const char* pgg_status_string(int status);

/* Copy the device error word to *host_out, synchronising `stream` first. */
int pgg_read_error(const int32_t* err_dev, int32_t* host_out, void* stream);

/* ---------------------------------------------------------------- BF16 */

/* Forward: Y_g = X_g . W_g^T for every group.
 *   X [M, K] bf16, W [G, N, K] bf16 (K contiguous), Y [M, N] bf16 (out).
 *   fp32 accumulation in tensor memory, bf16 round-to-nearest-even output.
 *   K >= 8, K % 8 == 0, N % 8 == 0.  M == 0 is a no-op. */
int pgg_grouped_gemm_fwd(const void* X, const void* W, const int32_t* group_lens, void* Y,
                         int64_t M, int64_t N, int64_t K, int G, int32_t* err, void* stream);

/* Dgrad: dX_g = dY_g . W_g (same grouping, weight used transposed; W is read
 * in place, no transposed copy -- cf. the transposed-weight cache that Pull
 * Request #891, "Changes", stops reusing).
 *   dY [M, N] bf16, W [G, N, K] bf16, dX [M, K] bf16 (out).
 *   N >= 8, N % 8 == 0, K % 8 == 0. */
int pgg_grouped_gemm_dgrad(const void* dY, const void* W, const int32_t* group_lens, void* dX,
                           int64_t M, int64_t N, int64_t K, int G, int32_t* err, void* stream);

/* Variable-K wgrad: dW_g = dY_g^T . X_g, reduced over group g's own len_g
 * rows; a group with len_g == 0 gets dW_g = 0 (the backward emits dW1/dW2:
 * "Enabling DeepSeek-V4-Flash ...", section "MegaMoE", backward order).
 *   X [M, K] bf16, dY [M, N] bf16, dW [G, N, K] bf16 (out, fully written).
 *   N % 8 == 0, K % 8 == 0. */
int pgg_grouped_gemm_wgrad(const void* X, const void* dY, const int32_t* group_lens, void* dW,
                           int64_t M, int64_t N, int64_t K, int G, int32_t* err, void* stream);

/* Variable-K wgrad accumulated into an fp32 gradient buffer ("main_grad"):
 *   dW_f32[g] += dY_g^T . X_g  for every group (an empty group adds nothing).
 * The weight-gradient bridge of "[Megatron-LM] feat: add grouped gemm fp4
 * support ... Pull Request #891", "Changes": the weight gradient is always
 * accumulated into weight.main_grad.  fp32 accumulation in tensor memory; the
 * add into dW_f32 is done by bulk tensor reduce-adds, one add per element per
 * call, so repeated calls (gradient accumulation over micro-batches) are
 * deterministic.
 *   X [M, K] bf16, dY [M, N] bf16, dW_f32 [G, N, K] fp32 (in/out).
 *   N % 8 == 0, K % 8 == 0.  Calls that overlap on the same dW_f32 race. */
int pgg_grouped_gemm_wgrad_accumulate(const void* X, const void* dY, const int32_t* group_lens,
                                      float* dW_f32, int64_t M, int64_t N, int64_t K, int G,
                                      int32_t* err, void* stream);

/* FC1 with SwiGLU folded into the epilogue ("Primus-Turbo" README, "What's
 * New": fused GroupedMLP with SwiGLU folded into the grouped GEMM; weight
 * layout w1 [g, 2I, H] "gate + up" from the MegaMoE section).
 *   H_g = X_g . W1_g^T  [len_g, 2I];  A = silu(H[:, :I]) * H[:, I:]
 *   X [M, K] bf16, W1 [G, 2I, K] bf16 (rows 0..I-1 gate, I..2I-1 up),
 *   A [M, I] bf16 (out), H [M, 2I] bf16 (out, optional: NULL skips it; it is
 *   the pre-activation the backward needs).  silu(x) = x / (1 + exp(-x)),
 *   evaluated in fp32 from the fp32 accumulators.  I % 8 == 0, K % 8 == 0. */
int pgg_grouped_fc1_swiglu(const void* X, const void* W1, const int32_t* group_lens, void* A,
                           void* H, int64_t M, int64_t I, int64_t K, int G, int32_t* err,
                           void* stream);

/* FC2 dgrad with the SwiGLU backward in the epilogue:
 *   dA_g = dY_g . W2_g  [len_g, I];  with g = H[:, :I], u = H[:, I:], s = sigmoid(g):
 *   dH[:, :I] = dA * u * s * (1 + g * (1 - s)),  dH[:, I:] = dA * g * s
 *   dY [M, Hd] bf16, W2 [G, Hd, I] bf16, H [M, 2I] bf16 (saved by FC1),
 *   dH [M, 2I] bf16 (out).  Hd % 8 == 0, I % 8 == 0. */
int pgg_grouped_fc2_dgrad_swiglu_bwd(const void* dY, const void* W2, const void* H,
                                     const int32_t* group_lens, void* dH, int64_t M, int64_t Hd,
                                     int64_t I, int G, int32_t* err, void* stream);

/* Clamped SwiGLU (the `swiglu_limit` knob of "Enabling DeepSeek-V4-Flash ...",
 * model-config table; the pages give no formula -- read here as): with L =
 * swiglu_limit > 0, gate <- min(gate, L) and up <- clamp(up, -L, L) before
 * A = silu(gate) * up.  H keeps the values before the clamp; the backward
 * applies the clamp to them again and passes no gradient where a clamp is
 * active (gate > L, |up| > L).  swiglu_limit == 0 is the plain SwiGLU (the two
 * calls above); a negative or non-finite limit returns PGG_ERR_INVALID_ARG.
 * Arguments otherwise as pgg_grouped_fc1_swiglu / pgg_grouped_fc2_dgrad_swiglu_bwd. */
int pgg_grouped_fc1_swiglu_clamped(const void* X, const void* W1, const int32_t* group_lens, void* A,
                                   void* H, int64_t M, int64_t I, int64_t K, int G, float swiglu_limit,
                                   int32_t* err, void* stream);
int pgg_grouped_fc2_dgrad_swiglu_bwd_clamped(const void* dY, const void* W2, const void* H,
                                             const int32_t* group_lens, void* dH, int64_t M, int64_t Hd,
                                             int64_t I, int G, float swiglu_limit, int32_t* err,
                                             void* stream);

/* ---------------------------------------------------------------- MX (microscaling) */

/* Row-wise MX quantization: one E8M0 scale per block of 32 consecutive
 * elements along C ("Primus-Turbo" README: MXFP8 / MXFP4 grouped GEMM; Pull
 * Request #891, "Changes": MXFP4 weights built as float4_e2m1fn_x2 buffers).
 * Rule (OCP Microscaling v1.0): E = clamp(floor(log2(amax)) - emax, -127, 127)
 * with emax 8 (e4m3) or 2 (e2m1), scale code E + 127, element code =
 * round-to-nearest-even(v * 2^-E) saturated to +-448 / +-6, sign of zero kept;
 * a block with a NaN or Inf gets scale 0xFF and zero codes.
 *   in [R, C] bf16; C % 32 == 0.
 *   codes [R, C] u8 (e4m3) or [R, C/2] u8 (e2m1: element 2j in the low
 *   nibble of byte j); scales [R, C/32] u8. */
int pgg_mx_quantize_rowwise(const void* in, int64_t R, int64_t C, int fmt, uint8_t* codes,
                            uint8_t* scales, void* stream);

/* Row-wise MX quantization with the scales in the blocked atom layout of the
 * block-scaled MMA -- the weight operand of the forward GEMM, quantized once
 * into the caller's weight cache.  Codes and the quantization rule are those of
 * pgg_mx_quantize_rowwise.
 *   in [R, C] bf16; C % 128 == 0.  codes as pgg_mx_quantize_rowwise.
 *   scales: round_up(R, 128) * C / 32 bytes; block j of row r sits at byte
 *   ((r / 128) * (C / 128) + j / 4) * 512 + 16 (r % 32) + 4 ((r % 128) / 32) + j % 4;
 *   rows past R hold scale 0. */
int pgg_mx_quantize_rowwise_blocked(const void* in, int64_t R, int64_t C, int fmt, uint8_t* codes,
                                    uint8_t* scales, void* stream);

/* Group-aware column-wise MX quantization (the wgrad operands, quantized
 * along the token axis).  Blocks of 32 rows run inside one group, starting at
 * the group's first row; group g is stored transposed in columns
 * [P_g, P_g + round_up(len_g, 32)) of the output, where P_g is the exclusive
 * prefix sum of round_up(len_h, PGG_MX_PAD).  Tail positions and everything
 * past the last group up to M_pad hold code 0 and scale 0.
 *   in [M, C] bf16; group_lens may be NULL for one group of M rows.
 *   codes_t [C, M_pad] u8 (e4m3) or [C, M_pad/2] (e2m1).
 *   scales_t: round_up(C, 128) * M_pad / 32 bytes in the blocked layout the
 *   block-scaled MMA reads: one 512-byte atom per 128-row block rb of C and
 *   per 128-column k-block p of [0, M_pad), at byte (rb * M_pad / 128 + p) * 512;
 *   inside it the scale of row 128 rb + m, 32-block 4 p + q sits at byte
 *   16 (m % 32) + 4 (m / 32) + q.  Rows past C hold scale 0.
 *   M_pad % PGG_MX_PAD == 0 and M_pad >= sum(round_up(len_g, PGG_MX_PAD))
 *   (else *err = PGG_ERR_PAD_OVERFLOW and nothing is written);
 *   M + G * (PGG_MX_PAD - 1) rounded up to PGG_MX_PAD always suffices. */
int pgg_mx_quantize_colwise(const void* in, int64_t M, int64_t C, const int32_t* group_lens,
                            int G, int fmt, uint8_t* codes_t, uint8_t* scales_t, int64_t M_pad,
                            int32_t* err, void* stream);

/* Block-scaled grouped GEMM on MX operands (both operands in `fmt`, scales
 * applied per 32-element block of the reduction axis, fp32 accumulation,
 * bf16 output):
 *   PGG_MODE_FWD:   out[M, N] = deq(A)_g . deq(B)_g^T
 *                   A [M, K] row-wise codes, SA [M, K/32];
 *                   B [G*N, K] row-wise codes (W) with SB in the blocked layout
 *                   of pgg_mx_quantize_rowwise_blocked.
 *                   epilogue PGG_EPI_SWIGLU: N = 2I, out = A_act [M, I],
 *                   out2 = H [M, 2I] or NULL (as pgg_grouped_fc1_swiglu).
 *   PGG_MODE_DGRAD: out[M, K] = deq(A)_g . W_g with A = dY [M, N] row-wise
 *                   codes (blocks along N), SA [M, N/32]; B = W quantized
 *                   along N and stored transposed, [K, G*N] codes, SB in the
 *                   blocked layout of pgg_mx_quantize_colwise (that call on W
 *                   viewed as [G*N, K] with G groups of N rows and M_pad =
 *                   G*N produces exactly this).
 *                   epilogue PGG_EPI_SWIGLU: the SwiGLU backward with the
 *                   saved bf16 H [M, 2K]; out = dH [M, 2K].
 *   PGG_MODE_WGRAD: out[G, N, K] = sum over group g's padded columns of
 *                   deq(A)[:, r] deq(B)[:, r]^T with A = dY column-wise
 *                   codes [N, M_pad], B = X column-wise codes [K, M_pad],
 *                   SA / SB their blocked scales (pgg_mx_quantize_colwise);
 *                   empty groups give 0.
 * Fused MX output (SwiGLU epilogues only; both NULL to skip): out_codes /
 * out_scales receive the row-wise MX quantization, in `fmt`, of the bf16 tensor
 * written to `out` (A of the forward, dH of the dgrad) -- bit-identical to
 * pgg_mx_quantize_rowwise(out) -- so the next GEMM's operand needs no separate
 * quantize pass ("Primus-Turbo" README, "What's New": fused GroupedMLP in
 * FP8 / MXFP8).  The width of `out` (I) must be a multiple of 32.
 * Row-major scales (fwd SA, dgrad SA) need 4-byte alignment, blocked ones
 * (fwd SB, dgrad SB, wgrad SA / SB) 16-byte alignment.
 * Sizes: the reduction axis is a multiple of 128 (fwd K, dgrad N); the other
 * dimensions are multiples of 8 (N of a SwiGLU forward a multiple of 16); e2m1
 * codes are packed two per byte.  fp32 accumulation, bf16 output. */
int pgg_mx_grouped_gemm(int mode, int fmt, int epilogue, const uint8_t* A, const uint8_t* SA,
                        const uint8_t* B, const uint8_t* SB, const void* H,
                        const int32_t* group_lens, void* out, void* out2, uint8_t* out_codes,
                        uint8_t* out_scales, int64_t M, int64_t N, int64_t K, int G,
                        int64_t M_pad, int32_t* err, void* stream);

/* ---------------------------------------------------------------- FP8 tensor-wise */

/* FP8 (e4m3) with one fp32 scale per tensor, computed from the tensor itself
 * ("current scaling": "[Megatron-LM] feat: add grouped gemm fp4 support ...
 * Pull Request #891", description and "Changes": the grouped linear layer's
 * FP8 path is the plain grouped_gemm_fp8 call, and under current scaling a
 * cached transposed weight must not be reused; "Primus-Turbo" README: FP8
 * GroupedGEMM).  The pages give no formula; the library takes the usual
 * per-tensor recipe:
 *   amax = max |x| over the tensor's finite elements;
 *   s = 448 / amax in fp32 (1 when amax is 0; clamped to the largest finite
 *       fp32 if the quotient overflows), so the largest element maps to +-448;
 *   code = e4m3 round-to-nearest-even of the fp32 product x * s, saturating
 *       at +-448 (+-Inf saturates too);
 *   deq(code) = decode(code) / s.
 * amax_scale is a device float[2] = {s, amax}, 16-byte aligned.  Every tensor
 * that the GEMM below reads takes its own amax_scale. */

/* amax and s of a bf16 tensor of n elements (n % 8 == 0; n == 0 gives s = 1,
 * amax = 0).  Writes amax_scale[0..1]; two small kernels and a 4-byte memset. */
int pgg_fp8_tensor_scale(const void* in, int64_t n, float* amax_scale, void* stream);

/* Row-major e4m3 codes [R, C] of bf16 in [R, C] with the scale amax_scale[0]
 * (from pgg_fp8_tensor_scale on the same tensor).  C % 8 == 0. */
int pgg_fp8_quantize_rowwise(const void* in, int64_t R, int64_t C, const float* amax_scale, uint8_t* codes,
                             void* stream);

/* Column-wise e4m3 codes for the wgrad GEMM: codes_t [C, M_pad], where group
 * g's row i of in [M, C] lands in column poff_g + i, poff the prefix sum of
 * round_up(len_g, PGG_MX_PAD), and every other column holds code 0 (the same
 * layout as pgg_mx_quantize_colwise's codes, with no scales).  group_lens NULL
 * means one group of M rows (G 0 or 1).  C % 8 == 0; M_pad a multiple of
 * PGG_MX_PAD; a layout past M_pad sets *err = PGG_ERR_PAD_OVERFLOW and writes
 * nothing.  W [G, N, K] for the dgrad GEMM is the same call on W viewed as
 * [G*N, K] with G groups of N rows and M_pad = G*N: codes_t = W^T [K, G*N]. */
int pgg_fp8_quantize_colwise(const void* in, int64_t M, int64_t C, const int32_t* group_lens, int G,
                             const float* amax_scale, uint8_t* codes_t, int64_t M_pad, int32_t* err,
                             void* stream);

/* Bytes of the workspace pgg_fp8_grouped_gemm needs: 0 (the FP8 MMAs read no
 * scale factors).  Kept so that callers sizing a workspace keep working. */
size_t pgg_fp8_workspace_size(int64_t N, int64_t K, int G, int64_t M_pad);

/* FP8 tensor-wise grouped GEMM (grouped_gemm_fp8): the operands, shapes and
 * epilogues of pgg_mx_grouped_gemm with fmt e4m3, each operand carrying one
 * scale instead of per-block scales:
 *   FWD    out[M, N]    = deq(A)_g . deq(B)_g^T   A = X codes [M, K], B = W codes [G*N, K]
 *   DGRAD  out[M, K]    = deq(A)_g . W_g          A = dY codes [M, N], B = W^T codes [K, G*N]
 *   WGRAD  out[G, N, K] = sum over group g's padded columns of deq(A)[:, r] deq(B)[:, r]^T
 *                         A = dY^T codes [N, M_pad], B = X^T codes [K, M_pad] (column-wise)
 * i.e. the sum of code products divided by s_A s_B, fp32 accumulation, bf16 out.
 * epilogue PGG_EPI_SWIGLU (fwd / dgrad, as pgg_mx_grouped_gemm): the fused
 * GroupedMLP in FP8 ("Primus-Turbo" README, "What's New": FP8 / MXFP8 expert
 * MLP with SwiGLU folded into the grouped GEMM).  FWD: N = 2I, out = A_act
 * [M, I], out2 = H [M, 2I] or NULL; DGRAD: the SwiGLU backward with the saved
 * bf16 H [M, 2K], out = dH [M, 2K].  swiglu_limit > 0 clamps as in
 * pgg_grouped_fc1_swiglu_clamped (0: none; SwiGLU epilogue only).  There is no
 * fused quantized output: a current-scaled operand needs the amax of the whole
 * tensor before any of its codes.
 * scale_a / scale_b point at each operand's s (its amax_scale).  The tensor
 * cores run the plain FP8 MMA (tcgen05 kind::f8f6f4, e4m3 x e4m3, fp32
 * accumulation); 1 / (s_A s_B) is applied in the epilogue.  ws / ws_bytes:
 * reserved, ignored (may be NULL / 0).  The size rules, errors and group
 * semantics are pgg_mx_grouped_gemm's (fwd K and dgrad N multiples of 128). */
int pgg_fp8_grouped_gemm(int mode, int epilogue, const uint8_t* A, const float* scale_a, const uint8_t* B,
                         const float* scale_b, const void* H, const int32_t* group_lens, void* out, void* out2,
                         int64_t M, int64_t N, int64_t K, int G, int64_t M_pad, float swiglu_limit, void* ws,
                         size_t ws_bytes, int32_t* err, void* stream);

/* ---------------------------------------------------------------- MoE glue (one GPU) */

/* Bytes of the scratch table pgg_moe_permute needs: ceil(T / 32) * E * 4. */
size_t pgg_moe_permute_workspace_size(int64_t T, int E);

/* Token permute into the expert-sorted layout the grouped GEMM consumes
 * ("Enabling DeepSeek-V4-Flash ...", section "Expert parallelism: DeepEP and
 * the grouped GEMM": the dispatch lays tokens out for the grouped GEMM; on one
 * GPU it has no communication).  Entry (t, j) -- token t's j-th routed expert
 * e = topk_ids[t, j] -- becomes row pos[t, j] of Xs; rows are ordered by expert,
 * then token, then choice (a stable sort of the flattened entries by expert),
 * so group g's rows are [sum_{h<g} len_h, sum_{h<=g} len_h).
 *   topk_ids [T, k] int32 in [0, E); X [T, H] bf16 (may be NULL: routing only);
 *   Xs [T * k, H] bf16 (out; rows past sum(group_lens) untouched);
 *   group_lens [E] int32 (out); pos [T, k] int32 (out);
 *   ws: device scratch of at least pgg_moe_permute_workspace_size(T, E) bytes,
 *   owned by the caller, 4-byte aligned, clobbered.
 *   1 <= k <= 32, 1 <= E <= 1024, T * k < 2^31, H % 8 == 0.
 * An id outside [0, E) sets *err = PGG_ERR_BAD_EXPERT; that entry gets
 * pos = -1, is not counted and not copied.  The result is deterministic. */
int pgg_moe_permute(const int32_t* topk_ids, const void* X, int64_t T, int k, int64_t H, int E,
                    void* Xs, int32_t* group_lens, int32_t* pos, void* ws, size_t ws_bytes,
                    int32_t* err, void* stream);

/* Combine ("Enabling DeepSeek-V4-Flash ...", section "MegaMoE": the second
 * grouped GEMM is followed by the combine and the weighted reduce):
 *   out[t] = sum_j w[t, j] * Ys[pos[t, j]], fp32 accumulation in choice order,
 *   bf16 output.  w NULL means weight 1, which makes this also the permute's
 *   backward: dX[t] = sum_j dXs[pos[t, j]].  Entries with pos < 0 are skipped.
 *   Ys [R, H] bf16 (R >= max pos + 1); pos [T, k] int32; w [T, k] fp32 or NULL;
 *   out [T, H] bf16.  1 <= k <= 32, H % 8 == 0. */
int pgg_moe_combine(const void* Ys, const int32_t* pos, const float* w, void* out, int64_t T, int k,
                    int64_t H, void* stream);

/* Backward of the weighted combine:
 *   dYs[pos[t, j]] = bf16(w[t, j] * dOut[t]);  dw[t, j] = <dOut[t], Ys[pos[t, j]]>
 *   (fp32 dot product in a fixed order: deterministic).  Entries with pos < 0
 *   get dw = 0 and leave dYs untouched.
 *   dOut [T, H] bf16, Ys [R, H] bf16, pos [T, k] int32, w [T, k] fp32,
 *   dYs [R, H] bf16 (out), dw [T, k] fp32 (out).  1 <= k <= 32, H % 8 == 0. */
int pgg_moe_combine_bwd(const void* dOut, const void* Ys, const int32_t* pos, const float* w,
                        void* dYs, float* dw, int64_t T, int k, int64_t H, void* stream);

/* Capacity of pgg_moe_permute_noalloc's fixed scratch, in int32 entries
 * (4 MiB of device memory in the library's module): ceil(T / 32) * E must not
 * exceed it, e.g. 131072 tokens over 256 experts or 32768 over 1024. */
#define PGG_MOE_NOALLOC_MAX_WS_INTS (1 << 20)

/* pgg_moe_permute without a caller workspace.  The pages have no counterpart:
 * it exists for callers that cannot provide device scratch -- a C or real-time
 * component without access to the framework's allocator and with a fixed
 * memory budget, or code that must not call cudaMalloc because it
 * synchronises the device.  The count table lives instead in a statically
 * sized array of the library's own module (PGG_MOE_NOALLOC_MAX_WS_INTS int32
 * entries per device), and the call allocates nothing.
 *   Arguments, layouts and results are those of pgg_moe_permute without ws /
 *   ws_bytes.  ceil(T / 32) * E > PGG_MOE_NOALLOC_MAX_WS_INTS returns
 *   PGG_ERR_TOO_LARGE and launches nothing.
 *   The first call on each device looks up the array's device address (with
 *   that device current) and caches it; make that first call before any
 *   stream capture.  The cache is keyed on the context: after a device reset
 *   (cudaDeviceReset) the next call looks the address up again, in the new
 *   context, so that call too should come before any stream capture.
 *   All calls on one device share the one array: calls that may overlap on
 *   the GPU (different streams without ordering between them) race and give
 *   wrong results.  Calls ordered on one stream are safe. */
int pgg_moe_permute_noalloc(const int32_t* topk_ids, const void* X, int64_t T, int k, int64_t H,
                            int E, void* Xs, int32_t* group_lens, int32_t* pos, int32_t* err,
                            void* stream);

/* The block-scaled grouped GEMM with the clamped SwiGLU epilogue (see
 * pgg_grouped_fc1_swiglu_clamped): mode PGG_MODE_FWD (FC1) or PGG_MODE_DGRAD
 * (FC2 dgrad + SwiGLU backward); the other arguments as pgg_mx_grouped_gemm
 * with epilogue PGG_EPI_SWIGLU. */
int pgg_mx_grouped_gemm_clamped(int mode, int fmt, const uint8_t* A, const uint8_t* SA, const uint8_t* B,
                                const uint8_t* SB, const void* H, const int32_t* group_lens, void* out,
                                void* out2, uint8_t* out_codes, uint8_t* out_scales, int64_t M, int64_t N,
                                int64_t K, int G, float swiglu_limit, int32_t* err, void* stream);

/* ---------------------------------------------------------------- around the experts: norm, routing, decode */

/* Element types and gate scores of the calls below. */
typedef enum { PGG_DTYPE_F32 = 0, PGG_DTYPE_BF16 = 1 } pgg_dtype;
typedef enum { PGG_SCORE_SOFTMAX = 0, PGG_SCORE_SIGMOID = 1 } pgg_score;

/* Longest row of the norm. */
#define PGG_NORM_MAX_COLS 16384

/* Residual addition, RMS norm and MX operand of the next product, in one pass:
 *   s = x + residual;  h = bf16(s);  rstd = 1 / sqrt(mean(s^2) + eps);  y = s rstd gamma
 * in fp32, every output rounded once.
 *   x [R, C], residual [R, C] or NULL, gamma [C] bf16.
 *   Outputs, each optional (NULL), at least one given: h [R, C] bf16 (the new residual stream),
 *   y [R, C] bf16, rstd [R] fp32 (the backward pass reads it), and with fmt PGG_FMT_E4M3 or
 *   PGG_FMT_E2M1 codes and scales: the row-wise MX quantization of y (the layout and the rule of
 *   pgg_mx_quantize_rowwise, applied to the fp32 y, not to its bf16 rounding; a block whose amax
 *   is an fp32 subnormal has scale code 0).  fmt 0: codes and scales are NULL.
 *   8 <= C <= PGG_NORM_MAX_COLS, C % 8 == 0, with codes C % 32 == 0; eps >= 0.  h may be x or
 *   residual (in place).  R == 0 is a no-op.  The sum of squares is fp32: a row whose sum leaves its
 *   range (elements of about 1.8e19 / sqrt(C)) has rstd 0 and y 0. */
int pgg_add_rmsnorm(const void* x, const void* residual, const void* gamma, int64_t R, int64_t C, float eps,
                    int fmt, void* h, void* y, uint8_t* codes, uint8_t* scales, float* rstd, void* stream);

/* Bytes of the workspace that pgg_add_rmsnorm_bwd needs, into *bytes. */
int pgg_add_rmsnorm_bwd_workspace_size(int64_t R, int64_t C, size_t* bytes);

/* Backward pass, with xh = h rstd and u = dy gamma:
 *   dx = dh + rstd (u - xh mean(u xh)), the gradient of x and of the residual alike;
 *   dgamma = sum over rows of dy xh, in fp32 and a fixed order.
 *   dy [R, C], dh [R, C] or NULL (the gradient of h), h [R, C], gamma [C] bf16, rstd [R] fp32;
 *   dx [R, C] bf16, dgamma [C] fp32.  dx may be dy or dh (in place).  ws: device scratch, 16-byte
 *   aligned.  R == 0 writes dgamma = 0. */
int pgg_add_rmsnorm_bwd(const void* dy, const void* dh, const void* h, const void* gamma, const float* rstd,
                        int64_t R, int64_t C, void* dx, float* dgamma, void* ws, size_t ws_bytes, void* stream);

/* The router: each token's k experts and their weights, what pgg_moe_permute, pgg_moe_combine and
 * pgg_moe_decode take.
 *   key_e = logit_e + bias_e (fp32; the bias decides the choice only);
 *   topk_ids: the k largest keys, largest first, ties to the lowest expert;
 *   w_j = scale a_j / Z with a = exp(logit - max) or sigmoid(logit); Z = the sum of a over all
 *   experts (softmax), over the k chosen (renormalize = 1; also where all of these are sigmoids below
 *   fp32's range), or 1 (sigmoid without it).  A sigmoid score counts as 0 below a logit of -700.
 * An expert whose key is -inf is masked: it counts in no sum, and where fewer than k are left it
 * fills the choice with weight 0 (a row that is masked whole has ids 0 .. k-1, weights 0).  A NaN
 * key ranks as -inf and makes the row's weights NaN; the ids are in range whatever the logits.
 *   logits [T, E] fp32 or bf16 (dtype), bias [E] fp32 or NULL; topk_ids [T, k] int32, w [T, k]
 *   fp32.  1 <= E <= 1024, 1 <= k <= min(32, E), T < 2^26. */
int pgg_moe_route(const void* logits, int dtype, const float* bias, int64_t T, int E, int k, int score,
                  int renormalize, float scale, int32_t* topk_ids, float* w, void* stream);

/* Gradient of the logits from dw [T, k], the gradient of w (pgg_moe_combine_bwd gives it), at the
 * experts that pgg_moe_route chose; the other arguments are that call's.  dlogits [T, E] in the
 * logits' type, fully written: zero outside the choice unless the score is a softmax over all
 * experts.  An id outside [0, E) has no part; a row with a NaN key gets NaN. */
int pgg_moe_route_bwd(const void* logits, int dtype, const float* bias, const int32_t* topk_ids, const float* dw,
                      int64_t T, int E, int k, int score, int renormalize, float scale, void* dlogits,
                      void* stream);

/* Most tokens of one pgg_moe_decode call. */
#define PGG_MOE_DECODE_MAX_T 128

/* Bytes of the workspace of the two calls below (fmt 0 for pgg_moe_decode), into *bytes. */
int pgg_moe_decode_workspace_size(int fmt, int64_t T, int k, int64_t H, int64_t I, int E, size_t* bytes);

/* A whole expert layer for a few tokens (decoding), in one kernel and without a permuted copy:
 *   out[t] = sum_j w[t, j] W2_e (silu(g) u),  [g; u] = W1_e X[t],  e = topk_ids[t, j]
 *   X [T, H] bf16; topk_ids [T, k] int32; w [T, k] fp32 or NULL (weight 1); W1 [E, 2I, H] (gate |
 *   up), W2 [E, H, I] bf16; out [T, H] bf16.  fp32 accumulation; the activation between the two
 *   products is kept as the sum of two bf16 numbers.  swiglu_limit as in
 *   pgg_grouped_fc1_swiglu_clamped (0: none).
 *   0 <= T <= PGG_MOE_DECODE_MAX_T (else PGG_ERR_TOO_LARGE: permute and use the grouped GEMMs, which
 *   are as fast from about 100 tokens on in bf16),
 *   1 <= k <= 32, H and I multiples of 8 up to 65536.  A token may name an expert twice.
 * An id outside [0, E) sets *err = PGG_ERR_BAD_EXPERT and has no part.
 * ws: device scratch of pgg_moe_decode_workspace_size bytes, 16-byte aligned, zeroed before the first
 * call.  Every call leaves it ready for the next, so one buffer serves any number of calls, of any
 * sizes and formats that it is large enough for, in the order of one stream.  Zero it again after a
 * call that set PGG_ERR_TIMEOUT: until then every call on it sets PGG_ERR_TIMEOUT, whatever it writes.
 * Calls that may overlap need a workspace each.
 * One cooperative launch: the CTAs wait for one another, so the call needs the whole GPU for its
 * time and starts when the kernels of other streams leave it. */
int pgg_moe_decode(const void* X, const int32_t* topk_ids, const float* w, const void* W1, const void* W2, void* out,
                   int64_t T, int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes,
                   int32_t* err, void* stream);

/* The same on MX operands in `fmt`: X row-wise codes [T, H] (e4m3) or [T, H/2] (e2m1) with scales
 * SX [T, H/32] (pgg_add_rmsnorm or pgg_mx_quantize_rowwise write them; 4-byte aligned); W1 codes
 * [E*2I, H], W2 codes [E*H, I] with blocked scales (pgg_mx_quantize_rowwise_blocked: the forward
 * weight operands of pgg_mx_grouped_gemm).  The activation between the products is quantized from
 * fp32 into MX codes of `fmt`.  H and I are multiples of 128. */
int pgg_mx_moe_decode(int fmt, const uint8_t* X, const uint8_t* SX, const int32_t* topk_ids, const float* w,
                      const uint8_t* W1, const uint8_t* SW1, const uint8_t* W2, const uint8_t* SW2, void* out,
                      int64_t T, int k, int64_t H, int64_t I, int E, float swiglu_limit, void* ws, size_t ws_bytes,
                      int32_t* err, void* stream);

/* ---------------------------------------------------------------- products with biases, joints between blocks */

/* Activations of the two calls below. */
typedef enum { PGG_ACT_NONE = 0, PGG_ACT_SILU = 1, PGG_ACT_GELU = 2, PGG_ACT_SWIGLU = 3 } pgg_act;

/* A matrix product per group with the bias, the activation and a residual in its epilogue:
 *   Z_g = X_g W_g^T + b_g,   Y = act(Z) + residual
 *   X [M, K], W [G, N, K] bf16; bias [G, N] bf16 or NULL; Z [M, N] bf16 (out) or NULL: what the
 *   backward pass reads; dtype: the type of Y and residual (PGG_DTYPE_BF16 or PGG_DTYPE_F32).
 *   Y and residual are [M, N], with PGG_ACT_SWIGLU [M, N/2]; residual may be NULL, and may be Y.
 *   group_lens NULL: one group of M rows (G = 1), a dense product.
 *   act: PGG_ACT_SILU z sigmoid(alpha z); PGG_ACT_GELU z Phi(z), exactly; PGG_ACT_SWIGLU of the halves
 *   z = [g | u]: g sigmoid(alpha g) (u + offset), with limit > 0 g <- min(g, limit) and u <-
 *   clamp(u, -limit, limit) first.  alpha, offset and limit are not read where act has no use for them,
 *   but must be finite, limit >= 0.  alpha = 1, offset = 0 is the SwiGLU of pgg_grouped_fc1_swiglu.
 *   Z is fp32 up to Y; Z, Y are each rounded once.  N % 8 == 0 (swiglu: % 16), K % 8 == 0,
 *   M <= 2^31 - 4097.
 * The result of a row does not depend on its group's other rows beyond the order in which K is summed
 * up, which follows the sizes of the call; it is deterministic. */
int pgg_grouped_linear(const void* X, const void* W, const int32_t* group_lens, const void* bias, const void* residual,
                       void* Y, int dtype, void* Z, int64_t M, int64_t N, int64_t K, int G, int act, float alpha,
                       float offset, float limit, int32_t* err, void* stream);

/* Bytes of the workspace that pgg_grouped_linear_bwd needs, into *bytes. */
int pgg_grouped_linear_bwd_workspace_size(int64_t M, int64_t N, int G, int act, size_t* bytes);

/* Its gradient up to the product:  dZ = dY act'(Z),  dbias_g = sum over group g's rows of dZ
 * (fp32, in a fixed order; 0 for an empty group).  dX and dW are pgg_grouped_gemm_dgrad and
 * pgg_grouped_gemm_wgrad on dZ; the residual's gradient is dY.
 *   dY [M, N] bf16 (PGG_ACT_SWIGLU: [M, N/2]), Z [M, N] bf16 as saved; dZ [M, N] bf16 (out; NULL: the
 *   bias' gradient alone; may be Z, and dY where they have one shape); dbias [G, N] fp32 (out).
 *   PGG_ACT_NONE: Z and dZ are NULL (dZ is dY).  No gradient passes where a clamp is active.
 *   ws: device scratch, 16-byte aligned; it holds nothing between calls, and calls that may overlap need
 *   one each.  M == 0 writes dbias = 0.
 *   Bad group_lens set *err and write nothing. */
int pgg_grouped_linear_bwd(const void* dY, const void* Z, const int32_t* group_lens, void* dZ, float* dbias, int64_t M,
                           int64_t N, int G, int act, float alpha, float offset, float limit, void* ws,
                           size_t ws_bytes, int32_t* err, void* stream);

/* Test hook, as pgg_test_stalled_fwd below for pgg_grouped_linear (bf16 Y, alpha 1, no bias). */
int pgg_test_stalled_linear(const void* X, const void* W, const int32_t* group_lens, void* Y, int64_t M, int64_t N,
                            int64_t K, int G, int act, int64_t stall_at, uint64_t wait_ns, int32_t* err, void* stream);

/* Test hooks: which kernel pgg_grouped_linear takes for these sizes (grouped: with group_lens), and the
 * call with a kernel of the tests' choice.
 *   plan[0]: 0 clusters that share a tile's reduction, 1 one CTA per SM, 2 pairs of CTAs; plan[1]: rows of X
 *   in a tile; plan[2]: CTAs that share a reduction (else 1); plan[3]: CTAs an SM.  sms: the SMs to plan
 *   for, 0: the current device's.
 *   A kernel that the sizes do not have is PGG_ERR_INVALID_ARG.  stall_at -1: no stall; wait_ns 0: the
 *   call's own limit; else as in pgg_test_stalled_linear. */
int pgg_test_linear_plan(int64_t M, int64_t N, int64_t K, int G, int grouped, int act, int dtype, int sms,
                         int32_t* plan);
int pgg_test_planned_linear(int kind, int tn, int splits, const void* X, const void* W, const int32_t* group_lens,
                            const void* bias, const void* residual, void* Y, int dtype, void* Z, int64_t M, int64_t N,
                            int64_t K, int G, int act, float alpha, float offset, float limit, int64_t stall_at,
                            uint64_t wait_ns, int32_t* err, void* stream);

/* Forms of a block's gate. */
typedef enum { PGG_GATE_NONE = 0, PGG_GATE_TOKEN = 1, PGG_GATE_CHANNEL = 2 } pgg_gate;

/* Between two blocks, in one pass: the norm of a block's output, dropout, its gate, the scaled
 * residual's addition, the next block's norm and the MX operand of its first product.
 *   t = x rstd_post gamma_post    rstd_post = 1 / sqrt(mean(x^2) + eps)   (gamma_post NULL: t = x)
 *   b = keep t / (1 - p)
 *   s = residual_scale residual + branch_scale gate b     h = bf16(s)     (residual NULL: 0)
 *   y = s rstd gamma              rstd = 1 / sqrt(mean(s^2) + eps)        (gamma NULL: no y, rstd, codes)
 *   in fp32, every output rounded once.  x, residual [R, C], gamma_post, gamma [C] bf16.
 *   gate: PGG_GATE_TOKEN [R] fp32, PGG_GATE_CHANNEL [C] bf16; NULL with PGG_GATE_NONE (1).
 *   Dropout, 0 <= p < 1 (0: none): rng is a device int64[2] {seed, offset}, 8-byte aligned, read when the
 *   call runs (a replayed graph takes what it holds then).  Element i of the row-major tensor is kept
 *   where word i % 4 of Philox4x32-10 with the counter (i / 4, offset), low words first, and the key
 *   seed is at least floor(p 2^32); a dropped element is 0 whatever it, its row's norm and a row's gate
 *   hold.  Calls with other offsets have independent masks.  The mask is not stored: pgg_block_join_bwd
 *   computes it again from the same rng and p.
 *   Outputs, each optional (NULL), at least one given: h, y [R, C] bf16, rstd_post, rstd [R] fp32, and
 *   with fmt codes and scales as in pgg_add_rmsnorm.  8 <= C <= PGG_NORM_MAX_COLS, C % 8 == 0, with codes
 *   C % 32 == 0; eps >= 0.  h may be x or residual (in place).  R == 0 is a no-op.  Sums of squares are
 *   fp32, with the range given at pgg_add_rmsnorm. */
int pgg_block_join(const void* x, const void* residual, const void* gamma_post, const void* gamma, const void* gate,
                   int gate_kind, const int64_t* rng, int64_t R, int64_t C, double p, float residual_scale,
                   float branch_scale, float eps, int fmt, void* h, void* y, uint8_t* codes, uint8_t* scales,
                   float* rstd_post, float* rstd, void* stream);

/* Bytes of the workspace that pgg_block_join_bwd needs, into *bytes. */
int pgg_block_join_bwd_workspace_size(int64_t R, int64_t C, size_t* bytes);

/* Backward pass, with xh = x rstd_post and hh = h rstd:
 *   d = dh + rstd (u - hh mean(u hh)), u = dy gamma          dgamma = sum over rows of dy hh
 *   dresidual = residual_scale d
 *   dgate = branch_scale sum of d b over the row (token), over the rows (channel)
 *   dt = branch_scale gate d keep / (1 - p)                  dgamma_post = sum over rows of dt xh
 *   dx = rstd_post (w - xh mean(w xh)), w = dt gamma_post    (without gamma_post: dx = dt)
 *   dy [R, C] bf16 (NULL without gamma), dh [R, C] bf16 or NULL, x, h, rstd_post, rstd as in and from the
 *   forward call (h and rstd NULL without gamma, rstd_post without gamma_post); the other arguments are
 *   that call's.  dx [R, C] bf16; dresidual [R, C] bf16 or NULL; dgamma_post, dgamma [C], dgate [R] or
 *   [C] fp32, each given where its operand is, summed up in a fixed order.
 *   What the mask drops passes nothing on, whatever it, its row's norm and a row's gate hold.
 *   dx and dresidual may be dy, dh, x or h (not the same of them).  ws: device scratch, 16-byte
 *   aligned; it holds nothing between calls, and calls that may overlap need one each.  R == 0 writes
 *   zero sums. */
int pgg_block_join_bwd(const void* dy, const void* dh, const void* x, const void* h, const float* rstd_post,
                       const float* rstd, const void* gamma_post, const void* gamma, const void* gate, int gate_kind,
                       const int64_t* rng, int64_t R, int64_t C, double p, float residual_scale, float branch_scale,
                       void* dx, void* dresidual, float* dgamma_post, float* dgamma, float* dgate, void* ws,
                       size_t ws_bytes, void* stream);

/* Test hook, as pgg_test_stalled_fwd below for the few-token layer (fmt 0: bf16, SX / SW1 / SW2
 * unused; weights 1): every CTA's load producer stops before the stall_at-th stage of its run, and
 * every wait is limited to wait_ns.  The kernel must give up, free its tensor memory, exit and write
 * PGG_ERR_TIMEOUT to *err.  The workspace has to be zeroed before its next use. */
int pgg_test_stalled_moe_decode(int fmt, const void* X, const uint8_t* SX, const int32_t* topk_ids, const void* W1,
                                const uint8_t* SW1, const void* W2, const uint8_t* SW2, void* out, int64_t T, int k,
                                int64_t H, int64_t I, int E, int64_t stall_at, uint64_t wait_ns, void* ws,
                                size_t ws_bytes, int32_t* err, void* stream);

/* Test hook; the pages have no counterpart.  Runs the forward grouped GEMM --
 * BF16 when fmt == 0 (A = X, B = W, SA and SB unused), else the block-scaled
 * forward in `fmt` (arguments as pgg_mx_grouped_gemm with PGG_MODE_FWD and
 * PGG_EPI_NONE) -- with every pipeline wait limited to `wait_ns` and the load
 * producer of each CTA told to stop before its `stall_at`-th k-block.  The MMA
 * and epilogue waits behind that k-block then run out, and the kernel must take
 * its failure path: raise the CTA's abort flag, drain what it issued, free its
 * tensor memory, exit, and write PGG_ERR_TIMEOUT to *err, leaving the device
 * usable for the next call.  It exists so that tests can run that path without
 * faulting or hanging the GPU.  stall_at >= 0; 100 us <= wait_ns <= 1 s.  The
 * output is incomplete. */
int pgg_test_stalled_fwd(int fmt, const void* A, const uint8_t* SA, const void* B, const uint8_t* SB,
                         const int32_t* group_lens, void* out, int64_t M, int64_t N, int64_t K, int G,
                         int64_t stall_at, uint64_t wait_ns, int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PGG_H_ */

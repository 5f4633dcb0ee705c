/*
 * moe_fp4 — block-scaled FP4 mixture-of-experts layer for AMD MI355X (gfx950).
 *
 * The layer (b12x PR #22, "rp-native tiny-decode kernel for w4a8_mx (M=1)",
 * What section, FC1 and FC2 bullets): for every token t and every route j of
 * its top-k, with expert e = ids[t][j],
 *     gate_n = sum_h x[t][h] * W13[e][n][h],        n in [0, I)
 *     up_n   = sum_h x[t][h] * W13[e][I + n][h]
 *     a_n    = gate_n / (1 + exp(-gate_n)) * up_n     (SiLU(gate) * up)
 *     y_h    = sum_n a_n * W2[e][h][n]
 *     out[t][h] = bf16( sum_j w[t][j] * y_h )         (fp32 sum, one rounding)
 * Weights are E2M1 nibbles with block scales:
 *   MXFP4: one UE8M0 scale byte (2^(b-127)) per 32 consecutive K elements;
 *   NVFP4: one E4M3 scale byte per 16 consecutive K elements, times an fp32
 *          global multiplier per expert per matrix (g13[e] for W13, g2[e]
 *          for W2).
 * A route whose id is negative or >= E reads no weights and contributes
 * nothing (b12x PR #311, commit message on the FC2-only endpoint, and its
 * review of tiny_decode.py); a token with no valid route yields +0.
 *
 * Logical weight layout (the input of moe_fp4_prepare), row-major, G = 32
 * (MXFP4) or 16 (NVFP4), for the gated activations (relu2: W13 has I rows):
 *   w13_codes  u8[E][2I][H/2]  rows [0, I) gate, [I, 2I) up; element 2b of a
 *                              row in the low nibble of byte b, 2b+1 in the high
 *   w13_scales u8[E][2I][H/G]
 *   w2_codes   u8[E][H][I/2]
 *   w2_scales  u8[E][H][I/G]
 *   g13, g2    f32[E]          NVFP4 only (NULL for MXFP4)
 *
 * Conventions for every entry point:
 *   - Device pointers are caller-owned device memory; the library allocates
 *     nothing, keeps no global state (except moe_fp4_forward_noalloc's
 *     workspace, below) and never synchronises.  Work is queued on `stream`
 *     (a hipStream_t; NULL is the default stream).
 *   - Inputs are never written.  Arguments are checked before any launch; a
 *     rejected call launches nothing.  A failed launch returns MOE_FP4_EHIP.
 *   - Data conditions are not errors: invalid ids contribute zero; NaN or Inf
 *     in scales, globals or activations of valid routes propagate.
 */
#ifndef MOE_FP4_H
#define MOE_FP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_FP4_OK = 0,
  MOE_FP4_EINVAL = 1,      /* null/misaligned pointer, bad size or count */
  MOE_FP4_EUNSUPPORTED = 2,/* valid request outside what the library handles */
  MOE_FP4_EWORKSPACE = 3,  /* workspace or prepared buffer too small */
  MOE_FP4_EHIP = 4         /* a HIP launch or runtime call failed */
} moe_fp4_status;

typedef enum {
  MOE_FP4_MXFP4 = 1, /* E2M1 + UE8M0 scale per 32 */
  MOE_FP4_NVFP4 = 2  /* E2M1 + E4M3 scale per 16, times an fp32 global */
} moe_fp4_format;

/* Activation format of the grouped path.
 *   BF16:  x and SiLU(gate) * up enter the GEMMs at bf16 precision or better
 *          (the layer as defined above).
 *   MXFP8: the W4A8-MX variant (b12x PR #22, Measured table and its note on
 *          the dynamic path, which quantises activations to MXFP8; MXFP4
 *          weights only).  x is quantised per token in blocks of 32 along H,
 *          and SiLU(gate) * up (from fp32 FC1 outputs, rounded to fp32) per
 *          route in blocks of 32 along I, each to MXFP8 as the OCP MX format
 *          defines it: one UE8M0 scale 2^(floor(log2(max |v|)) - 8) per
 *          block (clamped to 2^[-127, 127]; a zero block gets byte 0, a
 *          block with a NaN or an infinity byte 255), elements v / scale
 *          rounded to nearest-even E4M3 with magnitudes capped at 448 (a
 *          NaN/Inf block's codes are all 0x7F).  FC1 and FC2 then run on the
 *          scaled matrix instruction with fp32 accumulation.  The decode
 *          path (small M) keeps bf16 activations in both modes, as the
 *          pages' M = 1 kernel does. */
typedef enum {
  MOE_FP4_ACT_BF16 = 0,
  MOE_FP4_ACT_MXFP8 = 1
} moe_fp4_act_format;

/* Gated activation a = f(gate, up) between FC1 and FC2.  The pages name
 * SiLU (b12x PR #22, What: FC2 applies SiLU inline), gelu_tanh and
 * swigluoai_uninterleave with alpha, beta and limit (flashinfer #4285,
 * reviews of moe_activation.py and of the direct micro kernel's activation
 * coverage) without formulas; these are the standard definitions:
 *   SILU:      gate * sigmoid(gate) * up
 *   GELU_TANH: 0.5 * gate * (1 + tanh(sqrt(2/pi) * (gate + 0.044715 * gate^3))) * up
 *   SWIGLUOAI: g = min(gate, limit), u = max(min(up, limit), -limit),
 *              g * sigmoid(alpha * g) * (u + beta)
 *              (act_alpha, act_beta finite, act_limit > 0 or +inf; gate and
 *              up are the separate halves of W13; a NaN passes the clamps)
 *   RELU2:     not gated (b12x PR #311, commit message on the FP4 quantiser,
 *              which treats relu2 apart from the gated activations): W13 has
 *              I rows (w13_codes u8[E][I][H/2], w13_scales u8[E][I][H/G]),
 *              h = x . W13[n] and a_n = max(h, 0)^2; I must be a multiple
 *              of 64 (else MOE_FP4_EUNSUPPORTED)
 * Every path applies the same function. */
typedef enum {
  MOE_FP4_FN_SILU = 0,
  MOE_FP4_FN_GELU_TANH = 1,
  MOE_FP4_FN_SWIGLUOAI = 2,
  MOE_FP4_FN_RELU2 = 3
} moe_fp4_act_fn;

/* Resident form of the block scales (scale_format in moe_fp4_desc).
 *   PLAIN: the scale bytes as given.
 *   CSF:   in addition, each weight row's scale bytes compressed as a row
 *          base byte plus an offset per block, one bit (MXFP4, offset 0 or
 *          1) or four bits (NVFP4, 0..15), the byte being base + offset
 *          (b12x PR #459, "Reduce NVFP4-CSF scale reconstruction overhead",
 *          commit messages: one-bit MXFP4 and four-bit NVFP4 offsets from a
 *          row base byte).  The base is the row's smallest byte; a row whose
 *          bytes span more than the offsets reach, or whose smallest byte is
 *          255, is an exception read from the plain bytes.  Lossless: every
 *          result equals the PLAIN one bit for bit.  The decode path reads
 *          the compressed scales (one 4-byte word of base byte and offsets
 *          per row and 24 (MXFP4) or 3 (NVFP4) chunks of 32 weights, against
 *          1 or 2 plain bytes per chunk) and the plain bytes of exception
 *          rows only; the grouped path and moe_fp4_unprepare read the plain
 *          bytes.  The prepared buffer grows by the compressed blocks
 *          (moe_fp4_prepared_bytes). */
typedef enum {
  MOE_FP4_SCALES_PLAIN = 0,
  MOE_FP4_SCALES_CSF = 1
} moe_fp4_scale_format;

/* Shape of one MoE layer.  H and I must be multiples of 32 for both formats
 * (the kernels work in 32-element units); max_tokens is the largest M that
 * later forward calls will pass, used only to size the workspace.
 * act_format is a moe_fp4_act_format (0 keeps bf16 activations); MXFP8 with
 * NVFP4 weights returns MOE_FP4_EUNSUPPORTED.  act_fn and its parameters
 * choose the gated activation (0 and zeros: SiLU).  scale_format is a
 * moe_fp4_scale_format (0: plain). */
typedef struct {
  int32_t format;      /* moe_fp4_format */
  int32_t num_experts; /* E, resident experts; ids outside [0, E) are invalid */
  int32_t hidden;      /* H: K of FC1, N of FC2 */
  int32_t inter;       /* I: intermediate size */
  int32_t top_k;       /* k: routes per token */
  int32_t max_tokens;  /* capacity for workspace sizing */
  int32_t act_format;  /* moe_fp4_act_format */
  int32_t act_fn;      /* moe_fp4_act_fn (0: SiLU) */
  float act_alpha;     /* SWIGLUOAI only, else ignored */
  float act_beta;
  float act_limit;
  int32_t scale_format; /* moe_fp4_scale_format */
} moe_fp4_desc;

/* Human-readable name of a status code (static string).  A diagnostic hook
 * of this library's own; no page defines one. */
const char* moe_fp4_status_string(moe_fp4_status s);

/* Bytes of the prepared (resident) weight buffer for `desc`.  It holds the
 * same codes, scale bytes and fp32 globals as the logical tensors, reordered,
 * plus zero padding to whole tiles (b12x PR #459, "Reduce NVFP4-CSF scale
 * reconstruction overhead", commit messages: preparation keeps checkpoint
 * bytes and prepared memory sizes). */
moe_fp4_status moe_fp4_prepared_bytes(const moe_fp4_desc* desc, size_t* bytes);

/* Weight preparation, once per layer at load time (b12x PR #459, "Reduce
 * NVFP4-CSF scale reconstruction overhead", commit messages: keep the exact
 * FP4 nibbles and scale bytes, no requantisation, reorder resident offsets
 * for contiguous decoding).  A pure byte permutation of the logical tensors
 * above into `prepared` (device, 256-byte aligned, `prepared_bytes` >=
 * moe_fp4_prepared_bytes).  Logical inputs must be 16-byte aligned device
 * buffers; g13/g2 are required for NVFP4 and must be NULL for MXFP4. */
moe_fp4_status moe_fp4_prepare(const moe_fp4_desc* desc, const uint8_t* w13_codes,
                               const uint8_t* w13_scales, const uint8_t* w2_codes,
                               const uint8_t* w2_scales, const float* g13, const float* g2,
                               void* prepared, size_t prepared_bytes, void* stream);

/* Inverse of moe_fp4_prepare: writes the logical tensors back from a
 * prepared buffer (used to check that preparation is a bijection). */
moe_fp4_status moe_fp4_unprepare(const moe_fp4_desc* desc, const void* prepared,
                                 uint8_t* w13_codes, uint8_t* w13_scales, uint8_t* w2_codes,
                                 uint8_t* w2_scales, float* g13, float* g2, void* stream);

/* Workspace bytes for forward calls on `desc` (device scratch, 256-byte
 * aligned, caller-owned).  The size depends only on the descriptor, so one
 * workspace serves every M <= max_tokens; `M` is checked against max_tokens
 * (b12x PR #311, review comment on the intermediate_cache13 sizing: a
 * workspace must hold the largest requirement over every token count the
 * caller plans, or a smaller launch under-allocates).
 * The grouped path needs about 4I + 4H bytes per route (max_tokens * k
 * routes) with bf16 activations, and about I + 4H per route plus H per
 * token with MXFP8 activations.  Its contents on entry do not matter and
 * are overwritten. */
moe_fp4_status moe_fp4_workspace_bytes(const moe_fp4_desc* desc, int32_t M, size_t* bytes);

/* The layer.  x: bf16 [M][H]; topk_ids: int32 [M][k]; topk_w: fp32 [M][k]
 * (used as given, no renormalisation); out: bf16 [M][H], overwritten.  All
 * device pointers, 16-byte aligned except topk_ids (element size) and topk_w
 * (4-byte).  M may be 0 (nothing is launched).  Calls that share a workspace
 * must be ordered on one stream.
 *
 * Two execution paths, chosen by M (both compute the layer above):
 *   decode  FC1 and FC2 as streamed FP4 GEMVs in one launch each, FC1
 *           over chunks of up to C = min(16, 64 / k) tokens, each routed
 *           expert's weights read once per chunk (b12x PR #22, What);
 *           results are bit-reproducible.  Taken for M <= C; with bf16
 *           activations for M <= 2C, and for M <= 6C when the chunks'
 *           route slots ceil(M / C) * C * k are fewer than E (few routes
 *           per expert); and for every M when E > 8192.
 *   grouped (any other M): routes grouped by expert in route order, FC1 and
 *           FC2 as grouped GEMMs on the matrix cores over bf16 operands (FP4
 *           dequantised exactly) with fp32 accumulation, per-route fp32 rows
 *           summed per token in route order and cast once (flashinfer #4285,
 *           description: the prefill kernel's per-expert tiles; b12x PR #311,
 *           commit message on the prefill fused-sum epilogue).  The
 *           activation enters FC2 as a pair of bf16 values (hi + lo, 16
 *           significant bits), as in the decode path.  With act_format =
 *           MXFP8 both GEMMs instead take MXFP8 activations on the scaled
 *           FP8 x FP4 matrix instruction (the W4A8-MX variant above).
 *           Results are bit-reproducible.
 * The activation function (act_fn) is the same on both paths.
 * Returns MOE_FP4_EUNSUPPORTED when max_tokens * k > 2^22, or when the path
 * the call needs cannot run it: the grouped path with E > 8192, the decode
 * path with k > 64 or M > 65535. */
moe_fp4_status moe_fp4_forward(const moe_fp4_desc* desc, const void* prepared,
                               const uint16_t* x, int32_t M, const int32_t* topk_ids,
                               const float* topk_w, uint16_t* out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Same, with int64 route ids (any int64 value outside [0, E) is invalid).
 * Both id widths are served (b12x PR #459, "Reduce NVFP4-CSF scale
 * reconstruction overhead", commit messages: programs kept for both routing
 * integer types). */
moe_fp4_status moe_fp4_forward_i64(const moe_fp4_desc* desc, const void* prepared,
                                   const uint16_t* x, int32_t M, const int64_t* topk_ids,
                                   const float* topk_w, uint16_t* out, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under graph capture,
 * tight serving loops, harnesses that forbid allocation): moe_fp4_forward
 * (int32 ids) without a workspace argument.  The workspace is a block of
 * 64 MiB of device memory that the library itself holds, one per GPU it
 * runs on, from the first call on that GPU until the process ends; the call
 * allocates nothing.  `desc` must need at most that much workspace
 * (moe_fp4_workspace_bytes <= 64 MiB), else MOE_FP4_EWORKSPACE; other
 * arguments, checks and results are those of moe_fp4_forward.  The stream
 * must belong to the current device.  All calls on one GPU share that
 * GPU's block: calls that overlap on one GPU (other streams, other host
 * threads without ordering) race on it and give wrong results; calls
 * ordered on one stream are safe.  Its contents on entry do not matter. */
moe_fp4_status moe_fp4_forward_noalloc(const moe_fp4_desc* desc, const void* prepared,
                                       const uint16_t* x, int32_t M, const int32_t* topk_ids,
                                       const float* topk_w, uint16_t* out, void* stream);

/* Test hook of this library's own: dequantise one expert matrix from the
 * prepared buffer with the same decode instructions the forward kernels use,
 * into fp32 row-major `out` ([2I][H] for which = 0 (W13), [H][I] for
 * which = 1 (W2); device, 4-byte aligned, caller-owned).  Each value is
 * (E2M1 code * block scale) rounded to fp32, times the global (NVFP4), so
 * the tests can compare every prepared byte with the oracle's dequantisation
 * bit for bit (b12x PR #459, PR body: every arm is checked against an exact
 * byte oracle). */
moe_fp4_status moe_fp4_dequant_export(const moe_fp4_desc* desc, const void* prepared,
                                      int32_t expert, int32_t which, float* out,
                                      void* stream);

/* Execution path selector for moe_fp4_forward_ex. */
typedef enum {
  MOE_FP4_PATH_AUTO = 0,    /* by M, as moe_fp4_forward */
  MOE_FP4_PATH_DECODE = 1,  /* decode path (in chunks); MOE_FP4_EUNSUPPORTED when k > 64 or M > 65535 */
  MOE_FP4_PATH_GROUPED = 2  /* grouped path at any M */
} moe_fp4_path;

/* Launch shape of the decode kernels and the path; 0 in a field keeps the
 * built-in choice.
 *   fc1_chunks_per_wave: 32-element K chunks per FC1 wave (4, 8 or 16)
 *   fc1_rows: FC1 rows per workgroup, half gate and half up (16 or 32)
 *   fc2_rows: FC2 rows of H per workgroup (8, 16 or 32; at least 64 divided
 *             by FC2's chunk lanes, which is 4, 8 or 16 for I up to 128, 256
 *             or beyond)
 *   path: a moe_fp4_path */
typedef struct {
  int32_t fc1_chunks_per_wave;
  int32_t fc1_rows;
  int32_t fc2_rows;
  int32_t path;
} moe_fp4_tuning;

/* Measurement and test hook: moe_fp4_forward (int32 ids) with an explicit
 * launch shape and path (`tuning` may be NULL) and only part of the call
 * queued, so a caller can put events between the two halves: phases = 1
 * queues the first half (decode: FC1; grouped: routing and FC1), which fills
 * the workspace's activation; 2 queues the second half (FC2 and the combine
 * into `out`; it must follow a phase-1 call with the same arguments on the
 * same stream); 3 queues both.  On the grouped path, 4 queues only its
 * routing (the grouping of the routes by expert) and 8 only its combine
 * (which reads what a phase-2 call left), so the two GEMM launches can be
 * timed on their own; the decode path rejects 4 and 8. */
moe_fp4_status moe_fp4_forward_ex(const moe_fp4_desc* desc, const void* prepared,
                                  const uint16_t* x, int32_t M, const int32_t* topk_ids,
                                  const float* topk_w, uint16_t* out, void* workspace,
                                  size_t workspace_bytes, const moe_fp4_tuning* tuning,
                                  int32_t phases, void* stream);

/* The path and launch shape that moe_fp4_forward_ex takes for M tokens with
 * `tuning` (NULL: moe_fp4_forward's choice), written to `plan` with every
 * field resolved: path is MOE_FP4_PATH_DECODE or MOE_FP4_PATH_GROUPED, and
 * the decode shape fields are 0 on the grouped path.  Returns what
 * moe_fp4_forward_ex would return for an invalid or unsupported request;
 * launches nothing. */
moe_fp4_status moe_fp4_plan(const moe_fp4_desc* desc, int32_t M, const moe_fp4_tuning* tuning,
                            moe_fp4_tuning* plan);

/* The MXFP8 quantisation of the MXFP8 activation format (see
 * moe_fp4_act_format), as the grouped path applies it to x: bf16 `x`
 * [rows][cols] (device, 16-byte aligned, cols a multiple of 32) to E4M3
 * `codes` [rows][cols] (device, 8-byte aligned) and UE8M0 `scales`
 * [rows][cols / 32] (device), one scale per 32 consecutive values of a row.
 * rows may be 0 (nothing is launched). */
moe_fp4_status moe_fp4_mxfp8_quantize(const uint16_t* x, int64_t rows, int32_t cols, uint8_t* codes,
                                      uint8_t* scales, void* stream);

/* ------------------------------------------------------------------------
 * Operators around the layer: the router that gives it ids and weights, the
 * FP8 linear map of shared experts and projections, and the norms before and
 * after the block.  The conventions above hold for them too (caller-owned
 * device memory, no allocation, no synchronisation, checks before any
 * launch); calls that share a workspace must be ordered on one stream. */

typedef enum {
  MOE_FP4_TYPE_BF16 = 0,
  MOE_FP4_TYPE_F32 = 1
} moe_fp4_type;

typedef enum {
  MOE_FP4_SCORE_SOFTMAX = 0, /* p = softmax over all E logits */
  MOE_FP4_SCORE_SIGMOID = 1  /* p = 1 / (1 + exp(-z)) per expert */
} moe_fp4_scoring;

/* Router of a layer.  For a token x and router weights Wr [E][H]:
 *     z_e = sum_h x[h] * Wr[e][h],   p = softmax(z) or sigmoid(z),
 *     t_e = p_e + bias[e]                 (a bias is used for the choice only)
 *   groups: with num_groups > 1 the experts are num_groups runs of E /
 *     num_groups, a group's score is the sum of its two largest t, and only
 *     the top_groups best groups' experts can be taken;
 *   ids: the top_k experts of largest t (without a bias, of largest z, which
 *     is the same order), largest first, ties to the lowest index;
 *   weights: p of the taken experts, divided by their sum with renormalize,
 *     times scale.
 * The choice is that of z in exact arithmetic and t in 64 bits, whatever M:
 * logits are fp32 matrix products, and those that decide something within
 * their error bound are recomputed in 64 bits.  An expert whose t (without a
 * bias, whose z) is NaN or -infinity (a bias of -infinity masks one) is never
 * taken, and a group with fewer than two others has the score -infinity; a
 * token with fewer than top_k experts to take gets id -1 and weight 0 in the
 * slots left, which the layer's calls skip.  Weights that sum to 0 stay 0; a
 * softmax's, renormalised, are those of a softmax over the taken experts, also
 * where p itself is too small for a number. */
typedef struct {
  int32_t num_experts; /* E, at most 512 */
  int32_t hidden;      /* H, a multiple of 8, at most 65536 */
  int32_t top_k;       /* at most 64 and the experts of top_groups groups */
  int32_t max_tokens;  /* capacity for workspace sizing, at most 2^20 */
  int32_t weight_type; /* moe_fp4_type of Wr */
  int32_t scoring;     /* moe_fp4_scoring */
  int32_t num_groups;  /* 1 (no groups) to 64, divides E, 2 experts or more each */
  int32_t top_groups;  /* 1 to num_groups */
  int32_t renormalize; /* 0 or 1 */
  float scale;         /* finite */
} moe_fp4_router_desc;

/* Bytes of the prepared router weights, and the preparation, once per
 * router: a permutation of Wr ([E][H], device, 16-byte aligned; fp32 as three
 * bf16 terms that sum to it), the experts' 2-norms and Wr's rows as they are,
 * into `prepared` (device, 256-byte aligned, not overlapping Wr). */
moe_fp4_status moe_fp4_router_prepared_bytes(const moe_fp4_router_desc* desc, size_t* bytes);
moe_fp4_status moe_fp4_router_prepare(const moe_fp4_router_desc* desc, const void* weight, void* prepared,
                                      size_t prepared_bytes, void* stream);

/* Workspace bytes for route calls on `desc` (device, 256-byte aligned),
 * enough for every M <= max_tokens; M is checked against max_tokens. */
moe_fp4_status moe_fp4_router_workspace_bytes(const moe_fp4_router_desc* desc, int32_t M, size_t* bytes);

/* Routes M tokens.  x: bf16 [M][H], 16-byte aligned; bias: fp32 [E] or NULL;
 * topk_ids: int32 [M][k] and topk_w: fp32 [M][k], overwritten; logits: fp32
 * [M][E], overwritten, or NULL.  No output may overlap another, the workspace
 * or anything that is read, nor the workspace anything that is read.  M may be
 * 0 (nothing is launched). */
moe_fp4_status moe_fp4_route(const moe_fp4_router_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                             const float* bias, int32_t* topk_ids, float* topk_w, float* logits, void* workspace,
                             size_t workspace_bytes, void* stream);

/* act_fn of moe_fp4_fp8_desc besides the layer's activations */
#define MOE_FP4_FN_NONE (-1)

/* Linear map with E4M3 weights and an fp32 scale per block of 128 x 128:
 *     y[n] = sum_k q(x)[k] * codes[n][k] * scales[n / 128][k / 128],
 * where q(x) is x quantised in blocks of 128 along K: the least power of two
 * s >= 2^-127 with |x| <= 448 s over the block, values x / s rounded to
 * nearest-even E4M3, times s.  An activation where asked for
 * (moe_fp4_act_fn, the gated ones over gate and up rows), one rounding to
 * bf16.  A block of x that holds a NaN or an infinity makes its token's
 * outputs NaN; other tokens are not touched.
 *   Sums are not fp32 throughout: the matrix instruction adds 8 products of
 * codes first (k = 8 i to 8 i + 7), each cut towards zero to a multiple of
 * 2^-13 times the power of two at or below the largest of the 8; all that
 * follows is fp32.  Before the activation y is off by less than 2^-10 of the
 * sum over all such groups of their largest |q(x) * code * scale|, besides
 * fp32's own roundings.  Where the terms do not cancel that is 2 to 4 * 10^-4
 * of y, a tenth of a bf16 step; where they do, it is relative to the terms
 * and not to y. */
typedef struct {
  int32_t in_features;  /* K, a multiple of 8, at most 2^20 */
  int32_t out_features; /* N, a multiple of 8, at most 2^26; K * N at most 2^30 */
  int32_t max_tokens;   /* capacity for workspace sizing, at most 2^20 */
  int32_t act_fn;       /* MOE_FP4_FN_NONE or a moe_fp4_act_fn */
  float act_alpha;      /* SWIGLUOAI only, else ignored */
  float act_beta;
  float act_limit;
} moe_fp4_fp8_desc;

/* Bytes of the prepared weights, and the preparation, once per map: a
 * permutation of the bytes into `prepared` (device, 256-byte aligned, not
 * overlapping what is read).  codes: E4M3 bytes [N][K] (device, 16-byte
 * aligned), scales: fp32 [ceil(N / 128)][ceil(K / 128)]; for a gated
 * activation both hold the gate's and then the up's ([2N][K],
 * [2 ceil(N / 128)][ceil(K / 128)]). */
moe_fp4_status moe_fp4_fp8_prepared_bytes(const moe_fp4_fp8_desc* desc, size_t* bytes);
moe_fp4_status moe_fp4_fp8_prepare(const moe_fp4_fp8_desc* desc, const uint8_t* codes, const float* scales,
                                   void* prepared, size_t prepared_bytes, void* stream);

/* Workspace bytes for calls on `desc` (device, 256-byte aligned), enough for
 * every M <= max_tokens; M is checked against max_tokens. */
moe_fp4_status moe_fp4_fp8_workspace_bytes(const moe_fp4_fp8_desc* desc, int32_t M, size_t* bytes);

/* The map on M tokens.  x: bf16 [M][K], out: bf16 [M][N], overwritten; both
 * 16-byte aligned.  Neither may overlap the other or the workspace, nor out or
 * the workspace the prepared weights.  M may be 0 (nothing is launched). */
moe_fp4_status moe_fp4_fp8_linear(const moe_fp4_fp8_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                                  uint16_t* out, void* workspace, size_t workspace_bytes, void* stream);

/* What multiplies the branch before it joins the residual. */
typedef enum {
  MOE_FP4_GATE_NONE = 0,
  MOE_FP4_GATE_CHANNEL = 1, /* [H] */
  MOE_FP4_GATE_TOKEN = 2,   /* [M] */
  MOE_FP4_GATE_FULL = 3     /* [M][H] */
} moe_fp4_gate;

/* Norms before and after a block, fused with its gate and residual:
 *     b  = y + y2                                            (y2 may be absent)
 *     n  = b / sqrt(mean(b^2) + eps) * (post_weight + weight_offset)
 *                                                 (n = b without post_weight)
 *     h' = residual_scale * h + branch_scale * g * n     g: gate, sigmoid(gate)
 *                                                        or 1 without a gate
 *     x  = h' / sqrt(mean(h'^2) + eps) * (pre_weight + weight_offset)
 * in fp32, h' rounded once to the residual's type and x, which takes h' as
 * stored, once to bf16.  Without y, x is the norm of h itself. */
typedef struct {
  int32_t hidden;        /* H, a multiple of 8, at most 32768 */
  int32_t residual_type; /* moe_fp4_type of h and h_out */
  int32_t weight_type;   /* moe_fp4_type of post_weight, pre_weight and gate */
  int32_t gate;          /* moe_fp4_gate */
  int32_t gate_sigmoid;  /* 0 or 1 */
  float eps;             /* >= 0 */
  float residual_scale;  /* all finite */
  float branch_scale;
  float weight_offset;
} moe_fp4_norm_desc;

/* h: [M][H]; y, y2: bf16 [M][H] or NULL; gate: by desc->gate, NULL for
 * MOE_FP4_GATE_NONE; post_weight, pre_weight: [H] or NULL; h_out: [M][H],
 * given exactly when y is; x_out: bf16 [M][H], given exactly when pre_weight
 * is.  Device pointers, 16-byte aligned (a token gate: its element's size).
 * An output may be h, y or y2 itself where the types agree (h_out = h updates
 * the residual in place); any other overlap is refused, that with a gate of
 * [M][H] too.  M may be 0 (nothing is launched). */
moe_fp4_status moe_fp4_block_norm(const moe_fp4_norm_desc* desc, int32_t M, const void* h, const uint16_t* y,
                                  const uint16_t* y2, const void* gate, const void* post_weight,
                                  const void* pre_weight, void* h_out, uint16_t* x_out, void* stream);

/* ------------------------------------------------------------------------
 * From 16- and 32-bit experts to FP4 ones, and beside them: the quantisation
 * that makes the layer's weights, a linear map on FP4 activations, and the
 * parts of a layer whose experts are bf16, with their gradients (the routes'
 * grouping, products grouped by expert, the weighted join).  The conventions
 * above hold; outputs may not overlap anything that is read nor each other. */

/* FP4 quantisation of x [experts][rows][cols] (bf16 or fp32, a moe_fp4_type;
 * device, 16-byte aligned; rows `row_stride` values apart, a multiple of 8 (bf16)
 * or 4 (fp32) and cols at least, experts rows * row_stride) into codes
 * [experts][rows][cols / 2], the element of even index in the low nibble, and a
 * scale byte per block of G values along cols, [experts][rows][cols / G]: the
 * logical layout of moe_fp4_prepare.  cols: a multiple of G, at most 2^20.
 *   MXFP4 (G = 32): scale s = 2^(floor(log2(max |x|)) - 2) over the block, at
 *     least 2^-127 (OCP MX); code = x / s rounded to nearest-even E2M1, at most 6.
 *   NVFP4 (G = 16): s = max |x| / (6 g) rounded to nearest-even E4M3, at most 448;
 *     code = x / (s g) rounded to nearest-even E2M1, at most 6 (0 where s is 0);
 *     both roundings are those of the exact quotient.  g is the expert's global
 *     scale: global_scale [experts] where given (not negative, finite: a 0 makes
 *     codes and scales 0, anything else NaN scales), else the largest finite |x|
 *     of the expert over 2688 (= 6 * 448) in fp32, written to global_out
 *     [experts].  Exactly one of the two is given; MXFP4 takes neither.
 * A block that holds a NaN or an infinity gets the scale NaN (byte 255, E4M3
 * 0x7F) and codes 7.  The workspace is needed where global_out is
 * (moe_fp4_quantize_workspace_bytes; 0 otherwise and for MXFP4).  experts or
 * rows may be 0 (nothing is launched). */
moe_fp4_status moe_fp4_quantize_workspace_bytes(int32_t format, int64_t experts, size_t* bytes);
moe_fp4_status moe_fp4_quantize(int32_t format, int32_t type, const void* x, int64_t experts, int64_t rows,
                                int32_t cols, int64_t row_stride, uint8_t* codes, uint8_t* scales,
                                const float* global_scale, float* global_out, void* workspace, size_t workspace_bytes,
                                void* stream);

/* The values of codes and scales as moe_fp4_quantize lays them out: code *
 * scale in fp32, NVFP4 times global_scale [experts], rounded once more to bf16
 * where `type` says so.  out [experts][rows][cols], codes and out 16-byte aligned. */
moe_fp4_status moe_fp4_dequantize(int32_t format, int32_t type, const uint8_t* codes, const uint8_t* scales,
                                  const float* global_scale, int64_t experts, int64_t rows, int32_t cols, void* out,
                                  void* stream);

/* Linear map with MXFP4 weights and MXFP4 activations:
 *     y[n] = sum_k q(x)[k] * W[n][k]
 * where q(x) is x as moe_fp4_quantize gives it, on the matrix instruction's
 * form for two FP4 operands, with fp32 sums (a sum below 2^-126 may count as
 * zero).  An activation where asked for (the gated ones over gate and up rows),
 * one rounding to bf16.  M chooses the order of the sums and how the activation's
 * quotient is taken (divided, or multiplied by a reciprocal that may be off by
 * 2^-23 of itself), so that a token's last bit may change with M.  A block of x
 * that holds a NaN or an infinity makes its token's outputs NaN; other tokens
 * are not touched. */
typedef struct {
  int32_t in_features;  /* K, a multiple of 32, at most 2^20 */
  int32_t out_features; /* N, a multiple of 8, at most 2^26; K * N at most 2^31 */
  int32_t max_tokens;   /* capacity for workspace sizing, at most 2^20 */
  int32_t act_fn;       /* MOE_FP4_FN_NONE or a moe_fp4_act_fn */
  float act_alpha;      /* SWIGLUOAI only, else ignored */
  float act_beta;
  float act_limit;
} moe_fp4_linear_desc;

/* Bytes of the prepared weights, and the preparation, once per map: a
 * permutation of the bytes into `prepared` (device, 256-byte aligned).  codes
 * [N][K / 2] (device, 16-byte aligned), scales [N][K / 32]; for a gated
 * activation both hold the gate's rows and then the up's. */
moe_fp4_status moe_fp4_linear_prepared_bytes(const moe_fp4_linear_desc* desc, size_t* bytes);
moe_fp4_status moe_fp4_linear_prepare(const moe_fp4_linear_desc* desc, const uint8_t* codes, const uint8_t* scales,
                                      void* prepared, size_t prepared_bytes, void* stream);

/* Workspace bytes for calls on `desc` (device, 256-byte aligned), enough for
 * every M <= max_tokens; M is checked against max_tokens. */
moe_fp4_status moe_fp4_linear_workspace_bytes(const moe_fp4_linear_desc* desc, int32_t M, size_t* bytes);

/* The map on M tokens, x bf16 [M][K], or on tokens that are quantised already
 * (codes [M][K / 2], scales [M][K / 32]); out: bf16 [M][N], overwritten.  x,
 * codes and out are 16-byte aligned.  Neither out nor the workspace may overlap
 * each other or what is read.  M may be 0 (nothing is launched). */
moe_fp4_status moe_fp4_linear(const moe_fp4_linear_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                              uint16_t* out, void* workspace, size_t workspace_bytes, void* stream);
moe_fp4_status moe_fp4_linear_quantized(const moe_fp4_linear_desc* desc, const void* prepared, const uint8_t* codes,
                                        const uint8_t* scales, int32_t M, uint16_t* out, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Groups the routes topk_ids [tokens][top_k] by expert, in route order: expert
 * e's routes get the rows offsets[e] .. offsets[e + 1] - 1 (offsets int32 [E +
 * 1]); order int32 [tokens * top_k] holds each row's route t * top_k + j and
 * place int32 [tokens][top_k] each route's row.  A route whose id is negative or
 * >= E gets the place -1, and the rows from offsets[E] on the order -1.  E at
 * most 4096, tokens * top_k at most 2^22 (else MOE_FP4_EUNSUPPORTED).  Ids are
 * aligned to their size; tokens may be 0 (offsets are written). */
moe_fp4_status moe_fp4_group_routes_workspace_bytes(int32_t tokens, int32_t top_k, int32_t num_experts,
                                                    size_t* bytes);
moe_fp4_status moe_fp4_group_routes(const int32_t* topk_ids, int32_t tokens, int32_t top_k, int32_t num_experts,
                                    int32_t* offsets, int32_t* order, int32_t* place, void* workspace,
                                    size_t workspace_bytes, void* stream);
moe_fp4_status moe_fp4_group_routes_i64(const int64_t* topk_ids, int32_t tokens, int32_t top_k, int32_t num_experts,
                                        int32_t* offsets, int32_t* order, int32_t* place, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Rows in grouped order: out[p] = x[order[p] / top_k], zeros where order[p] is
 * negative.  x bf16 [tokens][hidden], out bf16 [tokens * top_k][hidden]; hidden
 * a multiple of 8, at most 2^15.  order and place (below) are what
 * moe_fp4_group_routes wrote; entries outside their range are not valid. */
moe_fp4_status moe_fp4_gather_routes(const uint16_t* x, const int32_t* order, int32_t tokens, int32_t top_k,
                                     int32_t hidden, uint16_t* out, void* stream);

/* The weighted join: out[t] = bf16(sum over j with place[t][j] >= 0, in the
 * order of j, of w[t][j] * y[place[t][j]]) in fp32; w fp32 [tokens][top_k], NULL
 * for ones (which makes it the gradient of moe_fp4_gather_routes).  y bf16
 * [tokens * top_k][hidden], out bf16 [tokens][hidden]. */
moe_fp4_status moe_fp4_combine_routes(const uint16_t* y, const int32_t* place, const float* w, int32_t tokens,
                                      int32_t top_k, int32_t hidden, uint16_t* out, void* stream);

/* Its gradients: dy[place[t][j]] = bf16(w[t][j] * dout[t]), zeros in the rows of
 * no route; dw[t][j] = sum_h dout[t][h] * y[place[t][j]][h] in fp32, 0 where
 * place is negative. */
moe_fp4_status moe_fp4_combine_routes_grad(const uint16_t* dout, const uint16_t* y, const int32_t* place,
                                           const int32_t* order, const float* w, int32_t tokens, int32_t top_k,
                                           int32_t hidden, uint16_t* dy, float* dw, void* stream);

/* Layout of a grouped weight: [E][out][in], or [E][in][out]. */
typedef enum {
  MOE_FP4_WEIGHT_OUT_IN = 0,
  MOE_FP4_WEIGHT_IN_OUT = 1
} moe_fp4_weight_layout;

/* Products grouped by expert over ragged rows, bf16 with fp32 sums.  Rows
 * offsets[e] .. offsets[e + 1] - 1 (offsets int32 [E + 1], device) belong to
 * expert e.  Offsets do not decrease and lie in [0, rows]; others give wrong
 * rows but no access out of range.  Rows of no expert (before offsets[0], from
 * offsets[E] on) are set to zeros. */
typedef struct {
  int32_t num_experts;   /* E, at most 4096 */
  int32_t in_features;   /* K, a multiple of 8, at most 2^20 */
  int32_t out_features;  /* N, a multiple of 8, at most 2^20 */
  int32_t weight_layout; /* moe_fp4_weight_layout */
} moe_fp4_grouped_desc;

/* y[t] = W[e(t)] x[t], rounded once to bf16.  x bf16 [rows][K], y bf16
 * [rows][N], rows at most 2^22, all 16-byte aligned.  The gradient of x is the
 * same call on dy with K and N swapped and the other weight layout. */
moe_fp4_status moe_fp4_grouped_linear(const moe_fp4_grouped_desc* desc, const uint16_t* x, int32_t rows,
                                      const uint16_t* weight, const int32_t* offsets, uint16_t* y, void* stream);

/* dW[e] = sum over e's rows t of dy[t] x[t]^T, [E][N][K] (MOE_FP4_WEIGHT_OUT_IN
 * only; for the other layout swap dy and x), bf16 or fp32 by `type`; zeros for
 * an expert without rows. */
moe_fp4_status moe_fp4_grouped_weight_grad(const moe_fp4_grouped_desc* desc, int32_t type, const uint16_t* dy,
                                           const uint16_t* x, int32_t rows, const int32_t* offsets, void* dw,
                                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP4_H */

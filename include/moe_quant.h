/*
 * moe_quant.h - C ABI of libmoe_quant.so: the routed MoE expert layer with
 * block-quantized expert weights on AMD Instinct MI355X (gfx950).
 *
 * What the layer computes.  The model cards describe the thinker's routed
 * experts kept packed in GPU memory and dequantized per layer "just in time"
 * for one grouped matmul ("clef-omni-fp8" card, section "How this checkpoint
 * runs"; "clef-omni-int4" card, section "How this checkpoint runs";
 * "clef-omni-NVFP4" card, section "How it was made").  For T tokens with
 * hidden states x[T, H] and router logits l[T, E]:
 *
 *   ids[t, 0..k)  = the k largest logits of token t, in descending order, ties
 *                   to the lower expert id;
 *   w[t, j]       = softmax over the k selected logits;
 *   y[t]          = sum_j w[t, j] * W2[e] (silu(G) * U),   e = ids[t, j],
 *                   [G; U] = W13[e] x[t]  (gate rows first, then up rows),
 *                   silu(z) = z / (1 + exp(-z));
 *   out[t]        = bf16(y[t])  or  bf16(residual[t] + y[t]).
 *
 * W13[e] is [2I, H], W2[e] is [H, I]; both are stored per expert, stacked over
 * experts, row major with the input dimension K contiguous, in one of three
 * packed formats (see mq_wformat).  The router itself is not part of the
 * path: it stays a BF16 linear layer on every card ("clef-omni-int4" card,
 * section "Recipe": ignore_layers=mlp.gate); moe_quant_forward takes its
 * logits as an input, and moe_quant_forward_with_router computes them from
 * the gate's weight in the same kernel as the top-k.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers, owned by the caller, row major
 *    and contiguous.  The library never allocates device memory, never copies
 *    weights and keeps no device state: init only borrows the weight pointers
 *    for the lifetime of the handle.
 *  - Every entry point returns an mq_status.  Argument checks run on the host
 *    before anything is enqueued; on failure nothing is enqueued and
 *    moe_quant_last_error() holds a one-line explanation (thread local).
 *    Nothing is printed and no exception crosses the ABI.
 *  - Work is enqueued asynchronously on the caller's HIP stream (a
 *    hipStream_t, passed as struct ihipStream_t *; NULL is the default stream).
 *  - A handle is immutable after init: concurrent forward calls, from any host
 *    threads, on different streams are safe as long as each uses its own
 *    workspace (the library's launch-shape caches are guarded by a lock).
 */
#ifndef MOE_QUANT_H
#define MOE_QUANT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_QUANT_ABI_VERSION 1u

struct ihipStream_t; /* hipStream_t */
struct ihipEvent_t;  /* hipEvent_t  */

typedef enum {
  MQ_OK = 0,
  MQ_E_NULL = 1,      /* a required pointer is NULL                                  */
  MQ_E_SHAPE = 2,     /* a dimension is out of range or not a multiple of the block  */
  MQ_E_ALIGN = 3,     /* a pointer is not aligned as required                        */
  MQ_E_FORMAT = 4,    /* unknown weight format                                       */
  MQ_E_DTYPE = 5,     /* unknown logits dtype                                        */
  MQ_E_WORKSPACE = 6, /* workspace NULL or smaller than moe_quant_workspace_size()   */
  MQ_E_ABI = 7,       /* descriptor built against another MOE_QUANT_ABI_VERSION      */
  MQ_E_HIP = 8,       /* a HIP launch or runtime call failed                         */
  MQ_E_OVERFLOW = 9   /* an FP16 intermediate saturated (moe_quant_check)           */
} mq_status;

/*
 * Packed weight formats.  N is a projection's output dim and K its input dim
 * (W13: N = 2I, K = H; W2: N = H, K = I).  4-bit codes are packed two per
 * byte, the even k in the low nibble.
 *
 * MQ_W_INT4_G128  INT4 W4A16, symmetric, one scale per 128 consecutive k of a
 *                 row ("clef-omni-int4" card, intro and section "What was
 *                 quantized").
 *     w      uint8   [E, N, K/2]    nibble c = q + 8 (offset binary)
 *     scale  float16 [E, N, K/128]
 *     weight = (c - 8) * scale[n, k/128]
 *
 * MQ_W_FP8_B128   FP8 E4M3 (OCP E4M3FN: bias 7, max 448, 0x7F/0xFF NaN) with
 *                 one FP32 scale per 128x128 block ("clef-omni-fp8" card,
 *                 sections "What was quantized" and "Recipe"; the stored scale
 *                 is weight_scale_inv, the dequantization multiplier).
 *     w      uint8   [E, N, K]      E4M3FN bits
 *     scale  float32 [E, N/128, K/128]
 *     weight = e4m3(w) * scale[n/128, k/128]
 *
 * MQ_W_NVFP4_G16  NVFP4: FP4 E2M1 values, one E4M3 scale per 16 weights along
 *                 k, one FP32 global scale per expert matrix
 *                 ("clef-omni-NVFP4" card, section "How it was made"; gate and
 *                 up are one concatenated matrix and share its global scale).
 *     w      uint8   [E, N, K/2]    E2M1 nibbles (bit 3 = sign)
 *     scale  uint8   [E, N, K/16]   E4M3FN bits
 *     gscale float32 [E]            global scale g = 448*6/amax
 *     weight = e2m1(c) * e4m3(scale[n, k/16]) / gscale[e]
 *
 * Dimension limits of this version: H and I multiples of 128 for every format,
 * 128 <= H, I <= 4608 (the decode GEMM stages 16 whole input rows of a
 * projection in the 160 KiB LDS of one workgroup), 1 <= k <= E <= 512, k <= 64.
 * The NVFP4 format itself only needs multiples of 16; this version's GEMM
 * tiles (128-wide k blocks and 128-row weight tiles) take multiples of 128
 * for NVFP4 too, which every Clef shape satisfies (hidden 2048, intermediate
 * 768).
 */
typedef enum { MQ_W_INT4_G128 = 1, MQ_W_FP8_B128 = 2, MQ_W_NVFP4_G16 = 3 } mq_wformat;

/* Router-logit element type; BF16 logits are widened exactly to FP32. */
typedef enum { MQ_F32 = 0, MQ_BF16 = 1 } mq_dtype;

typedef struct {
  uint32_t abi_version; /* must equal MOE_QUANT_ABI_VERSION                      */
  int32_t num_experts;  /* E                                                      */
  int32_t hidden;       /* H                                                      */
  int32_t intermediate; /* I (per expert)                                         */
  int32_t top_k;        /* k                                                      */
  int32_t format;       /* mq_wformat                                             */
  const void *w13;      /* gate_up weights [E, 2I, .], 16-byte aligned            */
  const void *w13_scale;/* its scales, 16-byte aligned                            */
  const float *w13_gscale; /* NVFP4 only: [E]; must be NULL for the other formats */
  const void *w2;       /* down weights [E, H, .], 16-byte aligned                */
  const void *w2_scale;
  const float *w2_gscale;
} mq_layer_desc;

typedef struct mq_layer mq_layer; /* opaque host object */

/* Stages of one forward call, in launch order (for mq_probe.events). */
enum {
  MQ_STAGE_ROUTE = 0,   /* top-k + softmax + FP16 staging of the hidden rows */
  MQ_STAGE_PERMUTE = 1, /* histogram, scan and stable grouping by expert     */
  MQ_STAGE_GATE_UP = 2, /* grouped gate/up GEMM with SwiGLU epilogue         */
  MQ_STAGE_DOWN = 3,    /* grouped down GEMM, routing-weighted per slot      */
  MQ_STAGE_COMBINE = 4, /* slot-ordered sum (+ residual), BF16 rounding      */
  MQ_NUM_STAGES = 5
};

/*
 * Optional extra outputs of a forward call, for tests and profiling.  Every
 * field may be NULL.  Device arrays are written in stream order:
 *   topk_ids         int32 [T, k]   selected experts, descending logit
 *   topk_w           float [T, k]   routing weights
 *   expert_offsets   int32 [E + 1]  grouped row range of each expert
 *   sorted_token_ids int32 [T * k]  token of each grouped row (experts
 *                                   ascending, tokens ascending inside one)
 *   inv_pos          int32 [T * k]  grouped row of slot t * k + j
 *   h                uint16 [T*k, I] FP16 bits of the SwiGLU intermediate in
 *                                   grouped row order
 * events[2 * s] / events[2 * s + 1] (hipEvent_t, created by the caller) are
 * recorded on the stream right before / after stage s; for the two GEMM
 * stages the runtime takes them at the start and the end of the GEMM kernel
 * itself (hipExtLaunchKernel), so they exclude the gap before its dispatch.
 */
typedef struct {
  int32_t *topk_ids;
  float *topk_w;
  int32_t *expert_offsets;
  int32_t *sorted_token_ids;
  int32_t *inv_pos;
  uint16_t *h;
  struct ihipEvent_t *events[2 * MQ_NUM_STAGES];
} mq_probe;

/*
 * Validate a layer descriptor and create a handle.  Host only: no HIP call is
 * made.  On MQ_OK *out holds a handle to release with moe_quant_destroy.
 * Errors: MQ_E_NULL (d, out or a weight pointer NULL; gscale NULL for NVFP4),
 * MQ_E_ABI, MQ_E_FORMAT, MQ_E_SHAPE (a dimension outside the limits above),
 * MQ_E_ALIGN.
 */
mq_status moe_quant_init(const mq_layer_desc *d, mq_layer **out);

/*
 * Device workspace bytes that one forward call over num_tokens tokens needs
 * (256-byte aligned start required).  num_tokens >= 0.  Host only.
 */
mq_status moe_quant_workspace_size(const mq_layer *L, int64_t num_tokens, size_t *bytes);

/*
 * Enqueue one layer forward on `stream`.
 *   router_logits  [T, E] of logits_dtype, 16-byte aligned
 *   hidden_bf16    [T, H] BF16 bits, 16-byte aligned
 *   residual_bf16  NULL, or [T, H]: then out = bf16(residual + moe(hidden))
 *   out_bf16       [T, H] BF16 bits, 16-byte aligned; may alias residual_bf16
 *   workspace      >= moe_quant_workspace_size(L, T) bytes, 256-byte aligned;
 *                  its contents on entry do not matter
 *   probe          NULL, or extra outputs (see mq_probe)
 * num_tokens == 0 returns MQ_OK without enqueuing anything.  Inputs must not
 * hold NaN or Inf; results are then unspecified but every access stays in
 * bounds.  Returns MQ_E_HIP if a launch fails.
 */
mq_status moe_quant_forward(const mq_layer *L, const void *router_logits, int32_t logits_dtype,
                            const uint16_t *hidden_bf16, const uint16_t *residual_bf16,
                            int64_t num_tokens, uint16_t *out_bf16, void *workspace,
                            size_t workspace_bytes, const mq_probe *probe,
                            struct ihipStream_t *stream);

/*
 * W8A8 block FP8: moe_quant_forward for an MQ_W_FP8_B128 layer with its
 * activations quantized to FP8 as the "clef-omni-fp8" card (table "What was
 * quantized") runs them in engines, "dynamic FP8 per 1x128 group": for each
 * token (gate/up input) and each grouped row (down input) and each 128
 * consecutive input features, s = amax / 448 (FP32) and code =
 * RNE-to-E4M3(x / s) saturated to +-448; the SwiGLU intermediate is quantized
 * from its FP32 value.  Both GEMMs run on the FP8 matrix units, the
 * activation and weight scales multiplying each 128-wide k block's FP32
 * partial sum.  Same arguments, workspace size and routing as
 * moe_quant_forward (the kernels are the many-rows-per-expert ones at every
 * batch size).  The probe's h buffer (T*k*I*2 bytes) receives h as kept
 * here: the E4M3 codes uint8 [T*k, I] in grouped row order, followed by their
 * FP32 scales [T*k, I/128].  Errors: as moe_quant_forward, plus MQ_E_FORMAT
 * for another weight format.
 */
mq_status moe_quant_forward_w8a8(const mq_layer *L, const void *router_logits, int32_t logits_dtype,
                                 const uint16_t *hidden_bf16, const uint16_t *residual_bf16,
                                 int64_t num_tokens, uint16_t *out_bf16, void *workspace,
                                 size_t workspace_bytes, const mq_probe *probe,
                                 struct ihipStream_t *stream);

/*
 * Test entry: the dynamic 1x128 FP8 activation quantizer of the W8A8 path on
 * FP32 rows x [rows, K] (device), writing codes uint8 [rows, K] (E4M3FN bits)
 * and scales float [rows, K/128] (device, caller-owned), with the same group
 * arithmetic the W8A8 kernels apply to hidden rows and to the SwiGLU
 * intermediate.  K a positive multiple of 128 (at most 65536).
 * Errors: MQ_E_SHAPE, MQ_E_NULL, MQ_E_ALIGN, MQ_E_HIP.
 */
mq_status moe_quant_quantize_act(const float *x, int64_t rows, int32_t K, uint8_t *codes, float *scales,
                                 struct ihipStream_t *stream);

/*
 * NVFP4 W4A4: moe_quant_forward for an MQ_W_NVFP4_G16 layer with its
 * activations quantized to NVFP4 as well, the format the
 * "clef-flash-NVFP4-Hybrid" card (section "Quantization details") gives its
 * W4A4 layers and the "clef-omni-fp8" card (table "Which Clef-Omni quant
 * should I use?") lists for the W4A4 build: E2M1 values, one E4M3 scale per
 * 16 consecutive values, one FP32 global scale per tensor, the activation
 * global scales calibrated.  act_gscale13 is the global scale g of the
 * gate/up input (the hidden rows), act_gscale2 that of the down input (the
 * SwiGLU intermediate), one per layer, shared by its experts.  For each
 * token (gate/up) or grouped row (down) and each 16 consecutive features
 * with maximum magnitude m, in FP32:
 *   s = RNE-to-E4M3(min((m * g) / 6, 448)),
 *   code = RNE-to-E2M1((x * g) / s) saturated to +-6 (0 where s = 0),
 * and the projection sees e2m1(code) * s / g; the intermediate is quantized
 * from its FP32 value.  The GEMMs multiply the exact products e2m1 * s on the
 * FP16 matrix units and apply 1 / g to their FP32 sums.  Same arguments,
 * workspace size and routing as moe_quant_forward (the kernels are the
 * many-rows-per-expert ones at every batch size).  The probe's h buffer
 * receives the down input as kept here: FP16 values e2m1(code) * s [T*k, I]
 * in grouped row order.  Errors: as moe_quant_forward, plus MQ_E_FORMAT for
 * another weight format and MQ_E_SHAPE for a global scale that is not
 * finite and positive.
 */
mq_status moe_quant_forward_w4a4(const mq_layer *L, const void *router_logits, int32_t logits_dtype,
                                 const uint16_t *hidden_bf16, const uint16_t *residual_bf16,
                                 int64_t num_tokens, uint16_t *out_bf16, void *workspace,
                                 size_t workspace_bytes, float act_gscale13, float act_gscale2,
                                 const mq_probe *probe, struct ihipStream_t *stream);

/*
 * Test entry: the NVFP4 activation quantizer of the W4A4 path on FP32 rows
 * x [rows, K] (device) with global scale gscale, writing the E2M1 codes
 * packed two per byte, even k in the low nibble, uint8 [rows, K/2], and the
 * E4M3FN block scales uint8 [rows, K/16] (device, caller-owned): the NVFP4
 * layout of MQ_W_NVFP4_G16 weights.  K a positive multiple of 16 (at most
 * 65536); gscale finite and positive.
 * Errors: MQ_E_SHAPE, MQ_E_NULL, MQ_E_ALIGN (x 16-byte, codes 4-byte), MQ_E_HIP.
 */
mq_status moe_quant_quantize_act_nvfp4(const float *x, int64_t rows, int32_t K, float gscale,
                                       uint8_t *codes, uint8_t *scales, struct ihipStream_t *stream);

/*
 * moe_quant_forward with the router in the library: the logits of the BF16
 * gate that stays unquantized on every card ("clef-omni-int4" card, section
 * "Recipe": ignore_layers=mlp.gate; "clef-omni-NVFP4" card, section "How it
 * was made": the router is copied unchanged), read as a linear layer without
 * bias, logits[t, e] = sum_h hidden[t, h] * router[e, h], are computed and
 * selected in one kernel from 4096 tokens up: each block of 16 or 32 tokens
 * keeps its FP32 logits on chip and runs the top-k there (same order, ties
 * and weights as moe_quant_forward).  Smaller batches run the router logits
 * kernel into the workspace and then the logits-driven routing kernel, which
 * is faster there.  The rest of the path is moe_quant_forward's.
 *   hidden_bf16   [T, H] BF16 bits, 16-byte aligned
 *   router_bf16   [E, H] BF16 bits (the gate's weight), 16-byte aligned
 *   residual_bf16, num_tokens, out_bf16, workspace, workspace_bytes, probe,
 *   stream        as for moe_quant_forward (same workspace size)
 *   logits_out    NULL, or float [T, E] (4-byte aligned): receives the FP32
 *                 logits the top-k decided on (for tests)
 * Products are exact in FP32 and summed in FP32 by the matrix units in a fixed
 * order, so repeated calls are bit-identical.  E at most 256.
 * Errors: as moe_quant_forward (MQ_E_NULL when router_bf16 is NULL,
 * MQ_E_SHAPE when E > 256).
 */
mq_status moe_quant_forward_with_router(const mq_layer *L, const uint16_t *hidden_bf16,
                                        const uint16_t *router_bf16,
                                        const uint16_t *residual_bf16, int64_t num_tokens,
                                        uint16_t *out_bf16, void *workspace,
                                        size_t workspace_bytes, float *logits_out,
                                        const mq_probe *probe, struct ihipStream_t *stream);

/*
 * Synchronize `stream` and report whether the last forward that used
 * `workspace` saturated one of its FP16 intermediates (the SwiGLU output h or a
 * routing-weighted per-slot expert output; values beyond +-65504 are clamped):
 * MQ_OK if not, MQ_E_OVERFLOW if it did.  workspace as passed to forward.
 * Batches of one or two tokens keep the per-slot outputs in FP32 (the down
 * projection adds them into the output itself), so there only h can saturate.
 */
mq_status moe_quant_check(const mq_layer *L, const void *workspace, struct ihipStream_t *stream);

/*
 * Test entry: enqueue the dequantization of one expert matrix through the
 * device unpack paths the GEMMs use, writing float32 [N, K] to `out`
 * (which: 0 = W13 [2I, H], 1 = W2 [H, I]).  Each value is the format's
 * definition evaluated in FP32 with at most one rounding: INT4 (c - 8) * s is
 * exact; FP8 e4m3 * scale is one FP32 multiply; NVFP4 (e2m1 * e4m3) is exact
 * and is then divided by gscale (one IEEE FP32 division).
 * Errors: MQ_E_NULL, MQ_E_SHAPE (which or expert out of range), MQ_E_HIP.
 */
mq_status moe_quant_dequantize(const mq_layer *L, int32_t which, int32_t expert, float *out,
                               struct ihipStream_t *stream);

/*
 * Router logits of the gate that stays in BF16 ("clef-omni-fp8" card, section
 * "What was quantized"; "clef-omni-NVFP4" card, section "How it was made"),
 * read as a linear layer without bias:
 *   logits_f32[t, e] = sum_h hidden_bf16[t, h] * router_bf16[e, h]
 *   hidden_bf16  [T, H] BF16 bits, row-major, 16-byte aligned
 *   router_bf16  [E, H] BF16 bits, row-major (the gate's weight), 16-byte aligned
 *   logits_f32   [T, E] float32, row-major, 16-byte aligned; written here, and
 *                ready for moe_quant_forward with logits_dtype MQ_F32
 * All three live in device memory owned by the caller; nothing is kept after
 * the call.  Products are exact in FP32 and summed in FP32 by the matrix
 * units (an order of their own).  hidden a positive multiple of 64 (at most
 * 65536), 1 <= num_experts <= 65536, 0 <= num_tokens <= 2^22; num_tokens == 0
 * returns MQ_OK without enqueuing anything.  No layer handle is needed.
 * Errors: MQ_E_SHAPE, MQ_E_NULL, MQ_E_ALIGN, MQ_E_HIP (launch failed).
 */
mq_status moe_quant_router_logits(const uint16_t *hidden_bf16, const uint16_t *router_bf16,
                                  int64_t num_tokens, int32_t hidden, int32_t num_experts,
                                  float *logits_f32, struct ihipStream_t *stream);

/*
 * The gate of a routed layer: which experts a token takes and with which
 * weights, from its router logits l[t, e].  In real arithmetic:
 *   s[t, e]  = sigmoid(l), or softmax of the token's logits over all E;
 *   c[t, e]  = s + bias[e], the selection score (without a bias the logits'
 *              own order, which is the scores');
 *   groups   : experts e / (E / num_groups) form a group; a group's score is the
 *              largest c in it (group_top 1) or the sum of its two largest
 *              (group_top 2), and the topk_groups best groups are kept, ties
 *              to the lower group;
 *   ids[t]   = the k largest c of the kept groups' experts, in descending
 *              order, ties to the lower expert id;
 *   w[t, j]  = s of the selected experts, divided by their sum if renormalize
 *              is not 0, times scale (the bias does not enter the weights).
 * The selection compares the scores in 64 bits, so scores that differ by less
 * than a 32-bit rounding are still told apart.
 * Masked experts: an expert whose logit or bias is -inf or NaN has c = -inf and
 * weight 0.  It is selected only where fewer than k experts of the kept groups
 * are left, lower ids first; a row without any live expert has weights 0 and k
 * distinct valid ids.  A logit or bias of +inf counts as the largest finite
 * float.
 */
typedef enum { MQ_SCORE_SOFTMAX = 0, MQ_SCORE_SIGMOID = 1 } mq_score;

typedef struct {
  uint32_t abi_version; /* must equal MOE_QUANT_ABI_VERSION                        */
  int32_t num_experts;  /* E, 1 to 512                                              */
  int32_t top_k;        /* k, 1 to min(64, topk_groups * E / num_groups)            */
  int32_t score;        /* mq_score                                                 */
  int32_t num_groups;   /* 1 (no groups) to 64, a divisor of E                      */
  int32_t topk_groups;  /* groups kept, 1 to num_groups                             */
  int32_t group_top;    /* 1 or 2 (2 needs groups of two experts or more)           */
  int32_t renormalize;
  float scale;          /* finite                                                   */
  const float *bias;    /* NULL, or [E] on the device, 4-byte aligned               */
} mq_gate;

/*
 * Enqueue the gate of num_tokens tokens on `stream`.
 *   logits   [T, E] of logits_dtype, 16-byte aligned
 *   ids      int32 [T, k], weights float [T, k]: written, 4-byte aligned
 * num_tokens == 0 returns MQ_OK without enqueuing anything.  No layer handle
 * and no workspace are needed.
 * Errors: MQ_E_NULL, MQ_E_ABI, MQ_E_SHAPE (a field outside its range, scale not
 * finite), MQ_E_DTYPE, MQ_E_ALIGN, MQ_E_HIP.
 */
mq_status moe_quant_gate_topk(const mq_gate *g, const void *logits, int32_t logits_dtype,
                              int64_t num_tokens, int32_t *ids, float *weights,
                              struct ihipStream_t *stream);

/*
 * moe_quant_forward under a gate: the experts and weights of mq_gate in the
 * place of the softmax over the k largest logits, the rest of the path the
 * same.  The gate's num_experts and top_k are the layer's.
 *   router_logits  [T, E] of logits_dtype, or NULL with
 *   router_bf16    [E, H] BF16 bits (the gate's weight): then the logits are
 *                  computed here, as moe_quant_router_logits does
 *   activations    mq_act: MQ_ACT_BF16 (moe_quant_forward), MQ_ACT_FP8
 *                  (moe_quant_forward_w8a8, FP8 layers) or MQ_ACT_NVFP4
 *                  (moe_quant_forward_w4a4, NVFP4 layers, with its act_gscales)
 *   logits_out     NULL, or float [T, E] that receives the logits computed here
 *   the others     as for moe_quant_forward; masked logits (-inf, NaN) are those
 *                  of mq_gate
 * The per-slot products of weight and expert output are rounded to FP16, which
 * has all of its digits between 2^-14 and 65504.  Where a token's largest weight
 * is above 1 or below 2^-7, a power of two that brings it to [1/2, 1) is taken out
 * of its weights first and multiplied back after the sum, so the size of the
 * weights costs no digits; largest weights from 2^-7 to 1 are taken as they are,
 * as moe_quant_forward takes its own.
 * A layer of one expert with top_k 1, MQ_SCORE_SIGMOID and renormalize 0 is a
 * shared expert with its sigmoid gate.
 * Errors: as moe_quant_forward and moe_quant_gate_topk, MQ_E_NULL unless
 * exactly one of router_logits and router_bf16 is given, MQ_E_SHAPE where gate
 * and layer differ, MQ_E_FORMAT for activations that the layer's format lacks.
 */
typedef enum { MQ_ACT_BF16 = 0, MQ_ACT_FP8 = 1, MQ_ACT_NVFP4 = 2 } mq_act;

mq_status moe_quant_forward_gated(const mq_layer *L, const mq_gate *gate, const void *router_logits,
                                  int32_t logits_dtype, const uint16_t *router_bf16,
                                  const uint16_t *hidden_bf16, const uint16_t *residual_bf16,
                                  int64_t num_tokens, uint16_t *out_bf16, void *workspace,
                                  size_t workspace_bytes, int32_t activations, float act_gscale13,
                                  float act_gscale2, float *logits_out, const mq_probe *probe,
                                  struct ihipStream_t *stream);

/*
 * Norms before and after a block in one pass over each row, with the block's
 * gate, the residual scale and the residual add between them:
 *   z  = x,  or with post_weight  x / sqrt(mean(x^2) + eps) * (offset + post_weight);
 *   r' = round(residual + scale * gate * z)        to residual_dtype;
 *   n  = bf16(r' / sqrt(mean(r'^2) + eps) * (offset + pre_weight)),
 * the mean over the row's hidden values, all in FP32.  x is a block's output
 * (the layer's, for instance), n the next block's input.  n is computed from
 * the rounded r', so one call gives the same bits as two (x and post_weight
 * first, then residual = r' and pre_weight).  Squares are summed in FP32:
 * values beyond 2^55 in magnitude are outside of this entry's range (eps covers
 * what small squares lose).
 */
typedef enum {
  MQ_GATE_NONE = 0,
  MQ_GATE_CHANNEL = 1, /* gate [H]: one factor per channel           */
  MQ_GATE_TOKEN = 2,   /* gate [T]: one factor per token             */
  MQ_GATE_FULL = 3     /* gate [T, H]                                */
} mq_gate_kind;

typedef struct {
  uint32_t abi_version;   /* must equal MOE_QUANT_ABI_VERSION              */
  int32_t hidden;         /* H, 1 to 32768                                  */
  int32_t residual_dtype; /* mq_dtype of residual and residual_out          */
  int32_t weight_dtype;   /* mq_dtype of post_weight and pre_weight         */
  float eps;              /* finite and at least 1e-30                      */
  float weight_offset;    /* finite: 0, or 1 where weights are stored as w - 1 */
  float scale;            /* finite                                         */
  const void *post_weight;/* NULL (no norm after the block) or [H]          */
  const void *pre_weight; /* NULL (no norm before the next block) or [H]    */
} mq_norm;

/*
 * Enqueue the norms of num_tokens rows on `stream`.  All arrays are 16-byte
 * aligned, a per-token gate to its element.
 *   x_bf16        [T, H] BF16 bits; NULL (then post_weight and gate are NULL
 *                 and r' = residual)
 *   residual      [T, H]; NULL counts as zero
 *   gate          NULL for MQ_GATE_NONE, else of gate_dtype and the kind's shape
 *   residual_out  [T, H], NULL if not wanted; may alias residual
 *   norm_out_bf16 [T, H]: given if and only if pre_weight is; may alias x_bf16
 * At least one of x and residual and one of the outputs is given.
 * num_tokens == 0 returns MQ_OK without enqueuing anything.
 * Errors: MQ_E_NULL, MQ_E_ABI, MQ_E_SHAPE (a field outside its range, an unknown
 * gate kind), MQ_E_DTYPE, MQ_E_ALIGN, MQ_E_HIP.
 */
mq_status moe_quant_norm(const mq_norm *n, const uint16_t *x_bf16, const void *residual,
                         const void *gate, int32_t gate_kind, int32_t gate_dtype, int64_t num_tokens,
                         void *residual_out, uint16_t *norm_out_bf16, struct ihipStream_t *stream);

/*
 * Matrix product on E4M3 weights with a scale for each block of 128: a dense
 * projection in the FP8 layer's weight format (its shared or dense layers, the
 * projections around the attention), the rows in E4M3 per 128 values:
 *   sa[t, g] = max |x[t, k]| * (1 / 448) over the k of block g = k / 128, an FP32
 *              product with the FP32 number next to 1 / 448 (1 where that is 0),
 *   a[t, k]  = RNE-to-E4M3(x[t, k] / sa[t, g]) saturated to +-448, one IEEE FP32
 *              division,
 *   y[t, n]  = sum_g (sa[t, g] * scale[n / 128, g]) * sum_{k in g} a[t, k] * w[n, k],
 *   out      = round(y + residual) to out_dtype,
 * sums, and the product of the two scales, in FP32.
 * The scale is what a division by the number 448 gives in PyTorch on a GPU, which
 * multiplies by the reciprocal.  forward_w8a8's sa is the quotient: for 71 of the 128
 * mantissas of a block's maximum it is the next smaller FP32 number, and one code in
 * 900 differs by a step (3e-3 of the rows in the 2-norm, where quantizing them costs
 * 2.6e-2).
 * For an FP32 output the products of codes are exact; for a BF16 one they come from
 * the FP8 matrix units, which cut the 128 products of a block at 2^-16 of their
 * largest: the block's sum is off by 6e-5 of the largest in the mean, by 2^-10.8 at
 * most on random codes.  N and K need not fill their last block.  A weight code of
 * NaN (0x7F, 0xFF) makes its output column NaN, a NaN or an infinity in x its output
 * row.
 */
typedef struct {
  uint32_t abi_version; /* must equal MOE_QUANT_ABI_VERSION                          */
  int32_t n;            /* N output features, 1 to 2^20                                */
  int32_t k;            /* K input features, a multiple of 16, 16 to 65536             */
  int32_t out_dtype;    /* mq_dtype of out                                             */
  const uint8_t *w;     /* E4M3FN bits [N, K], 16-byte aligned                         */
  const float *scale;   /* [ceil(N / 128), ceil(K / 128)], 4-byte aligned              */
} mq_linear;

/*
 * Device workspace bytes of moe_quant_linear over num_tokens tokens (the
 * activation codes and their scales).  Host only.
 */
mq_status moe_quant_linear_workspace_size(const mq_linear *l, int64_t num_tokens, size_t *bytes);

/*
 * Enqueue the product of num_tokens rows on `stream`.
 *   x_bf16        [T, K] BF16 bits, 16-byte aligned
 *   residual_bf16 NULL, or [T, N] BF16 bits, 2-byte aligned
 *   out           [T, N] of out_dtype, aligned to its element; a BF16 one may be
 *                 residual_bf16 itself; otherwise it overlaps nothing that is read
 *   workspace     >= moe_quant_linear_workspace_size bytes, 256-byte aligned; its
 *                 contents on entry do not matter; overlaps nothing else
 * num_tokens == 0 returns MQ_OK without enqueuing anything.
 * Errors: MQ_E_NULL, MQ_E_ABI, MQ_E_SHAPE, MQ_E_DTYPE, MQ_E_ALIGN,
 * MQ_E_WORKSPACE, MQ_E_HIP.
 */
mq_status moe_quant_linear(const mq_linear *l, const uint16_t *x_bf16, const uint16_t *residual_bf16,
                           int64_t num_tokens, void *out, void *workspace, size_t workspace_bytes,
                           struct ihipStream_t *stream);

/*
 * A paged cache of keys and values.  Page p holds page_size tokens of a request,
 * one head after the other; token s of it is "slot" p * page_size + s, and which
 * pages a request has, in order, stands in its row of a block table.
 */
typedef enum { MQ_KV_BF16 = 0, MQ_KV_FP8 = 1 } mq_kv_dtype;

typedef struct {
  uint32_t abi_version; /* must equal MOE_QUANT_ABI_VERSION                          */
  int32_t kv_heads;     /* 1 to 1024                                                   */
  int32_t head_dim;     /* D, a multiple of 16, 16 to 256                              */
  int32_t page_size;    /* a power of two, 1 to 1024                                   */
  int64_t num_pages;    /* at least 1; num_pages * page_size below 2^31                */
  int32_t dtype;        /* mq_kv_dtype                                                 */
  float k_scale;        /* MQ_KV_FP8: a key is e4m3 * k_scale, a value e4m3 * v_scale; */
  float v_scale;        /* finite and positive, 1 for MQ_KV_BF16                       */
  void *k, *v;          /* [num_pages, kv_heads, page_size, D], 16-byte aligned        */
} mq_kv_cache;

/*
 * What happens to a head's query and key before attention, in FP32 and rounded
 * once at the end:
 *   h = x,  or with a norm weight  x / sqrt(mean(x^2) + eps) * weight   (mean over D,
 *   finite values of any size);
 *   the first rot_dim values of h are turned by the angles of the token's
 *   position, in pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved:
 *     (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i).
 * cos_sin [max_positions, rot_dim] holds, for each position, the rot_dim / 2
 * cosines and then the sines, so any scaling of the angles is the caller's.
 */
typedef struct {
  uint32_t abi_version;  /* must equal MOE_QUANT_ABI_VERSION                         */
  int32_t head_dim;      /* D of the cache                                             */
  int32_t rot_dim;       /* 0 (no rotation) or a multiple of 16 up to D                */
  int32_t interleaved;
  int32_t max_positions; /* rows of cos_sin; not used if rot_dim is 0                  */
  float eps;             /* finite and at least 1e-30                                  */
  const float *cos_sin;  /* 16-byte aligned; NULL if and only if rot_dim is 0          */
  const uint16_t *q_norm, *k_norm; /* NULL, or [D] BF16 bits, 16-byte aligned          */
} mq_rotary;

/*
 * Enqueue, on `stream`, the queries of num_tokens tokens and the appending of
 * their keys and values to the cache.
 *   q           [T, q_heads, D] BF16 bits, tokens q_stride values apart, or NULL with
 *               q_heads 0: no queries
 *   k, v        [T, kv_heads, D] BF16 bits, tokens k_stride and v_stride values apart
 *               (so the three may lie in one row of a fused projection); all
 *               16-byte aligned, strides multiples of 8
 *   positions   int32 [T]: rows of cos_sin; NULL if rot_dim is 0
 *   slots       int32 [T]: where the token's key and value go.  A token whose slot
 *               is negative or behind the cache, or whose position is not a row of
 *               cos_sin, is padding: nothing of it is written
 *   q_out       [T, q_heads, D] BF16 bits, 16-byte aligned; may be q itself where
 *               q_stride is q_heads * D, and overlaps nothing else that is read
 * The cache's k and v overlap neither each other nor q_out nor what is read.
 * MQ_KV_FP8 keeps RNE-to-E4M3(value / scale), one IEEE FP32 division, saturated to
 * +-448.  The slots of one call are distinct: of a slot given twice it is
 * unspecified which token's values stay, per 8 values.
 * num_tokens == 0 returns MQ_OK without enqueuing anything.
 * Errors: MQ_E_NULL, MQ_E_ABI, MQ_E_SHAPE, MQ_E_DTYPE, MQ_E_ALIGN, MQ_E_HIP.
 */
mq_status moe_quant_kv_append(const mq_kv_cache *c, const mq_rotary *r, int32_t q_heads,
                              const uint16_t *q, int64_t q_stride, const uint16_t *k,
                              int64_t k_stride, const uint16_t *v, int64_t v_stride,
                              const int32_t *positions, const int32_t *slots, int64_t num_tokens,
                              uint16_t *q_out, struct ihipStream_t *stream);

/*
 * Device workspace bytes of moe_quant_attend over up to `batch` requests, for any
 * lengths: never less for more requests (256-byte aligned start required).  Host only.
 */
mq_status moe_quant_attend_workspace_size(const mq_kv_cache *c, int32_t q_heads, int64_t batch,
                                          size_t *bytes);

/*
 * Enqueue, on `stream`, the attention of one new token of each request over the
 * request's cached tokens (its own among them).  Query head h reads key and
 * value head h / (q_heads / kv_heads).  For a request of `length` tokens, over
 * its tokens j < length, with a window only the last `window` of them:
 *   s_j = scale * q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j),
 * statistics and sums in FP32.
 *   q_bf16      [B, q_heads, D] BF16 bits, 16-byte aligned
 *   block_table int32, rows table_stride apart: row b holds request b's pages in
 *               order, max_pages of them at most; what lies behind its last page
 *               is not read into the result
 *   lengths     int32 [B]; below 1 the request is empty: out 0, lse -inf.  More
 *               than max_pages pages hold counts as what they hold
 *   out_bf16    [B, q_heads, D] BF16 bits, 16-byte aligned; may be q_bf16 itself, and
 *               overlaps nothing else that is read
 *   lse         NULL, or float [B, q_heads], 4-byte aligned
 *   workspace   >= moe_quant_attend_workspace_size bytes, 256-byte aligned; its
 *               contents on entry do not matter; lse and it overlap nothing else
 * Tokens on a page outside of [0, num_pages) count as absent.  What the cache
 * holds behind a request's last token, NaN among it, does not reach the result;
 * queries, keys and values of the tokens themselves are finite.  Repeated calls
 * give the same bits.  Up to 1024 requests are cut into pieces where they are long;
 * of more, each goes whole to one workgroup per 16 query heads of a key head.
 * batch == 0 returns MQ_OK without enqueuing anything.
 * Limits: batch at most 65536, batch * kv_heads * ceil(q_heads / kv_heads / 16) at
 * most 2^23; q_heads a multiple of kv_heads, at most 1024; scale * k_scale * log2(e)
 * finite; window 0 (none) or positive; max_pages * page_size at most 2^30.  Scores
 * times log2(e), and the sums of exp(s_j - max s) |v_j| of the stored values, are below
 * FP32's largest number, 2^128.
 * Errors: MQ_E_NULL, MQ_E_ABI, MQ_E_SHAPE, MQ_E_DTYPE, MQ_E_ALIGN,
 * MQ_E_WORKSPACE, MQ_E_HIP.
 */
mq_status moe_quant_attend(const mq_kv_cache *c, int32_t q_heads, float scale, int32_t window,
                           const uint16_t *q_bf16, const int32_t *block_table, int64_t table_stride,
                           int32_t max_pages, const int32_t *lengths, int64_t batch,
                           uint16_t *out_bf16, float *lse, void *workspace, size_t workspace_bytes,
                           struct ihipStream_t *stream);

/*
 * Allocation-free variant of moe_quant_forward, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  It runs the same kernels; their scratch
 * (routing tables, the FP16 intermediate and the per-slot partials) lives in
 * a static device array inside the library, MOE_QUANT_NOALLOC_SCRATCH_BYTES
 * per GPU, held by each GPU the library runs on until the process ends.  No
 * hipMalloc, hipFree or allocating library routine is called.
 *   router_logits, hidden_bf16, residual_bf16, num_tokens, out_bf16, stream:
 *                  as for moe_quant_forward
 *   overflow_flag  NULL, or a caller-owned device uint32 (4-byte aligned):
 *                  set to 0 at the start of the call and to 1 if an FP16
 *                  intermediate saturated (read it after the stream syncs)
 * Every call on one GPU shares that GPU's array and leaves its contents
 * behind: calls that overlap on one GPU (different streams, or host threads
 * without ordering between them) race on it and must not be issued.
 * Errors: as moe_quant_forward, plus MQ_E_WORKSPACE when the batch needs more
 * scratch than the array holds (moe_quant_workspace_size(L, T) above
 * MOE_QUANT_NOALLOC_SCRATCH_BYTES; about 1350 tokens at hidden 2048,
 * intermediate 768, 128 experts, top-8), checked before anything is enqueued.
 */
#define MOE_QUANT_NOALLOC_SCRATCH_BYTES (64u << 20)
mq_status moe_quant_forward_noalloc(const mq_layer *L, const void *router_logits,
                                    int32_t logits_dtype, const uint16_t *hidden_bf16,
                                    const uint16_t *residual_bf16, int64_t num_tokens,
                                    uint16_t *out_bf16, uint32_t *overflow_flag,
                                    struct ihipStream_t *stream);

/*
 * Checkpoint import: one expert's gate_proj, up_proj and down_proj, each in
 * the tensor layout of the checkpoint format the model cards name for the
 * layer's weight format, written into the packed layouts above (gate and up
 * fused into W13, gate rows first).  Source and destination tensors are
 * device memory owned by the caller.  Per projection (N = out_features, K =
 * in_features: gate and up N = I, K = H; down N = H, K = I):
 *   MQ_W_FP8_B128   FineGrainedFP8 ("clef-omni-fp8" card, section "Recipe"):
 *                   weight = E4M3 [N, K], scale = weight_scale_inv float
 *                   [N/128, K/128]; copied into place (the same bytes).
 *   MQ_W_INT4_G128  auto_gptq packing ("clef-omni-int4" card, section "What
 *                   was quantized"): weight = qweight int32 [K/8, N] (word
 *                   [i, n] holds k = 8 i + j at bits 4 j), qzeros = int32
 *                   [K/128, N/8] (word [g, c] holds column 8 c + j at bits
 *                   4 j), scale = scales fp16 [K/128, N].  The stored zero
 *                   point plus gptq_zero_offset (1 in the auto_gptq
 *                   convention) must be 8 in every group (symmetric INT4);
 *                   weights and scales are transposed into place.
 *   MQ_W_NVFP4_G16  compressed-tensors NVFP4 ("clef-omni-NVFP4" card, section
 *                   "How it was made"): weight = weight_packed uint8 [N, K/2],
 *                   scale = weight_scale E4M3 [N, K/16], global_scale =
 *                   weight_global_scale (host float); copied into place, and
 *                   the global scales into w13_gscale[expert] (gate and up
 *                   must be equal: the card's quantizer fuses them) and
 *                   w2_gscale[expert].
 * dst: a descriptor of the destination layer (the same checks as
 * moe_quant_init); its weight and scale buffers are written.
 * bad_zero_points: INT4 only, NULL or a device uint32 that is set to 1 when
 * a group's zero point is not 8 (read it after the stream syncs; the weights
 * of such a group cannot be represented and the import must be discarded).
 * Asynchronous on `stream`.  Errors: the moe_quant_init errors for dst,
 * MQ_E_NULL (a source tensor NULL), MQ_E_SHAPE (expert out of range),
 * MQ_E_ALIGN (a source tensor not 16-byte aligned), MQ_E_FORMAT (NVFP4 gate
 * and up global scales differ), MQ_E_HIP.
 */
typedef struct {
  const void *weight;  /* see above, per format                            */
  const void *scale;
  const void *qzeros;  /* INT4 only; NULL for the other formats            */
  float global_scale;  /* NVFP4 only                                        */
} mq_src_proj;

mq_status moe_quant_import_expert(const mq_layer_desc *dst, int32_t expert, const mq_src_proj *gate,
                                  const mq_src_proj *up, const mq_src_proj *down,
                                  int32_t gptq_zero_offset, uint32_t *bad_zero_points,
                                  struct ihipStream_t *stream);

void moe_quant_destroy(mq_layer *L);

/* Static strings; never NULL. */
const char *moe_quant_status_string(mq_status s);
const char *moe_quant_last_error(void);
uint32_t moe_quant_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_QUANT_H */

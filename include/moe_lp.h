/*
 * moe_lp.h -- C ABI of the MI355X (gfx950) low-precision MoE expert forward.
 *
 * The operation (Orbit announcement, section 技术细节, "Active-expert-chunked
 * dequantization"): each token activates only the experts its router
 * selects; the selected experts are processed in fixed-size chunks whose
 * frozen low-precision weights are dequantized temporarily for a grouped
 * GEMM and released afterwards.  Weight formats: INT4 (Kimi INT4 base, same
 * page), FP8 E4M3 with [128,128] fp32 block scales and [1,128] activation
 * scales (NeMo RL FP8 post, Table 1), MXFP4 and NVFP4 (named as serving
 * formats in the mixed-precision sampler post, which defines neither; both
 * follow their public definitions).  The optional BF16 adapter is an OFT
 * orthogonal rotation of the expert input (Orbit analysis page, section on
 * why OFT matters); passing no adapter gives the frozen base, i.e. the
 * reference policy of that page.
 *
 * Conventions for every entry point
 *  - All array arguments are DEVICE pointers owned by the caller (e.g. torch
 *    tensors).  Only the descriptor structs live in host memory.  The library
 *    allocates nothing and keeps no state between calls.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  All
 *    work is enqueued on it; no call synchronises the host and no call copies
 *    device data to the host.  Buffers must stay alive until the work is done.
 *  - Arguments are validated on the host before anything is enqueued; on any
 *    error the call returns a non-zero moe_status and enqueues nothing.  Kernel
 *    launch failures return MOE_ERR_DEVICE.  Non-finite logits or activations
 *    are a precondition violation (not checked).
 *  - Device pointers must be 16-byte aligned.
 *  - Row-major everywhere; weights are stored K-contiguous (Y = X W^T).
 */
#ifndef MOE_LP_H
#define MOE_LP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LP_ABI_VERSION 6

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARGUMENT = 1,    /* null pointer, bad shape, misalignment */
  MOE_ERR_UNSUPPORTED = 2,         /* valid but outside the supported limits */
  MOE_ERR_WORKSPACE_TOO_SMALL = 3, /* ws_bytes < the matching *_workspace_bytes() */
  MOE_ERR_DEVICE = 4               /* a HIP launch reported an error */
} moe_status;

typedef enum {
  /* Two's-complement 4-bit codes, element 2i in the low nibble of byte i;
   * bf16 scale per (output row n, 32 consecutive k).  w = q * s.
   * Activations into the GEMMs: 16-bit floats (no activation quantization).
   * The GEMMs run on fp16 operands: w = q*s is exact in fp16 for bf16 scales
   * in [2^-17, 8188]; x (or x R_e with an adapter) and h = silu(gate)*up are
   * converted to fp16, exact in magnitude range [2^-14, 65504) for bf16 x.
   * Preconditions (not checked on the device): scales in that range and
   * |x|, |x R_e|, |h| < 65504 (larger values become infinite). */
  MOE_W_INT4_G32_BF16 = 1,
  /* OCP E4M3FN codes, one byte each; fp32 scale per [128,128] block
   * [n/128][k/128].  Activations (x and the SwiGLU output) are quantized to
   * E4M3 with an fp32 scale per [1,128] block: s = amax/448, q = RNE(v/s). */
  MOE_W_FP8_E4M3_B128 = 2,
  /* OCP MXFP4: E2M1 codes (low nibble first) with an E8M0 scale byte per
   * (n, 32 consecutive k).  Activations are quantized to MXFP8: E4M3 codes
   * with an E8M0 scale per 32, shared exponent floor(log2 amax) - 8. */
  MOE_W_MXFP4 = 3,
  /* As MOE_W_FP8_E4M3_B128 with power-of-two scales (the FP8 recipe's
   * power-of-two scaling-factor switches, NeMo RL FP8 post): weight block
   * scales must be exact powers of two (fp32, only their exponent is used);
   * activation scales are the smallest power of two >= fl32(amax/448).  The
   * GEMMs then apply both scales inside the block-scaled MFMA. */
  MOE_W_FP8_E4M3_B128_POW2 = 4,
  /* NVFP4 (named as a serving format in the mixed-precision sampler post;
   * this is the format's public definition): E2M1 codes (low nibble
   * first), an E4M3 scale byte per (n, 16 consecutive k), and one fp32
   * second-level scale per expert matrix (moe_scales.g13 / g2):
   * w = e2m1(q) * e4m3(s) * g.  Activations into the GEMMs: 16-bit floats,
   * as for INT4 (same range preconditions on x, x R_e and h; e2m1 * e4m3 is
   * exact in fp16 for every code, g multiplies the fp32 accumulators).
   * Forward, materialized forward and frozen-base backward. */
  MOE_W_NVFP4 = 5
} moe_wformat;

/* Storage order of the packed codes in w13 and w2 (every format). */
typedef enum {
  MOE_WL_ROWS = 0,   /* [E][N][K]: each output row's K codes contiguous */
  /* [E][N/16][K/128][16][B]: tiles of 16 rows x 128 codes, a row's 128
   * codes (B = 64 bytes of 4-bit codes in the usual nibble order, 128 bytes
   * of E4M3) contiguous within its tile, tiles K-fastest.  A GEMM step then
   * streams 1-2 KB runs instead of 64- or 128-byte pieces of rows K/2 or K
   * bytes apart.  Fused forward, materialized forward (its BF16 copy is in
   * rows either way) and frozen-base backward (the backward's transposed
   * copy is made from either order).  Written by moe_pack_weights_kblocked.
   * Scales keep their layout. */
  MOE_WL_KBLOCKED = 1
} moe_wlayout;

/* Layer description (host memory). */
typedef struct {
  /* T >= 0 (T = 0 is a no-op).  T*k*max(H, I)*2 must stay below 2^32 (the
   * grouped GEMMs address gathered activation rows with 32-bit byte offsets;
   * e.g. T <= 37449 at k = 8, H = 7168); larger: MOE_ERR_UNSUPPORTED. */
  int32_t num_tokens;
  int32_t hidden;      /* H: multiple of 256                                */
  int32_t inter;       /* I: multiple of 128 (expert intermediate size)     */
  int32_t num_experts; /* E: 1..1024                                        */
  int32_t top_k;       /* k: 1..min(16, E)                                  */
  int32_t wformat;     /* a moe_wformat value                               */
  int32_t oft_block;   /* 0: no adapter; 32: block-diagonal 32x32 rotation (every weight format) */
  int32_t tile_rows;   /* rows per grouped-GEMM tile: 0 = automatic, else 16, 32, 48, 64, 96, 128, 160 or 192 */
  int64_t adapter_expert_stride; /* elements between experts' R; 0 = one R shared by all */
  int32_t weight_layout;         /* a moe_wlayout value; other values: MOE_ERR_INVALID_ARGUMENT */
} moe_layer;

/* Packed expert weights.
 *   w13: [E][2I][H]  gate rows 0..I-1 then up rows I..2I-1 (packed bytes per format)
 *   w2 : [E][H][I]   down projection */
typedef struct {
  const void* w13;
  const void* w2;
} moe_qweights;

/* Scales, layouts per format.  Group scales (one per output row n and 32
 * or 16 consecutive k) are stored group-major, [K/32][N] per expert, so that
 * the scales of one K step for a block of output rows are contiguous:
 *   INT4 : s13 bf16 [E][H/32][2I],   s2 bf16 [E][I/32][H]
 *   FP8, FP8_POW2: s13 fp32 [E][2I/128][H/128], s2 fp32 [E][H/128][I/128]
 *   MXFP4: s13 u8   [E][H/32][2I],   s2 u8   [E][I/32][H]  (E8M0)
 *   NVFP4: s13 u8   [E][H/16][2I],   s2 u8   [E][I/16][H]  (E4M3, positive),
 *          g13, g2 fp32 [E] (device; 4-byte aligned).  g13 / g2 are read
 *          only for NVFP4 and may be NULL otherwise. */
typedef struct {
  const void* s13;
  const void* s2;
  const float* g13;
  const float* g2;
} moe_scales;

/* Routing result (all device arrays, caller-owned).  R = T*k.
 *   topk_ids[T][k]      int32, slots in descending logit order (ties: smaller id)
 *   topk_w[T][k]        fp32, softmax over the k selected logits
 *   expert_offsets[E+1] int32, exclusive scan of per-expert counts; [E] = R
 *   sorted_rows[R]      int32, permuted row -> flat pair t*k+j, stable in (t, j)
 *   row_of[R]           int32, flat pair -> permuted row (inverse of sorted_rows)
 *   active_experts[E]   int32, experts with >= 1 row in ascending id (first num_active valid)
 *   num_active[1]       int32 */
typedef struct {
  int32_t* topk_ids;
  float* topk_w;
  int32_t* expert_offsets;
  int32_t* sorted_rows;
  int32_t* row_of;
  int32_t* active_experts;
  int32_t* num_active;
} moe_route_out;

/* Workspace bytes moe_expert_forward needs for this layer (independent of
 * chunk_experts, which is accepted for symmetry; any value >= 1 gives the
 * same size).  Returns 0 for an invalid descriptor. */
size_t moe_workspace_bytes(const moe_layer* layer, int32_t chunk_experts);

/* Re-lays the codes from MOE_WL_ROWS (qweights, as described by
 * layer's dimensions and format; layer->weight_layout must be a valid value
 * but does not change what is read or written) into
 * MOE_WL_KBLOCKED: w13_out and w2_out (device, caller-owned, 16-byte
 * aligned, the same sizes as w13 and w2).  Bit-identical codes; a forward
 * with weight_layout = MOE_WL_KBLOCKED on the copy gives bit-identical
 * outputs.  Stream-ordered. */
moe_status moe_pack_weights_kblocked(const moe_layer* layer, const moe_qweights* qweights, void* w13_out,
                                     void* w2_out, void* stream);

/* Workspace bytes moe_route_permute needs (scan scratch only). */
size_t moe_route_workspace_bytes(const moe_layer* layer);

/* Rows per grouped-GEMM tile that moe_expert_forward uses for this layer
 * (layer->tile_rows if set, else the automatic choice); 0 if invalid. */
int32_t moe_tile_rows(const moe_layer* layer);

/* Router top-k + softmax over the selected logits, then the expert histogram,
 * exclusive scan and stable permutation by expert (Orbit announcement,
 * 技术细节: router-selected experts grouped dynamically).
 * logits: [T][E] fp32.  Outputs are bit-exact functions of the logits except
 * topk_w (fp32 softmax). */
moe_status moe_route_permute(const moe_layer* layer, const float* logits, const moe_route_out* out,
                             void* ws, size_t ws_bytes, void* stream);

/* The MoE expert forward (Orbit announcement, 技术细节, active-expert-chunked
 * dequantization): route, permute, then for each chunk of `chunk_experts`
 * consecutive active experts (ascending id) run the grouped
 * dequantize + GEMM1 (gate/up) + SwiGLU and the grouped dequantize + GEMM2
 * (down), and finally the weighted combine
 *   out[t] = sum_j topk_w[t][j] * y[t][j]   (fp32 sum in ascending j, bf16 out).
 * x: [T][H] bf16; logits: [T][E] fp32; adapter: NULL or bf16
 * R[E or 1][H/32][32][32] (x' = x R_e, rows of R index the input dim,
 * rotated per permuted row in fp32 and then given to the weight format's
 * GEMM1 input quantizer, as x is without an adapter); out: [T][H] bf16.  The launch count is fixed by (E, chunk_experts); the
 * result does not depend on chunk_experts.  ws: >= moe_workspace_bytes(). */
moe_status moe_expert_forward(const moe_layer* layer, const void* x_bf16, const float* logits,
                              const moe_qweights* qweights, const moe_scales* scales,
                              const void* adapter_bf16, int32_t chunk_experts, void* out_bf16,
                              void* ws, size_t ws_bytes, void* stream);

/* Stages reported by moe_expert_forward_timed. */
enum {
  MOE_STAGE_ROUTE = 0,   /* router top-k + softmax                          */
  MOE_STAGE_PERMUTE = 1, /* histogram, scan, stable scatter, tile lists      */
  MOE_STAGE_ACT = 2,     /* GEMM1 input: activation format and OFT rotation  */
  MOE_STAGE_GEMM1 = 3,   /* dequant + gate/up GEMM + SwiGLU                  */
  MOE_STAGE_GEMM2 = 4,   /* dequant + down GEMM (launch pairing: see below)  */
  MOE_STAGE_COMBINE = 5, /* weighted combine                                 */
  MOE_STAGE_DEQUANT = 6, /* materialized scheme only: chunk -> BF16 copy     */
  MOE_NUM_STAGES = 7
};

/* moe_expert_forward with per-stage timing, for measurement: a HIP event is
 * recorded on `stream` around every launch group, and the call synchronises
 * the stream before it returns (unlike moe_expert_forward).  stage_ms and
 * stage_launches are HOST arrays of MOE_NUM_STAGES entries, filled with the
 * summed event durations (milliseconds) and the number of launch groups of
 * each stage.  Same arguments, result and errors as moe_expert_forward.
 * The grouped GEMMs run one launch per chunk c = 0..n that does chunk c's GEMM1
 * together with chunk c-1's GEMM2 (n = number of chunks): launches 0..n-1
 * are reported under MOE_STAGE_GEMM1 and the last, GEMM2-only launch under
 * MOE_STAGE_GEMM2. */
moe_status moe_expert_forward_timed(const moe_layer* layer, const void* x_bf16, const float* logits,
                                    const moe_qweights* qweights, const moe_scales* scales,
                                    const void* adapter_bf16, int32_t chunk_experts, void* out_bf16,
                                    void* ws, size_t ws_bytes, void* stream, float* stage_ms,
                                    int32_t* stage_launches);

/* Workspace bytes moe_expert_forward_materialized needs: the routing arrays,
 * bf16 h [R][I] and y [R][H], the rotated input [R][H] bf16 when an adapter is
 * used, and one chunk's BF16 weight copy, min(chunk_experts, E) * 3*H*I * 2
 * bytes.  Returns 0 for an invalid descriptor or chunk_experts < 1. */
size_t moe_materialized_workspace_bytes(const moe_layer* layer, int32_t chunk_experts);

/* The materialized-chunk scheme (Orbit announcement, 技术细节: the chunk's
 * experts are dequantized temporarily to high precision, a grouped GEMM runs,
 * and the high-precision weights are released), for comparison with
 * moe_expert_forward.  Routing, permutation and combine are the same; then for
 * each chunk of chunk_experts consecutive active experts:
 *   1. dequantize the chunk's W13 and W2 into a BF16 copy in ws (each weight
 *      rounded once to bf16, nearest even),
 *   2. GEMM1 on bf16 MFMA: g, u = x~ W^T in fp32, h = silu(g) * u rounded to bf16,
 *   3. GEMM2: y = h W2^T in fp32, rounded to bf16,
 * and the next chunk overwrites the copy.  x~ is the bf16 token row, or x R_e
 * rounded to bf16 with the adapter; no activation quantizer is applied (the
 * copy is BF16, so the GEMMs are BF16 GEMMs for every weight format).
 * The copy's size, and so ws, grows with chunk_experts.
 * Same arguments and errors as moe_expert_forward, with
 * ws >= moe_materialized_workspace_bytes(layer, chunk_experts).  stage_ms and
 * stage_launches: both NULL (asynchronous, no host synchronisation), or both
 * HOST arrays of MOE_NUM_STAGES entries filled as by moe_expert_forward_timed
 * (the call then synchronises the stream); dequant launches are reported under
 * MOE_STAGE_DEQUANT, each chunk's GEMM1 and GEMM2 launch under GEMM1 and GEMM2. */
moe_status moe_expert_forward_materialized(const moe_layer* layer, const void* x_bf16, const float* logits,
                                           const moe_qweights* qweights, const moe_scales* scales,
                                           const void* adapter_bf16, int32_t chunk_experts, void* out_bf16,
                                           void* ws, size_t ws_bytes, void* stream, float* stage_ms,
                                           int32_t* stage_launches);

/* ---- Frozen-base backward --------------------------------------------------
 * The GEMM backward that bypasses the base weight gradient (Orbit
 * announcement, 技术细节): gradients for the layer inputs and the adapter only.
 * Its two GEMMs contract over the weights' output dimension, so they read a
 * transposed copy of the frozen weights, made once per base. */

/* Bytes of the transposed copy: W13^T [E][H][2I] and W2^T [E][I][H] in the
 * format's codes (INT4 / E2M1 nibbles, E4M3 bytes), stored in tiles of 16
 * rows x 128 codes as MOE_WL_KBLOCKED describes, plus scales (INT4, MXFP4,
 * NVFP4: one fp16 per group scale; FP8: the fp32 block scales transposed); 0 if the
 * layer is not supported by the backward (I multiple of 256; FP8 H and 2I at
 * most 8192). */
size_t moe_backward_weights_bytes(const moe_layer* layer);

/* Writes the transposed copy of (qweights, scales) into bwd_weights (device,
 * caller-owned, >= moe_backward_weights_bytes).  Codes are bit-identical
 * re-layouts; INT4 scales are converted to fp16 (exact for bf16 scales in
 * [2^-17, 8188]), MXFP4
 * scales to fp16 2^(e-127) (exact within fp16's range), NVFP4 E4M3 scales
 * to fp16 (exact), FP8 block scales are transposed.  NVFP4's fp32
 * second-level scales are not copied: moe_expert_backward reads them from
 * its moe_scales (g13 / g2 required there, 4-byte aligned). */
moe_status moe_prepare_backward_weights(const moe_layer* layer, const moe_qweights* qweights,
                                        const moe_scales* scales, void* bwd_weights, size_t bwd_bytes,
                                        void* stream);

/* Workspace bytes of moe_expert_backward (routing, recomputed gate/up
 * pre-activations fp32 [R][2I], their gradients fp16 [R][2I], dx' fp32
 * [R][H] (twice with an adapter), the fp16 copy of d_out, and for a shared
 * adapter the per-expert gradient partials fp32 [E][H/32][32][32]). */
size_t moe_backward_workspace_bytes(const moe_layer* layer, int32_t chunk_experts);

/* Backward of moe_expert_forward for given d_out = dL/dout [T][H] bf16:
 *   d_x      [T][H] bf16    dL/dx
 *   d_logits [T][E] fp32    dL/dlogits: w_tj (g_tj - sum_i w_ti g_ti) for the
 *                           selected experts, g_tj = <d_out_t, y_tj>; 0 elsewhere
 *   d_adapter fp32, shaped like the adapter, dL/dR (a shared R, stride 0,
 *                           gets the sum over all experts, added in ascending
 *                           active-expert order); NULL exactly when adapter is NULL
 * No gradient is formed for W13 or W2.  The forward is recomputed per chunk
 * (routing, gate/up pre-activations); per permuted row (t, j) of expert e:
 * u = d_out_t W2, dh = w_tj u, da = dh b silu'(a), db = dh silu(a),
 * dx' = da Wg + db Wu, dR_e += x_t^T dx' (32x32 diagonal blocks),
 * dx_tj = dx' R_e^T, d_x_t = sum_j dx_tj.  Activation quantizers of the
 * FP8 / MXFP4 formats pass gradients straight through; the router term uses
 * h as the forward quantized it.  GEMM operands are fp16 (INT4 and E2M1
 * weights times their scales exactly, NVFP4's second-level scale applied to
 * the fp32 accumulators, E4M3 times the block scale rounded once; d_out and the SwiGLU gradients rounded to fp16, so their magnitudes
 * must stay below 65504), accumulation fp32.
 * bwd_weights: from moe_prepare_backward_weights for the same weights.
 * Unsupported layers return MOE_ERR_UNSUPPORTED; the rest as moe_expert_forward.
 * Stream-ordered, no host synchronisation, nothing allocated, unless
 * stage_ms and stage_launches (HOST arrays of MOE_NUM_STAGES, both or
 * neither) are given: then per-stage event times are filled as by
 * moe_expert_forward_timed and the call synchronises the stream.  Stages:
 * ROUTE, PERMUTE; ACT = GEMM inputs (x or x R_e, d_out as fp16); GEMM1 =
 * gate/up recompute launches; GEMM2 = backward GEMM launches (chunk c's
 * u items with chunk c-1's dx' items); COMBINE = adapter backward,
 * un-permute sum and router gradient. */
moe_status moe_expert_backward(const moe_layer* layer, const void* x_bf16, const float* logits,
                               const moe_qweights* qweights, const moe_scales* scales, const void* bwd_weights,
                               const void* adapter_bf16, const void* d_out_bf16, int32_t chunk_experts,
                               void* d_x_bf16, float* d_logits, float* d_adapter, void* ws, size_t ws_bytes,
                               void* stream, float* stage_ms, int32_t* stage_launches);

/* The GEMM1 input quantizer of the layer's weight format applied to x, one
 * row per token (what moe_expert_forward feeds its first grouped GEMM when no
 * adapter is given), written to caller buffers:
 *   FP8 (NeMo RL FP8 post, Table 1, input activations): codes [T][H] E4M3FN,
 *     scales fp32 [T][H/128]: s = amax/448 (1 for an all-zero block),
 *     q = RNE-saturate(v/s), both quotients correctly rounded in fp32;
 *   FP8_POW2: as FP8 with s the smallest power of two >= amax/448;
 *   MXFP4: codes [T][H] E4M3FN, scales [T][H/32] E8M0 bytes: shared exponent
 *     X = floor(log2 amax) - 8 (0 for an all-zero block, clamped to
 *     [-127, 127]), q = RNE-saturate(v * 2^-X).
 * INT4 and NVFP4 layers take 16-bit activations and have no quantizer:
 * MOE_ERR_UNSUPPORTED.  x, codes: 16-byte aligned; scales: 4-byte aligned.
 * Stream-ordered, no host synchronisation. */
moe_status moe_quantize_activations(const moe_layer* layer, const void* x_bf16, void* codes, void* scales,
                                    void* stream);

/* Weighted combine on its own: out[t] = sum_{j<k} topk_w[t][j] *
 * y_perm[row_of[t*k+j]], fp32 sum in ascending j, RNE to bf16.  y_perm:
 * [T*k][H] bf16.  Atomic-free and deterministic. */
moe_status moe_combine(const moe_layer* layer, const void* y_perm_bf16, const float* topk_w,
                       const int32_t* row_of, void* out_bf16, void* stream);

/* Workspace bytes moe_lm_head_logprob needs: T*ceil(V/128)*2 fp32
 * log-softmax statistics (maximum and sum of exponentials per token and
 * block of 128 vocabulary rows) and T fp32 target logits, each 256-byte
 * aligned. */
size_t moe_lm_head_workspace_bytes(int32_t T, int32_t V);

/* Log-prob of target tokens under an LM head (the rollout log-probs whose
 * train/rollout agreement the NeMo RL FP8 post measures with its
 * token-mult-prob-error):  z = h / sqrt(mean(h^2) + 1e-6) (a final
 * parameter-free RMSNorm), logits = z W_lm^T (fp32 accumulation),
 * logprob[t] = logits[t][y_t] - logsumexp_v logits[t][v].
 * h: [T][H] bf16; w_lm: [V][H] bf16; targets: [T] int32 in [0, V);
 * logprob: [T] fp32.  H multiple of 128, T <= 4096. */
moe_status moe_lm_head_logprob(int32_t T, int32_t H, int32_t V, const void* h_bf16, const void* w_lm_bf16,
                               const int32_t* targets, float* logprob, void* ws, size_t ws_bytes,
                               void* stream);

/* ---- Training losses -------------------------------------------------------
 * The objectives an adapter on the frozen base is trained with, each with its
 * gradient: cross entropy and distillation through the LM head (their d_h is
 * what the layers below take as d_out), and the router's balance loss (its
 * gradient joins moe_expert_backward's d_logits).  A workspace serves one call
 * at a time: calls that may run at once, replayed graphs among them, need one
 * each. */

/* An LM head (host memory).  logits[t][v] = logit_scale * <z_t, W_v> with
 * z_t = h_t / sqrt(mean(h_t^2) + norm_eps), the parameter-free RMSNorm of
 * moe_lm_head_logprob, or z_t = h_t for norm_eps = 0.  The forward entries are
 * MOE_ERR_UNSUPPORTED where T V comes to 2^39 (more tiles than a launch holds). */
typedef struct {
  int32_t num_tokens; /* T: 0..2^20                                              */
  int32_t hidden;     /* H: multiple of 8, at most 32768                         */
  int32_t vocab;      /* V: 1..2^20                                              */
  float norm_eps;     /* finite, >= 0; 0: no norm                                */
  float logit_scale;  /* finite, > 0 (an inverse temperature)                    */
  int64_t h_stride;   /* elements between rows of h: 0 (= H), or a multiple of 8, H..2^22 */
  int64_t w_stride;   /* the same for W                                          */
} moe_lm_head;

/* Largest number of teacher logits per token. */
#define MOE_DISTILL_MAX_TOP 256

/* Workspace bytes of the loss entries below: top = 0 for cross entropy, else
 * the teacher logits per token; backward != 0 for the *_backward entry.
 * Returns 0 for an invalid or unsupported descriptor.  The logits are held
 * only where there are few (parts of their sums, fp32, at most 64 MB);
 * otherwise the forward keeps two floats per token and block of vocabulary
 * rows.  The backward keeps the scaled softmax gradient (bf16) of one piece of
 * the vocabulary at a time (at most about 512 MB, or 256 columns where more
 * tokens need more), partial sums of dL/dz (fp32, up to 64 [T][H]), and about
 * half a KB per target (at most 2^20 of them) for d_W. */
size_t moe_lm_head_loss_workspace_bytes(const moe_lm_head* head, int32_t top, int32_t backward);

/* Cross entropy of target ids: lse[t] = log sum_v exp(logits[t][v]),
 * loss[t] = lse[t] - logits[t][y_t] (the negative log-prob).
 * h: [T][H] bf16 (h_stride); w_lm: [V][H] bf16 (w_stride); targets: [T] int32;
 * loss, lse: [T] fp32.  A negative target marks a token that does not count:
 * loss = lse = 0, and its row of h has no part in anything, whatever it holds
 * (it may be read).  Above 256 tokens such rows are gathered out before the
 * products; up to 256 they take their place in the tiles.  A target >= V gives
 * loss = NaN, lse = 0, and is otherwise the same. */
moe_status moe_lm_head_loss(const moe_lm_head* head, const void* h_bf16, const void* w_lm_bf16,
                            const int32_t* targets, float* loss, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Its gradient for given d_loss = dL/dloss [T] fp32, with loss and lse from
 * moe_lm_head_loss of the same inputs (the logits are formed again, one piece
 * of the vocabulary at a time):
 *   d_h [T][H] bf16 (contiguous)       dL/dh; 0 for tokens that do not count
 *   d_w [V][H] bf16 (contiguous)       dL/dW; NULL: not formed (frozen head)
 * With p = softmax(logits), r = 1/sqrt(mean(h^2) + norm_eps) (1 without a norm):
 *   G[t][v] = logit_scale * r_t * d_loss[t] * (p[t][v] - [v = y_t])
 *   u = G W,  d_h = u - r^2 h mean(h u) (without a norm: u),  d_W = G^T h.
 * G is rounded to bf16 as the operand of the two products, and what that takes
 * off its entries at the targets is added to u and to d_W; sums, u and the norm's
 * terms are fp32, d_h and d_W are rounded once.  d_h and d_w must not overlap the
 * inputs.
 * T = 0 writes zeros to d_w. */
moe_status moe_lm_head_loss_backward(const moe_lm_head* head, const void* h_bf16, const void* w_lm_bf16,
                                     const int32_t* targets, const float* loss, const float* lse,
                                     const float* d_loss, void* d_h_bf16, void* d_w_bf16, void* ws, size_t ws_bytes,
                                     void* stream);

/* Distillation from a teacher's top logits: per token the teacher gives `top`
 * (1..MOE_DISTILL_MAX_TOP) vocabulary ids and logits; q = softmax of
 * teacher_scale * teacher_logits over the slots that are there (id in [0, V),
 * logit not -infinity), and
 *   logp[t][j] = logits[t][id_j] - lse[t]      (0 for absent slots)
 *   loss[t] = sum_j q_j (log q_j - logp[t][j]) (KL divergence; q = 0 elsewhere).
 * teacher_ids: [T][top] int32; teacher_logits: [T][top] fp32; loss, lse: [T]
 * fp32; logp: [T][top] fp32.  A token with no slot there does not count (as a
 * negative target above).  Slots may repeat an id; their q add up in the
 * gradient.  The student's softmax runs over the whole vocabulary. */
moe_status moe_lm_head_distill(const moe_lm_head* head, int32_t top, float teacher_scale, const void* h_bf16,
                               const void* w_lm_bf16, const int32_t* teacher_ids, const float* teacher_logits,
                               float* loss, float* lse, float* logp, void* ws, size_t ws_bytes, void* stream);

/* Its gradient: as moe_lm_head_loss_backward with
 *   G[t][v] = logit_scale * r_t * d_loss[t] * (p[t][v] - sum_j q_j [id_j = v]);
 * lse and logp from moe_lm_head_distill.  None for the teacher.  What rounding
 * takes off the entries at the slots' ids is added where those are few (top at
 * most V / 900, or T top at most V / 2 or 1024; to d_W up to T top = 2^20); past
 * that they stay rounded, as the rest of G (18% of a frozen gradient's time at 64
 * of 32000 ids). */
moe_status moe_lm_head_distill_backward(const moe_lm_head* head, int32_t top, float teacher_scale,
                                        const void* h_bf16, const void* w_lm_bf16, const int32_t* teacher_ids,
                                        const float* teacher_logits, const float* lse, const float* logp,
                                        const float* d_loss, void* d_h_bf16, void* d_w_bf16, void* ws,
                                        size_t ws_bytes, void* stream);

/* Workspace bytes of moe_balance_loss; 0 for an invalid layer or num_segs < 1. */
size_t moe_balance_loss_workspace_bytes(const moe_layer* layer, int32_t num_segs);

/* Router balance loss and per-expert counts, per segment of consecutive
 * tokens (a packed sequence; one segment: the whole batch).  With
 * p_t = softmax(logits[t]) over all E experts (an expert at -infinity has
 * p = 0; a row of them counts with p = 0):
 *   tokens[s]    tokens of segment s that count (token_mask != 0)
 *   counts[s][e] their routed slots: pairs (t, j) with topk_ids[t][j] = e
 *   probs[s][e]  mean of p_t[e] over them
 *   loss[s]      E / (k tokens[s]) * sum_e counts[s][e] probs[s][e]
 *                (1 for uniform routing; 0 for a segment without tokens)
 * logits: [T][E] fp32; topk_ids: [T][k] int32 (ids outside [0, E) are not
 * counted); token_mask: NULL (all tokens count) or [T] bytes (rows of tokens
 * that do not count are not used); seg_offsets: NULL (num_segs = 1, all
 * tokens), or [num_segs + 1] int32, non-decreasing; tokens outside
 * [seg_offsets[0], seg_offsets[num_segs]) belong to no segment.
 * loss: [S] fp32; counts: [S][E] int32; tokens: [S] int32; probs: [S][E] fp32.
 * Deterministic (no floating-point atomics).  num_segs at most 65536. */
moe_status moe_balance_loss(const moe_layer* layer, const float* logits, const int32_t* topk_ids,
                            const uint8_t* token_mask, const int32_t* seg_offsets, int32_t num_segs, float* loss,
                            int32_t* counts, int32_t* tokens, float* probs, void* ws, size_t ws_bytes, void* stream);

/* Its gradient for given d_loss = dL/dloss [S] fp32 (the counts are constants):
 *   dL/dlogits[t][e] = p_t[e] (a_e - sum_i p_t[i] a_i),
 *   a_e = d_loss[s] E counts[s][e] / (k tokens[s]^2)
 * for the tokens that count, 0 for the others.  d_logits: [T][E] fp32, written,
 * or with accumulate != 0 added to what it holds (moe_expert_backward's
 * d_logits). */
moe_status moe_balance_loss_backward(const moe_layer* layer, const float* logits, const uint8_t* token_mask,
                                     const int32_t* seg_offsets, int32_t num_segs, const int32_t* counts,
                                     const int32_t* tokens, const float* d_loss, int32_t accumulate,
                                     float* d_logits, void* stream);

/* ---- The gate ----------------------------------------------------------------
 * Routing of models whose gate scores every expert, chooses by score plus a
 * balance bias within the best groups of experts, and weighs by the scores:
 * what moe_route_permute (softmax over the chosen logits) does not do. */

enum { MOE_GATE_SOFTMAX = 0, MOE_GATE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };

/* The largest number of groups. */
#define MOE_GATE_MAX_GROUPS 64

/* A gate (host memory).  For the logits l of a token and the bias b (0 without
 * one), an expert is out where l or b is -infinity or NaN; then
 *   s_e = 1 / (1 + exp(-l_e)), or the softmax of l over the experts that are
 *         in; 0 for experts that are out
 *   c_e = s_e + b_e, formed in 64 bits
 * Experts lie in num_groups groups of E / num_groups consecutive ids.  A group
 * counts its largest c, or the sum of its two largest (of the experts that are
 * in; a single one counts alone).  The top_k experts with the largest c are
 * chosen within the top_groups best groups; equal values go to the lowest group
 * and the lowest id (c compared to 42 bits of its mantissa).  Experts that are
 * out come behind all others of the chosen groups.  The weights are
 *   w_j = scale s_j, or with renormalize scale s_j / sum_i s_i (0 where that sum
 *   is 0). */
typedef struct {
  int32_t score;       /* MOE_GATE_SOFTMAX or MOE_GATE_SIGMOID                        */
  int32_t num_groups;  /* divides num_experts; 1 (no groups) .. MOE_GATE_MAX_GROUPS   */
  int32_t top_groups;  /* 1..num_groups, with room for top_k experts                  */
  int32_t group_score; /* MOE_GROUP_MAX or MOE_GROUP_TOP2                             */
  int32_t renormalize; /* 0 or 1                                                      */
  float scale;         /* finite, > 0                                                 */
} moe_gate;

/* moe_route_permute through a gate.  bias: NULL or [E] fp32.  out->topk_ids in
 * descending order of c.  The arrays of the permutation (expert_offsets to
 * num_active) may be NULL, all of them together: then only topk_ids and topk_w
 * are written, and ws may be NULL.  ws: >= moe_route_workspace_bytes(). */
moe_status moe_route_gated(const moe_layer* layer, const moe_gate* gate, const float* logits, const float* bias,
                           const moe_route_out* out, void* ws, size_t ws_bytes, void* stream);

/* Its gradient for given d_topk_w = dL/dtopk_w [T][k] fp32, the choice being
 * constant: with ds_j = scale d_w_j, or with renormalize
 * ds_j = (scale d_w_j - sum_i d_w_i w_i) / sum_i s_i,
 *   sigmoid: d_logits[t][ids_j] = ds_j s_j (1 - s_j), 0 elsewhere
 *   softmax: d_logits[t][e] = s_e (ds_e - sum_j ds_j s_j)
 * (ds_e = 0 for experts not chosen).  Sigmoid scores are formed in 64 bits as in
 * the forward, softmax's with renormalize against the largest chosen, so that far
 * logits have their gradient too.  Ids outside [0, E) have no part; an id that
 * a token has twice takes both gradients.  The bias has no gradient.  d_logits:
 * [T][E] fp32 (over no input), written, or with accumulate != 0 added to what it
 * holds. */
moe_status moe_route_gated_backward(const moe_layer* layer, const moe_gate* gate, const float* logits,
                                    const float* bias, const int32_t* topk_ids, const float* d_topk_w,
                                    int32_t accumulate, float* d_logits, void* stream);

/* moe_expert_forward with its routing through a gate: the same arguments,
 * result and workspace. */
moe_status moe_expert_forward_gated(const moe_layer* layer, const moe_gate* gate, const void* x_bf16,
                                    const float* logits, const float* bias, const moe_qweights* qweights,
                                    const moe_scales* scales, const void* adapter_bf16, int32_t chunk_experts,
                                    void* out_bf16, void* ws, size_t ws_bytes, void* stream);

/* moe_expert_backward of moe_expert_forward_gated: d_logits through the gate
 * (moe_route_gated_backward of g_tj = <d_out_t, y_tj>; over neither the logits nor
 * the bias), the rest and the workspace as there; not timed. */
moe_status moe_expert_backward_gated(const moe_layer* layer, const moe_gate* gate, const void* x_bf16,
                                     const float* logits, const float* bias, const moe_qweights* qweights,
                                     const moe_scales* scales, const void* bwd_weights, const void* adapter_bf16,
                                     const void* d_out_bf16, int32_t chunk_experts, void* d_x_bf16, float* d_logits,
                                     float* d_adapter, void* ws, size_t ws_bytes, void* stream);

/* ---- The dense FP8 projection -------------------------------------------------
 * The linear layers beside the experts (a shared expert's among them) in the
 * experts' FP8 format: E4M3 codes W [N][K] with an fp32 scale per block of
 * 128 x 128, [ceil(N/128)][ceil(K/128)] (the last blocks may be smaller), and
 * activations quantized per 128 columns of a row as moe_quantize_activations
 * does (MOE_W_FP8_E4M3_B128, or MOE_W_FP8_E4M3_B128_POW2 with powers of two on
 * both sides, of which the exponent alone is used).  A NaN or an infinity in x makes
 * its whole row of y NaN, one in d_y its row of d_x and its column's row of d_w.
 * Results lie over no input.  A workspace serves one call at a time. */
typedef struct {
  int32_t num_tokens;   /* M: 0..2^20                                              */
  int32_t in_features;  /* K: multiple of 16, at most 2^17                         */
  int32_t out_features; /* N: the same                                             */
  int32_t wformat;      /* MOE_W_FP8_E4M3_B128 or MOE_W_FP8_E4M3_B128_POW2         */
  int64_t x_stride;     /* elements between rows of x: 0 (= K), or a multiple of 8, K..2^22 */
  int64_t dy_stride;    /* the same for d_y and N                                  */
} moe_linear;

/* What a call forms, for the workspace's size. */
enum { MOE_LINEAR_FORWARD = 0, MOE_LINEAR_D_X = 1, MOE_LINEAR_D_W = 2 };

/* Workspace bytes of moe_fp8_linear (grads = MOE_LINEAR_FORWARD) or of
 * moe_fp8_linear_backward (MOE_LINEAR_D_X, MOE_LINEAR_D_W, or both or-ed): the
 * codes and scales of the quantized operands, and parts of the sums (fp32) where
 * there are few tiles.  0 where none is needed (a few rows of x or d_y; ws may then
 * be NULL), and for an invalid or unsupported descriptor. */
size_t moe_fp8_linear_workspace_bytes(const moe_linear* lin, int32_t grads);

/* y = Q(x) W^T: x [M][K] bf16 (x_stride), y [M][N] bf16 (contiguous).  The
 * matrix cores add products of codes 8 at a time, aligned to the largest with 13
 * bits kept below it (1.4e-5 of a sum of normal values), everything else is added
 * in fp32; y is rounded once. */
moe_status moe_fp8_linear(const moe_linear* lin, const void* x_bf16, const void* w, const float* w_scale,
                          void* y_bf16, void* ws, size_t ws_bytes, void* stream);

/* W's transposed copy for the backward: w_t [K][N] codes and w_t_scale
 * [ceil(K/128)][ceil(N/128)]; num_tokens is not used. */
moe_status moe_fp8_linear_transpose(const moe_linear* lin, const void* w, const float* w_scale, void* w_t,
                                    float* w_t_scale, void* stream);

/* Gradients for given d_y = dL/dy [M][N] bf16 (dy_stride):
 *   d_x [M][K] bf16 = Q(d_y) W over the transposed copy; NULL: not formed (w_t
 *                     and w_t_scale are not read)
 *   d_w [N][K] bf16 = Qt(d_y)^T Qt(x), where Qt quantizes per column and block of
 *                     128 tokens; NULL: not formed (frozen; x is not read)
 * The quantizers pass gradients straight through.  Sums as in moe_fp8_linear,
 * each result rounded once.  num_tokens = 0 writes zeros to d_w. */
moe_status moe_fp8_linear_backward(const moe_linear* lin, const void* d_y_bf16, const void* w_t,
                                   const float* w_t_scale, const void* x_bf16, void* d_x_bf16, void* d_w_bf16,
                                   void* ws, size_t ws_bytes, void* stream);

/* ---- Clipping by the global norm ----------------------------------------------
 * Of the gradients that a step has formed (adapters, router, projections, head). */
typedef enum { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_F16 = 2 } moe_dtype;

/* One tensor of a list (host memory; the list is not needed after the call).
 * Addresses are aligned to the element (whole 16 bytes are faster). */
typedef struct {
  const void* data; /* device                                                         */
  void* out;        /* device: where the clipped values go; data itself: in place     */
  int64_t num;      /* elements, >= 0                                                 */
  int32_t dtype;    /* a moe_dtype value, of data and out                             */
} moe_tensor;

/* Workspace bytes of moe_grad_norm and moe_grad_clip for n tensors. */
size_t moe_grad_norm_workspace_bytes(int32_t n);

/* norm[0] = sqrt(sum of the squares of every element) in fp32 (device; 0 for an
 * empty list).  Squares and sums are formed in 64 bits, in an order that the sizes
 * fix.  `out` is not used. */
moe_status moe_grad_norm(const moe_tensor* tensors, int32_t n, float* norm, void* ws, size_t ws_bytes, void* stream);

/* The norm, and out = data c with c = max_norm / norm in fp32 where norm >
 * max_norm, else out = data (nothing is written in place).  A norm that is not
 * finite in fp32 clips nothing: the caller sees it and leaves the step out.
 * max_norm >= 0.
 * The tensors, norm and ws must not overlap. */
moe_status moe_grad_clip(const moe_tensor* tensors, int32_t n, float max_norm, float* norm, void* ws,
                         size_t ws_bytes, void* stream);

/* The second half alone, for a norm [1] that the caller holds on the device (one
 * joined over ranks); norm lies outside the tensors. */
moe_status moe_grad_scale(const moe_tensor* tensors, int32_t n, const float* norm, float max_norm, void* stream);

/* ---- Allocation-free forward -------------------------------------------
 * For callers that cannot allocate device memory or pass a workspace: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  Same computation, arguments (minus ws / ws_bytes) and result
 * as moe_expert_forward; the workspace is instead a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, reserved when
 * the library is loaded on that GPU and held until the process ends.  Layers
 * whose moe_workspace_bytes() exceeds it (e.g. more than a few thousand
 * tokens at hidden 7168) return MOE_ERR_WORKSPACE_TOO_SMALL with nothing
 * enqueued.  The call allocates nothing (no hipMalloc, no library
 * allocation); the first call on a device looks up that device's array
 * address once.  The stream must belong to the current device.  Every call on
 * one GPU uses the same array, whose contents persist between calls and are
 * overwritten by each call: calls that overlap on one GPU (other streams,
 * other host threads) race and must be serialised by the caller. */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)
moe_status moe_expert_forward_noalloc(const moe_layer* layer, const void* x_bf16, const float* logits,
                                      const moe_qweights* qweights, const moe_scales* scales,
                                      const void* adapter_bf16, int32_t chunk_experts, void* out_bf16,
                                      void* stream);

/* Static description of a status code (never NULL). */
const char* moe_status_str(moe_status status);

/* MOE_LP_ABI_VERSION of the built library. */
int32_t moe_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LP_H */

/*
 * moe.h -- C ABI of the single-GPU fused mixture-of-experts layer (GB300, sm_103a).
 *
 * The layer is the modular no-DP/EP pipeline described by the pages:
 *
 *   moe_route    -> topk_ids, topk_weights
 *   moe_align    -> per-expert grouping of the (token, choice) slots
 *   moe_prepare  -> a1q (+ a1q_scale)                         ("prepare")
 *   moe_experts  -> fused_expert_output, unweighted rows      ("experts")
 *   moe_finalize -> output (+ residual_out)                   ("finalize")
 *
 * with the experts also in other forms: moe_experts_act (other activations),
 * moe_experts_multi (routed and shared experts in the same launches),
 * moe_prepare_nvfp4 / moe_experts_nvfp4 (every operand NVFP4); and the whole
 * bf16 step as one launch for decode-sized problems: moe_layer_fused.  Around it: the
 * norm in front (moe_rmsnorm), projections and routers (moe_linear, moe_route_grouped), the
 * experts as separate calls (moe_grouped_linear, moe_activation), and the gradients.
 *
 * Sources: "[vLLM] MoE Oracle & Prepare/Finalize" blog, section "No DP/EP: the
 * simplest case" (prepare and finalize of MoEPrepareAndFinalizeNoDPEPModular);
 * "Fused MoE Kernel Features" (vLLM design doc), sections "Fused MoE Modular
 * All2All backends" and "Fused Experts Kernels"; "[flashinfer] MoE Finalize +
 * AllReduce fusion" page, introduction (finalize + shared row + residual +
 * RMSNorm + optional NVFP4 output).
 *
 * Conventions shared by every call
 *  - Every pointer argument is a DEVICE pointer on the current CUDA device,
 *    16-byte aligned, unless its comment says otherwise.  The caller owns and
 *    allocates every buffer, workspaces included; the library allocates no
 *    device memory.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and never synchronises (moe_device_status excepted).
 *  - Arguments are checked on the host before any launch; a bad argument
 *    returns an error status and launches nothing.  A launch failure returns
 *    MOE_ERR_CUDA.  No call aborts or throws.
 *  - Slot f = t * top_k + j names the j-th expert choice of token t.
 *  - Sizes are element counts; T (tokens) may be 0, in which case the call
 *    does nothing and returns MOE_OK.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *moe_stream_t; /* same type as cudaStream_t */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* null pointer, bad size or misaligned pointer   */
  MOE_ERR_UNSUPPORTED = 2,  /* valid request this library does not implement   */
  MOE_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required      */
  MOE_ERR_CUDA = 4,         /* a CUDA runtime/driver call or launch failed      */
  MOE_ERR_TIMEOUT = 5       /* a device-side wait gave up (see moe_device_status) */
} moe_status_t;

typedef enum {
  MOE_DT_BF16 = 0,
  MOE_DT_FP8_E4M3 = 1, /* OCP E4M3 ("e4m3fn"), saturating                    */
  MOE_DT_NVFP4 = 2,    /* E2M1 pairs + one E4M3 scale per 16 elements        */
  MOE_DT_FP32 = 3,
  MOE_DT_FP16 = 4 /* the linear and grouped products, moe_activation and the logits of moe_route_grouped only */
} moe_dtype_t;

typedef enum {
  MOE_SCORING_SOFTMAX_RENORM = 0, /* softmax over the chosen top-k logits     */
  MOE_SCORING_SIGMOID = 1         /* top-1, weight = sigmoid(logit)           */
} moe_scoring_t;

/* Activation between the two expert GEMMs: the activation column of the
 * "Fused Experts Kernels" table (vLLM design doc), which names them without
 * formulas.  With [g | u] = x . w13^T (gate rows first):
 *   MOE_ACT_SILU         h = silu(g) * u,  silu(g) = g / (1 + exp(-g))
 *   MOE_ACT_GELU         h = gelu(g) * u,  gelu(g) = g/2 (1 + erf(g / sqrt 2))
 *   MOE_ACT_GELU_TANH    h = g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) * u
 *   MOE_ACT_SWIGLUOAI    the clamped SwiGLU of the gpt-oss models:
 *                        g' = min(g, 7), u' = clamp(u, -7, 7),
 *                        h = (u' + 1) * g' * sigmoid(1.702 g')
 *   MOE_ACT_SILU_NO_MUL  h = silu(g); w13 holds the I gate rows only
 *   MOE_ACT_GELU_NO_MUL  h = gelu(g); w13 holds the I gate rows only */
typedef enum {
  MOE_ACT_SILU = 0,
  MOE_ACT_GELU = 1,
  MOE_ACT_GELU_TANH = 2,
  MOE_ACT_SWIGLUOAI = 3,
  MOE_ACT_SILU_NO_MUL = 4,
  MOE_ACT_GELU_NO_MUL = 5
} moe_activation_t;

/* act_group values for the quantisation formats of the "Fused MoE Kernel
 * Features" tables besides G(128): "A" (per activation token) and "T" (per
 * tensor). */
#define MOE_GROUP_TOKEN (-1)  /* one scale per token over all H channels   */
#define MOE_GROUP_TENSOR (-2) /* one scale over the whole activation tensor */

/* Quantisation of the expert inputs and weights.
 *   bf16:  {MOE_DT_BF16, 0, MOE_DT_BF16, 0, 0}   -- "no quantisation type"
 *   fp8:   {MOE_DT_FP8_E4M3, 128, MOE_DT_FP8_E4M3, 128, 128}
 *          activations: one fp32 scale per token per 128 channels ("G(128)"),
 *          a1q_scale [T, H/128]; weights: one fp32 scale per 128x128 block.
 *   fp8 with act_group MOE_GROUP_TOKEN: a1q_scale [T] ("A");
 *            act_group MOE_GROUP_TENSOR: a1q_scale [1] ("T").
 *          Every scale is s = fp32(max(amax, 1e-10) / 448) over its group and
 *          q = e4m3_rn_satfinite(fp32(x / s)).  In moe_experts the
 *          intermediate h is quantised in the same format: G(128) from fp32 h;
 *          A and T from h stored in bf16 (T: one scale over every expert's rows).
 * Other combinations return MOE_ERR_UNSUPPORTED. */
typedef struct {
  moe_dtype_t act;
  int act_group;
  moe_dtype_t weight;
  int w_block_n;
  int w_block_k;
} moe_quant_config;

/* Rows per expert tile in the tile map that moe_experts consumes. */
#define MOE_BLOCK_M 128

/* ------------------------------------------------------------------ route
 * Router: top-k experts per token and their weights.  The pages take
 * topk_ids/topk_weights as inputs of prepare and finalize ("No DP/EP"
 * listing); the router is the plainest reading of them:
 *   MOE_SCORING_SOFTMAX_RENORM: the top_k largest fp32 logits, ordered larger
 *     first, equal logits to the lower expert index; weight_j =
 *     exp(l_j - l_max) / sum over the chosen i of exp(l_i - l_max).
 *   MOE_SCORING_SIGMOID (top_k must be 1): argmax (lower index on ties),
 *     weight = 1 / (1 + exp(-l)) -- the Llama-type router whose weight is
 *     applied on the input ("Fused MoE Kernel Features", All2All section).
 * logits [T, E] fp32 row-major; topk_ids [T, top_k] int32; topk_weights
 * [T, top_k] fp32.  1 <= E <= 1024, 1 <= top_k <= min(E, 32).  NaN logits rank
 * below every number. */
moe_status_t moe_route(const float *logits, int T, int E, int top_k, int scoring,
                       int32_t *topk_ids, float *topk_weights, moe_stream_t stream);

/* ------------------------------------------------------------------ align
 * Per-expert token alignment and permutation: the slots are sorted by the key
 * (expert id, slot f), which groups each expert's rows contiguously in
 * ascending slot order (deterministic).
 *   expert_offsets [E + 1] int32: exclusive prefix sum of the per-expert
 *                  counts; expert_offsets[E] = T * top_k.
 *   sorted_slot    [T * top_k] int32: sorted_slot[p] = f.
 *   inv_slot       [T * top_k] int32: inv_slot[sorted_slot[p]] = p (may be NULL).
 *   tile_map       [moe_tile_map_capacity(T * top_k, E, block_m)] pairs of
 *                  int32 (expert, first row p) for each block_m-row tile of
 *                  each expert, expert by expert; entries past num_tiles are
 *                  left untouched.
 *   num_tiles      [1] int32: number of valid tile_map entries.
 *   ws             scratch of moe_align_workspace_size(T, top_k, E) bytes.
 * topk_ids values must lie in [0, E); 1 <= E <= 1024; block_m >= 1
 * (moe_experts needs MOE_BLOCK_M). */
moe_status_t moe_align(const int32_t *topk_ids, int T, int top_k, int E, int block_m,
                       int32_t *expert_offsets, int32_t *sorted_slot, int32_t *inv_slot,
                       int32_t *tile_map, int32_t *num_tiles, void *ws, size_t ws_bytes,
                       moe_stream_t stream);
size_t moe_align_workspace_size(int T, int top_k, int E);
int moe_tile_map_capacity(int num_slots, int E, int block_m);

/* ------------------------------------------------------------------ align, no allocation
 * Not part of the method: the pages have no counterpart of this call.  It is
 * moe_align for callers that cannot allocate device memory at call time --
 * runtimes that plan every device buffer ahead and forbid allocation while
 * serving, or plugin-style hosts whose per-call hook may not allocate -- and so
 * cannot supply the `ws` scratch that moe_align needs.
 *
 * Same arguments, layouts and results as moe_align, minus ws/ws_bytes.  The
 * scratch is a fixed array of MOE_ALIGN_NOALLOC_SCRATCH_BYTES inside the
 * library (every GPU that loads the library holds it until the process exits);
 * a problem needing more (moe_align_workspace_size(T, top_k, E) larger than
 * that) is rejected with MOE_ERR_WORKSPACE before anything is launched.  The
 * call allocates nothing.
 *  - The first call in each CUDA context looks up the array's device address
 *    (cudaGetSymbolAddress) with that context current and caches it for the
 *    context: normally once per device (its primary context), and once more
 *    after a cudaDeviceReset or in a caller's own context, where the library's
 *    device code is loaded again at another address.  Make that first call
 *    before any stream capture in the context.
 *  - All calls share the one array and it keeps the last call's contents (each
 *    call writes every entry it later reads, so nothing needs clearing).  Calls
 *    whose work overlaps on the GPU -- on different streams, or from different
 *    host threads without ordering -- race on it: order them on one stream. */
#define MOE_ALIGN_NOALLOC_SCRATCH_BYTES (256 * 1024)
moe_status_t moe_align_noalloc(const int32_t *topk_ids, int T, int top_k, int E, int block_m,
                               int32_t *expert_offsets, int32_t *sorted_slot, int32_t *inv_slot,
                               int32_t *tile_map, int32_t *num_tiles, moe_stream_t stream);

/* ------------------------------------------------------------------ prepare
 * Prepare ("No DP/EP" listing): when apply_router_weight_on_input is set
 * (top_k must be 1) the input is first multiplied by the token's weight cast to
 * bf16, a1 <- bf16(a1 * bf16(w)); then it is quantised per qc->act:
 *   MOE_DT_BF16:     a1q [T, H] bf16 (a copy; when a1q == a1 and no weight is
 *                    applied nothing is launched -- the passthrough);
 *   MOE_DT_FP8_E4M3: a1q [T, H] E4M3 codes (uint8), a1q_scale [T, H/128] fp32:
 *                    s = fp32(max(amax, 1e-10f) / 448) per 128 channels,
 *                    q = e4m3_rn_satfinite(x / s) (IEEE fp32 division);
 *                    act_group MOE_GROUP_TOKEN: a1q_scale [T], one s per token;
 *                    MOE_GROUP_TENSOR: a1q_scale [1], one s for the tensor
 *                    (a1q_scale is also the reduction's scratch until the call's
 *                    last launch writes the scale).
 * a1 [T, H] bf16.  topk_weights [T, top_k] fp32 (read only with the weight
 * flag).  topk_ids is accepted for parity with the pages' signature and unused
 * (may be NULL).  H % 128 == 0 for fp8, H % 8 == 0 for bf16. */
moe_status_t moe_prepare(const void *a1, const float *topk_weights, const int32_t *topk_ids,
                         int T, int H, int top_k, int apply_router_weight_on_input,
                         const moe_quant_config *qc, void *a1q, float *a1q_scale,
                         moe_stream_t stream);

/* ------------------------------------------------------------------ experts
 * Grouped expert MLPs ("Fused Experts Kernels": two GEMMs with SiLU-and-mul
 * between them).  For every expert e and sorted row p in
 * [expert_offsets[e], expert_offsets[e+1]), with slot f = sorted_slot[p] and
 * token t = f / top_k:
 *   [g | u] = a1q[t] . w13[e]^T          (w13 [E, 2I, H]: rows 0..I-1 gate,
 *                                          rows I..2I-1 up; K-contiguous)
 *   h       = silu(g) * u                 (bf16, or E4M3 G(128) with fp8)
 *   fused_expert_output[f] = h . w2[e]^T  (w2 [E, H, I]; bf16 [T*top_k, H],
 *                                          token-major, unweighted)
 * Accumulation is fp32.  fp8: a1q E4M3 + a1q_scale in the qc->act_group
 * format (G(128) [T, H/128], A [T], T [1]); w13/w2 E4M3
 * with w13_scale [E, 2I/128, H/128] and w2_scale [E, H/128, I/128] fp32; each
 * 128-deep K block is scaled by a1q_scale * w_scale before it is added.
 * expert_offsets / sorted_slot / tile_map / num_tiles come from moe_align with
 * block_m = MOE_BLOCK_M.  sorted_slot may be NULL when E == 1 and top_k == 1
 * (identity permutation; tile_map and expert_offsets are still required).
 * ws: moe_workspace_size(...) bytes.  H % 128 == 0, I % 128 == 0. */
moe_status_t moe_experts(const void *a1q, const float *a1q_scale, const void *w13,
                         const float *w13_scale, const void *w2, const float *w2_scale,
                         const int32_t *expert_offsets, const int32_t *sorted_slot,
                         const int32_t *tile_map, const int32_t *num_tiles, int T, int H,
                         int I, int E, int top_k, const moe_quant_config *qc,
                         void *fused_expert_output, void *ws, size_t ws_bytes,
                         moe_stream_t stream);
/* moe_experts with another activation (a moe_activation_t); moe_experts is
 * this call with MOE_ACT_SILU.  For the *_NO_MUL activations w13 is [E, I, H]
 * (fp8: w13_scale [E, I/128, H/128]).  Same arguments, workspace and errors
 * otherwise; an unknown activation returns MOE_ERR_UNSUPPORTED. */
moe_status_t moe_experts_act(const void *a1q, const float *a1q_scale, const void *w13,
                             const float *w13_scale, const void *w2, const float *w2_scale,
                             const int32_t *expert_offsets, const int32_t *sorted_slot,
                             const int32_t *tile_map, const int32_t *num_tiles, int T, int H,
                             int I, int E, int top_k, const moe_quant_config *qc, int activation,
                             void *fused_expert_output, void *ws, size_t ws_bytes,
                             moe_stream_t stream);
size_t moe_workspace_size(int T, int H, int I, int E, int top_k, const moe_quant_config *qc);

/* Where moe_experts / moe_experts_act leave the intermediate h in their workspace
 * (it stays there until the workspace is used again), for inspection of the stage
 * between the two GEMMs.  Rows are the S = T * top_k sorted rows p (expert order):
 *   *h_offset       byte offset in ws of h [S, I]: bf16, or E4M3 codes for fp8;
 *   *h_scale_offset fp8 only (0 otherwise): byte offset of h's fp32 scales --
 *                   G(128): [I/128][*scale_stride], transposed (the scale of row p and
 *                   128-column group g at g * *scale_stride + p); "A" and "T": [S],
 *                   one per row (*scale_stride = 1; "T" repeats the tensor's scale);
 *   *scale_stride   as above (0 for bf16).
 * Same sizes and qc as the moe_experts call.  Returns MOE_ERR_INVALID_ARG on a bad
 * size or null pointer, MOE_ERR_UNSUPPORTED for a qc moe_experts rejects.  The
 * pages have no counterpart: it exposes a stage of the experts to the caller. */
moe_status_t moe_workspace_intermediate(int T, int H, int I, int E, int top_k, const moe_quant_config *qc,
                                        size_t *h_offset, size_t *h_scale_offset, int *scale_stride);

/* Several expert problems with the same hidden size H in the same two GEMM
 * launches -- typically a layer's routed experts and its shared expert (E = 1,
 * top_k = 1, sorted_slot NULL).  Not in the pages: their shared-expert row is a
 * separate MLP the finalize adds; computing both in one pass of launches saves
 * each GEMM's start-up and tail once (decode-sized layers spend a large share
 * of a GEMM there).  Each problem as for moe_experts_act, all with the same
 * activation and qc.  num_problems is 1 or 2; two problems need bf16 (qc) and
 * the same I (the second GEMM's depth), else MOE_ERR_UNSUPPORTED.  Problems
 * with no rows (T == 0) are skipped.  ws: moe_workspace_size_multi(...) bytes;
 * every output and error as for moe_experts. */
typedef struct {
  const void *a1q;
  const float *a1q_scale;
  const void *w13;
  const float *w13_scale;
  const void *w2;
  const float *w2_scale;
  const int32_t *expert_offsets;
  const int32_t *sorted_slot;
  const int32_t *tile_map;
  const int32_t *num_tiles;
  int T, I, E, top_k;
  void *fused_expert_output;
} moe_experts_problem;

moe_status_t moe_experts_multi(const moe_experts_problem *problems, int num_problems, int H,
                               const moe_quant_config *qc, int activation, void *ws,
                               size_t ws_bytes, moe_stream_t stream);
size_t moe_workspace_size_multi(const moe_experts_problem *problems, int num_problems, int H,
                                const moe_quant_config *qc);

/* ------------------------------------------------------------------ NVFP4 experts
 * The experts with every operand in NVFP4 ("Fused MoE Kernel Features", experts
 * table: nvfp4 is a quantisation type of the cutlass_fp4 and trtllm experts),
 * in the encoding of the finalize page's packed output: E2M1 codes in pairs
 * (element 2i in the low nibble), one E4M3 scale code per 16 consecutive
 * elements of a row, and one fp32 global scale g per tensor, value =
 * e2m1(q) * e4m3(sf) * g.  Quantising a row (prepare, the intermediate):
 *   sf = e4m3_rn_satfinite(fp32(amax16 / fp32(6 g))),
 *   q  = e2m1_rn_satfinite(fp32(x / fp32(e4m3(sf) * g)))   (q = 0 when that is 0).
 *
 * moe_prepare_nvfp4: a1 [T, H] bf16 (optionally first a1 <- bf16(a1 *
 *   bf16(w)) with the top-1 weight, as moe_prepare) -> a1q [T, H/2] codes,
 *   a1q_sf [T, H/16] scale codes, with the global scale *a1_gscale (device
 *   pointer, fp32, > 0).  H % 16 == 0; a1 and a1q 16-byte aligned.
 *
 * moe_experts_nvfp4: for every expert e and its sorted rows (as moe_experts):
 *   [g | u] = dequant(a1q[t]) . dequant(w13[e])^T    fp32 accumulation; the
 *            tensor core applies the E4M3 block scales, the product of the two
 *            global scales *a1_gscale * w13_gscale[e] multiplies the sums
 *   h      = act(g, u) stored bf16, then quantised to NVFP4 with *h_gscale
 *   fused_expert_output[f] = dequant(h) . dequant(w2[e])^T   (bf16 [T*top_k, H],
 *            token-major, unweighted)
 * w13 [E, 2I, H/2] codes with w13_sf [E, 2I, H/16] (rows 0..I-1 gate, I..2I-1
 * up; the *_NO_MUL activations: [E, I, H/2] and [E, I, H/16]); w2 [E, H, I/2]
 * with w2_sf [E, H, I/16]; w13_gscale, w2_gscale [E] fp32; a1_gscale, h_gscale
 * [1] fp32 (all device pointers).  expert_offsets / sorted_slot / tile_map /
 * num_tiles as for moe_experts (sorted_slot NULL only when E == 1 and top_k ==
 * 1).  H % 256 == 0, I % 256 == 0; every code, scale and output pointer 16-byte
 * aligned.  ws: moe_workspace_size_nvfp4(...) bytes (MOE_ERR_WORKSPACE when
 * smaller); an unknown activation returns MOE_ERR_UNSUPPORTED.  The caller owns
 * every buffer; nothing is allocated. */
moe_status_t moe_prepare_nvfp4(const void *a1, const float *topk_weights, int T, int H, int top_k,
                               int apply_router_weight_on_input, const float *a1_gscale, void *a1q,
                               void *a1q_sf, moe_stream_t stream);
moe_status_t moe_experts_nvfp4(const void *a1q, const void *a1q_sf, const float *a1_gscale,
                               const void *w13, const void *w13_sf, const float *w13_gscale,
                               const void *w2, const void *w2_sf, const float *w2_gscale,
                               const float *h_gscale, const int32_t *expert_offsets,
                               const int32_t *sorted_slot, const int32_t *tile_map,
                               const int32_t *num_tiles, int T, int H, int I, int E, int top_k,
                               int activation, void *fused_expert_output, void *ws, size_t ws_bytes,
                               moe_stream_t stream);
size_t moe_workspace_size_nvfp4(int T, int H, int I, int E, int top_k);
/* Where moe_experts_nvfp4 leaves the intermediate in its workspace: byte offsets of
 * the bf16 h [S, I] that the first GEMM writes, and of its NVFP4 codes [S, I/2] and
 * scale codes [S, I/16] that the second GEMM reads (S = T * top_k sorted rows).
 * H % 256 == 0 and I % 256 == 0, else MOE_ERR_INVALID_ARG. */
moe_status_t moe_workspace_intermediate_nvfp4(int T, int H, int I, int E, int top_k, size_t *hb_offset,
                                              size_t *hq_offset, size_t *hsf_offset);

/* ------------------------------------------------------------------ batched activation format
 * The "batched" format of the prepare output ("Fused MoE Kernel Features", section "Fused MoE
 * Modular All2All backends": a prepare returns its activations in the standard or the batched
 * format and the finalize takes that format back to standard; "Fused Experts Kernels" lists
 * batched entry points).  The pages leave the layout to another document; the reading here:
 * one slab per expert, [E, max_tokens, H]: expert e's slab holds, in ascending slot order, the
 * prepared rows of the tokens that chose e, and expert_num_tokens[e] counts them.  Rows past a
 * count are neither written nor read.
 *
 * moe_prepare_batched: moe_prepare (same qc, same weight on the input) of every token, then
 *   token t's prepared row copied to the slab of each expert it chose.  expert_offsets and
 *   sorted_slot are moe_align's (they give each expert's slots in ascending order).  Outputs:
 *   a1q_b [E, max_tokens, H] (bf16 or E4M3 codes); a1q_b_scale: G(128) [E, max_tokens, H/128],
 *   "A" [E, max_tokens], "T" [1] (fp32; unused for bf16, may be NULL); expert_num_tokens [E]
 *   int32 (each count capped at max_tokens).  A slot past max_tokens in its expert's slab is
 *   left out and MOE_ERR_INVALID_ARG is recorded in the device status word (moe_device_status);
 *   nothing is written out of bounds.  ws: moe_prepare_batched_workspace_size(T, H, qc) bytes
 *   (bf16 without the weight on the input needs none: the rows come from a1 itself).
 * moe_experts_batched: the experts of moe_experts_act on the slabs: for every expert e and row
 *   m < expert_num_tokens[e] (taken as min(max(count, 0), max_tokens)), out_b[e, m] =
 *   expert_e(a1q_b[e, m]); out_b [E, max_tokens, H] bf16, unweighted; other rows untouched.
 *   Same weights, qc, activations and intermediate as moe_experts_act.  ws:
 *   moe_workspace_size_batched(E, max_tokens, H, I, qc) bytes.  H % 128 == 0, I % 128 == 0.
 * moe_finalize_batched: moe_finalize reading the expert row of slot f = t * top_k + j from
 *   expert_output_b [E, max_tokens, H] at (e = topk_ids[f], inv_slot[f] - expert_offsets[e])
 *   (moe_align's inv_slot and expert_offsets); every other argument, output and check as for
 *   moe_finalize. */
size_t moe_prepare_batched_workspace_size(int T, int H, const moe_quant_config *qc);
moe_status_t moe_prepare_batched(const void *a1, const float *topk_weights, const int32_t *expert_offsets,
                                 const int32_t *sorted_slot, int T, int H, int top_k, int E, int max_tokens,
                                 int apply_router_weight_on_input, const moe_quant_config *qc, void *a1q_b,
                                 float *a1q_b_scale, int32_t *expert_num_tokens, void *ws, size_t ws_bytes,
                                 moe_stream_t stream);
size_t moe_workspace_size_batched(int E, int max_tokens, int H, int I, const moe_quant_config *qc);
moe_status_t moe_experts_batched(const void *a1q_b, const float *a1q_b_scale, const void *w13,
                                 const float *w13_scale, const void *w2, const float *w2_scale,
                                 const int32_t *expert_num_tokens, int E, int max_tokens, int H, int I,
                                 const moe_quant_config *qc, int activation, void *out_b, void *ws,
                                 size_t ws_bytes, moe_stream_t stream);
moe_status_t moe_finalize_batched(void *output, const void *expert_output_b, int max_tokens,
                                  const float *topk_weights, const int32_t *topk_ids, const int32_t *inv_slot,
                                  const int32_t *expert_offsets, const void *shared, const void *residual,
                                  const void *rms_weight, float eps, int T, int H, int top_k,
                                  int apply_router_weight_on_input, moe_dtype_t out_dtype, uint8_t *out_scale,
                                  float out_global_scale, void *residual_out, moe_stream_t stream);

/* ------------------------------------------------------------------ single-launch layer
 * The whole bf16 layer step in one cooperative kernel launch -- the monolithic form of
 * the experts ("[vLLM] MoE Oracle & Prepare/Finalize", section "Modular vs
 * Monolithic": one kernel from the router logits to the layer output) -- for
 * decode-sized problems.  Its phases, separated by grid-wide barriers, compute what the
 * separate calls do: moe_route (scoring as there), moe_align (the same order),
 * prepare (bf16; a1 <- bf16(a1 * bf16(w)) with apply_router_weight_on_input, top_k 1),
 * the experts with SiLU-and-mul (the shared expert, when given, in the same GEMM units
 * on the unweighted a1), and moe_finalize's sum (weights skipped with the weight on the
 * input) + shared row + residual, RMSNorm when rms_weight is given, bf16 output.
 * logits [T, E] fp32; a1 [T, H] bf16; w13 [E, 2I, H], w2 [E, H, I] bf16; shared_w13
 * [2I, H] and shared_w2 [H, I] bf16, both or neither; residual [T, H] and rms_weight
 * [H] bf16 or NULL; topk_ids / topk_weights [T, top_k] are written as by moe_route;
 * output [T, H] bf16.  Limits: T * top_k <= 2048, E <= 256, H and I multiples of 128,
 * H <= 12288; beyond them, or on a device without cooperative launch,
 * MOE_ERR_UNSUPPORTED.  ws: moe_layer_fused_workspace_size(...) bytes, caller-owned;
 * every wait (the grid barriers included) gives up as described under "status". */
moe_status_t moe_layer_fused(const float *logits, const void *a1, int T, int H, int I, int E, int top_k,
                             int scoring, int apply_router_weight_on_input, const void *w13, const void *w2,
                             const void *shared_w13, const void *shared_w2, const void *residual,
                             const void *rms_weight, float eps, int32_t *topk_ids, float *topk_weights,
                             void *output, void *ws, size_t ws_bytes, moe_stream_t stream);
size_t moe_layer_fused_workspace_size(int T, int H, int I, int E, int top_k, int has_shared);

/* ------------------------------------------------------------------ finalize
 * Finalize: the top-k weight-and-reduce of the "No DP/EP" listing followed by
 * the single-GPU part of the flashinfer finalize fusion (introduction of its
 * page, all-reduce removed):
 *   o_t = sum_j w_tj * y[t*top_k + j]   (w_tj = 1 when the weights were
 *                                         applied on the input)
 *         + shared_t + residual_t        (each optional: NULL = absent)
 *   residual_out_t = bf16(o_t)           (optional, NULL = not written)
 *   o_t <- o_t * rsqrt(mean_h(o_t^2) + eps) * rms_weight  (when rms_weight)
 * Sums in fp32.  Output per out_dtype:
 *   MOE_DT_BF16:  output [T, H] bf16;
 *   MOE_DT_FP32:  output [T, H] fp32;
 *   MOE_DT_NVFP4: output [T, H/2] uint8, element 2i in the low nibble, and
 *                 out_scale [T, H/16] E4M3 codes: per 16 elements
 *                 sf = e4m3(amax / (6 g)), q = e2m1(x / (sf g)), g =
 *                 out_global_scale > 0.
 * fused_expert_output [T*top_k, H] bf16; topk_weights [T, top_k] fp32;
 * shared, residual, residual_out [T, H] bf16; rms_weight [H] bf16.  residual_out
 * may be residual itself (the sum is then written over the residual, in place);
 * any other overlap between inputs and outputs is not allowed.  topk_ids
 * is accepted for parity with the pages' signature and unused (may be NULL).
 * H % 8 == 0 (H % 16 == 0 for NVFP4), 1 <= top_k <= 32. */
moe_status_t moe_finalize(void *output, const void *fused_expert_output, const float *topk_weights,
                          const int32_t *topk_ids, const void *shared, const void *residual,
                          const void *rms_weight, float eps, int T, int H, int top_k,
                          int apply_router_weight_on_input, moe_dtype_t out_dtype,
                          uint8_t *out_scale, float out_global_scale, void *residual_out,
                          moe_stream_t stream);

/* ------------------------------------------------------------------ linear projection
 * A dense projection with its epilogue in the same launch -- the router's gate (bf16 hidden
 * states to fp32 logits) and the dense layers beside the experts:
 *   z   = x . w^T + bias                     fp32 accumulation
 *   out = act(z) + residual                  rounded once, to out_dtype
 *   preact = z in dtype                      (optional: what moe_linear_backward takes)
 * x [M, K], w [N, K] (K-contiguous) and bias [N] (NULL = none) in dtype (MOE_DT_BF16 or
 * MOE_DT_FP16); out [M, N] and residual [M, N] (NULL = none) in out_dtype (dtype itself or
 * MOE_DT_FP32); preact [M, N] in dtype, NULL = not written.  residual may be out itself (the
 * projection is then added in place); any other overlap of an output with another buffer is
 * not allowed.  activation: a moe_linear_activation_t.  0 <= M <= 2^30 (0: nothing is done),
 * 1 <= N <= 2^21, 8 <= K <= 2^30 and K % 8 == 0 (an N that is a multiple of 8 is stored by
 * 16-byte vectors); a product of over 2^27 tiles of 128 x 64 may be MOE_ERR_UNSUPPORTED.  Every pointer
 * 16-byte aligned.  A K that is no multiple of 64 (rows that do not start on 128 bytes) is
 * copied at about half the rate, which large products feel: a caller who can pad K should.
 * A row of x that holds a NaN or an infinity affects that row of out alone.  The tensor core's
 * own fp32 sums truncate; they are added with rounding to fp32 sums every 512 elements (fp32
 * outputs), 8192 (fp16 outputs and gradients) or 16384 (bf16), so that terms of one sign lose at
 * most about 5e-5 (fp16) and 1e-4 (bf16) of a sum however long: a tenth and a fortieth of the
 * rounding of the output.
 * The sums of a call have a fixed order: the same inputs give the same bits. */
typedef enum {
  MOE_LINEAR_NONE = 0,      /* act(z) = z                                            */
  MOE_LINEAR_SILU = 1,      /* z / (1 + exp(-z))                                     */
  MOE_LINEAR_GELU = 2,      /* z/2 (1 + erf(z / sqrt 2))                             */
  MOE_LINEAR_GELU_TANH = 3  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))         */
} moe_linear_activation_t;

moe_status_t moe_linear(const void *x, const void *w, const void *bias, const void *residual, int M,
                        int N, int K, moe_dtype_t dtype, int activation, moe_dtype_t out_dtype,
                        void *out, void *preact, moe_stream_t stream);

/* Gradients of moe_linear, given dout [M, N], the gradient of out, in dout_dtype (dtype or
 * MOE_DT_FP32):
 *   dz    = dout * act'(preact)             (act' is 1 or 0 far from 0 and at the infinities: of
 *                                            the preacts only a NaN makes a NaN)
 *   dx    = dz . w          [M, K] in dtype
 *   dw    = dz^T . x        [N, K] in dtype
 *   dbias = sum over m of dz  [N] in dtype (summed in fp32 from dz before any rounding)
 * Each of dx, dw and dbias may be NULL (not computed), not all three.  The gradient of the
 * residual is dout itself.  preact [M, N] in dtype is what moe_linear wrote (required unless
 * the activation is MOE_LINEAR_NONE, where it is not read).  The tensor cores take dz in
 * dtype: where it has to be computed, or dout is fp32, it is rounded to dtype once (with
 * fp16, the caller's loss scale keeps it in range).  A caller who wants an fp32 dout kept hands in
 * its two parts, dout rounded to dtype and what that leaves, rounded too, as 2M rows over x
 * twice: dw and dbias then sum both, and dx comes in two parts to add.  M == 0 sets dw and dbias to zero.
 * ws: moe_linear_backward_workspace_size(M, N, K) bytes (asked with the call's device
 * current: it depends on the number of SMs); it belongs to one call at a time -- calls, or
 * replayed graphs, that may run at once need one each.  Sizes, alignment and the order of sums as
 * for moe_linear; outputs overlap nothing. */
moe_status_t moe_linear_backward(const void *dout, moe_dtype_t dout_dtype, const void *x, const void *w,
                                 const void *preact, int M, int N, int K, moe_dtype_t dtype,
                                 int activation, void *dx, void *dw, void *dbias, void *ws,
                                 size_t ws_bytes, moe_stream_t stream);
size_t moe_linear_backward_workspace_size(int M, int N, int K);

/* ------------------------------------------------------------------ grouped route
 * Router with scores over all experts, a bias that balances their load, and expert groups:
 *   s_e = sigmoid(l_e)  or  softmax(l)_e over the E experts       (cfg->score)
 *   c_e = s_e + bias_e                       (bias [E] fp32, NULL = none: it steers the choice
 *                                             and does not enter the weights)
 *   the E experts form n_group groups of E / n_group consecutive ones; a group's score is the
 *   sum of its group_top largest c (1: its best expert, 2: its two best), and the topk_group
 *   groups of largest score are kept, equal scores to the lower group index
 *   topk_ids: the top_k experts of largest c in the kept groups, larger first, equal c to the
 *   larger logit and then to the lower index
 *   topk_weights_j = s_j * scale, with renormalize s_j / (sum of the chosen s) * scale (0 when
 *   that sum is 0)
 * The choice is the one of fp64 arithmetic on the given values: scores too close to be ordered
 * in fp32 are compared more exactly (without a bias and with group_top 1 the logits themselves
 * are ranked, which is exact; scores below 1e-300, which fp64 itself holds with few digits or not at
 * all, may count as 0).  (MoE routers of the DeepSeek-V3 kind: sigmoid, bias,
 * 4 of 8 groups by their two best, top 8, scale 2.5; plain softmax top-k: n_group 1.)
 * A logit or bias of -inf or NaN masks the expert: weight 0 (a softmax's denominator counts every
 * unmasked logit, whatever its bias), no share in its group's score (a
 * group of masked experts alone ranks last), chosen only when the kept groups have fewer than
 * top_k others, lower index first, with weight 0.  +inf counts as the largest finite number.
 * logits [T, E] in logits_dtype (MOE_DT_FP32, MOE_DT_BF16 or MOE_DT_FP16); topk_ids [T, top_k]
 * int32; topk_weights [T, top_k] fp32.  T <= 2^30, 1 <= E <= 1024, 1 <= top_k <= 32, n_group <= 32
 * divides E, 1 <= topk_group <= n_group, group_top 1 or 2 (at most the group's size), top_k <=
 * topk_group * E / n_group, scale finite. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;

typedef struct {
  int score;       /* a moe_score_t */
  int n_group;     /* 1: no groups  */
  int topk_group;
  int group_top;
  int renormalize;
  float scale;
} moe_route_config;

moe_status_t moe_route_grouped(const void *logits, moe_dtype_t logits_dtype, const float *bias, int T,
                               int E, int top_k, const moe_route_config *cfg, int32_t *topk_ids,
                               float *topk_weights, moe_stream_t stream);

/* Gradient of moe_route_grouped's weights with respect to the logits, the choice held fixed
 * (the bias has none): given dweights [T, top_k] fp32, the logits, bias and topk_ids of the
 * forward call, dlogits [T, E] in logits_dtype, every element written:
 *   renormalize, with p = s / (sum of the chosen s):
 *     dl_j = scale p_j f_j (dw_j - sum_i p_i dw_i),   f = 1 - s (sigmoid) or 1 (softmax)
 *   sigmoid otherwise:  dl_j = scale dw_j s_j (1 - s_j)
 *     (both 0 for the experts that were not chosen)
 *   softmax otherwise:  dl_e = s_e (g_e - sum_i g_i s_i), g = scale dw on the chosen, else 0
 * Only score, renormalize and scale of cfg are used (the others are checked as above).  An id
 * chosen twice in a row adds up; an id outside [0, E) is left out and recorded as
 * MOE_ERR_INVALID_ARG in the device status word.  A masked (-inf or NaN) logit gets 0, and the
 * constant weight of a masked expert has no gradient; bias is read for its masks alone (NULL: it
 * masks none). */
moe_status_t moe_route_grouped_backward(const float *dweights, const void *logits,
                                        moe_dtype_t logits_dtype, const float *bias, const int32_t *topk_ids,
                                        int T, int E, int top_k, const moe_route_config *cfg, void *dlogits,
                                        moe_stream_t stream);

/* ------------------------------------------------------------------ finalize, gradient
 * Gradients of moe_finalize with its bf16 output.  With o_t the sum that the forward call
 * normalised and r = 1 / sqrt(mean_h(o^2) + eps):
 *   G = r (gamma dout - o r^2 mean_h(gamma dout o))    with rms_weight (gamma)
 *     = dout                                           without
 *   G += dresidual_out                                 (optional)
 *   dy[t * top_k + j] = w_tj G                         (bf16 [T * top_k, H]; w = 1 when
 *                                                       topk_weights is NULL: the weights were
 *                                                       applied on the input)
 *   dweights[t, j] = sum_h G_h y[t * top_k + j, h]     (fp32 [T, top_k])
 *   dsum = G                                           (bf16 [T, H]: the gradient of the shared
 *                                                       row and of the residual)
 *   drms_h = sum_t dout o r                            (fp32 [H])
 * dout and dresidual_out [T, H] bf16 are the gradients of output and residual_out;
 * residual_out [T, H] bf16 is what the forward call wrote (o in bf16, read only with
 * rms_weight, then required); fused_expert_output (y) [T * top_k, H] bf16 is read for
 * dweights alone (may be NULL without it).  dy, dweights (needs topk_weights), dsum and drms
 * (needs rms_weight) may each be NULL: not computed; not all.  Sums in fp32, in a fixed order;
 * G stays in fp32 until an output is rounded.  T <= 2^30 (0 sets drms to zero), H % 8 == 0, H <=
 * 16384, 1 <= top_k <= 32.  ws: moe_finalize_backward_workspace_size(T, H) bytes (needed for
 * drms alone; as for moe_linear_backward it depends on the device and belongs to one call).  dsum
 * may be dout or dresidual_out itself; no other overlap. */
moe_status_t moe_finalize_backward(const void *dout, const void *dresidual_out, const void *residual_out,
                                   const void *rms_weight, float eps, const void *fused_expert_output,
                                   const float *topk_weights, int T, int H, int top_k, void *dy,
                                   float *dweights, void *dsum, float *drms, void *ws, size_t ws_bytes,
                                   moe_stream_t stream);
size_t moe_finalize_backward_workspace_size(int T, int H);

/* ------------------------------------------------------------------ RMSNorm
 * The norm in front of the layer, with the residual's addition before it and the 8-bit rows of
 * the fp8 experts behind it, in one pass over the rows:
 *   v = x + residual              (fp32; residual NULL: v = x)
 *   residual_out = bf16(v)        (optional, NULL = not written)
 *   n = v * weight / sqrt(mean_h(v^2) + eps)
 *   out = bf16(n)                 (optional)
 *   q, q_scale                    n quantised as by moe_prepare, from the fp32 n: s =
 *                                 fp32(max(amax, 1e-10) / 448), q = e4m3_rn_satfinite(n / s)
 * qc: NULL or act MOE_DT_BF16: no q (q and q_scale NULL).  act MOE_DT_FP8_E4M3: act_group 128
 * (q_scale [T, ceil(H / 128)]; a last group may be shorter) or MOE_GROUP_TOKEN (q_scale [T]); other
 * groups are MOE_ERR_UNSUPPORTED.  x, residual, residual_out, out [T, H] and weight [H] bf16, q
 * [T, H] E4M3 codes.  0 <= T <= 2^30, H % 8 == 0, 8 <= H <= 16384, eps >= 0; out or q is required.
 * The squares are summed in fp32 in an order that T, H, eps and the device fix: the same call gives the same bits, and a
 * row in a call with another T may differ by an fp32 rounding.  |v| beyond 1e19 / sqrt(H) overflows the sum; small
 * values keep their digits whatever eps is, and a row of zeros is NaN where eps is 0.  A row with a NaN or
 * an infinity affects that row alone.  residual_out may be residual or x, and out x or residual, itself (a row
 * is read before it is written); no other overlap.  The gradients, from residual_out (x without a residual),
 * are moe_finalize_backward's dsum and drms (topk_weights, dy and dweights NULL, top_k 1). */
moe_status_t moe_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int T, int H,
                         const moe_quant_config *qc, void *out, void *residual_out, void *q,
                         float *q_scale, moe_stream_t stream);

/* ------------------------------------------------------------------ grouped products
 * The experts' products over ragged groups of rows, as calls of their own: a training step keeps
 * what lies between them.  The S sorted rows are grouped by expert: those of expert e are p in
 * [expert_offsets[e], expert_offsets[e + 1]), with slot sorted_slot[p] and token slot / top_k
 * (moe_align's outputs).
 *   out_p = x_p . w[e]^T           w [E, N, K] (K-contiguous), fp32 accumulation
 * A tensor of rows comes in one of these orders:
 *   MOE_ROWS_SORTED  [S, .], row p               MOE_ROWS_SLOT  [S, .], row sorted_slot[p]
 *   MOE_ROWS_TOKEN   [S / top_k, .], row sorted_slot[p] / top_k (x and dout only)
 * x, w and out in dtype (MOE_DT_BF16 or MOE_DT_FP16).  expert_offsets [E + 1] int32 ascend within [0, S];
 * sorted_slot [S] int32, distinct values in [0, S), is read for the rows of a group alone (NULL where
 * every order is MOE_ROWS_SORTED); a value out of range is recorded as MOE_ERR_INVALID_ARG
 * in the device status word, its row of out (or dx) not written and its share in dw zero; offsets out of
 * order or range are recorded likewise, and nothing outside the buffers is touched.  Rows of out that belong to no group
 * (in front of expert_offsets[0] or behind expert_offsets[E]) are left as they were.  0 <= S <= 2^30 (0: nothing
 * is done), 1 <= E <= 1024, N and K multiples of 8 up to 2^21, S % top_k == 0 where MOE_ROWS_TOKEN is used; more
 * than 2^30 tiles may be MOE_ERR_UNSUPPORTED.  A row of x that holds a NaN or an infinity affects its row of out alone.
 * Long sums are treated as moe_linear's are; the order of a sum is fixed by the sizes and
 * the group, so the same inputs give the same bits.  ws: moe_grouped_linear_workspace_size(...)
 * bytes (may be 0 for MOE_ROWS_SORTED: ws may then be NULL), for one call at a time.  Outputs overlap nothing. */
typedef enum { MOE_ROWS_SORTED = 0, MOE_ROWS_SLOT = 1, MOE_ROWS_TOKEN = 2 } moe_rows_t;

moe_status_t moe_grouped_linear(const void *x, int x_rows, const void *w, const int32_t *expert_offsets,
                                const int32_t *sorted_slot, int S, int E, int N, int K, int top_k,
                                moe_dtype_t dtype, void *out, int out_rows, void *ws, size_t ws_bytes,
                                moe_stream_t stream);
size_t moe_grouped_linear_workspace_size(int S, int E, int N, int K, int x_rows);

/* Gradients of moe_grouped_linear, given dout, the gradient of out, in dtype:
 *   dx_p  = dout_p . w[e]                         (dx_rows: MOE_ROWS_SORTED or MOE_ROWS_SLOT; the gradient
 *                                                  of a token's row is the sum of its slots', which
 *                                                  moe_finalize with the weights on the input adds)
 *   dw[e] = sum over p of dout_p^T x_p            [E, N, K] in dw_dtype (dtype or MOE_DT_FP32); accumulate:
 *                                                  added to what dw holds (in fp32, rounded once), else
 *                                                  written, zeros for an expert without rows
 * dx (needs w) and dw (needs x) may each be NULL, not both.  S == 0 sets dw to zero (accumulate: leaves it).
 * ws: moe_grouped_linear_backward_workspace_size(...) bytes, for one call at a time.  Everything else as
 * for moe_grouped_linear. */
moe_status_t moe_grouped_linear_backward(const void *dout, int dout_rows, const void *x, int x_rows, const void *w,
                                         const int32_t *expert_offsets, const int32_t *sorted_slot, int S,
                                         int E, int N, int K, int top_k, moe_dtype_t dtype, void *dx,
                                         int dx_rows, void *dw, moe_dtype_t dw_dtype, int accumulate,
                                         void *ws, size_t ws_bytes, moe_stream_t stream);
size_t moe_grouped_linear_backward_workspace_size(int S, int E, int N, int K, int dout_rows, int x_rows);

/* ------------------------------------------------------------------ activation
 * The activation between an expert's two products (a moe_activation_t) as a call of its own:
 * gu [S, 2 I] = [g | u] (the *_NO_MUL activations: [S, I] = g) -> h [S, I], both in dtype (MOE_DT_BF16 or
 * MOE_DT_FP16), computed in fp32 and rounded once.  0 <= S <= 2^30, I % 8 == 0, 8 <= I <= 2^21.
 * The gate is 0 far below 0 and at -inf, where u is finite; a NaN affects its own h. */
moe_status_t moe_activation(const void *gu, int S, int I, moe_dtype_t dtype, int activation, void *h,
                            moe_stream_t stream);

/* Its gradient: dh [S, I] -> dgu, as gu,
 *   dg = dh act'(g) u,  du = dh act(g)
 * with MOE_ACT_SWIGLUOAI 0 where a clamp holds g or u (the border itself passes).  h: the activation's
 * output made again in the same pass (NULL: not written).  dgu may be gu itself, and h dh itself. */
moe_status_t moe_activation_backward(const void *dh, const void *gu, int S, int I, moe_dtype_t dtype,
                                     int activation, void *dgu, void *h, moe_stream_t stream);

/* ------------------------------------------------------------------ status
 * Every device-side wait in the library's kernels gives up after about two
 * seconds, records MOE_ERR_TIMEOUT in a device status word and lets the
 * kernel return.  moe_device_status synchronises the current device, returns
 * the recorded status (MOE_OK when none) and clears it when `clear` != 0. */
moe_status_t moe_device_status(int clear);

/* Self-test of that failure path (the pages have no counterpart; it is not a step of the
 * layer): launches one thread that waits, with the same bounded wait the GEMM kernels
 * use, on a barrier no thread ever arrives on, giving up after limit_ns nanoseconds
 * (1e3 .. 1e10) instead of the usual two seconds.  The wait runs out, MOE_ERR_TIMEOUT is
 * recorded in the device status word and the kernel returns normally: the context stays
 * usable, moe_device_status reports the timeout (and clears it when asked).  Nothing
 * faults, traps or hangs.  Asynchronous on stream; MOE_ERR_INVALID_ARG for a limit out of
 * range. */
moe_status_t moe_selftest_wait_timeout(uint64_t limit_ns, moe_stream_t stream);

/* Self-test of the division the fp8 GEMM1 epilogue uses to requantise h (each element
 * divided by its row group's scale s = max(amax, 1e-10) / 448, "[vLLM] MoE Oracle &
 * Prepare/Finalize", the G(128) quantisation): the correctly rounded quotient from the
 * divisor's correctly rounded reciprocal and one fma correction, compared bit for bit with
 * the IEEE division on n pseudo-random (dividend, divisor) pairs of that domain drawn
 * from seed on the device.  *mismatches (device memory, zeroed by the caller) receives the
 * count of differing results.  Asynchronous on stream; MOE_ERR_INVALID_ARG for n < 0 or a
 * NULL counter. */
moe_status_t moe_selftest_row_division(long long n, uint32_t seed, unsigned long long *mismatches,
                                       moe_stream_t stream);
const char *moe_status_string(moe_status_t status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H_ */

/*
 * qsmoe.h -- C ABI of the MI355X (gfx950) routed-expert MoE layer library.
 *
 * The layer is the DeepSeek-V4 MoE FFN as the following pages describe it
 * (cited by page title and section):
 *   [PR1192] mlx-lm pull request "Add DeepSeek-v4 (Flash/Pro)"
 *   [CARD4]  model card "mlx-community / DeepSeek-V4-Flash-4bit"
 *   [ALPHA]  model card "DeepSeek-V4-Flash-MLX-4bit"
 *   [PR1190] mlx-lm pull request "Add DeepSeek-V4 model and safetensors/tokenizer
 *            fallback handling"
 *   [SERVE]  model card "DeepSeek-V4-Flash-0731-MLX-Serve-mixed-2-3-8bit"
 *
 *   1. route    -- fp32 gate logits, sqrtsoftplus scores, per-expert bias,
 *                  top-k (or the tid2eid hash table), renormalised weights;
 *   2. permute  -- bucket the T*k (token, slot) assignments by expert;
 *   3. experts  -- per assignment, SwiGLU over group-quantised gate/up/down
 *                  projections (affine b-bit or MXFP4), plus the shared expert;
 *   4. combine  -- weighted sum of the k expert outputs (+ shared) per token.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All array pointers are DEVICE pointers owned by the caller. The library
 *    never allocates or frees device memory; all scratch comes from the
 *    caller's workspace `ws` (size from moe_workspace_size or the per-call
 *    sizes below). Descriptor structs are host memory, read during the call.
 *  - Every call only enqueues work on `stream` and returns: no host sync, no
 *    host readback of routing. Weights and inputs must stay valid until the
 *    enqueued work completes.
 *  - Host validation happens before anything is enqueued; a negative status
 *    means nothing was launched. T == 0 returns MOE_OK with no launch.
 *  - Device-side precondition violations (a token id outside [0, vocab), a
 *    tid2eid entry or a top-k id outside [0, E)) OR a code into the sticky
 *    error word at the start of `ws`; the offending id is replaced by 0 (and
 *    a hash-routed token's weights by 0) so that every access stays in
 *    bounds. Read it with moe_device_error, clear it with moe_workspace_init.
 *  - Layouts are row-major. A quantised projection is [rows = out][cols = in]
 *    per expert, codes packed along cols (the contraction dimension).
 *  - bf16 arrays are passed as uint16_t bit patterns.
 *  - Calls that share a workspace must not overlap in time.
 */
#ifndef QSMOE_H
#define QSMOE_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* null pointer, bad size, k > E, ...            */
  MOE_ERR_UNSUPPORTED = -2, /* a format/bits/group/shape the kernels lack      */
  MOE_ERR_ALIGNMENT = -3,   /* a pointer not 16-byte aligned                   */
  MOE_ERR_WORKSPACE = -4,   /* workspace null or smaller than required         */
  MOE_ERR_HIP = -5          /* a HIP launch or runtime call failed             */
} moe_status;

typedef enum { MOE_FMT_AFFINE = 0, MOE_FMT_MXFP4 = 1, MOE_FMT_MXFP8 = 2 } moe_format;
typedef enum { MOE_ROUTE_TOPK = 0, MOE_ROUTE_HASH = 1 } moe_route_mode;
typedef enum { MOE_OUT_BF16 = 0, MOE_OUT_F32 = 1 } moe_out_dtype;
/* Element types of the plain matrices of the block-scaled and grouped products
 * (the first two as in moe_out_dtype). */
typedef enum { MOE_DT_BF16 = 0, MOE_DT_F32 = 1, MOE_DT_F16 = 2 } moe_dtype;
/* ORed into out_dtype of moe_matmul_block and moe_grouped_matmul_block: exact
 * products and fp32 sums behind a bf16 result too (see there). */
#define MOE_SUMS_F32 0x100
/* How the rows of a matrix stand to the T*k assignments that moe_permute
 * bucketed; bucket position p is assignment perm[p].
 *   MOE_ROWS_BUCKET  [T*k] rows, row p belongs to position p (perm not read)
 *   MOE_ROWS_TOKEN   [T] rows, position p reads row perm[p] / k
 *   MOE_ROWS_SLOT    [T*k] rows, row perm[p] belongs to position p */
typedef enum { MOE_ROWS_BUCKET = 0, MOE_ROWS_TOKEN = 1, MOE_ROWS_SLOT = 2 } moe_rows;

/* Device error bits ORed into the workspace's error word. */
#define MOE_DEVERR_TOKEN_ID 1  /* token id outside [0, vocab)                  */
#define MOE_DEVERR_HASH_ID 2   /* tid2eid entry outside [0, E)                  */
#define MOE_DEVERR_EXPERT_ID 4 /* top-k id passed to moe_permute outside [0, E) */
#define MOE_DEVERR_QUANT_INPUT 8 /* moe_quantize_affine: a NaN/inf weight, or a group's
                                    scale or bias beyond fp16 (outputs unspecified);
                                    moe_quantize_block: a NaN/inf input */
#define MOE_DEVERR_ROW_INDEX 16 /* a perm entry of a grouped product outside its rows;
                                   a perm or positions entry of the row steps */

/*
 * One stacked quantised projection: num_experts matrices of [rows][cols].
 *
 * MOE_FMT_AFFINE ([PR1192] pre-stacked expert patch: {weight, scales, biases}
 * triplets; [SERVE]: packs byte-compatible with MLX's affine layout; bit
 * widths and groups from [CARD4] "Conversion" and the [SERVE] precision
 * table): element (e, r, c) has the unsigned code q = bits [c*b, c*b + b) of
 * row (e, r)'s LSB-first bit stream over little-endian uint32 words (a 3-bit
 * code may straddle two words), and the value
 *     w = scale[e][r][c / g] * q + bias[e][r][c / g]
 * with fp16 scale and bias.  bits in {2, 3, 4, 8}, g in {32, 64, 128}.
 *   codes  : uint32 [E][rows][cols * bits / 32]
 *   scales : fp16   [E][rows][cols / g]
 *   biases : fp16   [E][rows][cols / g]
 *
 * MOE_FMT_MXFP4 ([PR1192] mxfp4 dequantize with group_size 32, bits 4;
 * [ALPHA]: FP4 e2m1 packed two per byte; [PR1190]: e8m0 = 2^(b - 127)):
 * byte j of a row holds element 2j in its low nibble and 2j+1 in its high
 * nibble; nibble n decodes to (-1)^(n >> 3) * {0, .5, 1, 1.5, 2, 3, 4, 6}[n & 7]
 * (OCP MX e2m1), times 2^(s - 127) for the row's scale byte s of that group of
 * 32 (s = 255 is NaN).  bits = 4, g = 32.
 *   codes  : uint32 [E][rows][cols / 8]
 *   scales : uint8  [E][rows][cols / 32]
 *   biases : NULL
 *
 * MOE_FMT_MXFP8 ([PR1192] FP8-to-bf16 requantization report: E4M3 bytes
 * viewed as uint32 words with E8M0 block scales expanded to one per 32, read
 * by mx.dequantize with group_size 32, bits 8, mode "mxfp8"; [PR1190]:
 * MXFP8-quantized MoE layers, F8_E4M3 kept as uint8): byte j of a row holds
 * element j as OCP FP8 E4M3 (bit 7 sign, 4 exponent bits with bias 7, 3
 * mantissa bits; exponent 0 subnormal; S.1111.111 NaN; largest 448), times
 * 2^(s - 127) for the row's scale byte s of that group of 32.  bits = 8,
 * g = 32.
 *   codes  : uint32 [E][rows][cols / 4]
 *   scales : uint8  [E][rows][cols / 32]
 *   biases : NULL
 *
 * Requirements: cols % 32 == 0, cols % g == 0, cols <= 8192, rows >= 1;
 * codes 16-byte aligned, scales/biases 4-byte aligned.
 */
typedef struct {
  int32_t format;      /* moe_format                         */
  int32_t bits;
  int32_t group_size;
  int32_t rows;        /* output features                    */
  int32_t cols;        /* input features (contraction)       */
  int32_t num_experts;
  const uint32_t* codes;
  const void* scales;
  const void* biases;
} moe_qtensor;

/* SwiGLU expert weights: gate = w1 [I][d], up = w3 [I][d], down = w2 [d][I]
 * ([PR1192] pre-stacked rename: w1 -> gate_proj, w2 -> down_proj,
 * w3 -> up_proj). y = W2 (silu(W1 x) * (W3 x)), with the product rounded to
 * bf16 (round to nearest even) before the down projection. gate and up share
 * format, bits and group; down may differ ([SERVE] precision table: gate/up
 * 2-bit g128 with down 3-bit g128). */
typedef struct {
  moe_qtensor gate, up, down;
} moe_experts;

/*
 * Router.
 *  MOE_ROUTE_TOPK: l[t][e] = sum_i x[t][i] * weight[e][i] in fp32 ([PR1192]
 *    cross-reference table, row "MoE gate dtype"); s = sqrt(softplus(l))
 *    ([CARD4] "Architecture"), evaluated as sqrt(max(l,0) + log1p(exp(-|l|)))
 *    (the logaddexp form of [PR1192]'s review notes); key = s + bias[e]; the
 *    top_k experts by key descending, ties to the lower expert index, in that
 *    order; weights w_j = routed_scale * s_j / sum_j s_j (the bias ranks only;
 *    [ALPHA] "REAP-pruned builds": the router renormalises over the selected
 *    experts).
 *  MOE_ROUTE_HASH: ids[t][j] = tid2eid[token_ids[t]][j] in table order
 *    ([CARD4] "Architecture": deterministic tid2eid table for the first
 *    layers; [ALPHA]: tid2eid[vocab, 6]); weights as above from those experts'
 *    fp32 logits; no bias.
 *  weight : fp32 [E][hidden]; bias : fp32 [E] or NULL; tid2eid : int32
 *  [vocab][top_k] (hash mode only). 1 <= top_k <= min(E, 8), E <= 1024,
 *  hidden % 32 == 0.
 */
typedef struct {
  int32_t mode;        /* moe_route_mode */
  int32_t num_experts;
  int32_t top_k;
  int32_t hidden;
  int32_t vocab;       /* hash mode */
  const float* weight;
  const float* bias;
  const int32_t* tid2eid;
  float routed_scale;  /* 1.0f for the layers here */
} moe_router;

/* A whole layer. `shared` (nullable) is the always-on shared expert, added to
 * every token with weight 1 after the routed sum ([ALPHA] "Why mixed-4_8bit"
 * and the [SERVE] precision table name the shared experts). routed.*.num_experts
 * must equal router.num_experts; shared->*.num_experts must be 1. */
typedef struct {
  moe_router router;
  moe_experts routed;
  const moe_experts* shared;
} moe_layer;

/* Bytes of workspace moe_forward needs for every token count up to
 * max_tokens (0 on an invalid layer): never smaller for a larger max_tokens,
 * so a buffer sized once (e.g. before graph capture) serves every T <=
 * max_tokens. The same size serves every other entry point. */
size_t moe_workspace_size(const moe_layer* layer, int32_t max_tokens);

/*
 * Where moe_forward keeps its intermediates in the workspace, for inspection
 * after the call (tests, routing statistics). Byte offsets from the start of
 * `ws`; 0 marks a region the call does not write for this layer and T.
 *   ids      int32 [T][k]   routed expert ids, slot order (key descending)
 *   weights  fp32  [T][k]   combine weights
 *   logits   fp32  [T][E]   router logits (top-k routing; hash routing on the
 *                           fused path only)
 *   keys     uint64 [T][E]  ranking key of every expert: bits 63..32 are the
 *                           fp32 key s + bias mapped so that unsigned order is
 *                           numeric order (key >= 0: bits | 0x80000000; key < 0:
 *                           ~bits), bits 31..0 are 0xFFFFFFFF - e; the top-k
 *                           takes the k largest values (ties: lower index)
 *   scores   fp32  [T][E]   sqrtsoftplus scores s of every expert
 *   offsets  int32 [E+1], perm int32 [T*k]   buckets (general path only)
 *   h        bf16  [T*k][I]  silu(gate) * up rounded to bf16: bucket order
 *                           (row p belongs to assignment perm[p]) on the
 *                           general path, slot order t*k + j on the fused path
 *   h_shared bf16  [T][I_shared] (shared expert)
 *   y_slot   fp32  [T*k][d]  (general path only), y_shared fp32 [T][d] (general
 *            path, and the fused path of a single token)
 * fused = 1 when moe_forward takes the three-launch small-batch path. total =
 * the bytes moe_forward needs for exactly T tokens. Errors: INVALID_ARG (T <
 * 1, null out, invalid layer), UNSUPPORTED.
 */
typedef struct {
  size_t total;
  size_t ids, weights, logits, keys, scores, offsets, perm, h, h_shared, y_slot, y_shared;
  int32_t fused;
} moe_ws_layout;

moe_status moe_workspace_layout(const moe_layer* layer, int32_t T, moe_ws_layout* out);

/* Zero the workspace header, which holds the device error word (a small
 * kernel; capturable). */
moe_status moe_workspace_init(void* ws, size_t ws_bytes, hipStream_t stream);

/* Step 1 (the router as moe_router defines it). x_bf16 [T][hidden];
 * token_ids int32 [T] (hash mode, else may be NULL); outputs topk_ids int32
 * [T][top_k], topk_w fp32 [T][top_k]. In top-k mode ws needs 256 + A(4*T*E)
 * + A(8*T*E) + A(4*T*E) bytes, A() rounding up to a multiple of 256, and
 * holds after the call: logits fp32 [T][E] at byte 256, then the packed
 * ranking keys uint64 [T][E] and the scores fp32 [T][E] (formats as in
 * moe_ws_layout). Hash mode needs 256 bytes. */
moe_status moe_route(const moe_router* router, const uint16_t* x_bf16, const int32_t* token_ids,
                     int32_t T, int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/* Step 2. A stable counting sort of the T*k assignments a = t*k + j by
 * expert topk_ids[a], so that each of the stacked experts ([PR1192]: experts
 * pre-stacked as switch_mlp.{gate,up,down}_proj, one weight tensor per
 * projection over all experts) runs once over one contiguous bucket of its
 * assignments: expert_offsets int32 [E+1] (exclusive prefix sum of the
 * per-expert counts; offsets[E] = T*k), perm int32 [T*k] (assignment indices
 * bucketed by expert, ascending within a bucket). Ids outside [0, E) set
 * MOE_DEVERR_EXPERT_ID and count as expert 0. ws needs 256 bytes. */
moe_status moe_permute(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E,
                       int32_t* expert_offsets, int32_t* perm, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/* Step 3. For each bucketed assignment a (token t = a / k) of expert e:
 * y_slot[a] = expert_e(x[t]) in fp32, written in assignment order a, so row
 * t*k + j is token t's j-th expert. If `shared` is non-NULL, y_shared[t] =
 * shared(x[t]) for every token (y_shared may be NULL only when shared is).
 * y_slot fp32 [T*k][hidden], y_shared fp32 [T][hidden]. ws: see
 * moe_workspace_size. */
moe_status moe_expert_ffn(const moe_experts* routed, const moe_experts* shared,
                          const uint16_t* x_bf16, int32_t T, int32_t k,
                          const int32_t* expert_offsets, const int32_t* perm, float* y_slot,
                          float* y_shared, void* ws, size_t ws_bytes, hipStream_t stream);

/* Step 4. The weighted combine: each token's output is its selected
 * experts' outputs times their router weights ([ALPHA] "REAP-pruned builds":
 * router weight x expert output, renormalised over the kept experts), plus
 * the shared expert's output ([ALPHA] "Why mixed-4_8bit"):
 * out[t] = sum_{j=0..k-1} topk_w[t][j] * y_slot[t*k + j] (j in order) +
 * y_shared[t] (if non-NULL), accumulated in fp32 with one writer per output
 * element (no atomics); stored as bf16 (round to nearest even) or fp32 per
 * out_dtype. y_slot fp32 [T*k][d], topk_w fp32 [T][k], y_shared fp32 [T][d]
 * or NULL, out [T][d]. d % 4 == 0; y_slot, y_shared 16-byte aligned, out
 * 8-byte (bf16) or 16-byte (fp32) aligned. Errors: INVALID_ARG, UNSUPPORTED
 * (d), ALIGNMENT, HIP. */
moe_status moe_combine(const float* y_slot, const float* topk_w, const float* y_shared, int32_t T,
                       int32_t k, int32_t d, int32_t out_dtype, void* out, hipStream_t stream);

/* Steps 1-4 in one call: out [T][hidden] (bf16 or fp32). token_ids is needed
 * in hash mode only. ws >= moe_workspace_size(layer, T). */
moe_status moe_forward(const moe_layer* layer, const uint16_t* x_bf16, const int32_t* token_ids,
                       int32_t T, int32_t out_dtype, void* out, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/*
 * moe_forward for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same launches and results as moe_forward, with the workspace taken from a
 * library-owned device array of 64 MiB instead of a caller buffer. Each GPU
 * the library runs on holds its own copy of the array until the process ends;
 * its address is resolved on the first call on each device. The caller still
 * passes inputs and outputs (same rules as moe_forward). Every call on a GPU
 * shares that GPU's array: calls that overlap in time on one GPU (other
 * streams, other threads) race and must be serialised by the caller. The
 * device error word is cleared at the start of each call and is not reported
 * (out-of-range ids are still clamped in bounds). Allocates nothing, makes no
 * hipMalloc/hipFree and no host synchronisation. Errors: as moe_forward, and
 * MOE_ERR_WORKSPACE when moe_workspace_layout(layer, T).total exceeds the
 * 64 MiB (e.g. T = 512 at hidden 4096, intermediate 2048, top-6 fits; the
 * 4096-token prefill does not), before anything is launched.
 */
moe_status moe_forward_noalloc(const moe_layer* layer, const uint16_t* x_bf16, const int32_t* token_ids,
                               int32_t T, int32_t out_dtype, void* out, hipStream_t stream);

/* Test and inspection helpers (not on the hot path). */

/* Router logits only: logits fp32 [T][E] (top-k mode's first kernel). */
moe_status moe_router_logits(const moe_router* router, const uint16_t* x_bf16, int32_t T,
                             float* logits, hipStream_t stream);

/* moe_forward with timing probes: kernel i is launched with the event pair
 * events[2i] (start) and events[2i+1] (stop), which the dispatch itself
 * timestamps when the kernel begins and ends, so their elapsed time is the
 * kernel's execution time alone. Its name (a static string) goes to names[i]
 * and the number of kernels to *n_kernels. n_events must be at least twice
 * the number of kernels (at most 16 are launched, so 32 always suffice);
 * otherwise MOE_ERR_INVALID_ARG after the step has run. The caller creates
 * the events (timing enabled). Same results as moe_forward. */
moe_status moe_forward_probed(const moe_layer* layer, const uint16_t* x_bf16, const int32_t* token_ids,
                              int32_t T, int32_t out_dtype, void* out, void* ws, size_t ws_bytes,
                              hipStream_t stream, hipEvent_t* events, int32_t n_events, const char** names,
                              int32_t* n_kernels);

/* Measurement kernels (not part of the layer): the scale for HBM byte
 * counters and the achievable rates beside the nominal peaks.
 * moe_probe_stream: mode 0 reads every byte of buf [bytes] once (16 bytes per
 * lane, consecutive lanes on consecutive pieces: bytes of traffic); mode 1
 * reads the first 32 bytes of every 128-byte line (bytes / 4 requested);
 * mode 2 writes every byte once (bytes written). Modes 0 and 1 run 2048
 * workgroups; workgroup i stores the XOR of the words it read into sink[i]
 * (device uint32 [2048], overwritten), so the XOR of the 2048 words is that
 * of every word read. bytes > 0 and a multiple of 128; buf 16-byte aligned.
 * Errors: INVALID_ARG, ALIGNMENT, HIP. */
moe_status moe_probe_stream(void* buf, size_t bytes, int32_t mode, uint32_t* sink, hipStream_t stream);

/* moe_probe_mfma: `workgroups` workgroups of 4 waves, each wave `iters` rounds
 * of 8 independent V_MFMA_F32_32X32X16_BF16 (2 * 32 * 32 * 16 flops each), no
 * memory traffic. out: device uint64 [5], out[4] zeroed by the caller; wave 0
 * of workgroup 0 writes its shader-clock counter (s_memtime) before and after
 * its loop to out[0], out[1] and the 100 MHz wall clock to out[2], out[3]:
 * the sustained shader clock is (out[1] - out[0]) / ((out[3] - out[2]) / 1e8).
 * Errors: INVALID_ARG, ALIGNMENT, HIP. */
moe_status moe_probe_mfma(int32_t workgroups, int32_t iters, uint64_t* out, hipStream_t stream);

/* Synchronises `stream`, then copies the workspace error word to *code_out. */
moe_status moe_device_error(const void* ws, int32_t* code_out, hipStream_t stream);

/*
 * Plain min/max affine quantisation of bf16 weights: the conversion step
 * before the layer ([CARD4] "Conversion": mlx_lm.convert -q --q-bits b
 * --q-group-size g; [SERVE] contrasts its calibrated search with plain
 * min/max). Produces a MOE_FMT_AFFINE projection for one matrix (call per
 * expert, or once on E stacked matrices as rows = E * rows). Per group of g
 * inputs of a row, in fp32 with IEEE rounding (the pages give the recipe,
 * not its arithmetic; this is the reading taken):
 *     scale = fp16_rne((max - min) / (2^b - 1)),  bias = fp16_rne(min),
 *     q = clamp(rint((w - bias) / scale), 0, 2^b - 1), q = 0 if scale == 0.
 *   w_bf16 : device bf16 [rows][cols], 16-byte aligned
 *   codes  : device uint32 [rows][cols * bits / 32], 16-byte aligned (written)
 *   scales, biases : device fp16 [rows][cols / g], 2-byte aligned (written)
 *   err    : device int32 or NULL; MOE_DEVERR_QUANT_INPUT is ORed in for a
 *            NaN/inf weight or a group whose scale or bias overflows fp16.
 * bits in {2, 3, 4, 8}, g in {32, 64, 128}, cols % g == 0, rows >= 0.
 * Asynchronous on `stream`; allocates nothing. Errors: INVALID_ARG (null or
 * negative), UNSUPPORTED (bits, g, cols), ALIGNMENT, HIP.
 */
moe_status moe_quantize_affine(const uint16_t* w_bf16, int64_t rows, int32_t cols, int32_t bits, int32_t group_size,
                               uint32_t* codes, uint16_t* scales, uint16_t* biases, int32_t* err,
                               hipStream_t stream);

/*
 * mHC mix matrices (an op beside the MoE layer): [CARD4] "Architecture": the
 * residual stream is hc_mult = 4 parallel copies recombined by a
 * doubly-stochastic, Sinkhorn-normalised mix matrix; [PR1192] review notes:
 * unfused, a softmax followed by iterations of a sum and a division (~40
 * launches per call). For each of T tokens: m = softmax over each row of the
 * n x n logits, then `iters` rounds of dividing each column by its sum + eps
 * and then each row by its sum + eps (the pages give neither the round count
 * nor eps; 10 rounds and eps = 0 make the pages' ~40 unfused launches). fp32,
 * one launch, allocates nothing.
 *   logits : device fp32 [T][n][n]
 *   out    : device fp32 [T][n][n] (may be logits itself)
 * n in {2, 4, 8}; T >= 0; iters >= 0; eps >= 0 and finite. Rows whose
 * softmax leaves a column all zero (logit spreads beyond ~80 in fp32) give
 * NaN when eps = 0. Errors: INVALID_ARG, UNSUPPORTED (n), ALIGNMENT (4-byte),
 * HIP.
 */
moe_status moe_mhc_sinkhorn(const float* logits, int64_t T, int32_t n, int32_t iters, float eps, float* out,
                            hipStream_t stream);

/*
 * Block-scaled FP8 (ops beside the layer). A matrix is held as OCP E4M3 codes
 * (one byte per element, as in MOE_FMT_MXFP8) with one fp32 scale per block of
 * 128 columns and 1 or 128 rows; an element stands for code * scale.
 * Activations use 1 x 128 blocks, weights 128 x 128; blocks at the right and
 * lower edge may be smaller.
 *
 * moe_quantize_block: x [matrices][rows][cols] -> codes of the same shape and
 * scales [matrices][ceil(rows / block_rows)][ceil(cols / 128)]. Per block, in
 * fp32 with IEEE rounding, amax the largest |x| of the block:
 *     s = max(amax / 448, 2^-126),  code = e4m3_rne(x * (1 / s));
 * with pow2 != 0 the quotient amax / 448 is first raised to the next power of
 * two, which makes scaling and unscaling exact. A block that holds a NaN or an
 * infinity gets the scale NaN and codes 0, and MOE_DEVERR_QUANT_INPUT is ORed
 * into *err (err: device int32 or NULL); the other blocks are not affected.
 * dtype: moe_dtype of x. block_rows in {1, 128}; cols % 16 == 0; x and codes
 * 16-byte, scales and err 4-byte aligned. Nothing to do (MOE_OK, no launch)
 * when a size is 0. Errors: INVALID_ARG (null, negative, dtype), UNSUPPORTED
 * (block_rows, cols, more than 2^24 - 1 workgroups of 4096 elements or one
 * 128 x 128 block), ALIGNMENT, HIP.
 */
moe_status moe_quantize_block(const void* x, int32_t dtype, int64_t matrices, int64_t rows, int32_t cols,
                              int32_t block_rows, int32_t pow2, uint8_t* codes, float* scales, int32_t* err,
                              hipStream_t stream);

/* moe_swiglu_quantize_block: the step between an expert's two products. gu
 * [rows][2 * inner] holds gate in its first `inner` columns and up in the
 * others; h = silu(gate) * up in fp32, quantised as moe_quantize_block does
 * with block_rows = 1 (h itself is not rounded to 16 bits in between): codes
 * [rows][inner], scales [rows][ceil(inner / 128)]. inner % 16 == 0; the rest
 * as above (a block whose h holds a NaN or an infinity counts as such). */
moe_status moe_swiglu_quantize_block(const void* gu, int32_t dtype, int64_t rows, int32_t inner, int32_t pow2,
                                     uint8_t* codes, float* scales, int32_t* err, hipStream_t stream);

/*
 * moe_matmul_block: out[m][n] = sum_k a[m][k] * b[n][k] over the values the
 * codes stand for: the 128 products of a block are summed before the two scales
 * multiply the sum, sums of blocks are fp32, one rounding to the output. With
 * an fp32 or fp16 output, and with MOE_SUMS_F32 in out_dtype, every product is
 * exact and every sum fp32. With a bf16 output else the FP8 matrix instruction
 * forms a block's sum, at twice the rate: it adds 8 neighbouring products with
 * 13 bits below the largest of them and drops the rest, at most 7 * 2^-13 of
 * that largest product, and the groups in fp32. In the norm that is 1.3e-5 of
 * the result for normal inputs, 3e-6 for inputs of one sign (there all of it
 * towards zero) and 5e-5 where few channels outweigh the others; rounding to
 * bf16 is 1.7e-3. A result whose large products cancel can be off by more than
 * its rounding: MOE_SUMS_F32 is for callers who need those. The two scales are
 * multiplied with each other first, in fp32: a pair whose product leaves its
 * normal range loses accuracy.
 *   a [M][K] codes, a_scales [M][ceil(K / 128)]              (1 x 128)
 *   b [N][K] codes, b_scales [ceil(N / 128)][ceil(K / 128)]  (128 x 128)
 *   out [M][N], out_dtype MOE_DT_BF16, MOE_DT_F32 or MOE_DT_F16, MOE_SUMS_F32
 * K % 16 == 0, N % 8 == 0, N and K <= 2^20, M <= 2^30; a, b and out 16-byte,
 * scales 4-byte aligned. M, N or K of 0: MOE_OK (K == 0 writes zeros). Errors:
 * INVALID_ARG, UNSUPPORTED, ALIGNMENT, HIP.
 */
moe_status moe_matmul_block(const uint8_t* a, const float* a_scales, const uint8_t* b, const float* b_scales,
                            int32_t M, int32_t N, int32_t K, int32_t out_dtype, void* out, hipStream_t stream);

/*
 * Matrix products grouped by expert. offsets int32 [E+1] (device) and perm
 * int32 [T*k] (device) are those of moe_permute: positions offsets[e] ..
 * offsets[e+1] - 1 use expert e's weights. An expert may have no position;
 * positions outside every bucket (before offsets[0], from offsets[E] on) are
 * neither read nor written, so their output rows stay as they were. Offsets
 * are clamped to [0, T*k], and a bucket that runs backwards counts as empty;
 * where buckets overlap for that reason, their positions get the result of one
 * of their buckets or none. A perm entry outside [0, T*k) sets
 * MOE_DEVERR_ROW_INDEX in *err (device int32 or NULL); some row of the matrix
 * is read in its place, and an output row that it would name is not written.
 * perm may be NULL when no matrix is in token or slot order; it must not name
 * an output row twice.
 *
 * moe_grouped_matmul_block: out[p][n] = sum_k a[p][k] * w[e(p)][n][k] over
 * block-scaled FP8, as moe_matmul_block: a in a_order, w [E][N][K], w_scales
 * [E][ceil(N / 128)][ceil(K / 128)], out in out_order (BUCKET or SLOT).
 *
 * moe_grouped_matmul: the same for 16-bit x and w [E][N][K] of one type
 * (dtype MOE_DT_BF16 or MOE_DT_F16): out[p][n] = sum_k x[p][k] w[e][n][k], or
 * with transposed != 0 out[p][k] = sum_n x[p][n] w[e][n][k] (x has N columns:
 * the gradient in the rows). fp32 sums, one rounding to the output.
 *
 * moe_grouped_matmul_dw: the gradient in the weights, out[e][n][k] = sum over
 * expert e's positions of dy[p][n] * x[p][k]; x in x_order, dy in dy_order
 * (BUCKET or SLOT); out [E][N][K], zeros for an expert without a position.
 * fp32 sums in a fixed order (no atomics).
 *
 * T, k, E >= 1 sized as in moe_permute but for k, which only has to be >= 1
 * (T*k <= 2^30, E <= 1024). FP8: K % 16 == 0, N % 8 == 0; 16-bit: K % 8 == 0,
 * N % 8 == 0; N and K <= 2^20. out_dtype MOE_DT_BF16, MOE_DT_F32 or
 * MOE_DT_F16, in the FP8 product with MOE_SUMS_F32 too. Matrices 16-byte,
 * offsets, perm, scales and err 4-byte aligned.
 * T == 0, or nothing to write: MOE_OK without a launch, but dw still writes
 * its zeros; a contraction of length 0 gives zeros. No workspace; out must not
 * overlap an input. Errors: INVALID_ARG, UNSUPPORTED (sizes as above, or an
 * output of more tiles than a grid holds), ALIGNMENT, HIP.
 */
moe_status moe_grouped_matmul_block(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                                    int32_t T, int32_t k, int32_t N, int32_t K, int32_t E, const int32_t* offsets,
                                    const int32_t* perm, int32_t a_order, int32_t out_order, int32_t out_dtype,
                                    void* out, int32_t* err, hipStream_t stream);

moe_status moe_grouped_matmul(const void* x, const void* w, int32_t dtype, int32_t T, int32_t k, int32_t N, int32_t K,
                              int32_t E, const int32_t* offsets, const int32_t* perm, int32_t x_order,
                              int32_t out_order, int32_t transposed, int32_t out_dtype, void* out, int32_t* err,
                              hipStream_t stream);

moe_status moe_grouped_matmul_dw(const void* x, const void* dy, int32_t dtype, int32_t T, int32_t k, int32_t N,
                                 int32_t K, int32_t E, const int32_t* offsets, const int32_t* perm, int32_t x_order,
                                 int32_t dy_order, int32_t out_dtype, void* out, int32_t* err, hipStream_t stream);

/*
 * The steps around the experts' products, each a call of its own: rows brought
 * into bucket order and back with the router's weights, the activation between
 * the two products, the gradients of both, and products with 4-bit weights.
 * Assignments, offsets and perm are those of moe_permute. Types are moe_dtype;
 * everything is computed in fp32, sums in a fixed order, with one rounding to
 * the output; no workspace. Outputs must not overlap inputs.
 * Sizes: T*k and n <= 2^30, k >= 1, d and inner <= 2^20, any of them odd.
 * Pointers are aligned to their elements (err, perm, positions and weights to
 * 4 bytes).
 *
 * moe_invert_perm: the bucket position of every assignment. positions int32
 * [size] (written): positions[perm[p]] = p for p = 0 .. n - 1, -1 where perm
 * names no position, the last one where perm names an assignment twice. perm's
 * entries are -1 (a position without an assignment) or in [0, size); others set
 * MOE_DEVERR_ROW_INDEX in *err (device int32 or NULL) and count as -1.
 *
 * moe_gather_rows: out[p] = x[perm[p] / k] (x_order MOE_ROWS_TOKEN, x [T][d])
 * or x[perm[p]] (MOE_ROWS_SLOT, x [T*k][d]) for p = 0 .. n - 1, times
 * topk_w[perm[p]] if topk_w (fp32 [T*k]) is not NULL. out [n][d]. The row of an
 * entry -1 is not written; an entry outside [-1, T*k) sets
 * MOE_DEVERR_ROW_INDEX and its row is not written either. Without weights and
 * with one type the rows are copied bit for bit.
 *
 * moe_combine_rows: out[t] = sum over j = 0 .. k - 1, in order, of topk_w[t][j]
 * * y[positions[t * k + j]], plus y_shared[t] if not NULL. y [n][d] and
 * y_shared [T][d] of type dtype; topk_w NULL: ones; positions NULL: y is in
 * slot order, [T*k][d] (n == T*k). A position -1 adds nothing (y's row and its
 * weight are not read), one outside [-1, n) sets MOE_DEVERR_ROW_INDEX and adds
 * nothing. This is also the gradient of moe_gather_rows in x, for a perm that
 * names no assignment twice (moe_invert_perm keeps one position of each): in
 * token order with its k, in slot order with k = 1.
 *
 * moe_combine_rows_grad: the gradient of moe_combine_rows in y and the weights:
 * dy[p] = topk_w[a] * dout[a / k] and dw[a] = sum over columns of dout[a / k] *
 * y[p], p = positions[a]. dout [T][d] of type dout_dtype, dy [n][d] of y's type
 * dtype, dw fp32 [T][k] (zero for a position -1). Rows of dy that no position
 * names are not written. Where two assignments name one row, each element of
 * dy's row is of either one's gradient, not their sum, and which one is not
 * specified (moe_invert_perm gives no such positions); dw is as said.
 * y_shared's gradient is dout.
 * The gradient of moe_gather_rows (token order, no assignment named twice) in
 * its weights is this call's dw with x in the place of dout and the gathered
 * rows' gradient in the place of y.
 *
 * Nothing to write: MOE_OK without a launch (d == 0 still writes dw's zeros).
 * Errors: INVALID_ARG, UNSUPPORTED, ALIGNMENT, HIP.
 */
moe_status moe_invert_perm(const int32_t* perm, int32_t n, int32_t size, int32_t* positions, int32_t* err,
                           hipStream_t stream);

moe_status moe_gather_rows(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t d, int32_t x_order,
                           const int32_t* perm, int32_t n, const float* topk_w, int32_t out_dtype, void* out,
                           int32_t* err, hipStream_t stream);

moe_status moe_combine_rows(const void* y, int32_t dtype, int32_t n, const int32_t* positions, const float* topk_w,
                            const void* y_shared, int32_t T, int32_t k, int32_t d, int32_t out_dtype, void* out,
                            int32_t* err, hipStream_t stream);

moe_status moe_combine_rows_grad(const void* dout, int32_t dout_dtype, const void* y, int32_t dtype, int32_t n,
                                 const int32_t* positions, const float* topk_w, int32_t T, int32_t k, int32_t d,
                                 void* dy, float* dw, int32_t* err, hipStream_t stream);

/* moe_swiglu: h = silu(gate) * up of gu [rows][2 * inner], gate in its first
 * `inner` columns and up in the others (as moe_swiglu_quantize_block); h
 * [rows][inner] of gu's type. moe_swiglu_grad: its gradient, with s = 1 / (1 +
 * e^-gate): dgu [rows][2 * inner] of gu's type holds dh * up * s * (1 + gate *
 * (1 - s)) and dh * gate * s; dh [rows][inner] of type dh_dtype. Infinities and
 * NaN follow these formulas (gate = -inf gives NaN). */
moe_status moe_swiglu(const void* gu, int32_t dtype, int64_t rows, int32_t inner, void* h, hipStream_t stream);
moe_status moe_swiglu_grad(const void* gu, int32_t dtype, const void* dh, int32_t dh_dtype, int64_t rows,
                           int32_t inner, void* dgu, hipStream_t stream);

/*
 * moe_matmul_packed: out[m][n] = sum_k x[m][k] * W[n][k] for W held in 4 bits as
 * a moe_qtensor holds it: MOE_FMT_AFFINE (group 32, 64 or 128; fp16 scales and
 * biases) or MOE_FMT_MXFP4 (group 32; e8m0 scales, biases NULL). x bf16 or fp16
 * [M][K]; codes uint32 [N][K / 8], scales and biases [N][K / group].
 * moe_grouped_matmul_packed: the same with codes [E][N][K / 8] and so on, rows
 * grouped by expert as in moe_grouped_matmul (positions outside every bucket,
 * clamped offsets and perm entries out of range as described there).
 * Meant for few rows of x for each matrix (tokens being decoded): a pass over a
 * matrix takes up to 16 rows where there are few of them, 16 to 64 where there
 * are more, and one with K below 128. Products are exact, sums fp32: within a
 * group sum x * code and sum x are formed first and multiplied by the scale
 * and added with the bias then, so a row of x with an infinity or a NaN (or one
 * of 2^117 and more, of less with scales above 1 or biases above 16) gives
 * values that are not finite, and so does such a scale or bias; other rows are
 * not affected. One rounding to out_dtype.
 * K % 32 == 0, K % group == 0, K >= 32, N any; N and K <= 2^20, M and T*k <=
 * 2^30, E <= 1024, k >= 1. x and codes 16-byte, scales, biases and out aligned
 * to their elements, offsets, perm and err to 4 bytes. M, T or N of 0: MOE_OK.
 * Errors: INVALID_ARG, UNSUPPORTED (sizes as above, or an output of more tiles
 * than a grid holds, 2^23; format, group, fp32 x), ALIGNMENT, HIP.
 */
moe_status moe_matmul_packed(const void* x, int32_t dtype, const uint32_t* codes, const void* scales,
                           const uint16_t* biases, int32_t format, int32_t group, int32_t M, int32_t N, int32_t K,
                           int32_t out_dtype, void* out, hipStream_t stream);

moe_status moe_grouped_matmul_packed(const void* x, int32_t dtype, const uint32_t* codes, const void* scales,
                                   const uint16_t* biases, int32_t format, int32_t group, int32_t T, int32_t k,
                                   int32_t N, int32_t K, int32_t E, const int32_t* offsets, const int32_t* perm,
                                   int32_t x_order, int32_t out_order, int32_t out_dtype, void* out, int32_t* err,
                                   hipStream_t stream);

const char* moe_status_string(moe_status status);

/* Library version string. */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSMOE_H */

/*
 * moe_mxfp4.h -- C ABI of the MI355X (gfx950) MXFP4 mixture-of-experts
 * decode-layer library (libmoe_mxfp4.so).
 *
 * The operation.  One decode step of one mixture-of-experts layer of the kind
 * described in "Kimi K3 on GB300: 13 kernels a layer, and what 842 and 423
 * tokens a second measure" (ai.thesatyajit.com), section "What one decode
 * step of Kimi K3 does": per token a router scores 896 experts, 16 are routed
 * to, a shared expert runs beside them, and the experts are stored in MXFP4
 * (17,547,264 bytes each at hidden 7168, expert intermediate 1536).  For each
 * activation row b of a batch of 1..64 (the decode envelope of "vLLM reports
 * 842 tokens per second for Kimi decoding with NVIDIA DSpark", ai-primer.com,
 * list of the supported envelope):
 *
 *   logit[e] = fp32( sum_h x[b][h] * Wr[e][h] + bias[e] )
 *   S        = the top_k experts by (logit descending, index ascending)
 *   gate[j]  = exp(logit[S_j] - logit[S_0]) / sum_i exp(logit[S_i] - logit[S_0])
 *   FFN_W(x) = W_down ( silu(W_gate x) * (W_up x) ),   silu(z) = z / (1 + e^-z)
 *   residual[b] += FFN_shared(x[b]) + sum_j gate[j] * FFN_{S_j}(x[b])
 *
 * MXFP4 (OCP Microscaling Formats v1.0): each weight is a 4-bit E2M1 code
 * (sign, 2-bit exponent with bias 1, 1-bit mantissa: magnitudes 0, .5, 1,
 * 1.5, 2, 3, 4, 6), and each block of 32 consecutive elements along the
 * contraction dimension K of one output row shares an E8M0 scale byte
 * (2^(byte-127); 0xFF is NaN).  Codes are packed two per byte, element 2i in
 * bits 3:0 and element 2i+1 in bits 7:4.  A matrix [N][K] is stored as codes
 * [N][K/2] bytes and scales [N][K/32] bytes, both row-major.
 *
 * Expert blob.  Routed expert e occupies moe_expert_bytes(H, I) bytes at
 * experts + e * moe_expert_bytes(H, I), holding, each sub-array starting at a
 * multiple of 256 bytes (no padding occurs at H 7168, I 1536):
 *     gate codes [I][H/2] | up codes [I][H/2] | down codes [H][I/2] |
 *     gate scales [I][H/32] | up scales [I][H/32] | down scales [H][I/32]
 *
 * Precision.  Router products bf16 x bf16 are exact; they are summed in fp64
 * and rounded once to fp32 (so expert selection is reproducible bit for bit).
 * Expert and shared-expert dot products are accumulated in fp32; the SwiGLU
 * intermediate is kept in fp32; the combine is fp32.
 *
 * Conventions for every entry point.
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees or synchronises, and keeps no state
 *     between calls.  Work is enqueued on `stream` (a hipStream_t; NULL is the
 *     null stream) and runs asynchronously; results are visible after the
 *     caller synchronises that stream.
 *   - Argument errors are detected on the host before anything is enqueued
 *     and return MOE_ERR_INVALID_ARGUMENT; shapes outside the kernels'
 *     envelope return MOE_ERR_UNSUPPORTED (the caller runs something else);
 *     a failed launch returns MOE_ERR_HIP.  Device faults surface at the
 *     caller's next synchronisation.
 *   - Buffers must not alias unless stated.  Device pointers must be aligned
 *     to 16 bytes (bf16/fp32 tensors) and 256 bytes (expert blobs, workspace).
 *   - Concurrent calls are safe when they use distinct workspaces and
 *     outputs.  Non-finite inputs are not checked; a 0xFF scale byte makes
 *     NaN every output that depends on its block.
 */
#ifndef MOE_MXFP4_H
#define MOE_MXFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARGUMENT = -1,    /* NULL pointer, bad size, bad alignment   */
  MOE_ERR_UNSUPPORTED = -2,         /* valid, but beyond the kernels' envelope */
  MOE_ERR_WORKSPACE_TOO_SMALL = -3, /* ws_bytes < moe_workspace_size(...)      */
  MOE_ERR_HIP = -4                  /* a HIP runtime call or launch failed     */
} moe_status;

typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F32 = 1, MOE_DTYPE_F16 = 2, MOE_DTYPE_I8 = 3 } moe_dtype;

/* Largest batch (activation rows) of the decode-layer, router_topk, MXFP4,
 * norm and bf16 entry points.  moe_route and the 8-bit entry points below
 * take prompts too: their limits stand with them. */
#define MOE_MAX_BATCH 64
/* Largest top_k and number of experts the router/top-k kernels accept. */
#define MOE_MAX_TOPK 64
#define MOE_MAX_EXPERTS 4096
/* Largest number of rows (tokens) moe_route, quant_rows_i8, gemm_i8 and
 * moe_combine accept: 2^24 - 1. */
#define MOE_MAX_ROWS 0xFFFFFF

/* Layout of the experts buffer (moe_layer_weights.expert_layout). */
#define MOE_EXPERTS_CANONICAL 0 /* the blob layout described above             */
#define MOE_EXPERTS_PACKED 1    /* rewritten by moe_pack_experts (see below)    */

/*
 * One layer's weights: a host struct of device pointers.
 *   hidden H, inter I (routed expert intermediate), num_experts E, top_k k,
 *   shared_inter Is (0 = no shared expert).  H and I multiples of 32,
 *   Is a multiple of 8.
 *   router_w     bf16 [E][H] (row e scores expert e)
 *   router_bias  fp32 [E], added to the logits before selection and gates;
 *                NULL for none
 *   shared_gate, shared_up  bf16 [Is][H];  shared_down  bf16 [H][Is];
 *                all three NULL iff Is == 0
 *   experts      E blobs of moe_expert_bytes(H, I) bytes
 *   expert_layout  MOE_EXPERTS_CANONICAL or MOE_EXPERTS_PACKED: which layout
 *                the experts buffer holds (moe_decode_layer needs PACKED)
 * bf16 tensors are raw bfloat16 bit patterns (uint16_t).
 */
typedef struct {
  int32_t hidden, inter, num_experts, top_k, shared_inter;
  const uint16_t* router_w;
  const float* router_bias;
  const uint16_t* shared_gate;
  const uint16_t* shared_up;
  const uint16_t* shared_down;
  const uint8_t* experts;
  int32_t expert_layout;
} moe_layer_weights;

/* Bytes of one expert blob (17,547,264 at H 7168, I 1536); 0 if H or I is
 * not a positive multiple of 32. */
size_t moe_expert_bytes(int hidden, int inter);

/* Workspace bytes moe_decode_layer needs for this layer at this batch.
 * Returns MOE_ERR_INVALID_ARGUMENT for the same shape errors as
 * moe_decode_layer. */
moe_status moe_workspace_size(const moe_layer_weights* w, int batch, size_t* bytes);

/*
 * moe_pack_experts / moe_unpack_experts -- rewrite experts [0, num_experts)
 * of an experts buffer IN PLACE from the canonical blob layout into the
 * packed layout moe_decode_layer streams, or back.  Done once, when the
 * weights are loaded; not part of a decode step.  Each blob keeps its size
 * (moe_expert_bytes) and position; the rewrite is an exact byte permutation.
 *
 * Packed layout.  Each MXFP4 matrix [N][K] of a blob is cut into tiles of 16
 * rows x 16 scale blocks (16 x 512 elements; the last tile of a row group
 * holds the remaining K/32 mod 16 blocks).  A tile of SC blocks holds its
 * codes as [SC][16 rows] x 16 bytes followed by its scales as [16 rows][SC]
 * bytes (in a full tile, SC = 16, a row's scale of block 4 kb + q sits at
 * byte 4 q + kb of the row's 16); a row group's tiles are consecutive.  The blob holds, for every
 * 16-row group of the gate/up rows and every segment along H, the gate tile
 * then the up tile; then the down tiles (16-row groups of H, segments along
 * I); then zero padding up to moe_expert_bytes.  So a wave of 64 lanes reads
 * 16 rows x 128 elements of codes as one contiguous kilobyte, with the tile's
 * scales right behind it.
 *
 *   experts  device buffer of num_experts * moe_expert_bytes(H, I) bytes,
 *            256-byte aligned
 *   scratch  device buffer of >= moe_expert_bytes(H, I) bytes, not
 *            overlapping experts (one expert is staged through it at a time)
 * Enqueued on `stream`; the buffer must not be used by other work until the
 * stream has passed the call.
 */
moe_status moe_pack_experts(uint8_t* experts, int num_experts, int hidden, int inter, void* scratch,
                            size_t scratch_bytes, void* stream);
moe_status moe_unpack_experts(uint8_t* experts, int num_experts, int hidden, int inter, void* scratch,
                              size_t scratch_bytes, void* stream);

/*
 * router_topk -- router GEMV, top-k selection and renormalised gates.
 *   x          bf16 [batch][hidden]
 *   router_w   bf16 [num_experts][hidden]; bias fp32 [num_experts] or NULL
 *   topk_idx   out int32 [batch][top_k], experts in (logit desc, index asc)
 *              order -- ties resolve to the lower index
 *   topk_gate  out fp32 [batch][top_k], gates in the same order, sum 1
 *   logits     out fp32 [batch][num_experts] (the router scores), or NULL
 *   ws         device workspace of >= moe_router_workspace_size(...) bytes
 *              (may be NULL when that size is 0)
 * 1 <= batch <= 64, 1 <= top_k <= min(num_experts, 64),
 * num_experts <= 4096, hidden a multiple of 32 and <= 16384.
 */
size_t moe_router_workspace_size(int batch, int num_experts);
moe_status router_topk(const uint16_t* x, int batch, int hidden, const uint16_t* router_w, const float* bias,
                       int num_experts, int top_k, int32_t* topk_idx, float* topk_gate, float* logits, void* ws,
                       size_t ws_bytes, void* stream);

/*
 * expert_gemv_mxfp4 -- y[b][n] = sum_k dequant(W)[n][k] * x[b][k], fp32.
 *   codes   [n][k/2] bytes, scales [n][k/32] bytes (one MXFP4 matrix)
 *   x       [batch][k], bf16 (x_dtype MOE_DTYPE_BF16) or fp32
 *   y       out fp32 [batch][n]; must not alias x
 * k a multiple of 32 (<= 16384), 1 <= n, 1 <= batch <= 64.
 */
moe_status expert_gemv_mxfp4(const uint8_t* codes, const uint8_t* scales, int n, int k, const void* x,
                             moe_dtype x_dtype, int batch, float* y, void* stream);

/*
 * moe_workspace_init -- clear a workspace before its first use.
 * The first bytes of a layer workspace are a control block that
 * moe_decode_layer's single persistent kernel synchronises through: the
 * counters of its two work queues (zero between calls) and a call epoch that
 * every call advances.  Data that workgroups of one call hand to each other is tagged
 * with that call's epoch, so stale data of an earlier call is never taken
 * for the current call's.  A workspace therefore needs this (or any zero
 * fill of the whole buffer) once after allocation, and again after a call
 * that did not complete (a device fault).  Enqueued on `stream`.  ws
 * 256-byte aligned, ws_bytes a multiple of 16.
 * The uint32 at byte offset MOE_WS_STATUS_OFFSET of the workspace is a sticky
 * status word: nonzero means a synchronisation wait inside a call timed out
 * (about a second), which only happens if the workspace was not initialised
 * or the launch could not keep all of its workgroups resident; the outputs
 * of such a call are not valid.  It is cleared by moe_workspace_init.
 * Tags repeat after 2^32 calls on one workspace.
 */
#define MOE_WS_STATUS_OFFSET 28
moe_status moe_workspace_init(void* ws, size_t ws_bytes, void* stream);

/*
 * moe_workspace_status -- enqueue on `stream` a copy of the workspace's
 * sticky status word (above) into *status, a uint32 in device memory or in
 * pinned host memory; the value is there once the stream has passed the
 * call.  0: every synchronisation wait of every call since
 * moe_workspace_init completed, so their outputs are valid; nonzero: a wait
 * gave up and the outputs of that call (and of later calls on the
 * workspace, whose waits then give up at once) are not valid.  A call whose
 * wait gives up still runs to completion without reading or writing outside
 * its buffers.  ws 256-byte aligned with ws_bytes covering the control block
 * (512 bytes); status 4-byte aligned; else MOE_ERR_INVALID_ARGUMENT.
 */
moe_status moe_workspace_status(const void* ws, size_t ws_bytes, uint32_t* status, void* stream);

/* Batch > 1: the 8 bytes at this workspace offset hold, in their low 32 bits,
 * the number of distinct experts the last call routed its rows to (counted
 * on the device from the top-k indices) and, in their high 32 bits, that
 * call's tag.  Read it after the stream has passed the call. */
#define MOE_WS_ACTIVE_EXPERTS_OFFSET 384

/*
 * moe_decode_layer -- the whole layer for `batch` rows, as one kernel launch.
 *   x          bf16 [batch][hidden], the layer input (normalised activations)
 *   residual   fp32 [batch][hidden], read and overwritten with
 *              residual + shared + sum_j gate_j * expert_j; must not alias x
 *   topk_idx   out int32 [batch][top_k]; topk_gate out fp32 [batch][top_k]
 *   w          weights with expert_layout == MOE_EXPERTS_PACKED (a canonical
 *              experts buffer returns MOE_ERR_UNSUPPORTED: pack it once first)
 *   ws         workspace of >= moe_workspace_size(w, batch) bytes, 256-byte
 *              aligned, owned by the caller, cleared once by
 *              moe_workspace_init; calls that share a workspace must be
 *              ordered on one stream (they must not overlap)
 * Routing never leaves the device: no host synchronisation happens inside.
 */
moe_status moe_decode_layer(const moe_layer_weights* w, const uint16_t* x, float* residual, int batch,
                            int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_decode_layer_mxfp8 -- opt-in variant of moe_decode_layer whose routed
 * experts multiply their FP4 weights by MXFP8 activations, the precision the
 * expert kernel of "Kimi K3 on GB300: 13 kernels a layer, and what 842 and
 * 423 tokens a second measure" uses (section "Why batch 1 on a rack is not
 * only a bandwidth problem": FP4 x MXFP8 FC1/FC2 products).  The row entering
 * a routed expert's FC1 and the SwiGLU output entering its FC2 are each
 * quantised to MXFP8 (OCP Microscaling Formats v1.0: per block of 32
 * consecutive elements an E8M0 scale 2^(floor(log2 amax) - 8), elements the
 * nearest E4M3 value, ties to even, clamped to +-448) and the products run on
 * gfx950's scaled FP4 x FP8 matrix instruction with the dot products summed
 * in fp32.  The router, top-k, gates, the bf16 shared expert and the combine
 * are exactly those of moe_decode_layer, so expert indices and gates are
 * identical; the layer output differs from moe_decode_layer's by the
 * activation quantisation (a few 1e-2 relative on the experts' part).
 * Arguments, workspace and errors as moe_decode_layer; additionally
 * MOE_ERR_UNSUPPORTED when 16 columns of the FC2 input (inter rounded up to
 * 512, as E4M3 codes and scales) exceed 33,280 bytes of staging (inter above
 * 1536).
 */
moe_status moe_decode_layer_mxfp8(const moe_layer_weights* w, const uint16_t* x, float* residual, int batch,
                                  int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_decode_layer_noalloc -- moe_decode_layer for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  It takes no workspace: the library's
 * own static device array of MOE_NOALLOC_SCRATCH_BYTES serves instead, one
 * per GPU, held from the first call on that GPU until the process ends; the
 * call itself allocates nothing.  x, residual, topk_idx, topk_gate and w are
 * as for moe_decode_layer.
 *   status   device pointer to a uint32 (or NULL): after the layer, the
 *            array's sticky status word is copied there on `stream` (0: every
 *            wait of every no-allocation call on this GPU completed, see
 *            moe_workspace_status)
 * Errors: MOE_ERR_WORKSPACE_TOO_SMALL, before anything is enqueued, when
 * moe_workspace_size(w, batch) exceeds MOE_NOALLOC_SCRATCH_BYTES (24 MiB:
 * the K3 shape fits up to batch 20); MOE_ERR_UNSUPPORTED when the first call
 * on a GPU is made while `stream` is being captured (that call clears the
 * array once with a fill kernel, which must not be recorded into a graph);
 * otherwise as moe_decode_layer.
 * Every call on one GPU shares that GPU's array and leaves its contents for
 * the next (each call's data carries that call's tag, so nothing stale is
 * ever taken as current): calls on one GPU must be ordered -- two that
 * overlap, on different streams or threads, race on the array and their
 * results are undefined.
 */
#define MOE_NOALLOC_SCRATCH_BYTES (24u << 20)
moe_status moe_decode_layer_noalloc(const moe_layer_weights* w, const uint16_t* x, float* residual, int batch,
                                    int32_t* topk_idx, float* topk_gate, uint32_t* status, void* stream);

/*
 * Per-kernel timing of moe_decode_layer (for profiling and benchmarks).
 * moe_decode_layer_kernel_count() is the number K of kernels one call
 * launches; moe_decode_layer_kernel_name(i) the name of the i-th (NULL out
 * of range).  moe_decode_layer_timed() is moe_decode_layer that also records
 * K+1 caller-created hipEvent_t `events` on `stream`: events[0] before the
 * first kernel and events[i+1] right after kernel i, so the elapsed time
 * between events[i] and events[i+1] brackets kernel i.  n_events must be at
 * least K+1 and no entry may be NULL (else MOE_ERR_INVALID_ARGUMENT).
 */
int moe_decode_layer_kernel_count(void);
const char* moe_decode_layer_kernel_name(int i);
moe_status moe_decode_layer_timed(const moe_layer_weights* w, const uint16_t* x, float* residual, int batch,
                                  int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes, void* stream,
                                  void* const* events, int n_events);

/*
 * Dense-block pieces used between MoE layers of a decode-step stack.
 * rmsnorm_bf16:    out[b] = bf16( in[b] / sqrt(mean(in[b]^2) + eps) ), gain 1;
 *                  in fp32 [batch][hidden], out bf16 [batch][hidden].
 * dense_gemv_bf16: y[b][n] = bf16( sum_k W[n][k] * x[b][k] ) with fp32
 *                  accumulation; W bf16 [n][k], x bf16 [batch][k], y bf16
 *                  [batch][n]; y must not alias x.  k a multiple of 8.
 * residual_add_bf16: h[b][i] += float(t[b][i]) (h fp32, t bf16).
 * residual_add_rmsnorm_bf16: residual_add_bf16 then rmsnorm_bf16 of the
 *                  updated h into out, as one launch (same sums, same order).
 */
moe_status rmsnorm_bf16(const float* in, int batch, int hidden, float eps, uint16_t* out, void* stream);
moe_status dense_gemv_bf16(const uint16_t* w, int n, int k, const uint16_t* x, int batch, uint16_t* y,
                           void* stream);
moe_status residual_add_bf16(float* h, const uint16_t* t, int batch, int hidden, void* stream);
moe_status residual_add_rmsnorm_bf16(float* h, const uint16_t* t, int batch, int hidden, float eps, uint16_t* out,
                                     void* stream);

/*
 * moe_route -- scores of caller-computed router logits to experts and gates,
 * for any number of rows (one decoding token to a long prompt).
 *   logits      [rows][num_experts], bf16, fp16 or fp32 (`dtype`), row r at
 *               logits + r * row_stride elements (row_stride >= num_experts)
 *   bias        fp32 [num_experts] or NULL: added to the scores for the
 *               selection only, never to the gates (a balance bias)
 *   topk_idx    out int32 [rows][top_k]; topk_gate out fp32 [rows][top_k];
 *               they overlap neither the logits' rows, nor bias, nor each other
 * For row r with logits l, over the candidates: the experts whose logit (and
 * bias) is neither NaN nor -inf (a logit of +inf counts as the largest fp32):
 *   s[e]    = exp(l[e]) / sum_i exp(l[i])  (MOE_SCORE_SOFTMAX)  or
 *             1 / (1 + exp(-l[e]))         (MOE_SCORE_SIGMOID)
 *   c[e]    = s[e] + bias[e]
 *   groups  > 1: group g holds the num_experts / groups experts from
 *           g * num_experts / groups on; its worth is the sum of the
 *           group_top (1 or 2; fewer if it has fewer) largest c of its
 *           candidates; the top_groups groups of the largest worth stay
 *           (ties: the lower group; a group without candidates never stays).
 *           With group_top 1 and no bias the best logits are compared, the
 *           same order where the scores are told apart
 *   S       = the top_k candidates of the remaining groups by (c descending,
 *             index ascending); without a bias by (l descending, index
 *             ascending), the same order where the scores are told apart
 *   gate[j] = scale * s[S_j] / (renorm ? sum_i s[S_i] : 1); 0 if that sum is 0
 * A row with fewer than top_k such candidates (a padded row has none) ends in
 * index -1, gate 0.  Scores, sums and c are compared in fp64 (or so that the
 * comparison has the same result), so two experts are in the order of the
 * formula also where their fp32 scores would tie.  Gates are rounded once; of a
 * softmax without bias and renormalisation the sum over all its scores is
 * within 2^-29 of itself before that.
 * 1 <= rows <= MOE_MAX_ROWS, 1 <= top_k <= min(64, top_groups * num_experts / groups),
 * num_experts <= 4096 and a multiple of groups, 1 <= top_groups <= groups <=
 * 64, group_top 1 or 2; groups == 1 needs top_groups == 1; scale finite.  bias
 * 4-byte aligned, logits aligned to their element.
 */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
typedef struct {
  int32_t num_experts, top_k;
  int32_t score;                         /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID */
  int32_t groups, top_groups, group_top; /* 1, 1, 1: no groups                     */
  int32_t renorm;                        /* 0 or 1                                 */
  float scale;
} moe_route_params;
moe_status moe_route(const void* logits, moe_dtype dtype, size_t row_stride, int rows, const float* bias,
                     const moe_route_params* params, int32_t* topk_idx, float* topk_gate, void* stream);

/*
 * 8-bit integer products.  Activations are quantised per row (token), weights
 * per output channel, both symmetrically; the products are summed exactly in
 * int32 and scaled once.
 *
 * quant_rows_i8 -- rows to 8-bit codes with one scale each:
 *   scale[m] = fp32( max_k |x[m][k]| / 127 )
 *   q[m][k]  = the integer nearest to x[m][k] / scale[m] (the exact quotient,
 *              ties to even), within +-127
 *   x        [rows][k] bf16, fp16 or fp32, row m at x + m * x_stride elements
 *   q        out int8 [rows][k]; scale out fp32 [rows]; neither overlaps the
 *            rows of x, nor the other
 * A row of zeros (or so small that its scale rounds to 0) has scale 0 and
 * codes 0.  A row that holds a NaN or an infinity has scale NaN and codes 0,
 * so every product of it is NaN.  1 <= rows <= MOE_MAX_ROWS, 1 <= k <= 65536.
 */
moe_status quant_rows_i8(const void* x, moe_dtype dtype, size_t x_stride, int rows, int k, int8_t* q, float* scale,
                         void* stream);

/*
 * gemm_i8 -- y[m][n] = x_scale[m] * w_scale[n] * sum_k xq[m][k] * w[n][k]
 *   x         x_dtype MOE_DTYPE_I8: the codes xq, with x_scale fp32 [m];
 *             bf16, fp16 or fp32: rows that the call quantises as
 *             quant_rows_i8 does, x_scale NULL
 *             row i at x + i * x_stride elements, x_stride >= k
 *   w         int8 [n][k] codes, w_scale fp32 [n]
 *   swiglu    0, or 1: w is [2][n][k], gate then up, w_scale [2][n], and
 *             y[m][i] = silu(g) * u of the two products g and u
 *   y         out [m][n], bf16, fp16 or fp32 (y_dtype)
 *   ws        workspace of >= gemm_i8_workspace_size(...) bytes, 256-byte
 *             aligned (may be NULL where that is 0).  It needs no
 *             initialisation and holds nothing between calls.
 * Neither y nor the workspace's gemm_i8_workspace_size(...) bytes overlap the
 * rows of x, w, either scale or each other.
 * The sum is exact; it is rounded to fp32, multiplied by w_scale, then by
 * x_scale, a rounding each (so a w_scale up to 2^97 overflows only where the
 * result does), and rounded to y_dtype; SwiGLU runs in fp32 on the scaled sums,
 * within 11 roundings for every gate, also where exp(-gate) overflows.
 * 1 <= m <= MOE_MAX_ROWS, 1 <= n <= 2^20, k a multiple of 16 in 16 .. 65536;
 * MOE_ERR_UNSUPPORTED also where its tiles make 2^22 workgroups or more (an
 * output of some 10^11 elements, fewer with few rows an expert).  16-byte aligned x
 * (x_stride a multiple of 16) if it is int8, else aligned to its element; w
 * and y 16-byte aligned.
 */
size_t gemm_i8_workspace_size(int m, int n, int k, int swiglu, moe_dtype x_dtype);
moe_status gemm_i8(const void* x, moe_dtype x_dtype, size_t x_stride, const float* x_scale, int m, int k,
                   const int8_t* w, const float* w_scale, int n, int swiglu, void* y, moe_dtype y_dtype, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * moe_group_slots -- sort the slots s = t * top_k + j of a routing by expert.
 *   idx      int32 [tokens][top_k], as moe_route or router_topk leave it; a
 *            value outside 0 .. num_experts - 1 is a slot without an expert
 *   groups   out, device buffer of >= moe_slot_groups_size(...) bytes,
 *            256-byte aligned, holding
 *              int32 order[tokens * top_k] at byte 0: the slots by expert,
 *                ascending within one; slots without an expert come last
 *              int32 offsets[num_experts + 2] at byte
 *                MOE_GROUPS_OFFSETS(tokens, top_k): expert e has order[
 *                offsets[e]] up to order[offsets[e + 1]] exclusive, and
 *                num_experts names the slots without an expert
 *            and lists that experts_gemm_i8 works through; it does not overlap idx
 * 1 <= tokens, 1 <= top_k <= 64, num_experts <= 4096, tokens * top_k < 2^27.
 * moe_slot_groups_size is 0 outside these limits.
 */
#define MOE_GROUPS_OFFSETS(tokens, top_k) ((((size_t)(tokens) * (size_t)(top_k) * 4 + 255) / 256) * 256)
size_t moe_slot_groups_size(int tokens, int top_k, int num_experts);
moe_status moe_group_slots(const int32_t* idx, int tokens, int top_k, int num_experts, void* groups,
                           size_t groups_bytes, void* stream);

/*
 * experts_gemm_i8 -- gemm_i8 of every slot with its own expert's matrix:
 *   y[s] = product of x[r] with w[expert of slot s];  zeros for a slot
 *   without an expert
 *   x_rows   tokens (row r = s / top_k: FC1) or tokens * top_k (row r = s:
 *            FC2); with top_k 1 the two are the same
 *   groups   as moe_group_slots left it for the same tokens, top_k and
 *            num_experts
 *   w        int8 [num_experts][n][k], w_scale fp32 [num_experts][n]; with
 *            swiglu int8 [num_experts][2][n][k], w_scale [num_experts][2][n]
 *   y        out [tokens * top_k][n]
 * Types, alignments, limits, overlaps (groups among the inputs), sums and
 * workspace as gemm_i8; tokens, top_k and num_experts as moe_group_slots.
 */
size_t experts_gemm_i8_workspace_size(int tokens, int top_k, int num_experts, int x_rows, int n, int k, int swiglu,
                                      moe_dtype x_dtype);
moe_status experts_gemm_i8(const void* x, moe_dtype x_dtype, size_t x_stride, const float* x_scale, int x_rows, int k,
                           const void* groups, size_t groups_bytes, int tokens, int top_k, int num_experts,
                           const int8_t* w, const float* w_scale, int n, int swiglu, void* y, moe_dtype y_dtype,
                           void* ws, size_t ws_bytes, void* stream);

/*
 * moe_combine -- out[t][h] = residual[t][h] + sum_j gate[t][j] * y[t*top_k + j][h]
 *   y         [tokens * top_k][hidden], bf16, fp16 or fp32 (`dtype`)
 *   gate      fp32 [tokens][top_k]
 *   residual  fp32 [tokens][hidden], or NULL for zeros; may be out itself
 *   out       fp32 [tokens][hidden]; overlaps neither y, nor gate, nor
 *             otherwise residual
 * Summed in fp32, j ascending, then the residual.  1 <= tokens <=
 * MOE_MAX_ROWS, 1 <= top_k <= 64, 1 <= hidden <= 2^20.  Pointers aligned to
 * their element.
 */
moe_status moe_combine(const void* y, moe_dtype dtype, const float* gate, int tokens, int top_k, int hidden,
                       const float* residual, float* out, void* stream);

/*
 * moe_set_max_workgroups -- test and diagnostic knob, not needed for decoding:
 * caps the number of workgroups of the layer kernel (every moe_decode_layer*
 * entry point) launched after it returns, process-wide, at n; n = 0 restores
 * the default (two workgroups per compute unit).  The layer's work queue is
 * built to finish on any grid of at least one workgroup (a unit waits only
 * on units before it in the queue), and its results do not depend on the
 * grid; a small grid runs it in a different interleaving, which is what
 * the knob is for.  n < 0: MOE_ERR_INVALID_ARGUMENT.  Not synchronised
 * with launches in flight on other host threads.
 */
moe_status moe_set_max_workgroups(int n);

/*
 * moe_stream_read_probe -- measurement aid, not part of a decode step: one
 * kernel that reads `bytes` of `buf` once with 16-byte non-temporal loads
 * (blocks_per_cu 256-thread workgroups per compute unit, grid-stride), the
 * access pattern of a plain streaming read.  Timing it gives the device's
 * HBM read ceiling that the layer's weight streams are compared with.
 * `sink` (device, 4 bytes) is written only in the (never expected) case
 * that the xor of all data equals 0x9E3779B9, so nothing else is stored.
 * buf 16-byte aligned, bytes a positive multiple of 16, 1 <= blocks_per_cu
 * <= 32; else MOE_ERR_INVALID_ARGUMENT.
 */
moe_status moe_stream_read_probe(const void* buf, size_t bytes, int blocks_per_cu, uint32_t* sink, void* stream);

/*
 * moe_prefetch -- read a table of weight ranges once with ordinary
 * (allocating) loads, so that they sit in the device's memory-side
 * last-level cache (256 MB on MI355X) when a later kernel streams them: the
 * "prefetch on a third stream" of "Kimi K3 on GB300: 13 kernels a layer"
 * (section "What the fused path changes"), where a small kernel walks a
 * table of upcoming weight ranges.  Meant for a side stream, beside kernels
 * that leave HBM idle (norms, launch gaps); it writes nothing and its
 * results are not needed by anyone, so nothing has to wait for it.
 *   ranges   host array of n_ranges (1..MOE_PREFETCH_MAX_RANGES) device
 *            ranges, each 16-byte aligned with a size multiple of 16; the
 *            table is copied into the launch, so it need not outlive the call
 *   blocks   256-thread workgroups of the kernel (1..65536): how much of the
 *            device it occupies beside the other stream's work
 * Safe under stream capture (one kernel node, arguments by value).
 */
#define MOE_PREFETCH_MAX_RANGES 8
typedef struct {
  const void* ptr;
  size_t bytes;
} moe_range;
moe_status moe_prefetch(const moe_range* ranges, int n_ranges, int blocks, void* stream);

/* Static, human-readable name of a status code. */
const char* moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MXFP4_H */

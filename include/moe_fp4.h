/*
 * moe_fp4.h — C ABI of the FP4 routed mixture-of-experts layer for GB300 (sm_103a).
 *
 * The layer is the routed-expert block of DeepSeek-V4-Flash-style inference
 * ("DeepSeek-V4-Flash on AMD gfx90a: Correctness Recovery and Inference
 * Performance Engineering", abstract: FP4 routed mixture-of-experts with packed
 * FP4 weights and expert sorting; the "MXFP4 MoE" path of the vLLM-on-MI300X
 * write-up).  Per token it
 *   1. picks the top-k experts of the router logits, ordered by (logit desc,
 *      expert index asc), and weights them by the softmax over the k picked
 *      logits (fp32 comparison, ties to the lower expert id: MI250 correctness
 *      blog, section 4.1 table and section 4.2);
 *   2. sorts the T*k (token, slot) pairs by expert with a stable counting sort
 *      and builds per-expert offsets ("retuned expert sorting");
 *   3. for every expert, multiplies its tokens by the packed-FP4 W13 (gate and
 *      up) and applies SwiGLU, h = bf16(silu(g) * u);
 *   4. multiplies h by the packed-FP4 W2 (down) and combines the k expert
 *      outputs of each token with its routing weights (by default added into
 *      out in the W2 kernel's epilogue in no fixed order; in slot order with
 *      MOE_FP4_FLAG_DETERMINISTIC).
 *
 * Formats (MXFP4, OCP Microscaling v1.0):
 *   - weights: two E2M1 codes per byte along K, the LOW nibble holds the even
 *     K element; code bit 3 = sign, bits 0..2 index {0, .5, 1, 1.5, 2, 3, 4, 6};
 *   - scales: E8M0 bytes, value 2^(s-127), one per 32 consecutive K elements
 *     of a row; s in [0, 253].  Bytes 254 and 255 (NaN), and scales that push
 *     a product or sum past the fp32 range, are outside the contract: results
 *     are unspecified, nothing faults.
 *   - x is bf16 (raw IEEE binary32 upper halves), router logits and all
 *     outputs are fp32 except h (bf16).  Router logits must be finite.
 *
 * Tensor layouts (all row-major, C-contiguous, device memory unless stated):
 *   x              bf16   [T, d]
 *   router_logits  fp32   [T, E]
 *   w13            uint8  [E, 2I, d/2]   rows [0, I) = gate, rows [I, 2I) = up
 *   w13_scale      uint8  [E, 2I, d/32]
 *   w2             uint8  [E, d, I/2]    row n = output feature n, packed along I
 *   w2_scale       uint8  [E, d, I/32]
 *   out            fp32   [T, d]         fully overwritten
 *   topk_ids       int32  [T, k]         slot 0 = highest logit
 *   topk_weights   fp32   [T, k]
 *   expert_offsets int32  [E + 1]        expert e owns sorted rows [off[e], off[e+1])
 *   sorted_slot    int32  [T*k]          sorted row r -> flat slot t*k + j,
 *                                        increasing within each expert
 *   h              bf16   [T*k, I]       SwiGLU output in sorted-row order
 *
 * Ownership and threading: the caller owns every buffer and the stream.  The
 * library allocates nothing; all scratch lives in the caller's workspace
 * (moe_fp4_workspace_bytes).  moe_fp4_route and moe_fp4_forward only enqueue
 * work on the given stream and never synchronise.  Calls that use different
 * workspaces may run concurrently; calls sharing a workspace must be ordered
 * on one stream.  Inside a call the kernels after routing are launched with
 * programmatic dependent launch (each waits on the device for the one before
 * it); the call as a whole keeps ordinary stream order with the caller's work:
 * its first kernel starts after everything enqueued before it, and the last
 * kernel of moe_fp4_forward lets no later kernel start early.  (The routing
 * kernel of moe_fp4_route, T <= 32, does let a following kernel that the
 * caller launches early start before it ends; such a kernel must wait on the
 * device, griddepcontrol.wait, before it reads the routing outputs, as any
 * early-launched kernel must.)
 *
 * Errors: every function returns a moe_fp4_status.  Argument checks happen on
 * the host before anything is enqueued; on error nothing is launched.  A
 * failed launch returns MOE_FP4_ERR_CUDA (the CUDA error is left for the
 * caller's next CUDA call to see).  Kernels never trap.
 */
#ifndef MOE_FP4_H_
#define MOE_FP4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Problem sizes.  T tokens, d hidden size, I expert intermediate size,
 * E experts, k experts per token. */
typedef struct moe_fp4_dims {
  int32_t T, d, I, E, k;
} moe_fp4_dims;

typedef enum moe_fp4_status {
  MOE_FP4_OK = 0,
  MOE_FP4_ERR_INVALID_ARG = -1,  /* null pointer, bad size, misaligned pointer */
  MOE_FP4_ERR_UNSUPPORTED = -2,  /* sizes the kernels do not cover (see moe_fp4_workspace_bytes) */
  MOE_FP4_ERR_WORKSPACE = -3,    /* workspace too small */
  MOE_FP4_ERR_CUDA = -4,         /* a CUDA runtime call failed */
  MOE_FP4_ERR_DEVICE = -5        /* a kernel reported an error word (moe_fp4_check) */
} moe_fp4_status;

/* Flags for moe_fp4_forward.  Both expert paths give results within the same
 * tolerance of the definition; the default picks by shape (expected rows per
 * expert = T*k/E): the streaming GEMV path for few rows, the tensor-core path
 * otherwise. */
#define MOE_FP4_FLAG_FORCE_GEMV 0x1u    /* streaming path: weights streamed once, warp-level mma.sync
                                           (d, I multiples of 1024) */
#define MOE_FP4_FLAG_FORCE_TC   0x2u    /* tcgen05 tensor-core path */
/* On the streaming path: both projections in one persistent launch (W13 +
 * SwiGLU, a grid-wide arrival counter with a bounded wait, then W2), one CTA
 * per SM launched cooperatively, instead of two launches (the paper's
 * per-layer synchronisation and launch cost, abstract: limits).  The same
 * results; in moe_fp4_forward_profiled the W13 stage then covers both
 * projections and the W2 stage is empty.  May be combined with
 * MOE_FP4_FLAG_FORCE_GEMV; ignored on the tensor-core path. */
#define MOE_FP4_FLAG_PERSISTENT 0x4u
/* On the tensor-core path: run both projections on pairs of SMs (tcgen05
 * cta_group::2: one MMA instruction covers M = 256 weight rows, 128 from each
 * CTA's tensor memory, with the token tile split between the two CTAs), and
 * the weighted combine inside the W2 kernel (per-token counters; the CTA
 * that completes a token's k slots sums them in slot order, deterministic).
 * The same results within the layer's tolerance; slower than the default
 * one-SM kernels on GB300 (the dequantisers' tensor-memory stores wait while
 * the pair's MMAs read both SMs' tensor memory).  Ignored on the streaming
 * path. */
#define MOE_FP4_FLAG_CTA_PAIRS 0x8u
/* The weighted combine.  By default the W2 kernel adds each slot's weighted
 * output row into out in its epilogue (fp32 atomic adds, out zeroed first):
 * no y buffer round trip and no separate pass, but the k terms of an output
 * element are summed in whatever order the slots finish, so results may
 * differ in the last bits between calls.  With this flag the W2 kernel writes
 * y and a separate pass sums the k rows of each token in slot order:
 * bitwise reproducible.  CTA pairs always use their own in-epilogue combine in
 * slot order (reproducible); the fallback paths for sizes outside the
 * streaming kernel's use the separate pass. */
#define MOE_FP4_FLAG_DETERMINISTIC 0x10u

/* Bytes of device workspace a call with these sizes needs (256-byte aligned
 * base required).  Returns 0 when the sizes are invalid or unsupported:
 * T >= 1, 1 <= k <= min(E, 32), 1 <= E <= 1024, d and I multiples of 128,
 * 128 <= d <= 16384, 128 <= I <= 16384, T*k < 2^31, T*k*max(d, I) < 2^40. */
size_t moe_fp4_workspace_bytes(const moe_fp4_dims* dims);

/* Steps 1-2 only (routing and the expert sort), so that routing can be
 * checked bit-exactly on its own (the paper's fixed-token and hash checks).
 * topk_ids, topk_weights, expert_offsets and sorted_slot are required
 * device outputs.  Pointers: 4-byte aligned; workspace 256-byte aligned. */
int moe_fp4_route(const moe_fp4_dims* dims, const float* router_logits,
                  int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
                  int32_t* sorted_slot, void* workspace, size_t workspace_bytes,
                  void* cuda_stream);

/* The whole layer (steps 1-4) on device buffers.  out is required; the
 * routing outputs and h are optional (NULL: kept in the workspace only).
 * x, w13, w13_scale, w2, w2_scale, out and h must be 16-byte aligned,
 * the routing outputs 4-byte aligned, the workspace 256-byte aligned.  flags: 0 or one MOE_FP4_FLAG_FORCE_*,
 * optionally with MOE_FP4_FLAG_PERSISTENT. */
int moe_fp4_forward(const moe_fp4_dims* dims, const void* x_bf16, const float* router_logits,
                    const uint8_t* w13, const uint8_t* w13_scale,
                    const uint8_t* w2, const uint8_t* w2_scale, float* out,
                    int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
                    int32_t* sorted_slot, void* h_bf16, unsigned flags,
                    void* workspace, size_t workspace_bytes, void* cuda_stream);

/* The router (gate) projection, the step ahead of top-k routing:
 *   router_logits[t, e] = sum_K x[t, K] * w_gate[e, K]
 * with bf16 x [T, d] and bf16 w_gate [E, d] (row e = expert e's gate
 * vector), every product exact, fp32 accumulation, fp32 logits [T, E] (the
 * MI250 correctness blog, section 4.1: low-precision inputs with FP32
 * accumulation for the gate network, FP32 values for the top-k comparison).
 * The sum order is fixed, so the logits are the same on every call.  x and
 * w_gate 16-byte aligned, router_logits 4-byte aligned; dims as for
 * moe_fp4_forward (I and k are not used).  One kernel is enqueued; no
 * workspace. */
int moe_fp4_router(const moe_fp4_dims* dims, const void* x_bf16, const void* w_gate_bf16,
                   float* router_logits, void* cuda_stream);

/* The whole layer starting from x and the router weights: moe_fp4_router
 * writes router_logits (a required [T, E] fp32 device buffer owned by the
 * caller), then moe_fp4_forward runs on them.  Same arguments, checks and
 * results as moe_fp4_forward otherwise; every argument is checked before
 * anything is enqueued. */
int moe_fp4_forward_gated(const moe_fp4_dims* dims, const void* x_bf16, const void* w_gate_bf16,
                          float* router_logits, const uint8_t* w13, const uint8_t* w13_scale,
                          const uint8_t* w2, const uint8_t* w2_scale, float* out,
                          int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
                          int32_t* sorted_slot, void* h_bf16, unsigned flags,
                          void* workspace, size_t workspace_bytes, void* cuda_stream);

/* moe_fp4_forward that also records caller-created CUDA events (cudaEvent_t
 * handles, MOE_FP4_NUM_STAGE_EVENTS of them) on the stream between its
 * stages, so that a caller can time each kernel in place:
 *   events[0] before routing and the expert sort (3 kernels)
 *   events[1] before the token gather (tensor-core path only; else empty)
 *   events[2] before W13 + SwiGLU
 *   events[3] before W2
 *   events[4] before the combine pass
 *   events[5] after the combine pass (empty when the W2 kernel does the
 *   combine in its epilogue, the default)
 * Same arguments, checks and results as moe_fp4_forward. */
#define MOE_FP4_NUM_STAGE_EVENTS 6
int moe_fp4_forward_profiled(const moe_fp4_dims* dims, const void* x_bf16, const float* router_logits,
                             const uint8_t* w13, const uint8_t* w13_scale,
                             const uint8_t* w2, const uint8_t* w2_scale, float* out,
                             int32_t* topk_ids, float* topk_weights, int32_t* expert_offsets,
                             int32_t* sorted_slot, void* h_bf16, unsigned flags,
                             void* workspace, size_t workspace_bytes, void* cuda_stream,
                             void* const* stage_events);

/* Bytes of device workspace moe_fp4_forward_host needs: the forward workspace
 * plus device staging for x, router_logits and out. */
size_t moe_fp4_host_workspace_bytes(const moe_fp4_dims* dims);

/* The whole layer with HOST x, router_logits and out (weights stay on the
 * device).  Copies x to device staging inside the workspace, runs
 * moe_fp4_forward and synchronises the stream before returning.  Host buffers
 * may be pageable or pinned (pinned is faster).  router_logits and out in
 * memory the device can address (page-locked by the CUDA allocator or
 * registered with it; out 16-byte aligned) are used in place: the routing
 * kernel reads the logits and the combine writes out over the host link, with
 * no copy.  Otherwise they go through device staging too. */
int moe_fp4_forward_host(const moe_fp4_dims* dims, const void* x_bf16_host,
                         const float* router_logits_host,
                         const uint8_t* w13, const uint8_t* w13_scale,
                         const uint8_t* w2, const uint8_t* w2_scale, float* out_host,
                         unsigned flags, void* workspace, size_t workspace_bytes,
                         void* cuda_stream);

/* The whole layer without any workspace argument, for callers that cannot
 * allocate device memory: runtimes without an allocator, callers that must
 * not call cudaMalloc inside a stream-ordered or captured region, plugins
 * that are handed only input and output pointers.  (The paper has no
 * counterpart; this is a deployment convenience.)
 *
 * Scratch: a fixed device array of MOE_FP4_NOALLOC_SCRATCH_BYTES inside this
 * library, which every GPU that loads the library holds until the process
 * exits.  Problems whose moe_fp4_workspace_bytes exceeds it are rejected with
 * MOE_FP4_ERR_WORKSPACE before anything is enqueued.  With E = 256 and k = 8
 * that allows T <= 72 tokens at d = 4096, I = 2048 (the T = 32 decode batch
 * needs about 7.4 MB) and T <= 44 at d = 7168, I = 2048; prefill-sized
 * batches need a workspace (moe_fp4_forward).
 * The array's device address is looked up (with the call's device current)
 * on every call made outside a stream capture, so a device reset between calls
 * is harmless; a call made during a capture uses the address of the last call
 * outside one, so make one call on each device before capturing.
 * All calls share the array and it keeps the last call's contents: calls
 * that overlap on the GPU (other streams, other host threads) race and give
 * wrong results; order them on one stream.  Otherwise the same arguments,
 * checks and results as moe_fp4_forward, with no optional outputs.  The
 * device error word lives in the internal array: moe_fp4_noalloc_check reads
 * it. */
#define MOE_FP4_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)
int moe_fp4_forward_noalloc(const moe_fp4_dims* dims, const void* x_bf16, const float* router_logits,
                            const uint8_t* w13, const uint8_t* w13_scale,
                            const uint8_t* w2, const uint8_t* w2_scale, float* out,
                            unsigned flags, void* cuda_stream);

/* moe_fp4_check for the internal array of moe_fp4_forward_noalloc:
 * synchronises the stream, reads the device error word left by the calls
 * enqueued before it (bits as in moe_fp4_check) and clears it.  Returns
 * MOE_FP4_OK, MOE_FP4_ERR_DEVICE or MOE_FP4_ERR_CUDA.  Allocates nothing. */
int moe_fp4_noalloc_check(void* cuda_stream);

/* MXFP8 quantisation of bf16 rows: the activation operand of a block-scaled
 * (MX) tensor-core product.  The paper quantises its decode activations
 * (abstract: INT8 activation quantisation) and the MI250 blog names
 * block-wise FP8 quantisation as the next gain; this is the MX form, with
 * the blocks of the weights (OCP Microscaling v1.0 conversion, E4M3 element).
 * For each 32 consecutive elements of a row, with amax their largest
 * magnitude:
 *   scale byte  s = floor(log2(amax)) - 8 + 127, at least 0; an all-zero
 *               block gets 0 (the scale is 2^(s-127));
 *   codes       E4M3 (OCP FP8 "FN": bias 7, no infinities, largest 448) of
 *               x / 2^(s-127), rounded to nearest even, saturated at +-448;
 *               a negative zero gives 0x80.
 * Layouts (row-major, device memory):
 *   x_bf16  bf16   [rows, K]      16-byte aligned; K a positive multiple of 32
 *   codes   uint8  [rows, K]      16-byte aligned; fully overwritten
 *   scales  uint8  [rows, K/32]   fully overwritten
 * The caller owns the buffers and the stream.  One kernel is enqueued; for
 * rows = 0 nothing is, and the pointers may be null.  The call never
 * synchronises.  Returns MOE_FP4_ERR_INVALID_ARG, with nothing enqueued, for
 * rows < 0, K not a positive multiple of 32, or (rows > 0) a null pointer or
 * a misaligned x_bf16 / codes; MOE_FP4_ERR_CUDA if the launch fails. */
int moe_fp4_mxfp8_quantize(const void* x_bf16, int64_t rows, int32_t K, uint8_t* codes, uint8_t* scales,
                           void* cuda_stream);

/* Workspace bytes of moe_fp4_forward_mx (256-byte aligned base); 0 for the
 * sizes moe_fp4_workspace_bytes rejects. */
size_t moe_fp4_mx_workspace_bytes(const moe_fp4_dims* dims);

/* The layer with MXFP8 activations into both projections, on block-scaled
 * tensor cores (tcgen05.mma kind::mxf8f6f4: the E2M1 weights and their E8M0
 * scales as stored, E4M3 activations with one E8M0 scale per 32 elements,
 * fp32 accumulation).  Steps as in moe_fp4_forward, with two quantisations
 * added (the MXFP8 conversion of moe_fp4_mxfp8_quantize):
 *   x_q = MXFP8(x) per token row (blocks of 32 along d) before W13;
 *   h   = bf16(silu(g) * u) as in moe_fp4_forward, then
 *   h_q = MXFP8(h) per slot row (blocks of 32 along I) before W2;
 *   y   = h_q . W2_e^T; out = sum_j w_j y_j.
 * The paper quantises its decode activations (abstract: INT8 activation
 * quantisation) and the MI250 blog names block-wise FP8 as the next gain;
 * this is that layer in the weights' own MX block format, not the exact
 * layer: out differs from moe_fp4_forward by the activation rounding.
 * Routing and the sort are those of moe_fp4_route, bit for bit.
 * Arguments as in moe_fp4_forward, except: w13 and w2 must be 32-byte
 * aligned; there are no flags; the optional outputs (NULL: kept in the
 * workspace only) are, in sorted-row order (S = T*k, row r = the r-th row of
 * the expert sort):
 *   h_bf16    bf16  [S, I]     16-byte aligned
 *   h_codes   uint8 [S, I]     E4M3 codes of h_q, 16-byte aligned
 *   h_scales  uint8 [S, I/32]  E8M0 scales of h_q
 *   x_codes   uint8 [S, d]     E4M3 codes of x_q of the row's token, 16-byte aligned
 *   x_scales  uint8 [S, d/32]  E8M0 scales of x_q
 * Enqueues the routing kernel, the quantising gather, the W13 projection,
 * the quantiser of h, the W2 projection and the combine; never synchronises.  A block of x or h that
 * holds an infinity or a NaN gets the NaN scale 0xFF and NaN codes, and the
 * rows it feeds come out NaN.
 * stage_events: NULL, or 6 cudaEvent_t handles recorded on the stream as in
 * moe_fp4_forward_profiled (before routing, after routing, after the
 * quantising gather, after W13, after the quantiser of h and W2, after the
 * combine). */
int moe_fp4_forward_mx(const moe_fp4_dims* dims, const void* x_bf16, const float* router_logits,
                       const uint8_t* w13, const uint8_t* w13_scale, const uint8_t* w2, const uint8_t* w2_scale,
                       float* out, void* h_bf16, uint8_t* h_codes, uint8_t* h_scales, uint8_t* x_codes,
                       uint8_t* x_scales, void* workspace, size_t workspace_bytes, void* cuda_stream,
                       void* const* stage_events);

/* ---- Operators around the layer -------------------------------------------
 * MXFP4 quantisation, products of MXFP4 matrices (dense, and grouped by
 * expert) and the end of a block (norm, gate, residual, next norm).  As for
 * the layer: device buffers owned by the caller, work enqueued on the given
 * stream, nothing allocated, nothing synchronised, arguments checked on the
 * host before anything is enqueued.  They keep no state between calls but a
 * device's error words (moe_fp4_ops_check).  Their kernels are launched with programmatic
 * dependent launch: each is set up while the kernel before it on the stream
 * still runs and waits on the device until all work before has ended and is
 * visible, so that ordinary stream order holds; and each lets a kernel that the
 * caller launches early be set up while it runs (such a kernel must wait on the
 * device, griddepcontrol.wait, as any early-launched kernel must).  A quantiser,
 * read-back, scale layout or block end of fewer CTAs than the SMs hold asks for
 * shared memory that it does not use (up to 225 KB a CTA), which spreads its CTAs
 * over the SMs; kernels of other streams that need shared memory do not run
 * beside them on an SM for those microseconds. */

/* Element types of the operators' unquantised operands and results. */
#define MOE_FP4_TYPE_BF16 0
#define MOE_FP4_TYPE_F32 1

/* MXFP4 form of rows: for each 32 consecutive elements of a row, with amax
 * their largest magnitude (OCP Microscaling v1.0 conversion, E2M1 element),
 *   scale byte  s = floor(log2(amax)) - 2 + 127, at least 0; 0 for an
 *               all-zero block (the scale is 2^(s-127));
 *   codes       E2M1 of x / 2^(s-127), rounded to nearest (ties to the even
 *               code), saturated at +-6; two codes a byte, the LOW nibble the
 *               even element; a negative zero keeps its sign.
 * A block holding an infinity or a NaN gets the scale byte 0xFF (NaN).
 *
 *   x          bf16 or fp32, x_rows rows of K elements, row r at element
 *              r * x_stride (x_stride >= K; any alignment of whole elements,
 *              faster when rows start on 16 bytes)
 *   row_index  NULL: output row r is row r of x; else int32 [rows], output row
 *              r is row row_index[r] / index_div of x (the layer's sorted_slot
 *              with index_div = k gathers the tokens of the expert sort).  An
 *              index outside x gives a zero row and sets error bit 1.
 *   codes      uint8 [rows, K/2], 16-byte aligned
 *   scales     row-major (tiled = 0): uint8 [rows, K/32].
 *              tiled = 1, the layout of the products' scales: tiles of 128 rows
 *              by 4 scales, uint8 [row tiles][ceil(K/128)][512], the byte of
 *              row r and scale b of a tile at 16 (r % 32) + 4 (r / 32) + b;
 *              scales past K/32 are written as 0, those of rows past the end
 *              are left as they were.  Without groups row r is in tile r / 128.
 *              With group_offsets (int32 [groups + 1] on the device, groups <=
 *              1024, not decreasing, rows of group e in [off[e], off[e+1]))
 *              every group starts a tile: row r of group e is row r - off[e] of
 *              the tiles from off[e] / 128 + e on.  rows / 128 + groups tiles
 *              in all (moe_fp4_mxfp4_tiled_scale_bytes, 16-byte aligned).
 *              Rows in no group get codes and no scales.
 * K a positive multiple of 32, at most 32768; rows K < 2^35; rows = 0
 * enqueues nothing. */
int moe_fp4_mxfp4_quantize(const void* x, int x_type, int64_t x_rows, int64_t x_stride, int32_t K,
                           const int32_t* row_index, int32_t index_div, int64_t rows, const int32_t* group_offsets,
                           int32_t groups, uint8_t* codes, uint8_t* scales, int tiled, void* cuda_stream);

/* The values that codes [rows, K/2] with row-major scales [rows, K/32] stand
 * for: out [rows, K], bf16 or fp32 (both hold every value but those beyond
 * their range, which become infinities).  codes and out 16-byte aligned. */
int moe_fp4_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K, int out_type,
                             void* out, void* cuda_stream);

/* Bytes of the tiled scales of `rows` rows of K elements in `groups` groups
 * (1 when there are none): (rows / 128 + groups) ceil(K / 128) 512; 0 for
 * sizes moe_fp4_mxfp4_quantize rejects. */
size_t moe_fp4_mxfp4_tiled_scale_bytes(int64_t rows, int32_t groups, int32_t K);

/* Row-major scales [E, N, K/32] (the layer's w13_scale and w2_scale) in the
 * weights' layout of the products, once when weights are loaded: uint8
 * [E][ceil(N/128)][ceil(K/128)][512], tiles as above, zeros past the ends.
 * swiglu = 1: for a product with SwiGLU (N = 2I, gate rows then up rows), the
 * rows of a tile are gate and up rows in turn.  N at most 2^31 - 256; tiled
 * 16-byte aligned. */
int moe_fp4_mxfp4_tile_scales(const uint8_t* scales, int32_t E, int32_t N, int32_t K, int swiglu, uint8_t* tiled,
                              void* cuda_stream);

/* Sizes and form of a product: a has M rows, w is E matrices of N rows. */
typedef struct moe_fp4_mm_dims {
  int32_t M, N, K, E;   /* M >= 0, 1 <= N <= 2^31 - 256, K a multiple of 32 up to 32768, 1 <= E <= 1024 */
  int32_t swiglu;       /* 0: y [M, N]; 1: N = 2I even, y [M, I] = silu(first I features) * last I */
  int32_t y_type;       /* MOE_FP4_TYPE_BF16 or MOE_FP4_TYPE_F32 */
} moe_fp4_mm_dims;

/* y[m, n] = sum_K a[m, K] w_e[n, K] of MXFP4 matrices on block-scaled tensor
 * cores (tcgen05.mma kind::mxf4: products of codes and scales exact, fp32
 * sums, one rounding to y_type).
 *   a, a_scales  codes [M, K/2] and tiled scales of moe_fp4_mxfp4_quantize
 *   offsets      NULL (E = 1): all rows use the one matrix; else int32 [E + 1]
 *                on the device, not decreasing: rows [off[e], off[e+1]) use
 *                matrix e; empty groups are fine, rows in no group are not
 *                written.  a_scales are then in the grouped tiled layout.
 *   w, w_scales  codes [E, N, K/2], scales of moe_fp4_mxfp4_tile_scales
 * a, w, a_scales, w_scales 16-byte aligned, y aligned to its element.  A NaN
 * scale byte makes the results that it touches NaN.  The sums' order depends
 * on the sizes alone: the same call gives the same bits. */
int moe_fp4_mxfp4_matmul(const moe_fp4_mm_dims* dims, const uint8_t* a, const uint8_t* a_scales,
                         const int32_t* offsets, const uint8_t* w, const uint8_t* w_scales, void* y,
                         void* cuda_stream);

/* Device workspace of moe_fp4_mxfp4_linear (the codes and scales of the
 * quantised rows; 256-byte aligned base); 0 for unsupported sizes.  Products of
 * at most MOE_FP4_MXFP4_FEW_ROWS rows without offsets use none: it may be NULL. */
#define MOE_FP4_MXFP4_FEW_ROWS 16
size_t moe_fp4_mxfp4_linear_workspace_bytes(const moe_fp4_mm_dims* dims);

/* The same for a call that gathers its rows (row_index) from x_rows rows: with
 * this much, rows that are used several times are quantised once.  At least
 * moe_fp4_mxfp4_linear_workspace_bytes, which is enough too; the results are
 * the same. */
size_t moe_fp4_mxfp4_gathered_workspace_bytes(const moe_fp4_mm_dims* dims, int64_t x_rows);

/* The product from unquantised rows: moe_fp4_mxfp4_quantize of x (bf16 or
 * fp32, x_rows rows, stride x_stride; row_index / index_div as there, M output
 * rows), then moe_fp4_mxfp4_matmul.  The same bits as the two calls. */
int moe_fp4_mxfp4_linear(const moe_fp4_mm_dims* dims, const void* x, int x_type, int64_t x_rows, int64_t x_stride,
                         const int32_t* row_index, int32_t index_div, const int32_t* offsets, const uint8_t* w,
                         const uint8_t* w_scales, void* y, void* workspace, size_t workspace_bytes,
                         void* cuda_stream);

/* ---- Products with weights in 8-bit floating point ------------------------
 * E4M3 codes (OCP 8-bit, no infinities), one E8M0 scale for each 128 x 128 of a
 * weight matrix and for each 128 elements of a row of x, which is quantised in
 * the call: for 128 consecutive elements, with amax their largest magnitude,
 *   scale byte  s = e + 127, e the least integer >= -127 with amax <= 448 2^e
 *               (0 for an all-zero block)
 *   codes       E4M3 of x / 2^e, rounded to nearest (ties to the even code)
 * A block holding an infinity or a NaN becomes NaN.  K need not be a multiple
 * of 128: the last block of a row is then a shorter one. */

/* Weight scales [E, ceil(N/128), ceil(K/128)] in the product's layout, once when
 * weights are loaded: uint8 [E][ceil(N/128)][ceil(K/128)][512], tiles as for
 * MXFP4 with the same byte for the four times 32 elements of a block, zeros past
 * the end.  swiglu = 1: for a product with SwiGLU (N = 2I, gate rows then up
 * rows); N and K as in moe_fp4_mm_dims, tiled 16-byte aligned. */
int moe_fp4_fp8_tile_scales(const uint8_t* scales, int32_t E, int32_t N, int32_t K, int swiglu, uint8_t* tiled,
                            void* cuda_stream);

/* Device workspace of moe_fp4_fp8_linear (codes and scales of the quantised
 * rows; 256-byte aligned base); 0 for unsupported sizes.  None is used by at most
 * MOE_FP4_MXFP4_FEW_ROWS rows without offsets: it may be NULL. */
size_t moe_fp4_fp8_linear_workspace_bytes(const moe_fp4_mm_dims* dims);

/* y[m, n] = sum_K x_q[m, K] w_e[n, K], with SwiGLU, groups (offsets), sizes and y
 * as for moe_fp4_mxfp4_matmul: tcgen05.mma kind::mxf8f6f4, products of codes and
 * scales exact, fp32 sums, one rounding to y_type; the same call gives the same
 * bits.
 *   x         bf16 or fp32, x_rows >= M rows, row r at element r * x_stride
 *   w         E4M3 codes [E, N, K], 16-byte aligned
 *   w_scales  of moe_fp4_fp8_tile_scales, 16-byte aligned */
int moe_fp4_fp8_linear(const moe_fp4_mm_dims* dims, const void* x, int x_type, int64_t x_rows, int64_t x_stride,
                       const int32_t* offsets, const uint8_t* w, const uint8_t* w_scales, void* y, void* workspace,
                       size_t workspace_bytes, void* cuda_stream);

/* ---- Latent attention ------------------------------------------------------
 * Attention whose keys and values come from one latent vector a token (512
 * elements) and one rotary key that all heads share (64). */
#define MOE_FP4_LATENT_MAX_HEADS 1024

/* Absorbed form, one new token a sequence, over a paged cache of the latent
 * vectors: with c_j the 576 elements of token j of a sequence,
 *   s_j = scale q . c_j,   out = sum_j softmax(s)_j c_j[0 .. 511]
 * for j < lengths[b]; a sequence of no tokens gets zeros, a head whose scores are all
 * -infinity NaN.  fp32 scores,
 * statistics and sums; P is rounded to bf16 for its product, the result once to
 * bf16.  What the cache holds behind a sequence's end is not used, whatever it
 * is; its values up to there are to be finite (an infinity or a NaN reaches every
 * head of the sequence).  The same call gives the same bits; a sequence's last bits
 * depend on the lengths beside it.
 *   q        bf16 [B, H, 576] (latent part, rotary part), element strides
 *            q_stride and q_head_stride: multiples of 8, base 16-byte aligned
 *   cache    bf16 [pages, page, 576], contiguous, 16-byte aligned; page a multiple
 *            of 16 (64 and its multiples are read in one copy a tile)
 *   table    int32 [B, width], row stride table_stride: page of tokens [i page,
 *            (i + 1) page) of the sequence; entries behind its end are not read
 *   lengths  int32 [B], tokens in the cache (the new one included)
 *   out      bf16 [B, H, 512], contiguous, 16-byte aligned
 * A length below 0 or above width * page is taken as the nearest of the two, a page
 * outside the cache reads as zeros; both set error bit 1 (moe_fp4_ops_check).
 * pages * page and width * page below 2^31; scale finite. */
typedef struct moe_fp4_latent_decode_args {
  int32_t B, H, page, pages, width;  /* B 0 .. 2^24; H 1 .. 1024 */
  float scale;
  int64_t q_stride, q_head_stride, table_stride;
  const void *q, *cache;
  const int32_t *table, *lengths;
  void* out;
} moe_fp4_latent_decode_args;

/* Device workspace of moe_fp4_latent_decode (the pieces of sequences that several
 * SMs share; 256-byte aligned base), for the current device; 0 for unsupported
 * sizes.  It holds nothing between calls; calls that may overlap need one each. */
size_t moe_fp4_latent_decode_workspace_bytes(int32_t H);
int moe_fp4_latent_decode(const moe_fp4_latent_decode_args* args, void* workspace, size_t workspace_bytes,
                          void* cuda_stream);

/* Expanded form, for the new tokens of a ragged batch: sequence b has queries
 * [q_offsets[b], q_offsets[b+1]) and keys [k_offsets[b], k_offsets[b+1]) (those of
 * its cached tokens and of the new ones), nq and nk of them; for query i
 *   s_j = scale (q_i[0 .. 127] . kn_j + q_i[128 .. 191] . kr_j)
 *   out_i = sum_j softmax(s)_j v_j        over j < nk; causal: j <= i + nk - nq
 * for every head; a query that sees no key gets zeros (one whose scores are all
 * -infinity NaN, as the formula does), queries of no sequence are left as they were.  fp32 scores, statistics and sums; P is rounded to bf16 for
 * its product (not for sequences of at most 8 queries and 32 keys in batches of many
 * such, which have a kernel of their own), the result once to bf16.  Values (v) are to be
 * finite; what a sequence's neighbours hold does not reach it.  The same call gives the
 * same bits; a sequence's last bits depend on the sizes of the batch beside it.
 *   q         bf16 [Tq, H, 192], element strides q_stride, q_head_stride
 *   kv        bf16 [Tk, H, 256]: kn and v of a head side by side
 *   k_rope    bf16 [Tk, 64], the heads' shared rotary key kr
 *   q_offsets, k_offsets  int32 [B + 1] on the device, not decreasing, up to Tq and
 *             Tk: negative ones are taken as 0, INT32_MAX as the rows' end; decreasing
 *             ones and others behind the rows, taken as their end, set error bit 1
 *   out       bf16 [Tq, H, 128], contiguous
 * All bases 16-byte aligned, strides multiples of 8 elements; scale positive. */
typedef struct moe_fp4_latent_attention_args {
  int32_t B, H, causal;              /* B 0 .. 2^24; H 1 .. 1024 */
  float scale;
  int64_t Tq, Tk;
  int64_t q_stride, q_head_stride, kv_stride, kv_head_stride, rope_stride;
  const void *q, *kv, *k_rope;
  const int32_t *q_offsets, *k_offsets;
  void* out;
} moe_fp4_latent_attention_args;
/* Device workspace of moe_fp4_latent_attention (pieces of items that SMs share;
 * 256-byte aligned base), for the current device.  It holds nothing between calls;
 * calls that may overlap need one each. */
size_t moe_fp4_latent_attention_workspace_bytes(void);
int moe_fp4_latent_attention(const moe_fp4_latent_attention_args* args, void* workspace, size_t workspace_bytes,
                             void* cuda_stream);

/* Block tables and slots of a batch's new tokens in a paged cache.  Request b has
 * n = lengths[b] tokens in the cache and gets t = new_tokens[b] more; tokens are
 * numbered through in the requests' order.  The pages that its tokens n .. n + t - 1
 * need beyond its ceil(n / page) own ones are taken from free_pages, request after
 * request, and entered in its row of the table.
 *   slots      int64 [tokens]: table page * page + place in it, of each new token
 *   positions  int32 [tokens]: n, n + 1, ...
 *   out_lengths int32 [B]: n + t, of which the tokens that have a place (below)
 *   q_offsets, k_offsets  int32 [B + 1]: where a request's new tokens, and all those
 *              of out_lengths, begin if they are laid side by side
 *   taken      int32: pages taken, the first ones of free_pages, each entered
 * A batch of fewer than `tokens` new tokens (a padded one) gets slot -1 and position
 * 0 behind its last.  Negative lengths (taken as 0), a request that its row of the
 * table does not hold, more new tokens than `tokens`, too few free pages, and a negative
 * page in free_pages or in the table, where a new token lies in it, set error
 * bit 1 (moe_fp4_ops_check).  Tokens without a place get slot -1 and, but for those in a
 * negative page, are not counted in out_lengths and k_offsets: a later call may place
 * them, and nobody reads what a row of the table held behind its request.  (Beside its
 * queries, all of the new tokens, such a request then has fewer keys.)  The outputs
 * overlap no input; table is written in place. */
typedef struct moe_fp4_page_slots_args {
  int32_t B, page, width;            /* B 0 .. 8192, width * page below 2^31 */
  int64_t tokens, free_count, table_stride;
  const int32_t *lengths, *new_tokens, *free_pages;
  int32_t* table;                    /* [B, width], row stride table_stride */
  int64_t* slots;
  int32_t *positions, *out_lengths, *q_offsets, *k_offsets, *taken;
} moe_fp4_page_slots_args;
int moe_fp4_page_slots(const moe_fp4_page_slots_args* args, void* cuda_stream);

/* The end of a block in one pass over its rows.  With b = y (+ y2):
 *   post_norm:  b = b * rsqrt(mean(b^2) + eps)
 *   b = b * post_weight                      (NULL: 1)
 *   b = b * gate, or * sigmoid(gate)         (gate_shape: none, [T], [d], [T, d])
 *   out = residual + scale * b               (residual_type)
 *   normed = out * rsqrt(mean(out^2) + eps) * next_weight   (bf16; NULL weight: 1)
 * in fp32, each result rounded once (normed is of the unrounded sum).  y NULL:
 * normed = the norm of residual alone (the norm before a block); out, if
 * given, is then a copy of residual.  out may be residual itself; otherwise
 * outputs overlap no input.  normed NULL: no next norm.  Rows are T of d
 * elements, row t of an operand at element t * its stride (>= d); out and
 * normed are contiguous unless out is residual itself with its stride. */
#define MOE_FP4_GATE_NONE 0
#define MOE_FP4_GATE_TOKEN 1    /* [T] */
#define MOE_FP4_GATE_CHANNEL 2  /* [d] */
#define MOE_FP4_GATE_ELEMENT 3  /* [T, d], gate_stride */
typedef struct moe_fp4_block_norm_args {
  int64_t T;                    /* >= 0; 0 enqueues nothing */
  int32_t d;                    /* 1 .. 16384 */
  int32_t post_norm, gate_shape, gate_sigmoid;
  int32_t residual_type, y_type, y2_type, gate_type, post_weight_type, next_weight_type;
  int64_t residual_stride, y_stride, y2_stride, gate_stride, out_stride;
  float scale, eps;             /* eps >= 0 */
  const void *residual, *y, *y2, *gate, *post_weight, *next_weight;
  void *out, *normed;
} moe_fp4_block_norm_args;
int moe_fp4_block_norm(const moe_fp4_block_norm_args* args, void* cuda_stream);

/* Synchronises the stream and takes the errors of the operators above on the
 * current device: 1 = a row index out of range, 2 = a pipeline wait gave up
 * after 2 s (results incomplete).  Returns MOE_FP4_OK, MOE_FP4_ERR_DEVICE or
 * MOE_FP4_ERR_CUDA.  The error words are one set for all streams and threads of
 * a device: a check reports what calls on any of them have raised so far, and
 * each error is reported by one check, so that callers who share a device
 * share its checks too.  Not during a stream capture. */
int moe_fp4_ops_check(void* cuda_stream);

/* Fault injection, for tests of the failure path only (the layer's own
 * failure handling: every pipeline wait in the kernels is bounded, and a wait
 * that runs out sets bit 2 of the device error word, releases the kernel's
 * other roles, lets every copy and MMA in flight finish, frees tensor memory
 * and returns).  While a site other than MOE_FP4_FAULT_NONE is set, every
 * later moe_fp4_forward* call in this process, from any thread, plants the
 * fault on the host's instruction, and every pipeline wait gives up after
 * wait_limit_us microseconds instead of 2 s:
 *   MOE_FP4_FAULT_TC_TOKEN_TILE   the tensor-core W13 kernel's first CTA never
 *                                 loads its first token tile (in
 *                                 moe_fp4_forward_mx: the block-scaled W13
 *                                 kernel's first CTA never loads its first
 *                                 stage);
 *   MOE_FP4_FAULT_STREAM_STAGE    the streaming W13 kernel's first CTA never
 *                                 loads its first weight stage.
 * Nothing faults, traps or hangs: the waiting threads give up, the outputs of
 * that call are incomplete, and moe_fp4_check reports MOE_FP4_ERR_DEVICE.
 * The products (moe_fp4_mxfp4_matmul, moe_fp4_mxfp4_linear, moe_fp4_fp8_linear)
 * and latent attention take MOE_FP4_FAULT_TC_TOKEN_TILE too (the first CTA, or
 * pair, never loads its first stage; moe_fp4_ops_check reports it), and the limit; so does moe_fp4_block_norm
 * in its form for many rows (the first CTA never loads its first row).
 * MOE_FP4_FAULT_NONE (wait_limit_us ignored) restores normal operation.
 * Returns MOE_FP4_ERR_INVALID_ARG for an unknown site or a zero limit. */
#define MOE_FP4_FAULT_NONE 0
#define MOE_FP4_FAULT_TC_TOKEN_TILE 1
#define MOE_FP4_FAULT_STREAM_STAGE 2
int moe_fp4_set_fault_injection(int site, uint32_t wait_limit_us);

/* Synchronises the stream and reads the device error word of the workspace,
 * which the kernels OR bits into: 1 = an index out of range (e.g. a corrupted
 * expert id, whose slot is dropped); 2 = a pipeline wait gave up after 2 s
 * (the kernel skipped the rest of its work, so the outputs are incomplete).
 * Returns MOE_FP4_OK, MOE_FP4_ERR_DEVICE or MOE_FP4_ERR_CUDA, and clears the
 * word. */
int moe_fp4_check(void* workspace, void* cuda_stream);

/* Static text for a status code. */
const char* moe_fp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP4_H_ */

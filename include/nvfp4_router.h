/*
 * nvfp4_router.h -- C ABI of the MI355X (gfx950) NVFP4 dense-MoE router library
 * (libnvfp4_router.so).
 *
 * The path: runtime NVFP4 quantization of the activations, the block-scaled
 * gate projection to per-expert logits, and the fused six-step routing
 * epilogue. Sources are three commit pages of the nvfp4-megamoe-kernel
 * repository:
 *   - commit 04cf8ca8, dsv4/layers/router.py: runtime global scale
 *     gsa = max|x| / (6 * 448), the E4M3 block-scale ceiling of 448, the
 *     NVFP4 gate GEMM and the fused-router dispatch order;
 *   - commit e0f60b9f, dsv4/kernels/router/__init__.py: the six-step
 *     single-pass activation/top-k epilogue after the gate GEMM;
 *   - commit df05289d, dsv4/layers/grouped_linear.py: one flattened
 *     quantize launch with a device-only global scale, no host syncs and
 *     caller-owned pre-allocated buffers.
 * The NVFP4 format fixes the rest: 16-element blocks along the contraction
 * axis, E4M3 (OCP "FN", max 448) block scales, E2M1 element codes, one fp32
 * per-tensor global scale.
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; tensors
 *     are dense and row-major. The library allocates nothing and keeps no
 *     per-call state; it only enqueues work on `stream` (a hipStream_t, NULL
 *     for the default stream) and never synchronizes or copies to the host,
 *     so calls may be captured in a HIP graph.
 *   - A negative return value means the arguments were rejected on the host
 *     and nothing was enqueued, except ROUTER_EHIP (a launch failed).
 *   - Data pointers of an empty batch (rows or T == 0) may be NULL; the
 *     global scale output is still written (0, or the override).
 *   - Non-finite input values are a precondition violation: they make the
 *     global scale non-finite (the device-visible error flag) and leave the
 *     other outputs unspecified.
 *   - Calls that share one workspace must not overlap in time (enqueue them
 *     on one stream).
 *   - Tuning overrides, read once per process from the environment (results
 *     stay within the stated tolerances for any accepted value; invalid
 *     values are ignored): NVR_SPLIT_MAX_T (largest T on the 16x16-tile
 *     gate, default 256), NVR_MMA_BM (prefill tokens per workgroup: 32, 64
 *     or 128) with NVR_MMA_NTW (32-expert tiles per wavefront, 1..4). The
 *     workspace size follows the same settings, so set them before the first
 *     call and leave them.
 */
#ifndef NVFP4_ROUTER_H
#define NVFP4_ROUTER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ROUTER_OK 0
#define ROUTER_EINVAL (-1)       /* bad shape, null or misaligned pointer, workspace too small */
#define ROUTER_EUNSUPPORTED (-2) /* a documented size limit is exceeded */
#define ROUTER_EHIP (-3)         /* a kernel launch reported an error */
#define ROUTER_ESCRATCH (-4)     /* router_forward_noalloc: the call needs more than the static scratch */

#define ROUTER_MAX_EXPERTS 512
#define ROUTER_MAX_TOPK 32
#define ROUTER_MAX_GATE_D (1 << 22) /* largest hidden size of a gate call */
#define ROUTER_STATIC_SCRATCH_BYTES (16 << 20) /* router_forward_noalloc's scratch, per GPU */
#define ROUTER_WORKSPACE_STATE_BYTES (4096 + 131072) /* workspace prefix that stays zero between calls */

/*
 * Bytes of workspace that router_quantize and router_gate_topk need for a
 * call with these sizes (rows = T tokens, D hidden, E experts, k chosen).
 * One workspace sized by this function serves both calls. The caller
 * allocates it once, ahead of time, and reuses it for every call, so that no
 * call allocates or synchronizes and a decode loop can be captured in a
 * graph (commit df05289d, dsv4/layers/grouped_linear.py: the fixes that
 * pre-allocate the output buffer and the expert-offset range buffer once at
 * initialization instead of per call).
 *
 * The first ROUTER_WORKSPACE_STATE_BYTES bytes (arrival counters, then the
 * decode gate's flagged partials) must be zero before the first call
 * (allocate zero-filled memory or call router_workspace_init), and every call
 * leaves them zero again; the rest is per-call scratch. Every size this
 * function returns covers that state. Calls that share one workspace must be
 * ordered (one stream); concurrent calls need workspaces of their own.
 * Returns 0 for invalid sizes.
 */
size_t router_workspace_bytes(int64_t T, int64_t D, int64_t E, int64_t k);

/*
 * Zero-fills `bytes` of `workspace` on `stream` with a kernel (no memset
 * node, so it may be captured). Needed once per workspace allocation, at the
 * same initialization time as the allocation itself (the pre-allocated
 * buffers of commit df05289d, dsv4/layers/grouped_linear.py).
 * ROUTER_EINVAL if `workspace` is NULL or not 4-byte aligned, or `bytes` is
 * not a multiple of 4 (bytes == 0 does nothing).
 */
int router_workspace_init(void* workspace, size_t bytes, void* stream);

/*
 * Runtime NVFP4 quantization of x (the flattened single-launch quantizer
 * with a device-only global scale: commit df05289d,
 * dsv4/layers/grouped_linear.py; the scale rule: commit 04cf8ca8,
 * dsv4/layers/router.py, runtime-gsa paragraph).
 *
 *   x            [rows, D] bf16 bit patterns, 16-byte aligned.
 *   rows, D      rows >= 0, D >= 16, D % 16 == 0.
 *   gsa_override NULL: gsa = fp32(max|x|) / 2688 (one IEEE fp32 division).
 *                Else a device fp32 scalar used as gsa instead (reproduces a
 *                static scale; must be >= 0 and finite).
 *   codes        [rows, D/2] out: E2M1 codes, element 2i in the low nibble of
 *                byte i; each code is the E2M1 value nearest to
 *                |x| / (gsa * S) (ties to even, saturating at 6) with the
 *                sign bit of x. 8-byte aligned.
 *   scales       [rows, D/16] out: E4M3FN bytes; each is the E4M3 value nearest
 *                to bmax / (6 * gsa) over its 16-element block (ties to even,
 *                saturating at 448).
 *   gsa_out      [1] out: the global scale used (device fp32).
 * gsa == 0 gives zero scale bytes and sign-only codes. Every rounding is
 * exact (identical to the infinitely precise quotient's).
 *
 * Also used at load time on bf16 gate weights [E, D] (their gsa is gsw).
 */
int router_quantize(const void* x, int64_t rows, int64_t D, const float* gsa_override, uint8_t* codes,
                    uint8_t* scales, float* gsa_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gate projection plus the fused routing epilogue (gate GEMM on NVFP4
 * operands: commit 04cf8ca8, dsv4/layers/router.py; six-step epilogue:
 * commit e0f60b9f, dsv4/kernels/router/__init__.py).
 *
 *   x_codes, x_scales, gsa   router_quantize outputs for x [T, D].
 *   w_codes, w_scales, gsw   the gate weights in the same format, [E, D/2],
 *                            [E, D/16] and a device fp32 scalar.
 *   bias                     [E] fp32 selection bias.
 *   routed_scale             host fp32 factor applied after renormalization.
 *   T, D, E, k               T >= 0; 1 <= k <= E; D >= 16, D % 16 == 0
 *                            (ROUTER_EINVAL otherwise). The gate kernels
 *                            read K in 32-element chunks, so D % 32 != 0,
 *                            D > ROUTER_MAX_GATE_D, E > 512 and k > 32 give
 *                            ROUTER_EUNSUPPORTED.
 *   topk_idx                 [T, k] int32 out: experts by descending
 *                            s + bias, an exact tie going to the lower index.
 *   topk_w                   [T, k] fp32 out: routed_scale * s / sum(s) over
 *                            the chosen experts, s = sigmoid(logit).
 *   logits_out               NULL, or [T, E] fp32 out: the logits
 *                            gsa * gsw * sum_d xhat * what (fp32 accumulation).
 * Code and scale pointers must be 16- and 2-byte aligned.
 */
int router_gate_topk(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                     const uint8_t* w_scales, const float* gsw, const float* bias, float routed_scale, int64_t T,
                     int64_t D, int64_t E, int64_t k, int32_t* topk_idx, float* topk_w, float* logits_out,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * router_quantize followed by router_gate_topk, in one call and with the same
 * results: x_codes, x_scales and gsa_out are written exactly as
 * router_quantize writes them, and the routing is that of router_gate_topk on
 * them. For decode-size batches (T <= 4, D <= 16384) it is a single kernel
 * launch (the single-launch fused router that commit 04cf8ca8,
 * dsv4/layers/router.py, gives priority over the two-launch path): every
 * workgroup derives gsa from all of x and quantizes the blocks it multiplies
 * in registers. Batched decode (4 < T <= 256, D <= 16384) is two launches: a
 * pass that takes the partial maxima of x, then one kernel that quantizes,
 * multiplies and routes (each workgroup quantizes the x tile it multiplies).
 * Larger T runs the quantize kernels and then the gate kernels.
 *
 * Arguments as in the two calls above: x [T, D] bf16 (16-byte aligned);
 * x_codes (16-byte aligned), x_scales and gsa_out are outputs; the size
 * limits of router_gate_topk apply (ROUTER_EUNSUPPORTED beyond them).
 * The workspace must satisfy router_workspace_bytes(T, D, E, k).
 */
int router_forward(const void* x, int64_t T, int64_t D, const float* gsa_override, uint8_t* x_codes,
                   uint8_t* x_scales, float* gsa_out, const uint8_t* w_codes, const uint8_t* w_scales,
                   const float* gsw, const float* bias, float routed_scale, int64_t E, int64_t k, int32_t* topk_idx,
                   float* topk_w, float* logits_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * router_forward without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). It takes the same arguments as
 * router_forward minus the workspace and gives the same results from the same
 * kernels. Its scratch is a static device array of
 * ROUTER_STATIC_SCRATCH_BYTES (16 MiB) that each GPU the library runs on
 * holds until the process ends; the call itself allocates nothing and calls
 * no allocating routine. The first call on a device looks up that array's
 * address and enqueues one clear of its counters on `stream`.
 *
 * Calls whose router_workspace_bytes(T, D, E, k) exceeds 16 MiB (prefill
 * batches whose experts are split over workgroups with T * E * 4 above it,
 * e.g. T = 16384 at E = 256; batched-decode calls whose slice partials,
 * 4 * T * E * ceil(D / 256) bytes, exceed it, e.g. T = 256, D = 16384,
 * E = 512) return ROUTER_ESCRATCH before any launch;
 * invalid or unsupported sizes give router_forward's status. Every call on one
 * GPU shares that GPU's array: calls that overlap in time on one GPU (other
 * streams, other threads) race and give wrong results; enqueue them in order.
 */
int router_forward_noalloc(const void* x, int64_t T, int64_t D, const float* gsa_override, uint8_t* x_codes,
                           uint8_t* x_scales, float* gsa_out, const uint8_t* w_codes, const uint8_t* w_scales,
                           const float* gsw, const float* bias, float routed_scale, int64_t E, int64_t k,
                           int32_t* topk_idx, float* topk_w, float* logits_out, void* stream);

/*
 * Static text for a status code. The library reports every rejection as a
 * return value and never synchronizes to report one (the zero-host-sync rule
 * of commit df05289d, dsv4/layers/grouped_linear.py); this turns the value
 * into a message. Unknown codes give "unknown status".
 */
const char* router_status_string(int status);

/*
 * lm_head-shaped NVFP4 GEMV with a greedy (top-1) epilogue: for each of T
 * tokens, logits[t, n] = gsa * gsw * sum_d xhat[t, d] * what[n, d] (fp32
 * accumulation, the same arithmetic as the router's gate) over an N-row
 * vocabulary matrix, and the row with the largest logit (an exact tie going
 * to the lower row). The NVFP4 lm_head replaces a 1.8 GB BF16 weight (commit
 * df05289d, dsv4/layers/grouped_linear.py, weights paragraph); at decode
 * size the call streams the packed weights once.
 *
 *   x_codes, x_scales, gsa   router_quantize outputs for x [T, D] (16- and
 *                            2-byte aligned).
 *   w_codes, w_scales, gsw   the weights in the same format: [N, D/2],
 *                            [N, D/16] (16- and 2-byte aligned) and a device
 *                            fp32 scalar.
 *   T, D, N                  0 <= T <= 4; 32 <= D <= 16384, D % 32 == 0;
 *                            T * D <= 32768; 1 <= N <= 2^30.
 *   out_idx, out_logit       [T] int32 / fp32 out: the chosen row and its
 *                            logit.
 *   logits_out               NULL, or [T, N] fp32 out: every logit.
 *   workspace                256-byte aligned, lmhead_workspace_bytes(T, D,
 *                            N) bytes; its first
 *                            ROUTER_WORKSPACE_STATE_BYTES bytes are the state
 *                            shared with the router calls (zero between
 *                            calls, see router_workspace_bytes).
 * Returns ROUTER_EINVAL for bad shapes, pointers or workspace.
 */
size_t lmhead_workspace_bytes(int64_t T, int64_t D, int64_t N);
int lmhead_argmax(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                  const uint8_t* w_scales, const float* gsw, int64_t T, int64_t D, int64_t N, int32_t* out_idx,
                  float* out_logit, float* logits_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Group offsets of the grouped linear layer, on the device: offsets[g] =
 * range[g] * padded_rows for g = 0 .. G (G + 1 values), group g owning rows
 * offsets[g] .. offsets[g + 1] - 1 of the flattened activations. `range` is a
 * caller-owned device buffer of G + 1 int32 holding 0, 1, ..., G, filled once
 * at initialization and reused; computing the offsets from it on the device
 * is the fix of commit df05289d (dsv4/layers/grouped_linear.py, Section A
 * detector items 2 and 5) that removes the host loop, its per-group host
 * sync and the per-call allocation. One kernel launch on `stream`.
 *   1 <= G <= 2^24, padded_rows >= 0, G * padded_rows < 2^31; 4-byte aligned
 *   pointers; ROUTER_EINVAL otherwise.
 */
int grouped_offsets(const int32_t* range, int64_t G, int64_t padded_rows, int32_t* offsets, void* stream);

/*
 * Grouped NVFP4 GEMM (the grouped linear layer of commit df05289d,
 * dsv4/layers/grouped_linear.py): for every row r of group g,
 *   out[r, n] = gsa * gsw[g] * sum_d xhat[r, d] * what_g[n, d]
 * with fp32 accumulation over exact fp16 products (the gate's arithmetic).
 *
 *   x_codes, x_scales, gsa   router_quantize outputs for the flattened
 *                            activations of all groups, [R, D] (one launch,
 *                            one global scale: the pages' fused quantize
 *                            over (G * T, D)).
 *   w_codes, w_scales, gsw   the groups' weights, [G, N, D/2], [G, N, D/16]
 *                            (each group row-major (N, K_packed), as in the
 *                            checkpoint) and [G] fp32 device scales.
 *   offsets                  [G + 1] int32 device (e.g. from
 *                            grouped_offsets): 0 = offsets[0] <= ... <=
 *                            offsets[G] <= R. Values outside are clamped
 *                            (their rows are not defined).
 *   max_rows                 host bound on any group's row count; rows of a
 *                            group past max_rows are not computed. For the
 *                            padded layout it is padded_rows.
 *   out                      [R, N] fp32; rows of no group are not written.
 * Code pointers 16-byte, scale pointers 2-byte, the rest 4-byte aligned.
 * ROUTER_EINVAL for bad sizes or pointers; ROUTER_EUNSUPPORTED for D % 32 !=
 * 0, D > ROUTER_MAX_GATE_D or a grid beyond 2^31 workgroups. One launch on
 * `stream`, no workspace, no host sync: capturable. Decode-size groups
 * (max_rows <= 4, max_rows * D <= 32768, D <= 16384) run as a stream of the
 * weights with fp16 dot products on the VALU; larger groups on fp16 MFMA
 * tiles. Both give exact products and fp32 sums in a fixed order.
 */
int grouped_gemm(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                 const uint8_t* w_scales, const float* gsw, const int32_t* offsets, int64_t G, int64_t R,
                 int64_t max_rows, int64_t N, int64_t D, float* out, void* stream);

/*
 * The routed experts between the router's top-k and the next layer, on rows
 * sorted by expert: grouped_plan, then grouped_swiglu (gate and up
 * projections with the gated activation), router_quantize over its output,
 * and grouped_combine (down projection and the weighted sum per token). The
 * experts' sizes are ragged and stay on the device; every expert may have any
 * number of rows, none included. T tokens of k choices give R = T * k slots,
 * slot t * k + j being token t's j-th choice. An expert-parallel rank holds
 * the G experts first_expert .. first_expert + G - 1: slots of other experts
 * are left out, and the ranks' outputs add up to the layer's.
 *
 * Bytes of workspace for grouped_plan and grouped_combine with these sizes
 * (D: hidden size, the combined output's columns; F: the experts' inner
 * size); 0 for sizes that neither grouped_swiglu nor grouped_combine takes. A
 * layer of both needs D % 32 == 0 and F % 32 == 0. grouped_combine keeps
 * T * k * D fp32 products there, whatever share of the experts is held (7.5 GB
 * at T = 32768, k = 8, D = 7168). The workspace's state
 * prefix is the router calls' (see router_workspace_bytes); neither call
 * touches it.
 */
size_t grouped_workspace_bytes(int64_t T, int64_t k, int64_t G, int64_t D, int64_t F);

/*
 * Sorts the slots by expert, slots of one expert in slot order.
 *   topk_idx      [T, k] int32: router_gate_topk's choices (values outside
 *                 first_expert .. first_expert + G - 1, -1 for example, are
 *                 slots of no expert held here; a token may name an expert
 *                 twice).
 *   offsets       [G + 1] int32 out: expert first_expert + g owns rows
 *                 offsets[g] .. offsets[g + 1] - 1.
 *   rows          [T * k] int32 out: the slot of each row; -1 from offsets[G]
 *                 on.
 *   pos           [T * k] int32 out: the row of each slot; -1 for slots of no
 *                 expert held here.
 *   T, k, G       T >= 0, 1 <= k <= 32, 1 <= G <= 512, T * k < 2^30
 *                 (ROUTER_EUNSUPPORTED beyond the upper bounds);
 *                 first_expert >= 0.
 * Pointers 4-byte aligned, the workspace 256-byte aligned (needed for more
 * than 4096 slots). One launch up to 4096 slots, two beyond.
 */
int grouped_plan(const int32_t* topk_idx, int64_t T, int64_t k, int64_t first_expert, int64_t G, int32_t* offsets,
                 int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gate and up projections of the sorted rows with the SwiGLU activation: for
 * row p of expert g, with t = rows[p] / k,
 *   y[n] = gsa * gsw[g] * sum_d xhat[t, d] * what_g[n, d] + bias[g, n],  n < 2F
 *   out[p, f] = bf16(silu(y[f]) * y[F + f]),  silu(v) = v / (1 + e^-v)
 * with exact products and fp32 sums; rows from offsets[G] on are set to zero,
 * so that router_quantize over all T * k rows sees no stale values.
 *   x_codes, x_scales, gsa   router_quantize outputs for x [T, D] (not
 *                            gathered: the rows are read through `rows`).
 *   w_codes, w_scales, gsw   [G, 2F, D/2], [G, 2F, D/16], [G] fp32: each
 *                            expert's F gate rows, then its F up rows.
 *   bias                     NULL or [G, 2F] fp32.
 *   offsets, rows            grouped_plan's. Values that no plan gives are
 *                            clamped (their rows are not defined).
 *   F, D                     F >= 16, F % 16 == 0; D % 32 == 0; D and 2F at
 *                            most ROUTER_MAX_GATE_D; T * D / 2 and F * D
 *                            below 2^31 - 65536 (ROUTER_EUNSUPPORTED
 *                            otherwise).
 *   out                      [T * k, F] bf16.
 * Code pointers and out 16-byte, x_scales 2-byte, the rest 4-byte aligned. No
 * workspace.
 */
int grouped_swiglu(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                   const int32_t* rows, int64_t T, int64_t k, int64_t G, int64_t F, int64_t D, void* out,
                   void* stream);

/*
 * Down projection of the sorted rows and the weighted sum of each token's
 * rows, in slot order:
 *   y[p, n] = gsh * gsw[g] * sum_f hhat[p, f] * what_g[n, f] + bias[g, n]
 *   out[t, n] = bf16(residual[t, n] + sum_j topk_w[t, j] * y[pos[t, j], n])
 * over the j with pos[t, j] >= 0 (weights of other slots are not read); a
 * token without any gets its residual, or zeros. fp32 until the one rounding.
 *   h_codes, h_scales, gsh   router_quantize outputs for grouped_swiglu's
 *                            output [T * k, F].
 *   w_codes, w_scales, gsw   [G, D, F/2], [G, D, F/16], [G] fp32.
 *   bias                     NULL or [G, D] fp32.
 *   offsets, pos             grouped_plan's.
 *   topk_w                   [T, k] fp32: router_gate_topk's weights.
 *   residual                 NULL or [T, D] bf16; may be `out` itself.
 *   out                      [T, D] bf16.
 *   D, F                     D >= 16, D % 16 == 0; F % 32 == 0; both at most
 *                            ROUTER_MAX_GATE_D, D * F / 2 below 2^31 - 65536
 *                            (ROUTER_EUNSUPPORTED otherwise).
 *   workspace                grouped_workspace_bytes(T, k, G, D, F) bytes.
 * Code pointers, residual and out 16-byte, h_scales 2-byte, workspace
 * 256-byte, the rest 4-byte aligned.
 */
int grouped_combine(const uint8_t* h_codes, const uint8_t* h_scales, const float* gsh, const uint8_t* w_codes,
                    const uint8_t* w_scales, const float* gsw, const float* bias, const int32_t* offsets,
                    const int32_t* pos, const float* topk_w, const void* residual, int64_t T, int64_t k, int64_t G,
                    int64_t D, int64_t F, void* out, void* workspace, size_t workspace_bytes, void* stream);

#define ROUTER_F32 0  /* dtype of logits */
#define ROUTER_BF16 1

/*
 * Repetition, frequency and presence penalties, token biases and a grammar
 * mask on logits, and the greedy token: the constrained form of
 * lmhead_argmax's choice, on its logits_out or any others. For row t, in
 * fp32, each operation rounded by itself and in this order:
 *   tokens in history[t, :lengths[t]]:     x = x > 0 ? x / r : x * r
 *   tokens that occur c > 0 times in
 *   history[t, prompt[t]:lengths[t]]:      x = (x - f * c) - p
 *   tokens listed in the row's biases:     x = x + value
 *   tokens whose mask bit is clear:        x = -inf, whatever x is
 * The token with the largest x (a tie going to the lower one, -inf and NaN
 * never chosen) is the row's choice, made before the logits are rounded to
 * their type.
 *   logits, out    [T, N] of `dtype`, `ld` and `ld_out` >= N elements between
 *                  rows; out may be logits itself (with the same stride), and
 *                  must not overlap it otherwise.
 *   history        NULL or [T, L] int32 with ld_history >= L elements
 *                  between rows; tokens outside [0, N) are ignored.
 *   lengths        NULL (every row has L) or [T] int32, clamped to [0, L].
 *   prompt         NULL (0) or [T] int32: tokens before it count as seen
 *                  only, from it on also as made.
 *   repetition, frequency, presence   NULL (1, 0, 0) or [T] fp32: r, f, p.
 *   bias_start     NULL or [T + 1] int32: row t's biases are entries
 *                  bias_start[t] .. bias_start[t + 1] - 1 of bias_token
 *                  (int32) and bias_value (fp32), nbias entries in all
 *                  (starts are clamped to [0, nbias], an end before its start
 *                  is no entry, tokens outside [0, N) are ignored). A token
 *                  listed twice in a row takes its last value.
 *   mask           NULL or [T, ld_mask] 32-bit words, ld_mask >= N / 32
 *                  rounded up: bit n % 32 of word n / 32 is set where token n
 *                  is allowed.
 *   out_idx, out_logit   [T] int32 / fp32 out: the choice and its x; -1 and
 *                  -inf when nothing can be chosen.
 *   T, N           T >= 0, 1 <= N <= 2^30.
 *   workspace      lmhead_penalize_workspace_bytes(T, N) bytes, 256-byte
 *                  aligned, with the router calls' state prefix (not needed
 *                  for N <= 4096).
 * The other pointers are aligned to their element; 16-byte aligned rows of
 * logits and out are read and written 16 bytes at a time. One launch for each
 * 1024 rows. ROUTER_EINVAL for bad sizes, pointers or workspace.
 */
size_t lmhead_penalize_workspace_bytes(int64_t T, int64_t N);
int lmhead_penalize(const void* logits, int dtype, int64_t T, int64_t N, int64_t ld, const int32_t* history,
                    int64_t L, int64_t ld_history, const int32_t* lengths, const int32_t* prompt,
                    const float* repetition, const float* frequency, const float* presence,
                    const int32_t* bias_start, const int32_t* bias_token, const float* bias_value, int64_t nbias,
                    const uint32_t* mask, int64_t ld_mask, void* out, int64_t ld_out, int32_t* out_idx,
                    float* out_logit, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Losses of the lm_head over its whole vocabulary, with the gradient of x: z[t,
 * n] = gsa * gsw * sum_d xhat[t, d] * what[n, d], lmhead_argmax's logits. A loss
 * alone keeps T x N / 8 to / 4 bytes of sums and no logits. The gradient keeps its
 * softmax weights, fp16 [T, piece], for a piece of the vocabulary at a time:
 * 512 MB of them or 4096 columns, whichever is more, so up to T = 2^28 / N rows
 * that is all of T x N; beside them sums of [T, D] in fp32, for up to 256 splits
 * of a piece where tiles are few, and 8.2 KB for each row's named tokens.
 *
 * lmhead_loss, the cross entropy (the negative log-probability of a token):
 *   lse[t] = log sum_n e^z[t, n];  loss[t] = lse[t] - z[t, targets[t]]
 *   dx[t, d] = weight[t] * gsw * sum_n (e^(z[t, n] - lse[t]) - [n = targets[t]]) * what[n, d]
 * A target outside [0, N) (-100, for example) gives loss 0 and a gradient of
 * zeros.
 *
 * lmhead_distill, the divergence from a teacher of which K logits per token
 * are known, at a temperature tau:
 *   lse[t] = log sum_n e^(z[t, n] / tau)
 *   logq[t, j] = z[t, tokens[t, j]] / tau - lse[t]
 *   p[t, j] = softmax over j of teacher[t, j] / tau
 *   loss[t] = tau^2 * sum_j p[t, j] * (log p[t, j] - logq[t, j])
 *   dx[t, d] = weight[t] * gsw * tau * sum_n (e^(z[t, n] / tau - lse[t]) - sum_{j: tokens[t, j] = n} p[t, j]) * what[n, d]
 * Places whose token is outside [0, N) are left out whatever their teacher's
 * logit is, and have logq 0; -infinity is p = 0; a row without any place, or
 * with -infinity alone, has loss 0 and a gradient of zeros. A token may be
 * named more than once. Teacher logits of NaN or +infinity make their row's
 * loss and gradient NaN.
 *
 * A row with a logit of NaN or +infinity anywhere in the vocabulary has lse
 * NaN, and with it its loss and gradient, but for the zeros of ignored targets
 * and of rows without any place.
 *
 * dx is the gradient of sum_t weight[t] * loss[t] with respect to the
 * dequantized x (the quantization of x passes it through); the 4-bit weights
 * have none.
 *   x_codes, x_scales, gsa   router_quantize outputs for x [T, D] (16- and
 *                            2-byte aligned).
 *   w_codes, w_scales, gsw   the weights in the same format: [N, D/2],
 *                            [N, D/16] (16- and 4-byte aligned). Where N and
 *                            D/32 are odd the word that holds the last two
 *                            scales is read whole, 2 bytes past them.
 *   targets                  [T] int32.
 *   tokens, teacher          [T, K] int32 and [T, K] of `dtype`.
 *   temperature              2^-20 to 2^20.
 *   weight                   NULL (1) or [T] fp32; for dx alone.
 *   T, D, N, K               T >= 0; D >= 32, D % 32 == 0; N, K >= 1
 *                            (ROUTER_EINVAL otherwise); T >
 *                            ROUTER_MAX_LOSS_ROWS, D > ROUTER_MAX_GATE_D, N >
 *                            2^30 and K > ROUTER_MAX_TEACHER give
 *                            ROUTER_EUNSUPPORTED.
 *   loss, lse, logq          [T], [T], [T, K] fp32 out.
 *   dx                       NULL (no gradient) or [T, D] bf16 out (16-byte
 *                            aligned).
 *   workspace                lmhead_loss_workspace_bytes(T, D, N, dx != NULL)
 *                            bytes, 256-byte aligned, for either call; its
 *                            state prefix (see router_workspace_bytes) is not
 *                            touched. 0 for sizes that the calls refuse. A
 *                            workspace made for T rows takes every call with
 *                            fewer, one made for the gradient also those
 *                            without it.
 * Products are exact with fp32 sums in a fixed order, so results repeat bit for
 * bit. A named token's logit is the one that the sum over the vocabulary has in
 * it: no probability is above 1, no logq above 0 and no cross entropy below 0,
 * at any temperature. z / tau is rounded to 24 bits, an absolute error of
 * |z / tau| 2^-24 in each exponent beside that of the sum over D. In dx the
 * columns' softmax weights are rounded to 11 bits, those of the named tokens to
 * 24, and dx to bf16 at the end.
 */
#define ROUTER_MAX_LOSS_ROWS (1 << 18)
#define ROUTER_MAX_TEACHER 1024
size_t lmhead_loss_workspace_bytes(int64_t T, int64_t D, int64_t N, int grad);
int lmhead_loss(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                const uint8_t* w_scales, const float* gsw, const int32_t* targets, const float* weight, int64_t T,
                int64_t D, int64_t N, float* loss, float* lse, void* dx, void* workspace, size_t workspace_bytes,
                void* stream);
int lmhead_distill(const uint8_t* x_codes, const uint8_t* x_scales, const float* gsa, const uint8_t* w_codes,
                   const uint8_t* w_scales, const float* gsw, const int32_t* tokens, const void* teacher, int dtype,
                   int64_t K, float temperature, const float* weight, int64_t T, int64_t D, int64_t N, float* loss,
                   float* lse, float* logq, void* dx, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Routing on given logits: the rules of choice beside router_gate_topk's own
 * (which is ROUTER_SIGMOID with a bias, one group and renormalised weights,
 * fused behind the gate). For row t, with s = sigmoid(l) or softmax(l) over the
 * E logits l and key = s + bias:
 *   - the experts form `groups` groups of E / groups neighbours; a group's
 *     score is the sum of its group_top (1 or 2) largest keys, and experts
 *     outside the topk_groups groups with the largest scores (a tie going to
 *     the larger logit where a score is one key, then to the lower group) are
 *     left out;
 *   - topk_idx [T, k] int32: the k largest keys among the rest, in descending
 *     order, a tie going to the larger logit, then to the lower expert;
 *   - topk_w [T, k] fp32: routed_scale * s / (renormalize ? sum of the chosen
 *     s : 1), the bias left out.
 * The order is that of keys computed in 64 bits; with the ties' rule that is the
 * logits' own order wherever there is no bias, or the same one for all, also
 * where scores saturate (sigmoid logits of 40 and 50). An expert whose logit is
 * -infinity or NaN, or whose key is, is never chosen (it counts as -infinity
 * in its group); where fewer than k remain, the places left hold -1 and weight
 * 0, which grouped_plan takes as slots of no expert. Renormalised weights hold
 * for any finite logits, however small their s. A bias of +infinity puts its
 * experts before all others. A logit of +infinity makes its row's softmax
 * scores NaN: weights of NaN where the logits decide alone, and nothing chosen
 * where the order needs keys (with a bias, or groups by two keys).
 *   logits        [T, E] of `dtype`, ld >= E elements between rows.
 *   bias          NULL or [E] fp32.
 *   scoring       ROUTER_SIGMOID or ROUTER_SOFTMAX.
 *   T, E, k       T >= 0; 1 <= k <= topk_groups * (E / groups); E % groups == 0;
 *                 1 <= topk_groups <= groups (ROUTER_EINVAL otherwise); T >
 *                 ROUTER_MAX_SELECT_ROWS, E > 512, k > 32 and groups >
 *                 ROUTER_MAX_GROUPS give ROUTER_EUNSUPPORTED.
 * Pointers are aligned to their element. One launch, no workspace.
 */
#define ROUTER_SIGMOID 0
#define ROUTER_SOFTMAX 1
#define ROUTER_MAX_GROUPS 64
#define ROUTER_MAX_SELECT_ROWS (1 << 25)
int router_select(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, int scoring,
                  int64_t groups, int64_t topk_groups, int64_t group_top, int renormalize, float routed_scale,
                  int64_t k, int32_t* topk_idx, float* topk_w, void* stream);

/*
 * The gradient of router_select's logits, grad_logits [T, E] of the logits'
 * type, from that of its weights, grad_w [T, k] fp32, for the choice topk_idx
 * (places outside [0, E) are left out, whatever their grad_w; an expert named
 * twice takes part twice). The choice itself has no gradient, and so the bias
 * and the groups have none. Rows are written whole, with ld_grad >= E
 * elements between them; grad_logits must not overlap the logits. Without
 * renormalisation softmax scores give every expert a gradient, otherwise the
 * chosen ones alone have one. fp32 until the one rounding.
 */
int router_select_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const int32_t* topk_idx,
                           const float* grad_w, int scoring, int renormalize, float routed_scale, int64_t k,
                           void* grad_logits, int64_t ld_grad, void* stream);

/*
 * Measurement aid, not part of the router path: reads `bytes` of `buf`
 * (device, 16-byte aligned, bytes % 16 == 0) once with 16-byte loads in one
 * launch of min(bytes / 4096 rounded up, sink_words, 8192) workgroups of 256
 * threads, and stores one XOR of the data per workgroup into `sink` (device,
 * sink_words >= 1 words). Its duration is the time a kernel needs just to
 * read that footprint, against which the gate kernels' rates are read
 * (HBM bandwidth at a gigabyte; launch and cache latency at the decode
 * gate's megabyte). Returns ROUTER_EINVAL for bad arguments.
 */
int router_probe_read(const void* buf, size_t bytes, uint32_t* sink, size_t sink_words, void* stream);

/*
 * Measurement aid, not part of the router path: 1024 workgroups of 256
 * threads (four wavefronts per SIMD on 256 compute units) each run `iters`
 * rounds of four independent 32x32x16 fp16 MFMA chains with no memory
 * traffic, then store one float per thread into `sink` (device, at least
 * 262144 floats). Its duration gives the fp16 MFMA rate the chip sustains at
 * its running clock: 1024 * 4 * iters * 4 * 32768 FLOP per launch. 1 <= iters
 * <= 2^24; ROUTER_EINVAL otherwise.
 */
int router_probe_mfma(int64_t iters, float* sink, size_t sink_floats, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ROUTER_H */

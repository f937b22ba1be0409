/*
 * mxfp4_moe.h -- C ABI of the routed-expert MXFP4 mixture-of-experts layer
 * for one NVIDIA GB300 GPU (sm_103a).
 *
 * The layer reads each expert's weights in the served packed layout
 * ("MXFP4 MoE decode kernels", Design, "Read the served layout"):
 *   w13  uint8 [E, 2I, K/2]   two E2M1 values per byte, low nibble first
 *   s13  uint8 [E, 2I, K/32]  one E8M0 scale per 32 values along K
 *   w2   uint8 [E, K, I/2]
 *   s2   uint8 [E, K, I/32]
 * and computes, for every token t and slot j of its top-k routing,
 *   g, u = split([gate; up] rows of dequant(w13[e])) . x_t     (fp32 accumulate)
 *   h    = bf16( silu(g) * u )                                  (one bf16 rounding)
 *   o    = dequant(w2[e]) . h                                   (fp32 accumulate)
 *   y_t  = bf16( sum_{j=0..k-1} w_tj * o_(t,j) )                (slot order)
 * where dequant(v) = E2M1(nibble) * 2^(E8M0 - 127) ("GLM-5.2 and GLM-5.3 (744B)
 * in MXFP4 on Gaudi 2", What was built, "Byte-exact repack"; "MXFP4 MoE decode
 * kernels", Design, "Unpack in registers" and "Fused epilogues"; Beyond
 * gpt-oss, "mxk_w13x: SiLU without bias for [gate; up] row layouts").
 *
 * Conventions shared by every entry point:
 *  - Every pointer argument is a DEVICE pointer owned by the caller (for
 *    example a PyTorch CUDA tensor's data_ptr()), unless it is marked "host".
 *    The library never allocates device memory, never frees, and never
 *    synchronises the device: each call validates its arguments on the host,
 *    enqueues its kernels on `stream` (a cudaStream_t passed as void*, NULL =
 *    the legacy default stream) and returns.
 *  - A non-zero return value is an mxfp4_moe_status code and means nothing
 *    was enqueued (except MXFP4_MOE_ERR_CUDA, which reports a failed launch).
 *  - Conditions only the device can see are written to `status` (device
 *    int32[4]) by the enqueued work:
 *       status[0] = number of routes whose expert id is >= E (skipped)
 *       status[1] = number of distinct experts touched by the call
 *       status[2] = non-zero when a bounded wait inside a kernel gave up (the
 *                   output of that call is then not valid; never expected);
 *                   the bits name the wait: bits 0..7 the decode kernel's
 *                   producer, 8..15 its consumers, 16..23 the prefill path's
 *                   first GEMM, 24..31 its second. The workspace stays
 *                   usable after such a call: the decode kernel's last CTA
 *                   resets its counters on every exit path, and the prefill
 *                   path keeps no state in the workspace between calls
 *       status[3] = 1 + the first CTA that reported such a wait, else 0
 *    Negative expert ids are padding and are skipped silently.
 *  - Every call is deterministic: repeating it on the same inputs gives
 *    bit-identical outputs (no floating-point atomics anywhere).
 */
#ifndef MXFP4_MOE_H_
#define MXFP4_MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MXFP4_MOE_OK = 0,
  MXFP4_MOE_ERR_ARG = 1,        /* null pointer where one is required, negative size */
  MXFP4_MOE_ERR_SHAPE = 2,      /* shape outside the supported limits listed below */
  MXFP4_MOE_ERR_ALIGN = 3,      /* a pointer breaks its alignment rule */
  MXFP4_MOE_ERR_WORKSPACE = 4,  /* workspace missing or smaller than mxfp4_moe_workspace_size */
  MXFP4_MOE_ERR_CUDA = 5,       /* a CUDA runtime call failed (device query or launch) */
  MXFP4_MOE_ERR_DEVICE = 6      /* current device is not an sm_103 GPU */
} mxfp4_moe_status;

/* Shape limits (checked on the host, MXFP4_MOE_ERR_SHAPE otherwise):
 *   K % 32 == 0, I % 32 == 0, 32 <= K, I <= 16384
 *   1 <= E <= 1024, 1 <= topk <= 32, topk <= E, 0 <= T
 *   decode path: T <= 32, T * topk <= 1024, K % 64 == 0, I % 64 == 0 (scale
 *                rows are copied 8 rows at a time) and the kernel's shared-memory
 *                plan must fit: about 12 * max(K, I) + 20 * E + 2 * max(K, I)
 *                + 66 KB <= 227 KB (K, I <= 8192 always fit for E <= 256)
 *   prefill path: K % 64 == 0, I % 64 == 0 (tensor-core tiles), T * topk < 2^31 / K
 * Alignment (MXFP4_MOE_ERR_ALIGN otherwise): w13, s13, w2, s2, hidden and out
 * 16-byte aligned; workspace 256-byte aligned. */

/* Bytes of device workspace a forward call with these sizes needs (either
 * path). The bookkeeping part (the first mxfp4_moe_workspace_zero_bytes()
 * bytes) must be zero before the first call that uses a workspace; every call
 * leaves it zero again (also one whose bounded wait gave up), so a workspace
 * can be reused without clearing. Returns 0 for invalid sizes. */
size_t mxfp4_moe_workspace_size(int T, int K, int I, int E, int topk);

/* Bytes at the start of every workspace that hold the bookkeeping: they must
 * be zero before the first call (clearing only them is enough) and every call
 * leaves them zero. The same for all sizes (a few KB), so a workspace
 * sized for the largest call serves calls of any smaller size. */
size_t mxfp4_moe_workspace_zero_bytes(void);

/* Routing / permute ("MXFP4 MoE decode kernels", Design, "Routing inside the
 * kernel": a counting sort of the routes by expert; absent experts skipped).
 * Route r = t * topk + j. Outputs:
 *   expert_count  int32 [E]     routes per expert
 *   expert_offset int32 [E+1]   exclusive prefix sum, expert_offset[E] = valid routes
 *   route_list    int32 [T*topk] route ids grouped by expert in ascending
 *                 expert order, ascending r inside a group; entries past
 *                 expert_offset[E] are set to -1
 *   status        int32 [4]     as above (may be NULL)
 * topk_ids int32 [T, topk]. No workspace needed. */
int mxfp4_moe_route(const int32_t* topk_ids, int T, int topk, int E,
                    int32_t* expert_count, int32_t* expert_offset, int32_t* route_list,
                    int32_t* status, void* stream);

/* The same routing with device scratch for many routes: identical outputs
 * (bit for bit) to mxfp4_moe_route. From 8192 routes on it sorts over many
 * CTAs -- per-chunk expert counts, one prefix pass, an in-order placement per
 * chunk -- which is the form the prefill path runs; fewer routes take the
 * one-CTA sort. workspace: device memory of at least
 * mxfp4_moe_route_workspace_size(T, topk, E) bytes, 16-byte aligned
 * (MXFP4_MOE_ERR_WORKSPACE / MXFP4_MOE_ERR_ALIGN), no initial contents
 * required, not shared by calls that may run concurrently. Other arguments,
 * limits and errors as mxfp4_moe_route. */
size_t mxfp4_moe_route_workspace_size(int T, int topk, int E);
int mxfp4_moe_route_ws(const int32_t* topk_ids, int T, int topk, int E,
                       int32_t* expert_count, int32_t* expert_offset, int32_t* route_list,
                       int32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/* Router: the step before routing ("MXFP4 MoE decode kernels", Design, "Routing
 * inside the kernel" takes its top-k ids; the workload shapes fix the
 * scoring). Per token t:
 *   x_e = fp32(logits[t][e] + bias[e])   (bias may be NULL: x_e = logits[t][e];
 *                                          a NaN x ranks as -inf)
 *   topk_ids[t][0..k-1]  the k largest x in descending order, ties to the
 *                        lower expert index (sigmoid is increasing, so this is
 *                        also the top-k by sigmoid score)
 *   topk_weights[t][j]   scoring 0 ("softmax_topk"): exp(x_j - x_0) / sum over
 *                        the chosen; scoring 1 ("sigmoid_renorm"): sigmoid(x_j)
 *                        / sum of the chosen sigmoids; fp32
 *   logits fp32 [T, E], bias fp32 [E] or NULL, topk_ids int32 [T, k],
 *   topk_weights fp32 [T, k]: device pointers owned by the caller, 4-byte
 *   aligned (MXFP4_MOE_ERR_ALIGN). Limits: 1 <= E <= 1024, 1 <= k <= min(32, E),
 *   0 <= T (MXFP4_MOE_ERR_SHAPE); scoring 0 or 1 and non-NULL logits/outputs
 *   (MXFP4_MOE_ERR_ARG). T == 0 enqueues nothing. The outputs feed
 *   mxfp4_moe_forward directly. */
int mxfp4_moe_router(const float* logits, const float* bias, int T, int E, int topk, int scoring,
                     int32_t* topk_ids, float* topk_weights, void* stream);

/* Router with grouped top-k and a choice of what the bias moves ("GLM-5.2 and
 * GLM-5.3 (744B) in MXFP4 on Gaudi 2", Why it needed a port, item 4, names
 * grouped top-k without defining it). As mxfp4_moe_router, plus:
 *   n_group       the E experts form n_group equal groups of consecutive ids
 *                 (group of e = e / (E / n_group)); a group's score is its
 *                 largest x; only the topk_group highest-scoring groups (ties
 *                 to the lower group index) stay eligible, and the k largest x
 *                 among their experts are chosen as above. n_group = 1 is the
 *                 plain router.
 *   bias_in_weights  1: the weights use x (the bias moves selection and
 *                 weights, as mxfp4_moe_router); 0: the bias steers the
 *                 choice only, the weights use the chosen experts' unbiased
 *                 logits (a NaN logit as -inf); softmax over the chosen then
 *                 subtracts their largest value.
 * Limits (MXFP4_MOE_ERR_SHAPE): those of mxfp4_moe_router, 1 <= n_group <= 32,
 * E % n_group == 0, 1 <= topk_group <= n_group, k <= topk_group * E / n_group;
 * bias_in_weights 0 or 1 (MXFP4_MOE_ERR_ARG). */
int mxfp4_moe_router_grouped(const float* logits, const float* bias, int T, int E, int topk,
                             int scoring, int n_group, int topk_group, int bias_in_weights,
                             int32_t* topk_ids, float* topk_weights, void* stream);

/* The MoE layer, y = sum_j w_tj * W2[e] silu(W_gate[e] x) * (W_up[e] x).
 *   hidden        bf16  [T, K]
 *   topk_ids      int32 [T, topk]   (negative = padding, >= E = invalid, both skipped)
 *   topk_weights  fp32  [T, topk]
 *   w13/s13/w2/s2 packed weights and scales, layouts in the file header
 *   out           bf16  [T, K]      written completely (zero for tokens with no valid route)
 *   status        int32 [4]         may be NULL
 *   workspace     device scratch of at least mxfp4_moe_workspace_size(T,K,I,E,topk)
 *                 bytes, zero before first use (see above); not shared by
 *                 calls that may run concurrently
 *   path          0 = automatic (decode for T <= 32, else prefill),
 *                 1 = decode kernels, 2 = prefill (tensor-core grouped GEMM)
 * T == 0 returns MXFP4_MOE_OK and enqueues nothing. */
int mxfp4_moe_forward(const void* hidden, const int32_t* topk_ids, const float* topk_weights,
                      const uint8_t* w13, const uint8_t* s13,
                      const uint8_t* w2, const uint8_t* s2,
                      int T, int K, int I, int E, int topk,
                      void* out, int32_t* status,
                      void* workspace, size_t workspace_bytes,
                      int path, void* stream);

/* The layer over an expert-parallel window, optionally per route ("MXFP4 MoE
 * decode kernels", Design, "Routing inside the kernel": routes to experts on
 * other expert-parallel ranks are skipped and cost nothing; Beyond gpt-oss:
 * mxk_w2xr, a per-route w2 output for models that apply a per-route operation
 * before the token sum).
 *   w13/s13/w2/s2 hold the E local experts, global ids expert_base ..
 *                 expert_base + E - 1 (expert_base >= 0); a route whose id lies
 *                 outside that window is skipped silently (no status count)
 *   per_route 0   out bf16 [T, K]: y_t = sum over the window's routes of
 *                 w_tj * W2[e] h (this rank's part of the token sums)
 *   per_route 1   out bf16 [T * topk, K]: row t * topk + j = W2[e] h of route
 *                 (t, j), unweighted (topk_weights may be NULL), zero rows for
 *                 skipped routes
 * Everything else (paths, limits, alignment, workspace, errors) as
 * mxfp4_moe_forward; path, per_route or expert_base out of range give
 * MXFP4_MOE_ERR_ARG. */
int mxfp4_moe_forward_window(const void* hidden, const int32_t* topk_ids,
                             const float* topk_weights,
                             const uint8_t* w13, const uint8_t* s13,
                             const uint8_t* w2, const uint8_t* s2,
                             int T, int K, int I, int E, int topk,
                             int expert_base, int per_route,
                             void* out, int32_t* status,
                             void* workspace, size_t workspace_bytes,
                             int path, void* stream);

/* The gpt-oss form of the layer ("MXFP4 MoE decode kernels", Design, "Read
 * the served layout" and "Fused epilogues"):
 *   y_t = sum_j w_tj * (W2[e] h + b2[e]),  h = SwiGLU-OAI(W_gate[e] x + b_gate[e],
 *                                                     W_up[e] x + b_up[e])
 *   SwiGLU-OAI(g, u) = min(g, 7) * sigmoid(1.702 min(g, 7)) * (clamp(u, -7, 7) + 1)
 * with h rounded once to bf16 between the projections and all sums in fp32.
 *   w13 / s13     uint8 [E, 2I, K/2] / [E, 2I, K/32] with the gate and up rows
 *                 INTERLEAVED: row 2i is gate row i, row 2i + 1 is up row i
 *   b13           fp32  [E, 2I] in the same (interleaved) row order
 *   w2 / s2       as for mxfp4_moe_forward
 *   b2            fp32  [E, K]; each route adds its expert's b2 before the
 *                 routing weight, so a token gets sum_j w_tj * b2[e_tj]
 * Other arguments, paths (decode for T <= 32, else the tensor-core prefill),
 * limits and errors as mxfp4_moe_forward. b13 and b2 are device pointers, 4-byte
 * aligned (MXFP4_MOE_ERR_ALIGN), non-NULL (MXFP4_MOE_ERR_ARG); the caller owns
 * every buffer. NaN in a pre-activation stays NaN (the cap and clamp do not
 * replace it). */
int mxfp4_moe_forward_oai(const void* hidden, const int32_t* topk_ids, const float* topk_weights,
                          const uint8_t* w13, const uint8_t* s13, const float* b13,
                          const uint8_t* w2, const uint8_t* s2, const float* b2,
                          int T, int K, int I, int E, int topk,
                          void* out, int32_t* status,
                          void* workspace, size_t workspace_bytes,
                          int path, void* stream);

/* The forward call for callers that cannot allocate device memory. The pages
 * have no counterpart of this entry point: it is a convenience of this
 * library. Some callers may not call cudaMalloc at all -- code that runs under
 * a host framework that owns every device allocation (a plugin interface that
 * hands out no scratch space), latency-critical serving loops that must never
 * synchronise the device (cudaMalloc and cudaFree can), or pipelines that fix
 * their memory footprint before they start. This variant takes the same
 * arguments as mxfp4_moe_forward without the workspace, and uses instead a
 * fixed device array of MXFP4_MOE_NOALLOC_BYTES bytes compiled into the
 * library: every GPU that loads the library holds that array until the
 * process exits. Nothing is allocated by this call (no cudaMalloc, cudaFree or
 * allocating library routine).
 *  - Sizes whose mxfp4_moe_workspace_size(T, K, I, E, topk) exceeds
 *    MXFP4_MOE_NOALLOC_BYTES are rejected with MXFP4_MOE_ERR_WORKSPACE (the
 *    decode path of the four workload shapes fits up to T = 32).
 *  - The first call on a device performs the set-up for that device: it looks
 *    up the array's device address, which makes the CUDA driver load this part
 *    of the library and place the array on that device (a one-time driver
 *    allocation that may synchronise), and clears the array's bookkeeping part
 *    on `stream`. Make that first call in set-up code, before any stream
 *    capture and before any loop that must not synchronise; the promise that
 *    nothing is allocated holds for every later call.
 *  - The library leaves the array's bookkeeping part zero after every call,
 *    also after one whose bounded wait gave up (status[2] != 0), so the array
 *    never needs clearing by the caller (who could not reach it anyway).
 *  - All calls share the one array, and it keeps the last call's contents:
 *    calls whose work may overlap on the GPU (different streams without
 *    ordering) race on it; issue them on one stream or order them. */
#define MXFP4_MOE_NOALLOC_BYTES (16u * 1024u * 1024u)
int mxfp4_moe_forward_noalloc(const void* hidden, const int32_t* topk_ids,
                              const float* topk_weights,
                              const uint8_t* w13, const uint8_t* s13,
                              const uint8_t* w2, const uint8_t* s2,
                              int T, int K, int I, int E, int topk,
                              void* out, int32_t* status, int path, void* stream);

/* MXFP4 encoder ("GLM-5.2 and GLM-5.3 (744B) in MXFP4 on Gaudi 2", What was
 * built, "MXFP4 encoder"): bf16 rows -> the packed form the forward calls read.
 *   x       bf16  [rows, cols], cols % 32 == 0 (MXFP4_MOE_ERR_SHAPE), 16-byte aligned
 *   packed  uint8 [rows, cols/2]  value 2i in the low nibble of byte i, 4-byte aligned
 *   scale   uint8 [rows, cols/32] E8M0
 *   rule    0 = OCP: per 32-value block X = floor(log2(amax)) - 2;
 *           1 = Quark: the same, raised by one when amax / 2^X >= 7
 * X is clamped to [-127, 127] (an all-zero block gets byte 0); a block with a
 * NaN or infinite value gets byte 255 and codes 0. Each element v / 2^X is
 * rounded to the nearest E2M1 value, ties to the even code, saturating at 6,
 * keeping its sign (-0 stays -0). Device pointers owned by the caller;
 * rows == 0 enqueues nothing. */
int mxfp4_moe_encode(const void* x, int rows, int cols, int rule, uint8_t* packed,
                     uint8_t* scale, void* stream);

/* Dequantise packed rows to bf16 ("MXFP4 MoE decode kernels", Prefill:
 * mxk_deq unpacks an expert's MXFP4 weights straight to bf16).
 *   packed uint8 [rows, cols/2], scale uint8 [rows, cols/32] -> out bf16 [rows, cols]
 * Each value is E2M1(nibble) * 2^(s - 127) rounded once to bf16, which is
 * exact except that products beyond the bf16 range become +-inf and the
 * scale byte 255 gives NaN. cols % 32 == 0 (MXFP4_MOE_ERR_SHAPE); packed
 * 16-byte and out 4-byte aligned (MXFP4_MOE_ERR_ALIGN). Uses the decode
 * kernels' conversion (form 1 of mxfp4_moe_dequant_form). */
int mxfp4_moe_dequant(const uint8_t* packed, const uint8_t* scale, int rows, int cols,
                      void* out, void* stream);

/* The same dequantisation through the conversion of one path of the layer,
 * so that a bit-exact check pins the weights each path computes with:
 *   form 1  the decode kernels': hardware E2M1 -> f16 (exact), then an exact
 *           fp32 multiply by 2^(s - 127), rounded once to bf16;
 *   form 2  the prefill GEMM's operand A: the E2M1 fields placed in a bf16
 *           bit pattern (magnitude x 2^-126), then exact bf16 multiplies by
 *           2^(s - 1), or by 2^126 and 2^(s - 127) for bytes above 128 --
 *           the same device routine that feeds the GEMM's tensor memory.
 * Both give the value stated for mxfp4_moe_dequant, bit for bit; form
 * outside {1, 2} gives MXFP4_MOE_ERR_ARG; other rules as mxfp4_moe_dequant. */
int mxfp4_moe_dequant_form(const uint8_t* packed, const uint8_t* scale, int rows, int cols,
                           int form, void* out, void* stream);

/* ---------------------------------------------------------------------------
 * Operators around the layer. They follow the conventions above: device
 * pointers, contiguous rows, host checks before anything is enqueued, no
 * allocation and no synchronisation, bit-identical repeats. The pages have no
 * counterpart of them.
 * ------------------------------------------------------------------------- */

/* Residual addition and root-mean-square norm, with an MXFP8 output. Per row t:
 *   h = x + residual (fp32)            residual_out = bf16(h)
 *   y = h * rsqrt(mean(h^2) + eps) * gamma (fp32, from the unrounded h)
 *   out = bf16(y)
 *   out8, scale8: MXFP8 of y: per 32 values along the row X = floor(log2(amax)) - 8,
 *     clamped to [-127, 127], scale byte X + 127, code = E4M3(y / 2^X), nearest
 *     even, saturating at 448; an all-zero block has scale byte 0, a block with
 *     a NaN or infinite value byte 255 and codes 0.
 *     rule 0 = OCP (amax / 2^X lies in [256, 512): values above 448 saturate),
 *     rule 1 = "nosat": X raised by one when amax / 2^X > 448.
 *   x            bf16  [T, K]
 *   residual     bf16  [T, K] or NULL (h = x)
 *   gamma        bf16  [K]
 *   residual_out bf16  [T, K] or NULL; may be the same pointer as x or residual
 *   out          bf16  [T, K] or NULL
 *   out8         uint8 [T, K] (E4M3) or NULL; scale8 uint8 [T, K/32], both or neither
 * At least one of out, out8 and residual_out is needed. Limits
 * (MXFP4_MOE_ERR_SHAPE): 0 <= T, K % 32 == 0, 32 <= K <= 16384. eps finite and
 * >= 0, rule 0 or 1 (MXFP4_MOE_ERR_ARG). All pointers but scale8 16-byte
 * aligned (MXFP4_MOE_ERR_ALIGN). T == 0 enqueues nothing. */
int mxfp4_moe_add_rmsnorm(const void* x, const void* residual, const void* gamma, int T, int K,
                          float eps, int rule, void* residual_out, void* out, uint8_t* out8,
                          uint8_t* scale8, void* stream);

/* The norms after and before a block with the block's gate and the residual's
 * scale between them. Per row t:
 *   n = x * r1 * post_gamma, r1 = rsqrt(mean(x^2) + eps)   (post_gamma NULL: n = x)
 *   h = residual_scale * residual + g * n (fp32)            residual_out = bf16(h)
 *   y = h * r2 * pre_gamma, r2 = rsqrt(mean(h^2) + eps), from the unrounded h
 *   out = bf16(y); out8, scale8: MXFP8 of y in mxfp4_moe_add_rmsnorm's format and rules. y
 *   is two fp32 products here, where that call rounds once: codes beside a tie may differ
 *   x, residual    bf16 [T, K]
 *   post_gamma, pre_gamma  bf16 [K]; pre_gamma NULL: no y, out and out8 NULL
 *   gate           gate_kind 0: NULL (g = 1); 1: bf16 [K], a channel's; 2: fp32 [T],
 *                  a token's; 3: bf16 [T, K]. gate_act 0: g is the value, 1: its sigmoid
 *   residual_scale fp32 [1] or NULL (1)
 *   residual_out   bf16 [T, K] or NULL; may be the same pointer as x or residual
 *   x8, x8_scale / h8, h8_scale   what a backward pass keeps in 8 bits: MXFP8 of x
 *                  and of the unrounded h under checkpoint_rule; each pair or NULL
 *   rstd           fp32 [2, T] or NULL: r1 and r2 (1 where there is no norm)
 * rule and checkpoint_rule 0 = OCP or 1 = "nosat" as above; at least one output.
 * Limits, eps, T == 0 and alignment as mxfp4_moe_add_rmsnorm (scale bytes: any;
 * residual_scale, rstd and a token's gate 4 bytes). */
int mxfp4_moe_sandwich_norm(const void* x, const void* residual, const void* post_gamma,
                            const void* pre_gamma, const void* gate, int gate_kind, int gate_act,
                            const float* residual_scale, int T, int K, float eps, int rule,
                            int checkpoint_rule, void* residual_out, void* out, uint8_t* out8,
                            uint8_t* scale8, uint8_t* x8, uint8_t* x8_scale, uint8_t* h8,
                            uint8_t* h8_scale, float* rstd, void* stream);

/* Its gradient, from what the forward call kept. With H = h r2, X = x r1,
 * v = pre_gamma * grad_y, means over the row:
 *   d = grad_h + r2 (v - H mean(v H))       grad_residual = bf16(residual_scale * d)
 *   u = post_gamma * g * d                  grad_x = bf16(r1 (u - X mean(u X)))
 *                                           (post_gamma NULL: grad_x = bf16(g * d))
 *   grad_pre_gamma  fp32 [K]  sum_t grad_y * H
 *   grad_post_gamma fp32 [K]  sum_t g * d * X
 *   grad_gate       d * n * g' summed to the gate's shape: fp32 [K], fp32 [T] or bf16 [T, K]
 *   grad_residual_scale fp32 [1]  sum d * residual
 *   grad_h, grad_y  bf16 [T, K]; either may be NULL (zero), not both
 *   x, h            bf16 [T, K] (scale NULL), or E4M3 [T, K] with E8M0 [T, K/32],
 *                   each by itself; h may be NULL without grad_y
 *   rstd            fp32 [2, T], needed with post_gamma or grad_y
 *   post_gamma, pre_gamma, gate, gate_kind, gate_act, residual_scale as forward
 *   residual        bf16 [T, K], read for grad_residual_scale only
 * Outputs may be NULL where they are not wanted, at least one is needed, and none may
 * overlap an input. T == 0 zeroes the sums over rows that are asked for. workspace:
 * mxfp4_moe_sandwich_norm_backward_workspace_size bytes, 256-byte aligned, no
 * initial contents required, not shared by calls that may run concurrently. Limits
 * as forward; bf16 and E4M3 rows and fp32 [K] 16-byte aligned, the rest 4. */
size_t mxfp4_moe_sandwich_norm_backward_workspace_size(int T, int K);
int mxfp4_moe_sandwich_norm_backward(const void* grad_h, const void* grad_y, const void* x,
                                     const uint8_t* x_scale, const void* h, const uint8_t* h_scale,
                                     const float* rstd, const void* post_gamma,
                                     const void* pre_gamma, const void* gate, int gate_kind,
                                     int gate_act, const void* residual,
                                     const float* residual_scale, int T, int K, void* grad_x,
                                     void* grad_residual, float* grad_post_gamma,
                                     float* grad_pre_gamma, void* grad_gate,
                                     float* grad_residual_scale, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Router in the score domain (mxfp4_moe_router adds its bias to the logits; a
 * bias on the scores orders the experts differently). Per token:
 *   s_e = softmax over all E logits (scoring 0) or sigmoid(logit) (scoring 1)
 *   c_e = s_e + bias[e]     (bias NULL: the logits decide the choice, which
 *                            order as the scores do)
 *   n_group > 1: a group (equal runs of consecutive experts) scores the sum of
 *     its group_top (1 or 2) largest c; the topk_group best groups stay, ties
 *     to the lower group
 *   topk_ids[t]      the k largest c of the groups that stay, in descending
 *                    order, ties to the lower expert
 *   topk_weights[t]  s of the chosen (not c), divided by their sum when
 *                    renormalise is 1, times route_scale; fp32
 * An expert whose logit or c is NaN or -inf is never chosen; a slot with no
 * expert left gets id -1 (padding for the forward calls) and weight 0.
 *   logits fp32 [T, E], bias fp32 [E] or NULL, topk_ids int32 [T, k],
 *   topk_weights fp32 [T, k]; 4-byte aligned (MXFP4_MOE_ERR_ALIGN)
 * Limits (MXFP4_MOE_ERR_SHAPE): 1 <= E <= 1024, 1 <= k <= min(32, E), 0 <= T,
 * 1 <= n_group <= 32, E % n_group == 0, 1 <= topk_group <= n_group,
 * k <= topk_group * E / n_group. scoring 0 or 1, group_top 1 or 2, renormalise
 * 0 or 1, route_scale finite (MXFP4_MOE_ERR_ARG). T == 0 enqueues nothing. */
int mxfp4_moe_router_scored(const float* logits, const float* bias, int T, int E, int topk,
                            int scoring, int n_group, int topk_group, int group_top,
                            int renormalise, float route_scale, int32_t* topk_ids,
                            float* topk_weights, void* stream);

/* Balance losses and expert counts of a routing. s as mxfp4_moe_router_scored
 * scores the logits (NaN and -inf: masked, s = 0), p_e = s_e / sum s; rows of scores too
 * small for fp32 keep their quotients, but for one whose every score that call has as 0
 * (sigmoid, no logit above -88.7): p = 0. A token counts when
 * it has an id in [0, E) and a logit that is not masked; other ids are skipped,
 * the same id twice counts twice. Per sequence, over its n counting tokens:
 *   counts int32 [n_seq, E]  routes to each expert (C: their sum)
 *   prob   fp32  [n_seq, E]  mean of p
 *   slope  fp32  [n_seq, E]  E * counts / (C n), the gradient of the sequence's loss
 *                            E sum_e (counts / C) prob with respect to p of a token
 * (zeros for a sequence without tokens) and
 *   stats  fp32  [4]  the mean loss of the sequences that have tokens; the mean over
 *                     tokens of log(sum exp(logits))^2; tokens; such sequences
 *   logits fp32 [T, E], topk_ids int32 [T, topk]
 *   seq_offsets int32 [n_seq + 1], not decreasing: sequence i is the rows from
 *     seq_offsets[i] up to seq_offsets[i + 1]; rows in none are left out. NULL: all
 *     rows are one sequence (n_seq 1)
 * Limits (MXFP4_MOE_ERR_SHAPE): 0 <= T, T * topk < 2^31, 1 <= E <= 1024,
 * 1 <= topk <= min(32, E), 1 <= n_seq <= 2^20. T == 0 writes zeros. workspace as
 * mxfp4_moe_sandwich_norm_backward; all other pointers 4-byte aligned. */
size_t mxfp4_moe_router_balance_workspace_size(int T, int E, int n_seq);
int mxfp4_moe_router_balance(const float* logits, const int32_t* topk_ids, int T, int E, int topk,
                             int scoring, const int32_t* seq_offsets, int n_seq, float* stats,
                             int32_t* counts, float* prob, float* slope, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Gradient of the logits of mxfp4_moe_router_scored's weights (the choice is
 * fixed) and of mxfp4_moe_router_balance's losses (the counts are):
 *   sum grad_weights * topk_weights + grad_losses[0] * stats[0] + grad_losses[1] * stats[1]
 *   topk_ids      the chosen experts; an id outside [0, E) or of a masked expert
 *                 takes no part, the same id twice twice. Renormalised weights have
 *                 their gradient where the largest chosen score is not 0 in fp32; the
 *                 others' is 0 for scores below 2^-126
 *   grad_weights  fp32 [T, topk] or NULL (zero)
 *   grad_losses   fp32 [2] or NULL (zero; stats, slope and seq_offsets are then not
 *                 read); stats, slope, seq_offsets, n_seq as that call's
 *   grad_logits   fp32 [T, E], written completely (0 for masked logits and for rows
 *                 without a valid id)
 * Limits and alignment as mxfp4_moe_router_balance; T == 0 enqueues nothing. */
int mxfp4_moe_router_backward(const float* logits, const int32_t* topk_ids,
                              const float* grad_weights, int T, int E, int topk, int scoring,
                              int renormalise, float route_scale, const float* grad_losses,
                              const float* stats, const float* slope, const int32_t* seq_offsets,
                              int n_seq, float* grad_logits, void* stream);

/* Gradient of the layer's combination y_t = sum_j w_tj o_tj of its routes'
 * outputs o (mxfp4_moe_forward_window with per_route):
 *   grad_weights fp32 [T, topk]       sum over the row of grad_out_t * o_tj
 *   grad_routes  bf16 [T * topk, K] or NULL   bf16(w_tj * grad_out_t): for a caller whose
 *   routes come from something that trains; the MXFP4 experts have no gradient here
 *   grad_out bf16 [T, K], routes bf16 [T * topk, K], topk_weights fp32 [T, topk]
 *   (needed with grad_routes)
 *   topk_ids int32 [T, topk] or NULL (every route counts). A negative id, or one outside
 *   expert_base .. expert_base + n_experts - 1 (n_experts 0: no window, whatever expert_base
 *   is), is a skipped route: its row is not read, its gradients are 0
 * No output may overlap an input (MXFP4_MOE_ERR_ARG).
 * Limits (MXFP4_MOE_ERR_SHAPE): K as above, 1 <= topk <= 32, T * topk < 2^31.
 * bf16 rows 16-byte aligned, the rest 4. T == 0 enqueues nothing. */
int mxfp4_moe_combine_backward(const void* grad_out, const void* routes, const int32_t* topk_ids,
                               const float* topk_weights, int T, int K, int topk, int expert_base,
                               int n_experts, float* grad_weights, void* grad_routes,
                               void* stream);

/* A shared projection from packed MXFP4 weights, with the low-rank adapters of
 * many requests beside it:
 *   y_t = W x_t + adapter_scale[a] * B[a] (A[a] x_t),   a = adapter_ids[t]
 * fp32 sums, one rounding to bf16. The inner products v = adapter_scale (A x)
 * are rounded to 17 significant bits on their way to the second product, an error
 * of at most 2^-17 sum_r |B[n][r] v[r]|. MXFP8 values are taken as bf16: exact,
 * but for codes of scale bytes 0 to 2 whose last bits are below bf16's smallest
 * step (2^-133), and infinite past its largest value.
 *   x             bf16 [T, K] (x_scale NULL), or MXFP8 as mxfp4_moe_add_rmsnorm
 *                 writes it: E4M3 uint8 [T, K] with x_scale E8M0 uint8 [T, K/32]
 *   w / s         uint8 [N, K/2] / [N, K/32], the packed layout of one expert's w2
 *   adapter_ids   int32 [T] or NULL (no adapters; the next four are ignored).
 *                 A negative id: no adapter for this token; an id >= n_adapters:
 *                 none either, counted in status[0]
 *   adapter_a     bf16 [n_adapters, rank, K]
 *   adapter_b     bf16 [n_adapters, N, rank] (adapters of a smaller rank: padded
 *                 with zeros)
 *   adapter_scale fp32 [n_adapters] or NULL (1)
 *   out           bf16 [T, N], written completely
 *   status        int32 [4] or NULL; status[1] = 0, status[2] and [3] as in the
 *                 file header (status[2] bit 0: this call's bounded waits)
 *   workspace     device scratch of mxfp4_moe_linear_workspace_size bytes, no
 *                 initial contents required, not shared by calls that may run
 *                 concurrently
 * Limits (MXFP4_MOE_ERR_SHAPE): 0 <= T <= 2^20, K % 64 == 0, 64 <= K <= 16384,
 * N % 8 == 0, 8 <= N <= 2^20, and with adapters rank % 8 == 0, 8 <= rank <= 256,
 * 1 <= n_adapters <= 1024. x and adapter_a 32-byte aligned (their rows are
 * read 32 bytes a thread), the workspace 256, adapter_ids, adapter_scale and
 * status 4, all others 16 (MXFP4_MOE_ERR_ALIGN). T == 0 enqueues nothing. */
size_t mxfp4_moe_linear_workspace_size(int T, int K, int N, int rank, int x_is_mxfp8);
int mxfp4_moe_linear(const void* x, const uint8_t* x_scale, const uint8_t* w, const uint8_t* s,
                     int T, int K, int N, const int32_t* adapter_ids, const void* adapter_a,
                     const void* adapter_b, const float* adapter_scale, int n_adapters, int rank,
                     void* out, int32_t* status, void* workspace, size_t workspace_bytes,
                     void* stream);

/* Profiling hook: when events (host array of n cudaEvent_t handles, n >= 2)
 * is non-NULL, each later forward call on this process records events[0]
 * before its first kernel and events[i] after its i-th kernel (while i < n),
 * on its stream; the decode path runs 1 kernel (one cooperative launch), the
 * prefill path 5 (the first two events bracket route + gather). Pass NULL to
 * turn it off.
 * Not thread-safe; meant for benchmarks. */
void mxfp4_moe_set_phase_events(void* const* events, int n);

/* Test only: from the next forward call on, the decode kernel's CTA `cta`
 * does not arrive at the grid barrier between its two phases, so every
 * bounded wait on that barrier (in all CTAs) runs out and the call reports it
 * in status[2] and status[3] instead of computing the output; a negative cta
 * turns this off (the default). It exists so tests can exercise the failure
 * reporting without faulting or hanging a GPU. Not thread-safe. */
void mxfp4_moe_test_skip_grid_arrival(int cta);

/* Test only: from the next mxfp4_moe_linear call of more than 16 tokens on, CTA
 * `cta` of its tile kernel leaves out its first copy of packed weights, so the waits
 * that depend on it run out (0.2 s each) and the call reports it in
 * status[2] and status[3] instead of computing the output; a negative cta turns
 * this off (the default). Not thread-safe. */
void mxfp4_moe_test_skip_linear_copy(int cta);

/* Test only: the warps per CTA of the decode kernel form that a decode call of
 * this shape and T would run on a device with max_smem bytes of opt-in shared
 * memory per block: 12, 11 or 10 (every warp a consumer), 7 (7 consumer warps
 * and a producer warp), or 0 when no form fits. The form is the one the call's
 * own T needs, except that every T of a layer shape runs the form of its
 * largest decode T when that is a 10- to 12-warp form. Host only; no device
 * is touched. -1 for shapes the decode path does not take (T outside 1..32,
 * T * topk > 1024, K or I not a multiple of 64, E or topk out of range). */
int mxfp4_moe_test_decode_form(int T, int K, int I, int E, int topk, int max_smem);

/* Static description of an error code (never NULL). */
const char* mxfp4_moe_strerror(int code);

/* Library ABI version: 100 * major + minor. */
int mxfp4_moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_MOE_H_ */

/*
 * skinny_gemm.h - C ABI of the MI355X (gfx950) decode-phase linear layer.
 *
 * Operation (every entry point):  y[M x N] = x[M x K] . W^T,  M = 1..16 tokens.
 *
 *   The decode-phase linear layer is a tall-skinny product of a few token
 *   rows with a weight matrix that is read from HBM once per step
 *   ("Developing a custom Qwen2.5 72B inference engine from scratch - what is
 *   the real bottleneck?", section 2 "The two-phase reality" and section 6.1
 *   "Decode GEMV: already near the roofline").  A linear layer computes
 *   y = x W with one row of x per token ("Multi-GPU Inference and Serving at
 *   Scale", Example 2); here W is stored one row per output feature, so the
 *   product is x . W^T.
 *
 *   FP8 weights are weight-only: activations stay 16-bit and each FP8 weight
 *   is dequantized with the fp32 scale of the 128 x 128 block it lies in
 *   ("9% faster GLM-5.3-Flash prefill with GPU-to-GPU IPC (and why TileLang
 *   didn't help)", section "TileLang: twice as fast, and no faster"; the
 *   Qwen2.5 72B engine report, section 6.2).
 *
 * Layouts (all row-major, contiguous, device memory):
 *   x        [M][K]                    bf16
 *   W        [N][K]                    bf16, or OCP E4M3FN bytes (FP8)
 *   w_scale  [ceil(N/128)][ceil(K/128)] fp32; weight (n, k) uses
 *                                       w_scale[n/128][k/128] (FP8 only)
 *   y        [M][N]                    bf16, round-to-nearest-even
 *   Accumulation is fp32.  Results are within 2e-3 * sum_k |x w| + 1e-6 of
 *   the exact product, and bitwise reproducible for a given device and plan.
 *
 * Requirements checked on the host before anything is enqueued:
 *   1 <= M <= SKINNY_MAX_M, N >= 1, K >= 1; K % 8 == 0 (bf16) or
 *   K % 16 == 0 (FP8); x, W, y and the workspace 16-byte aligned; w_scale
 *   4-byte aligned; no NULL operand.  Violations return a status and enqueue
 *   nothing.
 *
 * Ownership and concurrency:
 *   The caller owns every buffer (x, W, w_scale, y, workspace) and keeps it
 *   alive until the work on `stream` has finished.  The library allocates
 *   nothing and keeps no pointer after a call returns.  Host arrays passed in
 *   (the `linears` of a stack) are read during the call only.  y must not
 *   overlap x, W, w_scale, the workspace or another linear's y, and the
 *   workspace must not overlap x, W or w_scale (checked:
 *   SKINNY_ERR_INVALID_ARG).  Calls enqueue work on `stream` (a hipStream_t;
 *   NULL is the default stream) and return without waiting for it; execution
 *   faults surface at the caller's next synchronization.  Calls on different streams need separate workspaces.
 *   Workspace contents are undefined after a call.  Entry points may be
 *   called from several host threads at once: the library's only shared
 *   state is a per-device cache of device properties, occupancy results and
 *   granted LDS sizes, filled on first use under a lock.
 */
#ifndef SKINNY_GEMM_H
#define SKINNY_GEMM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SKINNY_ABI_VERSION 2
#define SKINNY_MAX_M 16
/* Linears whose descriptors travel in a main-kernel launch's arguments; a
 * launch over more linears reads them from a table in the workspace. */
#define SKINNY_MAX_LINEARS_PER_LAUNCH 32
/* Smallest workspace any call asks for (bytes). */
#define SKINNY_MIN_WORKSPACE_BYTES 256

typedef enum skinny_status {
  SKINNY_OK = 0,
  SKINNY_ERR_INVALID_ARG = 1, /* NULL operand, M outside 1..16, N < 1, K < 1, count < 1,
                                 unknown dtype or variant, overlapping output             */
  SKINNY_ERR_UNSUPPORTED = 2, /* K not a multiple of 8 (bf16) / 16 (FP8), misaligned
                                 pointer, shape too large, device is not gfx950            */
  SKINNY_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than the *_workspace_bytes value */
  SKINNY_ERR_HIP = 4          /* a HIP call failed (device query or kernel launch)          */
} skinny_status;

enum skinny_dtype { SKINNY_BF16 = 0, SKINNY_FP8_BS128 = 1 };

/* Compute variant of the main kernel.  VECTOR streams one row per wave and
 * multiplies on the vector ALUs (M <= 8); MFMA streams 16-row tiles and
 * multiplies on the matrix cores (any M).  AUTO picks per (dtype, M) from
 * measurement. */
enum skinny_variant { SKINNY_VARIANT_AUTO = 0, SKINNY_VARIANT_VECTOR = 1, SKINNY_VARIANT_MFMA = 2 };

/* One linear of a stack.  All pointers are device pointers. */
typedef struct skinny_linear {
  int dtype;            /* SKINNY_BF16 or SKINNY_FP8_BS128                  */
  int N;                /* output features: rows of W, columns of y         */
  int K;                /* input features: columns of W and x               */
  int reserved;         /* must be 0                                        */
  const void* w;        /* W[N][K] bf16 or E4M3FN bytes                     */
  const float* w_scale; /* FP8: [ceil(N/128)][ceil(K/128)] fp32; bf16: NULL */
  const void* x;        /* x[M][K] bf16                                     */
  void* y;              /* y[M][N] bf16                                     */
} skinny_linear;

/* Main kernel of a launch, as the plan queries report it. */
enum skinny_kernel {
  SKINNY_KERNEL_NONE = 0,
  SKINNY_KERNEL_ROWS = 1,         /* skinny_rows (VECTOR), deep instance; MoE form      */
  SKINNY_KERNEL_ROWS_LEAN = 2,    /* skinny_rows, lean instance (bf16 launches >= 0.4 GB) */
  SKINNY_KERNEL_ROWS_FLAT = 3,    /* skinny_rows_flat (loads streamed across units):
                                     launches < 0.4 GB of up to 4 (bf16) or 2 (FP8)
                                     tokens, one-token FP8 launches >= 1 GB             */
  SKINNY_KERNEL_TILES = 4,        /* skinny_tiles (MFMA), 4-wave workgroups; MoE form  */
  SKINNY_KERNEL_TILES_WIDE = 5,   /* skinny_tiles, 8-wave workgroups                    */
  SKINNY_KERNEL_TILES_KSPLIT = 6, /* skinny_tiles' K-split form (one-token MoE slices)  */
  SKINNY_KERNEL_MOE_MLP1 = 7      /* skinny_moe_mlp1 (the experts' MLP in one launch)   */
};

/* Launch plan override, for tests and benchmarks.  Zero-initialised = automatic. */
typedef struct skinny_plan {
  int variant;          /* enum skinny_variant                               */
  int waves;            /* persistent waves per main launch; 0 = automatic   */
  int kernel;           /* enum skinny_kernel, filled by the plan queries;
                           ignored on input                                  */
  int reserved[5];      /* must be 0                                         */
} skinny_plan;

/* Bytes of workspace a single linear needs: at least SKINNY_MIN_WORKSPACE_BYTES
 * for valid arguments, 0 for invalid ones.  Pure host arithmetic, no HIP call.
 * The workspace holds the fp32 partial sums of K-chunks that the second pass
 * adds: for every row group of a linear that the launch splits into C > 1
 * K-chunks, C slots of [M][band rows] floats.  The value covers the largest
 * split either variant may choose.  The split is the long dimension cut
 * across workgroups so that a skinny launch still streams on the whole chip
 * ("9% faster GLM-5.3-Flash prefill with GPU-to-GPU IPC (and why TileLang
 * didn't help)", section "TileLang: twice as fast, and no faster"); a
 * K-split's partial results add up to the product ("Multi-GPU Inference and
 * Serving at Scale", Example 3, the row-split second linear). */
size_t skinny_workspace_bytes(int dtype, int M, int N, int K);

/* Bytes of workspace decode_linear_stack needs for these linears at this M:
 * the partial sums of its launches (for a launch of more than
 * SKINNY_MAX_LINEARS_PER_LAUNCH linears, bounded at the largest grid any
 * launch runs) plus that launch's descriptor table. */
size_t skinny_stack_workspace_bytes(const skinny_linear* linears, int count, int M);

/* y = x . W^T with bf16 W: one linear layer of the decode step, x the
 * [M][K] activations of M tokens, W the layer's [N][K] weights ("Multi-GPU
 * Inference and Serving at Scale", Example 2: a linear's product, worked on
 * a small matrix; "Developing a custom Qwen2.5 72B inference engine from
 * scratch - what is the real bottleneck?", section 6.1: the decode GEMV).
 *   x, y       device, [M][K] and [M][N] bf16 row-major, 16-byte aligned
 *   w          device, [N][K] bf16 row-major (the nn.Linear layout)
 *   workspace  device, >= skinny_workspace_bytes(SKINNY_BF16, M, N, K)
 * Argument errors are returned before anything is enqueued; the call is
 * asynchronous on `stream`. */
skinny_status skinny_gemm_bf16(const void* x, const void* w, void* y, int M, int N, int K,
                               void* workspace, size_t workspace_bytes, void* stream);

/* y = x . (e4m3(W) * block scale)^T: weight-only FP8, each weight an OCP
 * E4M3FN byte times the fp32 scale of its 128 x 128 block, activations and
 * outputs bf16 ("9% faster GLM-5.3-Flash prefill with GPU-to-GPU IPC (and why
 * TileLang didn't help)", section "TileLang: twice as fast, and no faster":
 * FP8 weights with 128 x 128 block scales against 16-bit activations).
 *   w_fp8      device, [N][K] bytes row-major
 *   w_scale    device, [ceil(N/128)][ceil(K/128)] fp32 row-major; the scale
 *              of W[n][k] is w_scale[n / 128][k / 128]
 *   x, y, workspace as skinny_gemm_bf16 (workspace for SKINNY_FP8_BS128) */
skinny_status skinny_gemm_fp8_bs128(const void* x, const void* w_fp8, const float* w_scale,
                                    void* y, int M, int N, int K, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Runs `count` independent linears that share M, e.g. the QKV, O, gate_up
 * and down projections of every decoder layer: the decode step streams every
 * layer's weights once per generated token ("Developing a custom Qwen2.5 72B
 * inference engine from scratch - what is the real bottleneck?", section 1
 * (80 layers, each with attention and MLP projections) and section 2 "The
 * two-phase reality" (decode reads the whole model from HBM per token)).
 *   linears    host array of `count` >= 1 skinny_linear, read during the call
 *   M          tokens, 1..SKINNY_MAX_M, the rows of every x and y
 *   workspace  device, 16-byte aligned, >= skinny_stack_workspace_bytes(linears,
 *              count, M); contents undefined afterwards
 * Each linear reads its own x and writes its own y; no y may overlap any x,
 * W, w_scale, other y or the workspace (checked).  The linears of each dtype,
 * in call order, are streamed by one persistent launch (one per 4096 linears
 * of a dtype, should a call have more); a launch of more than
 * SKINNY_MAX_LINEARS_PER_LAUNCH linears reads their descriptors from a table
 * that the call copies from host memory into the workspace on `stream` just
 * before it.  On a stream under graph capture (where such a copy would read
 * this call's host memory at every replay) the call instead makes launches of
 * at most SKINNY_MAX_LINEARS_PER_LAUNCH linears.  Each launch's split-K
 * partial sums are combined by a second, deterministic pass.  Errors (any
 * linear failing the checks of a single linear) are returned before anything
 * is enqueued. */
skinny_status decode_linear_stack(const skinny_linear* linears, int count, int M,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* decode_linear_stack for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): no workspace argument; the split-K partial sums go to a static
 * device buffer of SKINNY_STATIC_SCRATCH_BYTES that the library holds on each
 * GPU it runs on until the process ends.  Nothing is allocated on the call
 * path (the first call on a device only looks up the buffer's address there),
 * and nothing is copied: its launches hold at most
 * SKINNY_MAX_LINEARS_PER_LAUNCH linears each, descriptors in the arguments.
 *   A call is accepted only if skinny_stack_workspace_bytes of each of its
 *   launches (every SKINNY_MAX_LINEARS_PER_LAUNCH consecutive linears of one
 *   dtype, in call order) is <= SKINNY_STATIC_SCRATCH_BYTES (a bound from the
 *   shapes alone, so the same call is accepted on every device); otherwise
 *   SKINNY_ERR_WORKSPACE, returned before anything is enqueued.  Every other argument rule and
 *   error is that of decode_linear_stack.
 *   All calls on one GPU share its buffer, which keeps the last call's
 *   contents: calls on one stream are ordered and safe, but calls that may
 *   overlap on one GPU (other streams, other host threads) race on it and
 *   give wrong results.  No part of the buffer needs to start at zero. */
#define SKINNY_STATIC_SCRATCH_BYTES (64u << 20)
skinny_status decode_linear_stack_noalloc(const skinny_linear* linears, int count, int M,
                                          void* stream);

/* decode_linear_stack with an explicit plan (plan may be NULL = automatic). */
skinny_status skinny_linear_run(const skinny_linear* linears, int count, int M,
                                const skinny_plan* plan, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Number of main-kernel launches a call over these linears makes on a stream
 * not under graph capture: one per dtype present (per 4096 linears of it);
 * 0 if invalid. */
int skinny_launch_count(const skinny_linear* linears, int count);

/* skinny_linear_run that also records events around each main-kernel launch,
 * for benchmarks: events[2 g] just before and events[2 g + 1] just after
 * launch g, on `stream`.  `events` is a host array of hipEvent_t created by
 * the caller; event_count must be >= 2 * skinny_launch_count(linears, count).
 * The second (combine) pass of each launch is enqueued after events[2 g + 1]. */
skinny_status skinny_linear_run_timed(const skinny_linear* linears, int count, int M,
                                      const skinny_plan* plan, void* const* events,
                                      int event_count, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Rows of W in one row group of the main kernel of this dtype, variant
 * (VECTOR or MFMA; 0 for AUTO, whose choice depends on the shapes) and M; 0 if
 * invalid.  For MFMA this is the 4-wave workgroup's 64; FP8 launches of M >= 2
 * tokens with at least 8 row groups of 128 rows per compute unit run 8-wave
 * workgroups with 128-row groups instead.  The split-K workspace holds fp32 partial sums laid out
 * [slot][M][band rows]: one slot per K-chunk of each row group of a linear the
 * launch splits; linears in order, then row groups, then K-chunks in K order. */
int skinny_band_rows(int dtype, int variant, int M);

/* The automatic plan (fills *out) of the launch of linears[0]'s dtype on
 * the current device: a call launches its linears grouped by dtype (one
 * launch per dtype, or launches of at most SKINNY_MAX_LINEARS_PER_LAUNCH under
 * graph capture), and each launch chooses its own variant (it can depend on
 * the launch's size).  out->variant, ->waves
 * (persistent waves of the main launch) and ->kernel (its form) are set. */
skinny_status skinny_plan_query(const skinny_linear* linears, int count, int M,
                                skinny_plan* out);

/* Greedy next token: idx[m] = the smallest n such that y[m][n] is the largest
 * of y[m][0..N), comparing the bf16 values (NaN ranks below every number,
 * -inf included, so a row of NaNs gives 0).  This is the decode step's on-device argmax
 * ("Developing a custom Qwen2.5 72B inference engine from scratch - what is
 * the real bottleneck?", section 5, third lever: pick the next token on the
 * GPU rather than copying the logits back to the host).
 *   y          [M][N] bf16, device, 2-byte aligned (read 16 bytes at a time
 *              when y is 16-byte aligned and N % 8 == 0)
 *   idx        [M] int32, device, 4-byte aligned, written
 *   workspace  device, 16-byte aligned, >= skinny_argmax_workspace_bytes(M, N)
 *              (a (value, index) pair per 4096 logits of a row)
 * y, idx and the workspace must not overlap.  1 <= M <= SKINNY_MAX_M, N >= 1;
 * errors are returned before anything is enqueued.  Two launches, no
 * atomics; the result does not depend on the launch. */
size_t skinny_argmax_workspace_bytes(int M, int N);
skinny_status skinny_argmax_bf16(const void* y, int M, int N, int* idx, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* The vocabulary projection and its greedy token in one call (same section
 * and lever): runs the one linear `head` (N = vocabulary size, K = hidden
 * size, head->y = the logits [M][N], written) exactly as decode_linear_stack
 * would, and writes into next_token[M] (device int32) what skinny_argmax_bf16
 * over those logits gives.  Where the linear runs on the vector kernel with K
 * unsplit, its launch also leaves one (value, index) pair per workgroup and
 * token and a single pass reduces them; otherwise the two argmax passes run
 * after the linear.  next_token must not overlap x, W, w_scale, y or the
 * workspace.  The workspace serves the linear and the argmax (stream order),
 * so it needs skinny_lm_head_workspace_bytes(head, M) bytes (0 for invalid
 * arguments); less returns SKINNY_ERR_WORKSPACE before anything is enqueued. */
size_t skinny_lm_head_workspace_bytes(const skinny_linear* head, int M);
skinny_status skinny_lm_head_argmax(const skinny_linear* head, int M, int* next_token,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* One gated MLP of a decoder layer (Qwen2.5's SiLU-gated unit): y = down(h),
 * h = silu(g) * u, [g | u] = x . W_gate_up^T ("Multi-GPU Inference and
 * Serving at Scale", Example 3: a column-split linear, the activation, then a
 * row-split linear; the Qwen2.5 72B engine report, section 3, the MLP of each
 * layer).  All pointers are device pointers:
 *   x          [M][H] bf16                    y          [M][H] bf16, written
 *   w_gate_up  [2I][H] bf16 or E4M3FN: rows 0..I-1 the gate, I..2I-1 the up
 *   w_down     [H][I] bf16 or E4M3FN
 *   s_gate_up  [ceil(2I/128)][ceil(H/128)] fp32, s_down [ceil(H/128)][ceil(I/128)]
 *              fp32 (FP8 only; NULL for bf16)
 * g and u are the gate_up linear's bf16 outputs; h = bf16(silu(g) * u) is
 * computed in fp32 (silu(g) = g / (1 + e^-g)) while down stages its input, so
 * no separate activation pass runs.  Both linears accumulate in fp32 and are
 * within the bound of each linear.  The intermediate [M][2I] bf16 lives in
 * the workspace (skinny_mlp_workspace_bytes(mlp, M), 0 for invalid
 * arguments).  H % 8 == 0 and I % 8 == 0 (bf16) or % 16 (FP8); y must not
 * overlap x, the weights, the scales or the workspace, and x must not overlap
 * the workspace.  reserved must be 0. */
typedef struct skinny_mlp {
  int dtype;
  int H;
  int I;
  int reserved;
  const void* w_gate_up;
  const float* s_gate_up;
  const void* w_down;
  const float* s_down;
  const void* x;
  void* y;
} skinny_mlp;
size_t skinny_mlp_workspace_bytes(const skinny_mlp* mlp, int M);
skinny_status skinny_mlp_swiglu(const skinny_mlp* mlp, int M, void* workspace,
                                size_t workspace_bytes, void* stream);

/* One linear of a mixture-of-experts layer over the routes of a decode or
 * verify batch.  A router sends each of T tokens to topk experts, every
 * expert being its own small network ("Multi-GPU Inference and Serving at
 * Scale", Example 8); a verify step passes a handful of tokens through the
 * weight-only FP8 expert matmuls ("9% faster GLM-5.3-Flash prefill with
 * GPU-to-GPU IPC (and why TileLang didn't help)", section "TileLang: twice as
 * fast, and no faster").  Route r = t * topk + j is token t's j-th choice,
 * e = ids[r]:
 *   y[r] = x_r . W_e^T, x_r = x[t] (default) or x[r] (SKINNY_MOE_X_PER_ROUTE),
 *   y[r] = 0 for every r whose e is outside [0, E).
 * With SKINNY_MOE_SWIGLU each x row holds [g | u] (2K values) and x_r is
 * bf16(silu(g) * u) computed in fp32 as the input is staged: the experts'
 * down projection reads their gate_up outputs directly.
 *   experts->w        [E][N][K] bf16 or E4M3FN (expert e at e * N * K)
 *   experts->w_scale  [E][ceil(N/128)][ceil(K/128)] fp32 (FP8), NULL (bf16)
 *   x                 [T][K] bf16, or [T * topk][K]; 2K columns with SWIGLU
 *   ids               [T][topk] int32, device, read by the kernel (no host
 *                     synchronization); any values (duplicates included)
 *   y                 [T * topk][N] bf16, written
 * Each chosen expert's weights are streamed once for all of its routes, in
 * one persistent launch that finds the routes per expert itself (plus a
 * second pass when K is split).  Accumulation is fp32 with the single-linear
 * bound per route.  Requirements as for a linear (K % 8 or % 16, 16-byte
 * aligned x, y, w and workspace; 4-byte aligned ids and w_scale), plus
 * 1 <= T <= SKINNY_MAX_M, 1 <= topk <= SKINNY_MAX_TOPK, E >= 1; y must not
 * overlap x, ids, the weights, the scales or the workspace, and the
 * workspace must not overlap x or ids.  Workspace:
 * skinny_moe_workspace_bytes(experts, T, topk, flags), 0 for invalid
 * arguments. */
#define SKINNY_MAX_TOPK 16
enum skinny_moe_flags { SKINNY_MOE_X_PER_ROUTE = 1, SKINNY_MOE_SWIGLU = 2 };
typedef struct skinny_experts {
  int dtype;            /* SKINNY_BF16 or SKINNY_FP8_BS128 */
  int E;                /* experts                          */
  int N;                /* rows of each expert's W          */
  int K;                /* columns of each expert's W       */
  const void* w;
  const float* w_scale;
} skinny_experts;
size_t skinny_moe_workspace_bytes(const skinny_experts* experts, int T, int topk, int flags);
skinny_status skinny_moe_linear(const skinny_experts* experts, const void* x, const int* ids,
                                int T, int topk, int flags, void* y, void* workspace,
                                size_t workspace_bytes, void* stream);
/* skinny_moe_linear recording events[0] / events[1] (hipEvent_t, created by
 * the caller) just before and after its main launch, for benchmarks. */
skinny_status skinny_moe_linear_timed(const skinny_experts* experts, const void* x,
                                      const int* ids, int T, int topk, int flags, void* y,
                                      void* const* events, void* workspace,
                                      size_t workspace_bytes, void* stream);
/* The main kernel skinny_moe_linear takes for these experts and routes, for
 * tests and benchmarks: out->variant is SKINNY_VARIANT_VECTOR (the row
 * kernel, for one-token slices of rows long enough to keep its loads in
 * flight) or SKINNY_VARIANT_MFMA (the tile kernel); out->kernel names the
 * kernel's form; out->waves and out->reserved are 0.  Host logic only (no device call).  Errors: the
 * argument checks of skinny_moe_linear on experts, T, topk and flags, and
 * SKINNY_ERR_INVALID_ARG for a NULL out. */
skinny_status skinny_moe_plan_query(const skinny_experts* experts, int T, int topk, int flags,
                                    skinny_plan* out);

/* The experts' gated MLP over the routes of a batch (the same sources as
 * skinny_moe_linear: the router's top-k experts, each its own small MLP whose
 * SiLU-gated activation sits between its two linears, "Multi-GPU Inference
 * and Serving at Scale", Examples 3 and 8).  For route r = t * topk + j,
 * e = ids[r]:
 *   [g | u] = bf16(x[t] . Wgu_e^T),  y[r] = bf16(silu(g) * u) . Wdn_e^T,
 * exactly skinny_moe_linear(gate_up, x, ids, ..., flags 0) into a
 * [T * topk][2I] buffer followed by skinny_moe_linear(down, that buffer, ids,
 * ..., SKINNY_MOE_X_PER_ROUTE | SKINNY_MOE_SWIGLU, y).  y[r] = 0 for routes
 * whose e is outside [0, E).
 *   gate_up  E experts of N = 2I rows, K = H columns
 *   down     the same E experts (same dtype or not) of N rows, K = I columns
 *   x        [T][H] bf16;  ids [T][topk] int32, device;  y [T * topk][N] bf16
 * One token (T = 1, topk <= 16, both linears of one dtype, and each
 * workgroup's rows within the one-token kernel's registers) runs as one
 * launch: every wave issues the loads of all its gate_up and down rows at its
 * start, and the workgroups (one or two per CU, all resident) meet once
 * between the linears through a counter in the workspace.  A wait there gives
 * up after a bounded number of polls (skinny_moe_mlp_set_spin_limit) and then
 * sets the flag word, leaving y invalid; it never hangs.  Other calls make the
 * two launches.
 *   Workspace: skinny_moe_mlp_workspace_bytes(gate_up, down, T, topk) bytes,
 * 256-byte aligned; 0 for invalid arguments.  Its first
 * SKINNY_MOE_MLP_COUNTER_BYTES hold a counter (bytes 0-7: workgroups of the
 * one-launch form finished over all calls, a multiple of the grid between
 * calls) and a flag (bytes 8-11, nonzero once a wait gave up; the caller
 * clears it): zero them once before the first call on that workspace, do not
 * hand the workspace to other calls in between, and do not run two calls on
 * it at once.  The gate_up outputs follow: [T * topk][2I] bf16 (two launches),
 * or [topk][I] 64-bit words, each this call's number (low 32 bits of the
 * counter / grid + 1) above two bf16 values (one launch; rows of routes with
 * no expert keep what they held). */
#define SKINNY_MOE_MLP_COUNTER_BYTES 256
/* Requirements and errors as for skinny_moe_linear on both linears, plus gate_up->E ==
 * down->E and gate_up->N == 2 * down->K (else SKINNY_ERR_INVALID_ARG); y
 * must not overlap x, ids, the weights, the scales or the workspace, and the
 * workspace must not overlap x, ids, the weights or the scales. */
size_t skinny_moe_mlp_workspace_bytes(const skinny_experts* gate_up, const skinny_experts* down,
                                      int T, int topk);
skinny_status skinny_moe_mlp_swiglu(const skinny_experts* gate_up, const skinny_experts* down,
                                    const void* x, const int* ids, int T, int topk, void* y,
                                    void* workspace, size_t workspace_bytes, void* stream);
/* skinny_moe_mlp_swiglu recording events[0] / events[1] just before and after
 * its main launch (the one launch, or gate_up's), for benchmarks. */
skinny_status skinny_moe_mlp_swiglu_timed(const skinny_experts* gate_up,
                                          const skinny_experts* down, const void* x,
                                          const int* ids, int T, int topk, void* y,
                                          void* const* events, void* workspace,
                                          size_t workspace_bytes, void* stream);
/* Polls before the one-token launch's wait gives up (default 4194304; a
 * negative value makes it give up without waiting).  Process-wide; read when
 * a call is enqueued.  For tests of that path. */
void skinny_moe_mlp_set_spin_limit(long long polls);
/* The plan of skinny_moe_mlp_swiglu's main launch on the current device:
 * kernel SKINNY_KERNEL_MOE_MLP1 (variant VECTOR, waves of its grid) for the
 * one launch, else skinny_moe_plan_query's answer for the gate_up launch. */
skinny_status skinny_moe_mlp_plan_query(const skinny_experts* gate_up, const skinny_experts* down,
                                        int T, int topk, skinny_plan* out);

/* ------------------------------------------------------------------------
 * The step's operators between the QKV linear and the O linear: the paged
 * key/value cache and the attention over it (grouped query heads: "Developing
 * a custom Qwen2.5 72B inference engine from scratch - what is the real
 * bottleneck?", section 6.3).
 *
 * A pool of `pages` pages of `page_tokens` tokens holds the keys and values of
 * all sequences, one layer's at a time; all pointers are device pointers:
 *   k, v              [pages][kv_heads][page_tokens][head_dim], bf16 or e4m3
 *   k_scale, v_scale  [pages][kv_heads] fp32 (FP8 only, else NULL): an e4m3
 *                     code of that page and head stands for code * scale
 * page_tokens is a power of two from SKINNY_KV_MIN_PAGE to SKINNY_KV_MAX_PAGE,
 * head_dim 64, 128 or 256, kv_heads at most SKINNY_KV_MAX_HEADS; k and v are
 * 16-byte aligned.  reserved must be 0. */
enum skinny_kv_dtype { SKINNY_KV_BF16 = 0, SKINNY_KV_FP8 = 1 };
#define SKINNY_KV_MIN_PAGE 16
#define SKINNY_KV_MAX_PAGE 128
#define SKINNY_KV_MAX_HEADS 1024
#define SKINNY_KV_MAX_SEQS 65536
#define SKINNY_KV_MAX_TOKENS 1048576
typedef struct skinny_kv_cache {
  int dtype;            /* SKINNY_KV_BF16 or SKINNY_KV_FP8 */
  int pages;
  int kv_heads;
  int page_tokens;
  int head_dim;
  int reserved;
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
} skinny_kv_cache;

/* The sequences of a step, ragged (device arrays, read by the kernels):
 *   q_start     [seqs + 1] int32, ascending: sequence s owns rows q_start[s] ..
 *               q_start[s + 1] - 1 of the step's `tokens` rows (none if equal);
 *               rows from q_start[seqs] on belong to no sequence
 *   kv_len      [seqs] int32: the sequence's tokens with this step's included,
 *               so row i of its n rows stands at position kv_len - n + i
 *   page_table  [seqs][max_pages] int32: page j holds positions j * page_tokens
 *               .. (j + 1) * page_tokens - 1
 * One token per sequence is plain decode, several are a verify step or a
 * prompt.  The values are not trusted: row ranges are cut to 0 .. tokens,
 * lengths to the page table, and a page outside the pool is one that is
 * neither written nor seen.  Entries of page_table past a sequence's length
 * are not used.  reserved must be 0. */
typedef struct skinny_kv_batch {
  int seqs;             /* 1 .. SKINNY_KV_MAX_SEQS   */
  int tokens;           /* 1 .. SKINNY_KV_MAX_TOKENS */
  int max_pages;        /* >= 1, max_pages * page_tokens <= 2^30 */
  int reserved;
  const int* q_start;
  const int* kv_len;
  const int* page_table;
} skinny_kv_batch;

/* Appends a step's keys and values to the cache, rotating queries and keys by
 * their positions on the way.
 *   qkv       [tokens][(q_heads + 2 kv_heads) head_dim] bf16, the QKV linear's
 *             y: query heads, then key heads, then value heads; 16-byte aligned
 *   inv_freq  [rotary_dim / 2] fp32, or NULL with rotary_dim 0 (no rotation)
 *   q_out     [tokens][q_heads head_dim] bf16, written, 16-byte aligned
 * Of each query and key head the first rotary_dim values (a multiple of 16) are
 * rotated in pairs (a, b) = (x[i], x[i + rotary_dim / 2]), or (x[2i], x[2i + 1])
 * with interleaved = 1, by the angle t = position * inv_freq[i]:
 * a' = a cos t - b sin t, b' = a sin t + b cos t, angles and products in fp64.
 * Queries, and a bf16 cache's keys and values, are rounded once, to bf16.
 *   An FP8 cache keeps one scale per page, head and k or v.  Rows that begin a
 * page set it to the smallest power of two s, 2^-64 at least, with |x| <= 448 s
 * for all of this step's rows in the page; rows that continue a page set it to
 * the larger of that and the scale the page has, and where it grows the
 * sequence's earlier codes in the page are rounded again to the new scale
 * (exact but for codes that become subnormal, unless the caller had set a scale
 * that is no power of two; that one is kept while it is large enough).  Codes are
 * x / scale to nearest even; infinities, and values that the rotation takes past
 * fp32's largest number, become the largest code and take no part in the scale,
 * NaN stays NaN.
 *   Written are q_out's rows that belong to a sequence and the cache's slots of
 * their positions (and, as above, earlier codes in the same page), nothing
 * else: positions below 0 or past the page table have no slot.  A page that
 * receives rows must belong to one sequence only (shared full pages are fine:
 * they receive none); if two sequences, or two places of one, write one
 * page, its contents are undefined.  A second call with the same inputs changes nothing.
 * q_heads is a multiple of kv_heads.  No buffer that is written may overlap
 * another operand.  No workspace; one launch. */
skinny_status skinny_kv_append(const skinny_kv_cache* cache, const skinny_kv_batch* batch,
                               const void* qkv, int q_heads, const float* inv_freq,
                               int rotary_dim, int interleaved, void* q_out, void* stream);

/* Each row's attention over its sequence's cache, up to and including the
 * row's own position (kv_append has put it there):
 *   out[row][head] = sum_j p_j v_j,  p = softmax_j(scale * q[row][head] . k_j)
 * over the positions j <= kv_len - n + i of row i, query head `head` reading KV
 * head head / (q_heads / kv_heads).
 *   q, out  [tokens][q_heads head_dim] bf16, 16-byte aligned; out is written
 *   scale   usually 1 / sqrt(head_dim); finite, and times log2 e too
 * Scores, the softmax's statistics and sums are fp32; the probabilities go into
 * the product with v as two bf16 numbers each, within 2^-16.  Keys and values of positions that a
 * row does not see do not reach it, whatever they hold; an infinite value that
 * it sees gives that infinity, however small its probability.  A row that sees no
 * position gets zeros, one that sees scores of -inf only NaN (0 / 0); rows that
 * belong to no sequence are left as they were.
 * Results are reproducible bitwise for the same lengths, shapes and device.
 *   workspace  >= skinny_kv_attention_workspace_bytes(cache, batch, q_heads)
 *              bytes (0 for invalid arguments; pure host arithmetic on the
 *              shapes, for which a step of fewer sequences can need more: its
 *              sequences have more rows), 16-byte aligned; contents undefined
 *              before and after, so calls that may overlap need their own
 * out must not overlap q, the cache, the batch's arrays or the workspace, nor
 * the workspace any of them.  A step that could be more blocks of work than 32 bits
 * count is refused (SKINNY_ERR_UNSUPPORTED, and 0 for its workspace); none is while
 * kv_heads * (tokens * q_heads / kv_heads / 16 + seqs) * (max_pages * page_tokens
 * / 32 + 1) stays below 2^31 - 1. */
size_t skinny_kv_attention_workspace_bytes(const skinny_kv_cache* cache,
                                           const skinny_kv_batch* batch, int q_heads);
skinny_status skinny_kv_attention(const skinny_kv_cache* cache, const skinny_kv_batch* batch,
                                  const void* q, int q_heads, float scale, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* The end of a verify step: which drafted tokens the target keeps, and the one
 * that follows them, from the target's logits and given random numbers, so that
 * the tokens are distributed as the target's own ("9% faster GLM-5.3-Flash
 * prefill with GPU-to-GPU IPC (and why TileLang didn't help)", section
 * "TileLang: twice as fast, and no faster": a verify step of drafted tokens).
 *   Sequence s has rows q_start[s] .. q_start[s + 1] - 1 (device int32, as in
 * skinny_kv_batch, values not trusted); tokens[row] is the token that the step
 * read at that row: a sequence's first one is its last sure token, the others
 * are drafted.  logits[row] are the target's for the place after it, and
 * draft_logits[row] those that the token at row + 1 was drawn from (the rows of a
 * greedy sequence, a sequence's last row and rows of none are not read).  With p = softmax(logits[row] / t), q =
 * softmax(draft_logits[row] / t), t = temperature[s] and d = tokens[row + 1]:
 *   row by row, d is kept while accept_u[row] * q(d) < p(d);
 *   at the first row that keeps none, the next token is drawn from max(0, p - q)
 *   (from p if that is zero everywhere), and at a sequence's last row, all
 *   drafts kept, from p: the smallest v whose running sum, v included, is above
 *   sample_u[s] times the total.
 * draft_logits NULL: the drafts are given, not drawn (q = 1 at d).  temperature
 * NULL: 1 for all.  t <= 0 (or NaN): greedy, p is 1 at the lowest index of the
 * largest logit, and draft_logits are not asked.  A NaN logit counts as -inf; a row
 * without any logit above -inf keeps nothing and gives token 0.  A drafted token
 * outside 0 .. vocab - 1 is not kept.
 *   out_tokens [rows] int32: at a sequence's rows its kept drafts, the next
 *     token, then -1; rows of no sequence are left as they were
 *   accepted [seqs] int32: drafts kept, so accepted + 1 tokens are new (0, and
 *     none, for a sequence without rows).  -1, and -1 in all of its out_tokens, if
 *     a wait inside the launch gave up (skinny_verify_set_spin_limit; by default
 *     after polls of many times what a launch takes): the step is to be repeated
 * Probabilities and sums are fp64, and an entry below 2^-1000 of its row's largest
 * probability has none: it is neither drawn nor kept (so masks of the type's lowest
 * value hold for a random number of 0, too).  The tokens are then those of exact
 * arithmetic unless a random number lies within about 2e-13 of a boundary,
 * relative to it.
 *   accept_u [rows], sample_u [seqs] fp32, uniform on [0, 1)
 *   logits, draft_logits [rows][vocab] bf16 or fp32, aligned to their type (read
 *     16 bytes at a time when 16-byte aligned and rows are multiples of 16 bytes)
 *   workspace >= skinny_verify_workspace_bytes(rows, seqs, vocab) bytes (0 for
 *     invalid arguments; more rows, sequences or entries never need less),
 *     16-byte aligned, contents undefined before and after, so calls that may
 *     overlap need their own
 * out_tokens, accepted and the workspace must not overlap anything else. */
enum skinny_logits_dtype { SKINNY_LOGITS_BF16 = 0, SKINNY_LOGITS_F32 = 1 };
#define SKINNY_VERIFY_MAX_ROWS 65535
#define SKINNY_VERIFY_MAX_VOCAB 16777216
typedef struct skinny_verify {
  int dtype;            /* enum skinny_logits_dtype              */
  int vocab;            /* 1 .. SKINNY_VERIFY_MAX_VOCAB          */
  int rows;             /* 1 .. SKINNY_VERIFY_MAX_ROWS           */
  int seqs;             /* 1 .. SKINNY_VERIFY_MAX_ROWS           */
  const int* q_start;
  const void* logits;
  const void* draft_logits;
  const int* tokens;
  const float* temperature;
  const float* accept_u;
  const float* sample_u;
  int* out_tokens;
  int* accepted;
} skinny_verify;
size_t skinny_verify_workspace_bytes(int rows, int seqs, int vocab);
skinny_status skinny_verify_draft(const skinny_verify* verify, void* workspace,
                                  size_t workspace_bytes, void* stream);
/* Polls for another workgroup's sums before a sampling sequence gives up (default
 * 65536; a negative value makes it give up without waiting).  Process-wide; read
 * when a call is enqueued.  For tests of that path. */
void skinny_verify_set_spin_limit(long long polls);

/* ------------------------------------------------------------------------
 * What a layer computes between and beside its linears.  Values of two types
 * share one enum; arrays need the alignment of their type only. */
enum skinny_values_dtype { SKINNY_VALUES_BF16 = 0, SKINNY_VALUES_F32 = 1 };

/* The residual's update with a block's output, and the norm that makes the next
 * linear's x, for every row t of a step (each layer's attention and MLP blocks
 * add to the residual between their linears: "Developing a custom Qwen2.5 72B
 * inference engine from scratch - what is the real bottleneck?", section 3):
 *   b  = sum_j route_weights[t][j] * block[t * routes + j]
 *   b  = norm(b) * (weight_offset + post_weight) + post_bias    (post_weight given)
 *   b  = gate * b                                               (gate given)
 *   h  = residual_scale * residual[t] + block_scale * b
 *   residual_out[t] = h
 *   out[t] = norm(h) * (weight_offset + weight) + bias
 *   norm(v) = v / sqrt(mean(v^2) + eps)                         SKINNY_NORM_RMS
 *           = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) SKINNY_NORM_LAYER
 * What is NULL takes no part: no block (b = 0), no residual (h = block_scale * b),
 * weights of norm(h) and route_weights 1, biases 0; residual_out or out NULL: not
 * written.  One of block and residual, and one of residual_out and out, are needed;
 * post_weight, post_bias, gate and route_weights need a block, post_bias a
 * post_weight, bias an out.
 *   block         [rows * routes][width] bf16: the O linear's, mlp_swiglu's (routes
 *                 1) or moe_mlp_swiglu's y; routes 1 .. SKINNY_MAX_TOPK
 *   route_weights [rows][routes] fp32
 *   residual, residual_out  [rows][width] of residual_dtype; residual_out may be
 *                 residual itself (same address), and overlaps nothing else
 *   gate          [width], or [rows][width] with gate_rows = 1; weights, biases
 *                 [width]; all of weight_dtype
 *   out           [rows][width] bf16, overlaps nothing else
 * Values are fp32 from the load on (out is made of h before residual_out's
 * rounding), means and sums of squares fp64, so they neither overflow nor vanish;
 * outputs are rounded once, to nearest even.  A value or sum that passes fp32's
 * largest number is infinite.  A row whose mean of squares plus eps is 0 gives NaN
 * (0 / 0); a row with a NaN or an infinity does not touch other rows.
 * Bitwise reproducible.  No workspace; one launch.  reserved must be 0; eps >= 0
 * and finite, the scales and the offset finite. */
enum skinny_norm_kind { SKINNY_NORM_RMS = 0, SKINNY_NORM_LAYER = 1 };
#define SKINNY_NORM_MAX_ROWS 1048576
#define SKINNY_NORM_MAX_WIDTH 32768
typedef struct skinny_norm {
  int kind;             /* enum skinny_norm_kind          */
  int rows;             /* 1 .. SKINNY_NORM_MAX_ROWS      */
  int width;            /* 1 .. SKINNY_NORM_MAX_WIDTH     */
  int routes;           /* 1 .. SKINNY_MAX_TOPK           */
  int residual_dtype;   /* enum skinny_values_dtype       */
  int weight_dtype;     /* enum skinny_values_dtype       */
  int gate_rows;        /* 0 or 1                         */
  int reserved;
  float eps;
  float residual_scale;
  float block_scale;
  float weight_offset;
  const void* block;
  const float* route_weights;
  const void* post_weight;
  const void* post_bias;
  const void* gate;
  const void* residual;
  void* residual_out;
  const void* weight;
  const void* bias;
  void* out;
} skinny_norm;
skinny_status skinny_block_norm(const skinny_norm* norm, void* stream);

/* The low-rank adapters of many requests beside a shared projection ("Multi-GPU
 * Inference and Serving at Scale", Example 15: several adapters over one model's
 * weights).  Row t has adapter e = ids[t]:
 *   y[t] = base[t] + scale[e] * B_e (A_e x[t]),
 * and y[t] = base[t] for every t whose e is outside [0, adapters).  A projection
 * of several parts (q, k and v; gate and up) has an A and a B for each: slice i
 * covers the n[i] columns of y behind those of the slices before it.
 *   x         [rows][K] bf16, the projection's x; K % 8 == 0, 16-byte aligned;
 *             rank * K at most 2^30
 *   base, y   [rows][N] bf16, N = n[0] + .. + n[slices - 1]: the projection's y and
 *             the result; base NULL: y itself (added in place; rows without an
 *             adapter are then left as they were); base overlaps y in no other way
 *   a[i]      [adapters][rank][K] bf16, b[i] [adapters][n[i]][rank] bf16, 16-byte
 *             aligned; both NULL: a slice without adapters
 *   rank      of the pool, a multiple of 8 up to SKINNY_LORA_MAX_RANK
 *   ranks     [adapters] int32 or NULL: adapter e uses its first ranks[e] (cut to
 *             0 .. rank) rows of A and columns of B; the others are not used,
 *             whatever they hold
 *   scale     [adapters] fp32, or NULL: 1
 *   ids       [rows] int32, device, read by the kernels; any values
 * Rows of one adapter share the reading of its weights, 64 at a time.  Sums are fp32;
 * scale * (A x), as fp32, enters the product with B without another rounding (numbers
 * below 2^-110 within 2^-133); y is rounded once.  Infinities and NaN come out as fp32
 * sums of those products have them.  A row's result does not depend on the other rows'
 * values; results are bitwise reproducible for the same sizes.
 *   workspace >= skinny_lora_workspace_bytes(lora, rows) bytes (0 for invalid
 *             arguments), 16-byte aligned, contents undefined before and after, so
 *             calls that may overlap need their own
 * Up to 64 rows take two launches, more three, more than 512 four.  A call of more
 * workgroups than a launch may have threads for (2^32) is refused
 * (SKINNY_ERR_UNSUPPORTED).  y and the workspace must not overlap anything else. */
#define SKINNY_LORA_MAX_ROWS 1048576
#define SKINNY_LORA_MAX_RANK 256
#define SKINNY_LORA_MAX_ADAPTERS 8192
#define SKINNY_LORA_MAX_SLICES 4
typedef struct skinny_lora {
  int adapters;         /* 1 .. SKINNY_LORA_MAX_ADAPTERS  */
  int rank;             /* 8 .. SKINNY_LORA_MAX_RANK      */
  int K;
  int slices;           /* 1 .. SKINNY_LORA_MAX_SLICES    */
  int n[SKINNY_LORA_MAX_SLICES];
  const void* a[SKINNY_LORA_MAX_SLICES];
  const void* b[SKINNY_LORA_MAX_SLICES];
  const int* ranks;
  const float* scale;
} skinny_lora;
size_t skinny_lora_workspace_bytes(const skinny_lora* lora, int rows);
skinny_status skinny_lora_linear(const skinny_lora* lora, const void* x, const int* ids, int rows,
                                 const void* base, void* y, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* A router's choice: the ids that skinny_moe_linear and skinny_moe_mlp_swiglu
 * take, and the weights with which skinny_block_norm sums their outputs ("Multi-GPU
 * Inference and Serving at Scale", Example 8: each token goes to its top experts).
 * For row t with logits l:
 *   s = softmax(l), or 1 / (1 + e^-l) with SKINNY_ROUTE_SIGMOID
 *   c = s + bias (bias [experts] fp32; only the choice sees it); without a bias
 *       the choice goes by l itself, whose order s shares
 *   with groups > 1, the experts are `groups` equal runs; those of the top_groups
 *       best groups are chosen from, a group being worth its largest c (with a
 *       bias the sum of its two largest)
 *   ids[t]     = the topk largest c, descending; equal ones (and groups) by the lowest
 *                index
 *   weights[t] = scale * s[ids], over their sum first with renormalize = 1 (where
 *                that sum is 0, they are 0)
 * A NaN logit counts as -inf, +inf as fp32's largest number.  A row of -inf alone
 * has s = 0.  A c or a sum of two that is NaN (by its bias) counts as -inf.
 * s, c and sums are fp64; weights are rounded once.
 *   logits  [rows][experts] bf16 or fp32;  ids [rows][topk] int32 and weights
 *           [rows][topk] fp32, written, neither overlapping anything else
 * experts % groups == 0, topk <= top_groups * (experts / groups).  No workspace;
 * one launch.  reserved must be 0; scale finite. */
enum skinny_route_scoring { SKINNY_ROUTE_SOFTMAX = 0, SKINNY_ROUTE_SIGMOID = 1 };
#define SKINNY_ROUTE_MAX_ROWS 1048576
#define SKINNY_ROUTE_MAX_EXPERTS 1024
#define SKINNY_ROUTE_MAX_GROUPS 64
typedef struct skinny_route {
  int dtype;            /* enum skinny_values_dtype, of the logits */
  int scoring;          /* enum skinny_route_scoring               */
  int rows;             /* 1 .. SKINNY_ROUTE_MAX_ROWS              */
  int experts;          /* 1 .. SKINNY_ROUTE_MAX_EXPERTS           */
  int topk;             /* 1 .. SKINNY_MAX_TOPK                    */
  int groups;           /* 1 .. SKINNY_ROUTE_MAX_GROUPS            */
  int top_groups;       /* 1 .. groups                             */
  int renormalize;      /* 0 or 1                                  */
  float scale;
  int reserved;
  const void* logits;
  const float* bias;
  int* ids;
  float* weights;
} skinny_route;
skinny_status skinny_moe_route(const skinny_route* route, void* stream);

/* Static text for a status code; never NULL. */
const char* skinny_status_string(int status);

/* SKINNY_ABI_VERSION of the loaded library. */
int skinny_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_GEMM_H */

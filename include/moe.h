/*
 * moe.h -- C ABI of a single-GPU mixture-of-experts layer for NVIDIA GB300
 * (sm_103a): router top-k, device-side schedule, dispatch gather, grouped
 * expert GEMMs (BF16 or OCP MXFP8) with fused SwiGLU and quantisation,
 * deterministic combine, an optional BF16 shared expert, and the backward
 * pass.
 *
 * The method is the one described by the "Mixture-of-Kittens" pages (Cursor's
 * MoE training megakernel): token routing, a device-side schedule kernel with
 * no CPU synchronisation, dispatch, expert grouped GEMMs with SwiGLU and
 * activation quantisation fused in, and a bitwise-deterministic combine
 * ("Mixture-of-Kittens" wiki page, TL;DR, flowchart and Key claims).  The
 * pages' inter-GPU dispatch/combine become intra-GPU gathers here.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All pointers are DEVICE pointers unless stated otherwise; the caller owns
 *   every buffer.  The library allocates nothing and keeps no per-call state.
 * - Every tensor is row-major and contiguous.  bf16 = IEEE bfloat16 bits.
 *   Pointers must be 16-byte aligned (MOE_ERR_ALIGN otherwise).
 * - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *   default stream): no host synchronisation, no device-to-host copy.  Only
 *   moe_get_status synchronises.
 * - Return value: MOE_OK (0), or a negative moe_status for errors detected on
 *   the host before anything is launched.  Errors detected on the device
 *   (a bounded wait that ran out) are recorded in the status word inside the
 *   workspace and read with moe_get_status.
 * - Results are bitwise reproducible: the same inputs give the same bits on
 *   every call (fixed floating-point operation order, no atomics on floats).
 *
 * MXFP8 format (OCP Microscaling v1.0, as the layer's MXFP8 configurations
 * state): codes are E4M3 bytes; every 32 consecutive elements along the
 * reduction axis K share one E8M0 scale byte (2**(byte-127)); the shared
 * exponent is floor(log2(amax)) - 8, clamped to [-127, 127] (an all-zero
 * block gets byte 0); codes are round-to-nearest-even and saturate to +-448.
 *
 * MXFP8 scale layouts.  A matrix with `rows` rows and reduction length K has
 * rows*K/32 scale bytes.
 *   Canonical (every scale this ABI takes from or returns to the caller):
 *     [rows, K/32] row-major, the scale of (row r, block b = column/32) at
 *     byte r*(K/32) + b.  Batched matrices stack along rows.
 *   Prepared (the expert GEMMs' operand layout; internal): the same bytes in
 *     the order the tensor cores' scale-factor copy reads them, made from
 *     canonical scales by moe_prepare_scales and turned back by
 *     moe_canonical_scales (rows and K multiples of 128).  moe_weights'
 *     *_scale fields and the scale buffers inside the workspace use it.  For
 *     reference, byte ((r/128)*(K/128) + b/4)*512 + (r%32)*16 + ((r%128)/32)*4
 *     + b%4 holds the scale of (r, b): 512-byte atoms of 128 rows x 4 blocks.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *moe_stream_t; /* same type as cudaStream_t */

typedef enum { MOE_BF16 = 0, MOE_MXFP8 = 1, MOE_NVFP4 = 2 } moe_dtype;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_ARG = -1,     /* NULL pointer, non-positive size, k > E, unknown name */
  MOE_ERR_SHAPE = -2,   /* shape outside what the kernels tile (see moe_config) */
  MOE_ERR_ALIGN = -3,   /* a pointer is not 16-byte aligned (around the layer: not as its entry point says) */
  MOE_ERR_CUDA = -4,    /* a CUDA runtime / driver call or a launch failed */
  MOE_ERR_DEVICE = -5,  /* current device is not sm_103 / sm_100 family */
  MOE_ERR_TIMEOUT = -6, /* device side: a bounded wait inside a kernel ran out */
  MOE_ERR_BOUNDS = -7   /* device side: an index read from a buffer fell outside its range; the
                           access was skipped (the layer: debug builds only, compiled with
                           -DMOE_DEBUG; the grouped products' offsets: every build) */
} moe_status;

/* moe_config.flags bits */
#define MOE_FLAG_BACKWARD 1 /* size the workspace for moe_backward as well */
/* Test hook for the device-side failure path: in moe_forward the gate/up
 * GEMM's load warp issues nothing (with a ring: the gather CTAs publish no
 * tile), so the waits for its data run out (limit 50 ms instead of 4 s); the
 * kernels drain and return, moe_get_status then reports MOE_ERR_TIMEOUT, and
 * the outputs of that call are undefined.  The CUDA context stays usable. */
#define MOE_FLAG_DEBUG_STARVE 2
/* Test hook for the fused quantisation points (MXFP8 experts; ignored with
 * BF16 experts): moe_forward also stores the fp32 SwiGLU output h -- the
 * values the gate/up GEMM's epilogue quantises -- in the workspace buffer
 * "h_dump" [padded rows, m] fp32, and moe_backward stores the bf16 dG|dU
 * values the SwiGLU-backward epilogue quantises in "dGU_dump" [padded rows,
 * 2m] bf16 (moe_buffer_info gives their offsets).  Quantising those dumps
 * with the format's definition must reproduce the codes and scales the
 * kernels wrote, byte for byte.  Nothing else changes.  Not available with a
 * dispatch ring (ring_rows > 0: MOE_ERR_ARG). */
#define MOE_FLAG_DEBUG_DUMP 4

/*
 * Layer shape.  T tokens, hidden d, expert intermediate m, E experts, top-k k.
 * Supported: 1 <= k <= min(E, 16), E <= 1024, d % 256 == 0, m % 128 == 0,
 * m_shared % 128 == 0 (0 = no shared expert), T*k < 2^31 - 127*E.  dtype is
 * the routed experts' arithmetic; the shared expert is always BF16.
 * MOE_NVFP4 (the NVFP4 variant of the expert GEMMs; the pages say the method
 * has none -- "Mixture-of-Kittens" wiki page, Key claims, MXFP8 bullet -- so
 * the format is NVIDIA's published NVFP4): packed E2M1 codes with an E4M3
 * scale per 16 along K and an fp32 second-level scale per tensor (2688 /
 * amax): x's over all T tokens, each expert matrix's own, and 1 for h.
 * Forward only (inference: MOE_FLAG_BACKWARD, a ring or a `saved` buffer give
 * MOE_ERR_ARG) and m % 256 == 0.  flags:
 * any of MOE_FLAG_BACKWARD, MOE_FLAG_DEBUG_STARVE and MOE_FLAG_DEBUG_DUMP, or 0
 * (moe_backward needs a workspace sized with MOE_FLAG_BACKWARD).
 *
 * Dispatch ring (MXFP8 only; "Mixture-of-Kittens" wiki page, flowchart, and
 * daily-ai-frontier summary, TL;DR: a fixed-size token ring between the
 * dispatch and the expert GEMMs, and an SM split between data movement and
 * GEMM work handing off through device counters):
 *   ring_rows  = 0: the dispatch writes every routed row to the workspace
 *                (one row per routed (token, expert) pair, padded per expert);
 *              > 0: a multiple of 128.  The forward's dispatch and gate/up
 *                GEMM run as one persistent launch: `gather_sms` SMs gather
 *                and quantise 128-row tiles of expert-sorted rows into a ring
 *                of ring_rows rows in the workspace, the other SMs run the
 *                GEMM on the ring, and each slot is refilled once every GEMM
 *                tile has loaded it.  Experts with more rows than the ring
 *                pass through it in pieces.  Results are bitwise identical to
 *                ring_rows = 0 for every ring size and SM split.
 *   gather_sms = gather SMs of the ring launch (0 = 8; at most 64).
 *   The ring needs d <= 8192 (MOE_ERR_SHAPE otherwise).
 *
 * Load-balancing term (aux_alpha > 0; the pages define none, so this is the
 * Switch-Transformer auxiliary loss taken over the k routed slots):
 *   L = aux_alpha * E * sum_e f_e * P_e,  f_e = counts_e / (T k),
 *   P_e = (1/T) sum_t softmax(logits_t)_e over all E experts.
 * moe_forward computes it after the schedule (fixed-order sums, bitwise
 * reproducible) into the workspace buffer "aux" = [L, P[E], f[E]] fp32
 * (moe_buffer_info); a training forward also keeps dL/dlogits =
 * aux_alpha E / T * p (f - sum_e f_e p_e), which moe_backward adds to
 * dlogits (the loss enters the objective with weight 1; f is piecewise
 * constant, so no gradient flows through the counts).
 */
typedef struct {
  int32_t T, d, m, E, k;
  int32_t m_shared;
  int32_t dtype; /* moe_dtype */
  int32_t flags;
  int32_t ring_rows;
  int32_t gather_sms;
  float aux_alpha; /* 0 = no load-balancing term */
} moe_config;

/*
 * Expert weights.  BF16 path: `gu` [E, 2m, d] bf16 (rows 0..m-1 of each
 * expert are the gate projection, m..2m-1 the up projection), `dn` [E, d, m]
 * bf16; the *_scale pointers are unused.
 * MXFP8 path: `gu` = E4M3 codes [E*2m, d] with prepared scales `gu_scale`
 * (rows E*2m, K d); `dn` = codes [E*d, m], `dn_scale` (rows E*d, K m) --
 * the codes from moe_quantize_weights(blocks_along_rows = 0) (or
 * moe_quantize_mx(transpose = 0)) of the bf16 masters, the scales that call's
 * canonical scales passed through moe_prepare_scales (an MXFP8 checkpoint's
 * codes and canonical scales can be used the same way).
 * Backward operands (NULL for a forward-only layer):
 *   BF16:  gu_t = [E, d, 2m] bf16 = per-expert transpose of gu,
 *          dn_t = [E, m, d] bf16 = per-expert transpose of dn
 *          (moe_transpose_bf16);
 *   MXFP8: gu_t = codes [E*d, 2m] + prepared gu_t_scale, dn_t = codes
 *          [E*m, d] + prepared dn_t_scale (moe_quantize_weights(
 *          blocks_along_rows = 1) of the masters, then moe_prepare_scales;
 *          moe_quantize_mx_both writes both orientations at once).
 * NVFP4 path: `gu` = packed E2M1 codes [E*2m, d/2] (element 2i in the low
 * nibble of byte i) with prepared E4M3 scales `gu_scale` (rows E*2m, 16-blocks
 * along d), `dn` = [E*d, m/2] with `dn_scale`, and the experts' second-level
 * scales gu_gscale [E], dn_gscale [E] fp32 -- all from moe_prepare_weights.
 * Shared expert (BF16 always; NULL when m_shared == 0): s_gu [2m_s, d],
 * s_dn [d, m_s]; for backward also s_gu_t [d, 2m_s], s_dn_t [m_s, d].
 */
typedef struct {
  const void *gu, *gu_scale;
  const void *dn, *dn_scale;
  const void *gu_t, *gu_t_scale;
  const void *dn_t, *dn_t_scale;
  const void *s_gu, *s_dn;
  const void *s_gu_t, *s_dn_t;
  const float *gu_gscale, *dn_gscale; /* NVFP4 only: second-level scales [E] */
} moe_weights;

/* Bytes of scratch (`ws`) that moe_route / moe_forward / moe_backward need
 * for this config (one buffer serves all three; 0 on invalid config). */
size_t moe_workspace_bytes(const moe_config *cfg);

/* Bytes of the activations a training forward saves for the backward
 * (`saved`; 0 on invalid config). */
size_t moe_saved_bytes(const moe_config *cfg);

/* Byte offset and size of a named sub-buffer of `saved` (which = 0) or of the
 * workspace (which = 1), for inspection by tests and tools.  Names include
 * "idx", "w", "counts", "offsets", "perm", "inv", "poff", "o", "GU", "s_GU",
 * "s_h", with BF16 experts "h" and with MXFP8 experts "xT", "xT_sf", "hT",
 * "hT_sf" (saved: column-blocked codes of the wgrad operands); "xs",
 * "xs_sf", "hq", "hq_sf", "s_out", "dX", "g" and, with MXFP8 experts,
 * "dOq", "dOq_sf", "dOT", "dOT_sf", "dGUq", "dGUq_sf", "dGUT", "dGUT_sf"
 * and, with MOE_FLAG_DEBUG_DUMP, "h_dump" and "dGU_dump"
 * (workspace; "dO" and "dGU" exist only with BF16 experts, whose backward
 * materialises them in bf16).  Row-indexed buffers use padded rows (see
 * moe_forward).  Returns MOE_OK or MOE_ERR_ARG (unknown name / buffer absent
 * for this config). */
int moe_buffer_info(const moe_config *cfg, int which, const char *name, size_t *offset,
                    size_t *bytes);

/* Number of padded expert-sorted rows the buffers are sized for:
 * roundup(T*k + 127*E, 128). */
int64_t moe_padded_rows(const moe_config *cfg);

/*
 * S0: MXFP8 weight quantisation ("Mixture-of-Kittens" wiki page, Key claims,
 * MXFP8 bullet: MXFP8 is the default expert format).
 * src: [batch, rows, cols] bf16.
 *   transpose = 0: codes [batch*rows, cols], blocks of 32 along cols;
 *                  canonical scales [batch*rows, cols/32].
 *   transpose = 1: codes [batch*cols, rows] = per-batch transpose, blocks of
 *                  32 along the original rows; canonical scales
 *                  [batch*cols, rows/32].
 * rows and cols must be multiples of 128.  Inputs must be finite.
 */
int moe_quantize_mx(const void *src, int batch, int rows, int cols, int transpose, void *codes,
                    void *scales, moe_stream_t stream);

/* S0 in the layer's own terms: the MXFP8 codes of the layer's stacked expert
 * weights, one bf16 master matrix [rows, cols] per expert (cfg->E of them,
 * back to back at w_bf16).
 *   blocks_along_rows = 0: the forward operand, blocks of 32 along cols
 *     (W_gu [E*2m, d] with rows = 2m, cols = d; W_dn [E*d, m]): as
 *     moe_quantize_mx(w_bf16, cfg->E, rows, cols, 0, ...).
 *   blocks_along_rows = 1: the backward operand, each expert's matrix
 *     transposed and quantised in blocks of 32 along its rows (W_gu^T
 *     [E*d, 2m], W_dn^T [E*m, d]): as moe_quantize_mx(..., 1, ...).
 * cfg must be a valid MXFP8 config (MOE_ERR_ARG otherwise); rows and cols
 * multiples of 128; inputs finite.  Asynchronous on `stream`. */
int moe_quantize_weights(const moe_config *cfg, const void *w_bf16, int rows, int cols, int blocks_along_rows,
                         void *codes, void *scales, moe_stream_t stream);

/* S0 for a training layer: both orientations from one read of the bf16
 * masters.  codes/scales exactly as moe_quantize_mx(transpose = 0) and
 * codes_t/scales_t exactly as moe_quantize_mx(transpose = 1) would write them
 * (bit-identical, canonical scales).  rows and cols multiples of 128; inputs
 * finite. */
int moe_quantize_mx_both(const void *src, int batch, int rows, int cols, void *codes, void *scales,
                         void *codes_t, void *scales_t, moe_stream_t stream);

/* S0 for the whole layer, straight into the operands moe_forward and
 * moe_backward read (one read of each bf16 master; "Mixture-of-Kittens" wiki
 * page, Key claims, MXFP8 bullet: MXFP8 expert weights with BF16 masters).
 * w_gu [E, 2m, d] and w_dn [E, d, m] bf16 masters of cfg's experts.
 *   MXFP8: gu / dn = E4M3 codes [E*2m, d] / [E*d, m] with PREPARED scales
 *     gu_scale / dn_scale (as moe_quantize_weights(blocks_along_rows = 0)
 *     followed by moe_prepare_scales, bit for bit); with gu_t and dn_t given,
 *     also the backward operands gu_t [E*d, 2m] + gu_t_scale and dn_t [E*m, d]
 *     + dn_t_scale (blocks_along_rows = 1), from the same read of the masters.
 *   BF16: the masters are the forward operands (copied into gu / dn when
 *     those name other buffers; NULL = use the masters); with gu_t and dn_t
 *     given, the per-expert transposes of the masters (the *_scale pointers are
 *     unused).
 *   NVFP4: gu / dn = packed codes [E*2m, d/2] / [E*d, m/2] with prepared
 *     scales and the experts' second-level scales gu_gscale / dn_gscale [E]
 *     fp32 (2688 / the expert matrix's amax); no backward operands.
 * gu_t and dn_t are both NULL (forward only) or both given (MOE_ERR_ARG
 * otherwise).  gu_gscale / dn_gscale are required with NVFP4 (4-byte
 * aligned suffices: they hold one fp32 per expert) and ignored otherwise.
 * Re-run after every update of the masters.  Asynchronous on `stream`. */
int moe_prepare_weights(const moe_config *cfg, const void *w_gu, const void *w_dn, void *gu, void *gu_scale,
                        void *dn, void *dn_scale, void *gu_t, void *gu_t_scale, void *dn_t, void *dn_t_scale,
                        float *gu_gscale, float *dn_gscale, moe_stream_t stream);

/* MXFP8 scales from the canonical order to the prepared operand layout that
 * moe_weights' *_scale fields take (a permutation of bytes, part of S0):
 * scales [rows, K/32] -> prepared (rows*K/32 bytes).  rows and K multiples of
 * 128 (MOE_ERR_SHAPE otherwise); the two buffers must not overlap
 * (MOE_ERR_ARG if they are the same pointer).  Asynchronous on `stream`. */
int moe_prepare_scales(const void *scales, int64_t rows, int32_t K, void *prepared, moe_stream_t stream);

/* The inverse of moe_prepare_scales: prepared -> canonical [rows, K/32]
 * (e.g. to read the scale buffers moe_buffer_info names, or to save prepared
 * weights in the format's own order).  Same rules. */
int moe_canonical_scales(const void *prepared, int64_t rows, int32_t K, void *scales, moe_stream_t stream);

/* Per-batch transpose of bf16 matrices: src [batch, rows, cols] ->
 * dst [batch, cols, rows] (rows, cols multiples of 32). */
int moe_transpose_bf16(const void *src, int batch, int rows, int cols, void *dst,
                       moe_stream_t stream);

/*
 * S1 + S2: router top-k and the device-side schedule (daily-ai-frontier
 * summary, TL;DR: routing fused into the layer; wiki page, flowchart and Key
 * claims: the device-side schedule kernel never talks to the host).
 * logits [T, E] fp32 (finite).  Outputs (device, caller-owned):
 *   idx [T, k] int32: experts ordered by (logit desc, index asc), first k;
 *   w [T, k] fp32: softmax over the k chosen logits (= softmax over E
 *                  renormalised to the chosen k);
 *   counts [E] int32; offsets [E+1] int32 (exclusive prefix sum);
 *   perm [T*k] int32: perm[t*k+j] = expert-sorted row of slot (t, j); rows of
 *                  one expert keep ascending slot order (stable).
 * Any output pointer may be NULL, in which case that output stays in `ws`.
 */
int moe_route(const moe_config *cfg, const float *logits, int32_t *idx, float *w, int32_t *counts,
              int32_t *offsets, int32_t *perm, void *ws, moe_stream_t stream);

/*
 * Router projection in front of the layer (daily-ai-frontier summary, TL;DR:
 * routing is the first fused stage; the pages do not define the projection,
 * so it is a bias-free linear map): logits [T, E] fp32 = x [T, d] bf16 *
 * W_r [E, d] bf16 ^T with fp32 accumulation, on the library's own tcgen05
 * GEMM (fp32 epilogue) through a zero-padded [roundup(T,128), roundup(E,128)]
 * buffer inside `ws`.  Bitwise reproducible.
 */
int moe_router_forward(const moe_config *cfg, const void *x, const void *W_r, float *logits, void *ws,
                       moe_stream_t stream);

/*
 * Router backward: dlogits [T, E] fp32 (moe_backward's output, including the
 * load-balancing term) is rounded to bf16 g; then dx [T, d] bf16 is updated in
 * place to bf16(dx + g W_r) (the layer's dx plus the router's, one rounding)
 * and dW_r [E, d] bf16 = bf16(g^T x).  Both on the library's own tcgen05 GEMM
 * (the first with an add-into-bf16 epilogue), over zero-padded copies of g,
 * g^T, W_r^T and x^T inside `ws`, which must be sized with MOE_FLAG_BACKWARD.
 */
int moe_router_backward(const moe_config *cfg, const float *dlogits, const void *x, const void *W_r, void *dx,
                        void *dW_r, void *ws, moe_stream_t stream);

/*
 * Forward pass: route -> schedule -> dispatch gather (MXFP8: x quantised in
 * the gather) -> gate/up grouped GEMM with SwiGLU (MXFP8: h quantised in the
 * epilogue) -> down grouped GEMM -> shared expert -> combine
 *     y[t] = bf16( sum_{j<k} w[t,j] * o[row(t,j)] + s[t] )   (fixed j order)
 * x [T, d] bf16; logits [T, E] fp32; y [T, d] bf16 output.
 * saved: NULL for inference, else moe_saved_bytes() bytes that the backward
 * reads.  ws: moe_workspace_bytes() bytes.
 * Expert-sorted rows are padded per expert to multiples of 128: the rows of
 * expert e occupy [poff[e], poff[e] + counts[e]) with
 * poff[e] = sum_{e'<e} roundup(counts[e'], 128).
 */
int moe_forward(const moe_config *cfg, const void *x, const float *logits, const moe_weights *W,
                void *y, void *saved, void *ws, moe_stream_t stream);

/*
 * Backward pass (wiki page, Key claims: reverse-combine, then the expert
 * GEMMs' dgrad/wgrad, then reverse-dispatch).  Inputs: dy [T, d] bf16, the
 * forward's x, weights (including the backward operands) and `saved`.
 * Outputs: dx [T, d] bf16; dlogits [T, E] fp32 (w_j (g_j - sum_i w_i g_i) at
 * the chosen experts, g_j = <dy_t, o_j>, 0 elsewhere); dW_gu [E, 2m, d] and
 * dW_dn [E, d, m] bf16, every element written (all zeros for an expert that
 * received no rows, so the buffers need no clearing beforehand); dWs_gu
 * [2m_s, d], dWs_dn [d, m_s] bf16 (shared expert; NULL when absent).
 */
int moe_backward(const moe_config *cfg, const void *dy, const void *x, const moe_weights *W,
                 const void *saved, void *dx, float *dlogits, void *dW_gu, void *dW_dn,
                 void *dWs_gu, void *dWs_dn, void *ws, moe_stream_t stream);

/*
 * Router top-k + schedule without a workspace, for callers that cannot call
 * cudaMalloc: code inside a host framework that owns every device byte through
 * its own arena, or a latency-critical path on which an allocation (which can
 * synchronise the device) is not acceptable.  The pages have no counterpart:
 * this is an extra entry point of this library, not a step of the method.
 * Computes exactly what moe_route computes (same kernels, same bits); all
 * seven pointers are required (no output can stay in a workspace).
 * Scratch: a fixed array in the library's device memory, sized for at most
 * MOE_ROUTE_NOALLOC_MAX_SLOTS routed slots (T*k) and
 * MOE_ROUTE_NOALLOC_MAX_EXPERTS experts (about 2 MiB, held by every GPU that
 * loads the library until the process exits); larger shapes return
 * MOE_ERR_SHAPE.  Every call shares that array and leaves its contents behind
 * (nothing in it needs to start at zero): calls that overlap on the GPU (on
 * different streams, or from several host threads) race and corrupt each
 * other's results.  Calls on one stream are ordered and safe.  The first call
 * on a device looks up the array's device address (cudaGetSymbolAddress); make
 * that first call before any stream capture.  The address is kept for the life
 * of the process: calls made after cudaDeviceReset (or anything else that
 * destroys and re-creates the device's primary context) are not supported.
 * Allocates nothing.
 */
#define MOE_ROUTE_NOALLOC_MAX_SLOTS 262144
#define MOE_ROUTE_NOALLOC_MAX_EXPERTS 1024
int moe_route_noalloc(const moe_config *cfg, const float *logits, int32_t *idx, float *w,
                      int32_t *counts, int32_t *offsets, int32_t *perm, moe_stream_t stream);

/*
 * ======================================================================
 * Around the layer: what a model needs next to the block.  The pages have no
 * counterpart; these entry points are additions of this library.
 * ======================================================================
 * They follow the conventions at the top with these differences, which hold
 * for every entry point below: element types are moe_elem values; the rows of
 * a matrix may be strided (ld_* in elements, 0 = contiguous; the elements of a
 * row are always adjacent); pointers need only their element's alignment
 * (MOE_ERR_ALIGN otherwise; offsets, ids and fp32 statistics 4 bytes or their
 * own size, workspaces 16 bytes), and 16-byte aligned rows take the faster
 * kernels; a call over zero rows is valid and writes what does not depend on
 * rows (zero weight gradients).  Sums, norms and statistics are fp32; each
 * output is rounded once.
 */
typedef enum { MOE_ELEM_BF16 = 0, MOE_ELEM_FP16 = 1, MOE_ELEM_FP32 = 2 } moe_elem;

/*
 * Matrix products grouped by expert, ragged sizes.  Rows r of expert e are
 * [offsets[e], offsets[e+1]) (int32 [E+1] on the device, ascending, as
 * moe_route writes them; no padding); w [E, N, K].
 *   forward:   y[r] = x[r] w[e]^T              x [rows, K] -> y [rows, N]
 *   backward:  dx[r] = dy[r] w[e]              dy [rows, N] -> dx [rows, K]
 *              dw[e] = sum_r dy[r]^T x[r]      -> dw [E, N, K] contiguous
 * Rows below offsets[0] or at and above offsets[E] belong to no expert: their
 * y and dx are written as zeros and what x and dy hold there (NaN included)
 * is not used.  An expert without rows gets dw[e] = 0.
 * dtype is the type of x, w, dy and dx (BF16 or FP16); out_dtype that of y or
 * dw: dtype, or FP32.  accumulate = 1 adds to what dw holds instead of
 * overwriting it (FP32 dw only; an expert without rows is left alone).
 * ld_x: row stride of x and dx; ld_y: of y and dy; ld_w: of w's rows;
 * ld_e: elements from one expert's matrix to the next.
 * Offsets that descend or leave [0, rows] never cause an access out of range;
 * moe_get_status(ws) then reports MOE_ERR_BOUNDS (in every build) and the
 * outputs are unspecified.
 * Limits: 1 <= E <= 32767, 1 <= N, K <= 2^20, rows < 2^31 - 256, strides below 2^31
 * (MOE_ERR_SHAPE).  16-byte aligned rows and pointers run on the tensor cores
 * through TMA, few rows in all (a generated token) on a kernel that streams
 * the experts' weights, everything else on a plain tiled kernel.
 */
typedef struct {
  int64_t rows;
  int32_t E, N, K;
  int32_t dtype, out_dtype; /* moe_elem */
  int32_t accumulate;
  int64_t ld_x, ld_y, ld_w, ld_e; /* 0 = contiguous */
} moe_grouped_config;

/* Bytes of scratch for one grouped call (0 on an invalid config). */
size_t moe_grouped_workspace_bytes(const moe_grouped_config *cfg);
int moe_grouped_forward(const moe_grouped_config *cfg, const void *x, const void *w, const int32_t *offsets, void *y,
                        void *ws, moe_stream_t stream);
/* dx or dw may be NULL (not both); x is not read without dw, w not without dx. */
int moe_grouped_backward(const moe_grouped_config *cfg, const void *dy, const void *x, const void *w,
                         const int32_t *offsets, void *dx, void *dw, void *ws, moe_stream_t stream);

/*
 * The norms around a block, fused with its gate and the residual:
 *   n = w_post * f / rms(f)   with MOE_NORM_POST, else n = f
 *   z = alpha * x + g * n     (z = alpha * x when f is NULL)
 *   h = w_pre * z / rms(z)    with MOE_NORM_PRE: the next block's input
 *   rms(v) = sqrt(mean(v^2) + eps) over the d elements of a row
 * x is the residual stream, f the block's output; the gate g is none (1), one
 * value per channel [d], per row [rows] or per element [rows, d].  w_post and
 * w_pre are [d] or NULL (ones).  All of dtype (BF16, FP16 or FP32), ld_x of x
 * and dx, ld_f of f and df, ld_z of z and dz, ld_h of h and dh, ld_g of a
 * full gate and its gradient.
 * forward writes z (may be NULL with MOE_NORM_PRE), h, and the reciprocal roots
 * r_post = 1 / rms(f), r_pre = 1 / rms(z) [rows] fp32 that a backward needs
 * (each may be NULL).  h comes from z before z is rounded.
 * backward takes the gradients dz (NULL = none, with MOE_NORM_PRE) and dh, the
 * forward's z, f, r_post and r_pre, and writes
 *   dx = alpha * t, df, dgate (in the gate's shape), dw_post, dw_pre,
 *   t = dz + the pre norm's gradient; any output may be NULL.
 * Sums over rows run in a fixed order (bitwise reproducible).  z and r_pre are
 * needed with MOE_NORM_PRE, f for df / dgate / dw_post, r_post with
 * MOE_NORM_POST.  dx may be dz's buffer and df f's.
 * Limits: 1 <= d <= 65536, rows < 2^31, eps >= 0 (MOE_ERR_SHAPE, MOE_ERR_ARG).
 */
#define MOE_NORM_POST 1
#define MOE_NORM_PRE 2
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_ROW = 2, MOE_GATE_FULL = 3 } moe_gate;
typedef struct {
  int64_t rows;
  int32_t d;
  int32_t dtype; /* moe_elem */
  int32_t flags; /* MOE_NORM_POST | MOE_NORM_PRE */
  int32_t gate;  /* moe_gate */
  float alpha, eps;
  int64_t ld_x, ld_f, ld_z, ld_h, ld_g; /* 0 = d */
} moe_norm_config;

int moe_norm_forward(const moe_norm_config *cfg, const void *x, const void *f, const void *gate, const void *w_post,
                     const void *w_pre, void *z, void *h, float *r_post, float *r_pre, moe_stream_t stream);
/* Bytes of scratch of one moe_norm_backward call (0 on an invalid config). */
size_t moe_norm_workspace_bytes(const moe_norm_config *cfg);
int moe_norm_backward(const moe_norm_config *cfg, const void *dz, const void *dh, const void *z, const void *f,
                      const void *gate, const void *w_post, const void *w_pre, const float *r_post,
                      const float *r_pre, void *dx, void *df, void *dgate, void *dw_post, void *dw_pre, void *ws,
                      moe_stream_t stream);

/*
 * Token embedding: out[t] = scale * table[ids[t]], a zero row for an id outside
 * [0, V) (padding), and its gradient
 *   dtable[v] = scale * sum of dout[t] over the t with ids[t] = v
 * by sorting the tokens: each table row's sum runs over ascending t in fp32 in a
 * fixed order and is rounded once (bitwise reproducible).  Ids outside [0, V)
 * take no gradient.  accumulate = 0 writes every row of dtable (zeros where no
 * token points); accumulate = 1 adds to the rows that tokens point to and
 * leaves the others alone.
 * ids: int32 or (ids64 = 1) int64 [rows].  table and out / dout are of dtype
 * (BF16, FP16, FP32), dtable of grad_dtype (dtype or FP32).  ld_t: row stride
 * of table and dtable; ld_o: of out and dout.
 * Limits: rows < 2^30, 1 <= V < 2^31 - 1, 1 <= d <= 2^20 (MOE_ERR_SHAPE).
 */
typedef struct {
  int64_t rows;
  int64_t V;
  int32_t d;
  int32_t dtype, grad_dtype; /* moe_elem */
  int32_t ids64, accumulate;
  float scale;
  int64_t ld_t, ld_o; /* 0 = d */
} moe_embed_config;

int moe_embed_forward(const moe_embed_config *cfg, const void *ids, const void *table, void *out,
                      moe_stream_t stream);
/* Bytes of scratch of one moe_embed_backward call (0 on an invalid config). */
size_t moe_embed_workspace_bytes(const moe_embed_config *cfg);
int moe_embed_backward(const moe_embed_config *cfg, const void *ids, const void *dout, void *dtable, void *ws,
                       moe_stream_t stream);

/*
 * Gated products grouped by expert, ragged sizes: the first half of a gated
 * feed-forward block in one kernel.  Rows r of expert e as for moe_grouped_*;
 * w [E, 2m, K]: an expert's m rows of the gate, then its m of the up projection.
 *   forward:   g = x[r] w[e][0:m]^T, u = x[r] w[e][m:2m]^T,  h[r] = act(g) u
 *              x [rows, K] -> h [rows, m], and gu [rows, 2m] = [g | u] unless NULL
 *   backward:  dg = dh u act'(g), du = dh act(g) from the forward's gu,
 *              dx[r] = dg w[e][0:m] + du w[e][m:2m]           -> dx [rows, K]
 *              dw[e] = sum_r [dg | du][r]^T x[r]               -> dw [E, 2m, K] contiguous
 * act: SiLU g / (1 + e^-g), GELU g Phi(g), its form by tanh, or ReLU.  h comes from
 * g and u before they are rounded; dg and du are rounded to dtype in front of
 * their products.  Rows of no expert: h, gu and dx zeros, what x, dh and gu hold
 * there is not used; an expert without rows gets dw[e] = 0; bad offsets, dtype,
 * grad_dtype (dw's), accumulate and limits (1 <= m <= 2^19) as for moe_grouped_*.
 * ld_x: row stride of x and dx; ld_h: of h and dh; ld_gu: of gu; ld_w, ld_e of w.
 */
typedef enum { MOE_ACT_SILU = 0, MOE_ACT_GELU = 1, MOE_ACT_GELU_TANH = 2, MOE_ACT_RELU = 3 } moe_act;
typedef struct {
  int64_t rows;
  int32_t E, m, K;
  int32_t dtype, grad_dtype; /* moe_elem */
  int32_t act;               /* moe_act */
  int32_t accumulate;
  int64_t ld_x, ld_h, ld_gu, ld_w, ld_e; /* 0 = contiguous */
} moe_gated_config;

/* Bytes of scratch of one call in each direction (0 on an invalid config). */
size_t moe_gated_forward_workspace_bytes(const moe_gated_config *cfg);
size_t moe_gated_backward_workspace_bytes(const moe_gated_config *cfg);
int moe_gated_forward(const moe_gated_config *cfg, const void *x, const void *w, const int32_t *offsets, void *h,
                      void *gu, void *ws, moe_stream_t stream);
/* dx or dw may be NULL (not both); x is not read without dw, w not without dx. */
int moe_gated_backward(const moe_gated_config *cfg, const void *dh, const void *x, const void *w, const int32_t *offsets,
                       const void *gu, void *dx, void *dw, void *ws, moe_stream_t stream);

/*
 * The loss over a vocabulary straight from the last hidden rows, in pieces of the
 * vocabulary: the logits z = x w^T are never in memory.
 *   forward:   lse[t] = log sum_v exp z[t, v],  loss[t] = lse[t] - z[t, labels[t]]   (fp32)
 *   backward:  dz[t, v] = (dloss[t] + dlse[t]) exp(z[t, v] - lse[t]) - dloss[t] [v = labels[t]]
 *              dx[t] = sum_v dz[t, v] w[v]      -> dx [rows, d] of dtype
 *              dw[v] = sum_t dz[t, v] x[t]      -> dw [V, d] contiguous, of grad_dtype
 * x [rows, d] and w [V, d] of dtype (BF16 or FP16), labels int32 or (labels64 = 1)
 * int64 [rows].  A row whose label lies outside [0, V) (padding) does not count:
 * loss, lse and dx are zero and what x holds there (NaN included) is not used.
 * So it is in the backward for rows whose dloss and dlse are both zero.
 * dloss or dlse [rows] fp32 may be NULL (zeros), lse is the forward's.  With
 * dlse the loss may hold terms in lse (a penalty lse^2).
 * accumulate = 1 adds to dw (FP32 only).  dz is formed in fp32 and rounded to
 * dtype relative to the largest coefficient of all rows, in front of its two
 * products.  Sums run in a fixed order (bitwise reproducible).
 * The tensor cores read w through TMA: w and its rows must start on 16-byte
 * boundaries (MOE_ERR_ALIGN otherwise), or copy_w = 1 takes a padded copy in the
 * workspace.  ld_x, ld_w, ld_dx: row strides.
 * Workspace (256-byte aligned): a copy of the rows that count; forward 16 bytes
 * per row and 256 vocabulary entries; backward about 512 MB for a piece of dz
 * (4096 entries for all rows at least) and the fp32 sums of dx.
 * moe_get_status(ws) reports a wait that timed out.
 * Limits: rows, V < 2^30, 1 <= d <= 2^20, 2^30 tiles of 256 x 256 (MOE_ERR_SHAPE).
 */
typedef struct {
  int64_t rows, V;
  int32_t d;
  int32_t dtype, grad_dtype; /* moe_elem */
  int32_t labels64, accumulate, copy_w;
  int64_t ld_x, ld_w, ld_dx; /* 0 = d */
} moe_vocab_config;

/* Bytes of scratch of one call in each direction (0 on an invalid config). */
size_t moe_vocab_forward_workspace_bytes(const moe_vocab_config *cfg);
size_t moe_vocab_backward_workspace_bytes(const moe_vocab_config *cfg);
int moe_vocab_forward(const moe_vocab_config *cfg, const void *x, const void *w, const void *labels, float *loss,
                      float *lse, void *ws, moe_stream_t stream);
/* dx or dw may be NULL (not both). */
int moe_vocab_backward(const moe_vocab_config *cfg, const float *dloss, const float *dlse, const void *x, const void *w,
                       const void *labels, const float *lse, void *dx, void *dw, void *ws, moe_stream_t stream);

/*
 * The global norm of many gradients, and their clipping:
 *   norm = sqrt(sum of all elements' squares),  c = min(1, max_norm / (norm + eps))
 *   outs[i] = c grads[i]
 * The arrays are host arrays of n entries, read before the call returns: device
 * addresses, element counts, types (moe_elem; outs' type is the tensor's or FP32).
 * An out may be its own gradient (of one type: in place; nothing is written when c = 1);
 * otherwise outs share memory neither with one another nor with a gradient
 * (MOE_ERR_ARG).  The same gradient twice counts twice in moe_grad_norm.
 * norm: one fp32 on the device.  Sums are held in 64 bits over short fp32 sums, in
 * a fixed order; no squares overflow or vanish.  A norm that is not finite makes
 * c zero (infinite norm) or NaN, as the formula says.
 * max_norm >= 0, eps > 0; n <= 2^24, counts <= 2^42, 2^45 bytes in all.
 * An infinite max_norm is no limit: c = 1, for an infinite norm too (a NaN among
 * the gradients: c NaN).
 */
typedef struct {
  double max_norm, eps;
} moe_clip_config;

size_t moe_grad_workspace_bytes(int32_t n);
int moe_grad_norm(const void *const *grads, const int64_t *counts, const int32_t *dtypes, int32_t n, float *norm,
                  void *ws, moe_stream_t stream);
int moe_grad_clip(const moe_clip_config *cfg, const void *const *grads, void *const *outs, const int64_t *counts,
                  const int32_t *dtypes, const int32_t *out_dtypes, int32_t n, float *norm, void *ws,
                  moe_stream_t stream);

/* Synchronises `stream`, returns the device status word recorded in `ws`
 * (MOE_OK, MOE_ERR_TIMEOUT, or MOE_ERR_BOUNDS -- from the layer only in a debug
 * build; a timeout is reported first when both happened) and clears it.  Returns MOE_ERR_CUDA if
 * the stream reports a CUDA error. */
int moe_get_status(void *ws, moe_stream_t stream);

/* Static description of a status code (never NULL). */
const char *moe_status_string(int status);

/*
 * Optional per-launch timing (process-wide, for benchmarks and profilers).
 * moe_trace_enable(n) creates n pairs of CUDA events (n = 0 disables tracing
 * and destroys them); while enabled, every kernel launch made by moe_route,
 * moe_forward and moe_backward is bracketed by an event pair recorded on the
 * call's stream, in launch order, until n launches are recorded.  Tracing
 * adds two event records per launch and changes nothing else.
 * moe_trace_clear() restarts at slot 0; moe_trace_count() is the number of
 * recorded launches; moe_trace_name(i) names launch i (static string, NULL
 * when i is out of range); moe_trace_ms(i) synchronises on launch i's end
 * event and returns its duration in milliseconds (negative on error).
 * Not thread-safe: trace from one host thread.
 */
int moe_trace_enable(int capacity);
void moe_trace_clear(void);
int moe_trace_count(void);
const char *moe_trace_name(int i);
float moe_trace_ms(int i);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */

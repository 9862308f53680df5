/*
 * moe.h - C ABI of the GB300 (sm_103a) quantized routed-expert MoE FFN.
 *
 * One decode step of a Mixture-of-Experts layer, as the pulsar README states
 * it ("MoE resolve" passage and the model table):
 *   1. moe_quantize_q8K : activations -> q8 blocks (integer dots follow,
 *                         "activations quantized to q8_0/q8_K").
 *   2. moe_route        : router GEMV, softmax or sigmoid top-k (README model
 *                         table: "softmax router", "sigmoid-gated router").
 *   3. moe_expert_ffn   : per (token, slot) the chosen expert's gate/up GEMVs
 *                         over block-quantised weights, SwiGLU, requantised h,
 *                         the down GEMV, the routing-weight scale and the
 *                         fixed-order per-token sum, plus the shared expert.
 *                         Experts arrive as explicit per-expert device
 *                         pointers and a NULL gate pointer means "not mine"
 *                         (README, "MoE resolve": the kernels receive
 *                         per-(token, slot) pointers; NULL means not mine).
 *
 * Conventions for every call:
 *  - All pointers named "device" are CUDA device pointers; the library never
 *    dereferences them on the host.  Host pointers are marked "host".
 *  - The caller owns every buffer.  The library allocates nothing, keeps no
 *    state between calls and never synchronises the host, except
 *    moe_read_device_status, which does.
 *  - Calls are asynchronous and ordered on the given stream (0 = legacy
 *    default stream).  Argument errors are returned before anything is
 *    launched; a failed launch returns MOE_ERR_CUDA.
 *  - Inputs must be finite.  Weights and expert tables are read-only for the
 *    duration of a call.
 *  - Results are deterministic: identical inputs give bit-identical outputs,
 *    whatever the batch composition (see moe_expert_ffn).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* NULL where a buffer is required, bad size or shape */
    MOE_ERR_UNSUPPORTED = 2,   /* valid but not implemented (format/shape pairing)   */
    MOE_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required          */
    MOE_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed                */
    MOE_ERR_DEVICE_STATUS = 5, /* a kernel recorded a data error (see status word)    */
    MOE_ERR_TIMEOUT = 6        /* reserved: a bounded device-side wait gave up        */
} moe_status;

/* Weight formats (GGUF-style blocks; see moe_pack_weights for the bytes). */
typedef enum {
    MOE_F32 = 0,    /* plain fp32 (router only)                                   */
    MOE_Q8_0 = 1,   /* 32 weights: f16 d, i8 q[32]               w = d*q   (34 B)  */
    MOE_Q4_K = 2,   /* 256 weights: f16 d, f16 dmin, 6-bit sc/m x 8, 4-bit q (144 B) */
    MOE_Q2_K = 3,   /* 256 weights: 4-bit sc/m x 16, 2-bit q, f16 d, f16 dmin (84 B) */
    MOE_MXFP4 = 4,  /* 32 weights: E8M0 scale e, FP4 E2M1 q[32]  w = 2^(e-127)*q (17 B) */
    MOE_Q6_K = 5,   /* 256 weights: 4+2-bit q (offset 32), i8 sc x 16, f16 d     (210 B) */
    MOE_Q3_K = 6    /* 256 weights: 2+1-bit q (offset 4), 6-bit sc x 16, f16 d   (110 B) */
} moe_qtype;

typedef enum { MOE_GATE_SOFTMAX = 0, MOE_GATE_SIGMOID = 1 } moe_gating;

/* Element types of the calls around the experts. */
typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1 } moe_dtype;

/* What moe_matmul does with its products (v: the product plus the bias). */
typedef enum {
    MOE_ACT_NONE = 0,        /* v                                                              */
    MOE_ACT_SILU = 1,        /* v sigma(v)                                                     */
    MOE_ACT_GELU = 2,        /* v Phi(v), Phi(v) = (1 + erf(v / sqrt 2)) / 2                   */
    MOE_ACT_SWIGLU = 3,      /* silu(gate) up: v has 2N columns, gate then up                  */
    MOE_ACT_SILU_GRAD = 4,   /* v silu'(z)                                                     */
    MOE_ACT_GELU_GRAD = 5,   /* v gelu'(z)                                                     */
    MOE_ACT_SWIGLU_GRAD = 6  /* z = [gate up], 2N columns: y = [v up silu'(gate), v silu(gate)] */
} moe_act;

/* Device status word bits (moe_read_device_status). */
#define MOE_DEV_BAD_ID 0x1u       /* an expert id outside [0, E): that slot was skipped     */
#define MOE_DEV_DUP_ID 0x2u       /* an id repeated within one token: the repeat was skipped */
#define MOE_DEV_TIMEOUT 0x4u      /* a bounded wait in moe_layer_forward, moe_fp8_matmul or moe_matmul gave
                                     up: y is invalid, zero the workspace before the next call */
#define MOE_DEV_BAD_ROW 0x8u      /* moe_fp8_matmul, moe_matmul: a row index outside x (its products are
                                     zero) or offsets that fall or leave [0, M] (rows of those groups
                                     are left out or computed with one group or another)        */

/* Limits of this build. */
#define MOE_MAX_TOKENS 16          /* T per call (small-batch decode)        */
#define MOE_MAX_K 32               /* top-k                                  */
#define MOE_MAX_EXPERTS 1024       /* E                                      */
#define MOE_MAX_RANKS 64           /* partial outputs summed by moe_sum_partials */
#define MOE_MAX_ROWS (1 << 24)     /* T, M, X of the calls around the experts  */
#define MOE_MAX_PAIRS (1 << 22)    /* T*k of moe_expert_order and the row calls */
#define MOE_MAX_NORM_WIDTH 16384   /* n of moe_add_rmsnorm                     */
#define MOE_FP8_GROUP 128          /* values that share a scale of an e4m3 row */

/* ------------------------------------------------------------------ sizes */

/* Activation quantisation block for a width n: 256 if n % 256 == 0, 32 if
 * n % 32 == 0 (the README's "multiple of 32 but not 256 -> q8_0" rule),
 * else 0 (unsupported). */
int moe_act_block(int n);

/* Bytes of one token's q8 activation record of width n (a multiple of 16):
 *   offset 0          : float d[n/B]        block scales, B = moe_act_block(n)
 *   offset A          : int8  q[n]          codes, A = 16-aligned 4*n/B
 *   offset A + n      : int16 bsum[n/16]    sum of each 16 consecutive codes
 * T tokens are T records back to back.  Returns 0 if n is unsupported. */
size_t moe_q8_row_bytes(int n);

/* Bytes of a packed weight matrix (rows x cols), 0 if unsupported.
 * rows % 32 == 0; cols % 256 == 0 for Q4_K, Q2_K, Q8_0, Q6_K and Q3_K;
 * cols % 32 == 0 for MXFP4.  The packed size equals the GGUF size except for
 * MXFP4 matrices whose cols/32 is not a multiple of 8, Q6_K (4 bytes per row
 * and 256 columns for d instead of 2) and Q3_K (112 bytes per row and 256
 * columns instead of 110). */
size_t moe_packed_bytes(moe_qtype qtype, int rows, int cols);

/* ------------------------------------------------------------- one-time pack */

/*
 * Lossless re-layout of a row-major matrix of GGUF-style blocks (device,
 * rows x cols/QK blocks, QK = 256 or 32) into the packed layout the FFN
 * kernels stream with 128-bit coalesced loads (device, moe_packed_bytes).
 * Same bits per weight; run once at load time.  This mirrors the README's
 * load-time tensor transforms (K-quant dense tensors are requantised when
 * loaded); here nothing is requantised, only moved.
 *
 * Packed layout: rows are cut into tiles of 32; a tile is a sequence of
 * records along the columns; a record is a set of 512-byte planes, plane p
 * holding 16 bytes for each of the 32 rows (row r of the tile at byte 16*r):
 *   Q4_K  : record = 1 block (256 cols); planes 0..8 = the block's bytes
 *           [16p, 16p+16) (plane 0: d, dmin, scales; 1..8: qs).      4608 B
 *   Q2_K  : record = 1 block; planes 0..4 = bytes [16p, 16p+16) (scales,
 *           qs), then one 128-byte plane of {d, dmin} (4 B per row). 2688 B
 *   Q8_0  : record = 8 blocks (256 cols); planes 2b, 2b+1 = q of block b,
 *           plane 16 = the 8 f16 d of the row.                       8704 B
 *   MXFP4 : record = nb <= 8 blocks (the last record of a row takes the
 *           remainder); planes 0..nb-1 = qs of block b, then a 256-byte
 *           plane of 8 scale bytes per row (unused bytes zero). nb*512+256 B
 *   Q6_K  : record = 1 block; planes 0..12 = bytes [16p, 16p+16) (ql, qh,
 *           the 16 int8 scales), then a 128-byte plane of {d, 0, 0}.  6784 B
 *   Q3_K  : record = 1 block; planes 0..5 = hmask and qs, plane 6 = the
 *           12 scale bytes, d and two zero bytes.                    3584 B
 * Errors: MOE_ERR_UNSUPPORTED for F32 or shapes outside the rules above.
 */
moe_status moe_pack_weights(const void *blocks, moe_qtype qtype, int rows, int cols,
                            void *packed, cudaStream_t stream);

/* ---------------------------------------------------------- hot-path calls */

/*
 * Activation quantisation (README "MoE resolve": activations quantised to
 * q8_0/q8_K before integer dots).  x: device fp32 [T][n]; xq: device, T
 * records of moe_q8_row_bytes(n); both 16-byte aligned.  Per block of
 * B = moe_act_block(n): amax = max|x|, d = amax/127, q = rint(x*(127/amax))
 * (round half to even; IEEE division), d = 0 and q = 0 for an all-zero
 * block; bsum = sums of 16 codes.  T in [0, MOE_MAX_TOKENS*64]; T == 0 is a
 * no-op.
 * Errors: MOE_ERR_UNSUPPORTED if moe_act_block(n) == 0; MOE_ERR_INVALID_ARG
 * for T out of range or a NULL or unaligned x or xq.
 */
moe_status moe_quantize_q8K(const float *x, int T, int n, void *xq, cudaStream_t stream);

/*
 * Router GEMV + top-k + gating (README intro: the router stays resident;
 * model table: softmax and sigmoid-gated routers, top-k of E).
 *   hidden      : device fp32 [T][H], 16-byte aligned (read by an F32 router)
 *   xq          : device q8 records of hidden (moe_quantize_q8K), required
 *                 for a Q8_0 router, ignored (may be NULL) for F32
 *   w_router    : device, F32 [E][H] row-major, or Q8_0 blocks [E][H/32]
 *                 (GGUF row-major, not packed; rows must be 16-byte aligned,
 *                 i.e. (H/32) % 8 == 0)
 *   router_bias : device fp32 [E] added to the logits, or NULL
 *   ids         : device int32 [T][k] out: the k largest logits, largest
 *                 first, the lower index first on equal logits
 *   weights     : device fp32 [T][k] out.  Softmax: exp(l - lmax) over the
 *                 chosen k, normalised to sum 1 (renormalize != 0) or over all
 *                 E (renormalize == 0).  Sigmoid: s = 1/(1+exp(-l)), divided
 *                 by the sum over the chosen k when renormalize != 0.
 *   logits_out  : device fp32 [T][E] out, or NULL
 *   shared_gate : device fp32 [H], 16-byte aligned, or NULL: the shared
 *                 expert's gate vector (the README's gate_inp_shexp, an f32
 *                 tensor; its use is not stated there, and the reading taken
 *                 is a per-token scalar gate on the shared expert's output)
 *   shared_scale: device fp32 [T] out with shared_gate (NULL without it):
 *                 sigma(shared_gate . hidden[t]), the logit in the fixed order
 *                 below (a one-row F32 router, hidden required), then
 *                 1/(1+exp(-l)); moe_expert_ffn takes it as the shared
 *                 expert's weight
 *   ws          : device workspace of moe_route_workspace_bytes(T, E, H) bytes,
 *                 zero-filled before its first use; every completed call
 *                 leaves it ready for the next one
 * Logits are fp32 in one fixed summation order, so ids are reproducible bit
 * for bit: the row is cut into 1024-element segments; in a segment, lane l of
 * 32 accumulates float4 chunks l, l+32, ... with fused multiply-adds in
 * element order; the 32 lane values are combined by an xor butterfly
 * (offsets 16, 8, 4, 2, 1); segment values are added in order, then the bias.
 * A Q8_0 router uses 32-block segments with lane l taking block l of the
 * segment, value (d_w*d_x)*isum.
 * Limits: 1 <= k <= min(E, MOE_MAX_K), E <= MOE_MAX_EXPERTS, T <= MOE_MAX_TOKENS,
 * H % 32 == 0.
 * Errors: MOE_ERR_INVALID_ARG for limits, gating, a NULL or unaligned
 * buffer, or shared_gate and shared_scale not given together (or a shared
 * gate without hidden); MOE_ERR_UNSUPPORTED for a router type other than F32/Q8_0 or a Q8_0
 * router with H % 256 != 0; MOE_ERR_WORKSPACE for a missing, short or
 * unaligned ws.
 */
moe_status moe_route(const float *hidden, const void *xq, int T, int H,
                     const void *w_router, moe_qtype rtype, int E, const float *router_bias,
                     int k, moe_gating gating, int renormalize,
                     int32_t *ids, float *weights, float *logits_out,
                     const float *shared_gate, float *shared_scale,
                     void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_route_workspace_bytes(int T, int E, int H);

/* One expert: packed device matrices (moe_pack_weights) and optional biases.
 * A fused gate_up tensor (one [2I][H] matrix, gate rows first, as the README's
 * GGUF notes allow) packed as one matrix serves both projections: gate = its
 * start, up = gate + moe_packed_bytes(qtype, I, H), since packed tiles of 32
 * rows are stored one after another. */
typedef struct {
    const void *gate;     /* packed [I][H]; NULL: this expert is not owned here  */
    const void *up;       /* packed [I][H]                                        */
    const void *down;     /* packed [H][I]                                        */
    const float *b_gate;  /* device fp32 [I] or NULL                              */
    const float *b_up;    /* device fp32 [I] or NULL                              */
    const float *b_down;  /* device fp32 [H] or NULL (scaled by the routing weight) */
} moe_expert;

/* A set of experts of one format.  `experts` is a DEVICE array of E entries
 * (the per-expert pointer table stays on the device; the host never walks it). */
typedef struct {
    moe_qtype qtype;
    int H, I, E;
    const moe_expert *experts;
} moe_pool;

/*
 * Routed + shared expert FFN for T tokens (README "MoE resolve": integer
 * dots on q8 activations with per-block rescale; SwiGLU; per-slot weighted
 * sum; shared expert always on).
 *   xq      : device q8 records of the T hidden states (width pool->H),
 *             16-byte aligned
 *   ids     : device int32 [T][k]; weights: device fp32 [T][k]
 *   pool    : host pointer to the routed pool (qtype Q8_0, Q4_K, Q2_K, MXFP4,
 *             Q6_K or Q3_K)
 *   shared  : host pointer to a pool with E == 1 (no biases read), or NULL
 *   shared_scale: device fp32 [T], the shared expert's weight per token
 *             (moe_route's shared_scale), or NULL for weight 1; requires
 *             shared
 *   y       : device fp32 [T][H] out, 16-byte aligned, overwritten:
 *             y[t] = sum over slots s in slot order of w[t][s]*o(ids[t][s])
 *                    + g[t]*o_shared (added last; g = shared_scale or 1),
 *             o = W_down . q8(h) + b_down,  h = silu(g) * u,
 *             g = W_gate . xq + b_gate, u = W_up . xq + b_up (fp32 h is
 *             requantised with the moe_quantize_q8K rule, width I).
 *             Slots whose expert is not owned (gate == NULL) add nothing: an
 *             expert-parallel rank passes a pool with its non-owned entries
 *             NULL and receives a partial y.
 *   ws      : device workspace of moe_ffn_workspace_bytes() bytes, zero-filled
 *             before its first use.  The first 4 bytes are the device status
 *             word (MOE_DEV_* bits): an id outside [0, E) or repeated within a
 *             token is skipped and flagged there, without failing the call.
 * Every token's result is computed with the same arithmetic and order
 * whatever the other tokens of the batch, so a token's y is bit-identical
 * between T = 1 and any batch that contains it.
 * Limits: T <= MOE_MAX_TOKENS, k <= MOE_MAX_K, E <= MOE_MAX_EXPERTS;
 * H and I multiples of 32 (of 256 for Q4_K, Q2_K, Q8_0).
 * Errors: MOE_ERR_INVALID_ARG for limits, a pool with no expert table, an
 * unknown expert format, a NULL or unaligned buffer, or shared_scale without
 * a shared pool; MOE_ERR_UNSUPPORTED for widths the format cannot hold or a
 * shared pool of another H;
 * MOE_ERR_WORKSPACE for a missing, short or unaligned ws.
 */
moe_status moe_expert_ffn(const void *xq, int T, const int32_t *ids, const float *weights, int k,
                          const moe_pool *pool, const moe_pool *shared, const float *shared_scale,
                          float *y, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_ffn_workspace_bytes(int T, int k, const moe_pool *pool, const moe_pool *shared);

/*
 * moe_expert_ffn for callers that cannot allocate device memory: code bound
 * to a device-memory plan fixed at start-up, plugin hosts that pass inputs
 * and outputs but offer no allocator, and paths where cudaMalloc/cudaFree are
 * not allowed because they can synchronise the device or fail under memory
 * pressure.  The pages have no counterpart to this call; it exists for
 * deployment.  Arguments and results are those of moe_expert_ffn, without
 * the workspace.
 *  - Scratch is one fixed array of 2 MiB in the library's device image, held
 *    on every device that loads the library until the process exits.  A
 *    shape whose moe_ffn_workspace_bytes() exceeds 2 MiB returns
 *    MOE_ERR_WORKSPACE before anything is enqueued.
 *  - Allocates nothing.  The first call on a device looks up the array's
 *    device address; make that first call before any stream capture.
 *  - Every call uses the same array and finds the previous call's contents
 *    there (the status word and tickets are cleared by each call).  Calls
 *    that overlap on the GPU (other streams, other host threads) race and
 *    corrupt each other's results: order them.
 *  - The status word lives in that array and is not reported; out-of-range
 *    or repeated ids are still skipped.
 */
moe_status moe_expert_ffn_noalloc(const void *xq, int T, const int32_t *ids, const float *weights, int k,
                                  const moe_pool *pool, const moe_pool *shared, const float *shared_scale,
                                  float *y, cudaStream_t stream);

/*
 * The whole layer: quantise (moe_quantize_q8K's rule), route (moe_route's
 * fixed-order logits, top-k and gating) and the routed + shared expert FFN
 * (moe_expert_ffn's arithmetic), for decode where the three steps sit back to
 * back.  For T <= 4 this is one launch, described below; larger batches run
 * the three calls in turn (their kernels keep more warps per SM busy once
 * every weight record is dotted with many tokens), inside the same workspace.
 * One persistent block per SM: every block quantises x and
 * computes the logits of its own router rows, every block reads all logits,
 * selects the same top-k and streams its share of the chosen experts' packed
 * weights with TMA bulk copies into a shared-memory ring.  Logits, h and the
 * per-slot o rows pass between blocks through the workspace as 8-byte words
 * that carry the value and a per-call epoch (launch counters kept in the
 * workspace), so readers poll the data itself.  Results equal those of the
 * three calls (same arithmetic and summation orders).
 *   hidden      : device fp32 [T][H]; w_router/rtype/router_bias/k/gating/
 *                 renormalize as in moe_route; pool/shared as in moe_expert_ffn
 *   shared_gate : device fp32 [H] or NULL, as in moe_route: the shared
 *                 expert's output is scaled per token by sigma(gate . hidden)
 *                 (requires shared; 16-byte aligned)
 *                 (shared: the same format as pool or Q8_0)
 *   y           : device fp32 [T][H] out
 *   ids_out, weights_out, logits_out, xq_out: optional outputs (NULL to skip)
 *   hidden, w_router, y and xq_out must be 16-byte aligned
 *   ws          : device workspace of moe_layer_workspace_bytes() bytes,
 *                 zero-filled before its first use and after any call that set
 *                 MOE_DEV_TIMEOUT; completed calls leave it ready for the next
 *                 call with the same T (zero-fill it again before a call with
 *                 another T: the layouts differ)
 *   flags       : (T <= 4) MOE_LAYER_OVERLAP_PREVIOUS lets this launch start while the
 *                 previous kernel in the stream is still running (programmatic
 *                 dependent launch): before that kernel has finished, the call
 *                 reads only weights, router and expert tables, so none of those
 *                 may be written by the previous kernel; hidden and everything
 *                 else are read only after it completes.
 * Every device-side wait is bounded (8e8 SM cycles, under a second): on timeout the call sets
 * MOE_DEV_TIMEOUT in the status word (moe_read_device_status) and returns.
 * Limits as moe_route and moe_expert_ffn; additionally the blocks must all be
 * resident at once (checked: MOE_ERR_UNSUPPORTED otherwise).
 * Errors: as moe_route and moe_expert_ffn (argument errors before any launch),
 * and MOE_ERR_UNSUPPORTED for a shared pool whose format is neither the
 * routed pool's nor Q8_0.
 */
#define MOE_LAYER_OVERLAP_PREVIOUS 0x1u
moe_status moe_layer_forward(const float *hidden, int T, const void *w_router, moe_qtype rtype,
                             const float *router_bias, int k, moe_gating gating, int renormalize,
                             const moe_pool *pool, const moe_pool *shared, const float *shared_gate, float *y,
                             int32_t *ids_out, float *weights_out, float *logits_out, void *xq_out,
                             void *ws, size_t ws_bytes, unsigned flags, cudaStream_t stream);
size_t moe_layer_workspace_bytes(int T, int k, const moe_pool *pool, const moe_pool *shared);

/*
 * Expert-parallel reduction (README "MoE resolve": each tier card computes
 * the slots of the experts it holds and the partial outputs are summed).  An
 * expert-parallel rank passes moe_expert_ffn / moe_layer_forward a pool whose
 * non-owned entries are NULL and gets a partial y; with the R partials side
 * by side (for example gathered from every rank):
 *   parts : device fp32 [R][n], rank r's partial at parts + r*n
 *   y     : device fp32 [n] out: y[i] = ((parts[0][i] + parts[1][i]) + ...)
 *           + parts[R-1][i], added in rank order, so the result does not
 *           depend on how the partials arrived
 * Both 16-byte aligned; n % 4 == 0; 1 <= R <= MOE_MAX_RANKS.
 * Errors: MOE_ERR_INVALID_ARG for R, n or a NULL or unaligned buffer.
 */
moe_status moe_sum_partials(const float *parts, int R, size_t n, float *y, cudaStream_t stream);

/* --------------------------------------------------- around the experts */

/*
 * Residual addition, root-mean-square norm and the 8-bit rows that the
 * products take, in one pass: per row of n values
 *   s = x + residual                  (residual NULL: s = x)
 *   v = s * (1 / sqrt(mean(s*s) + eps)) * weight
 * in fp32, from the sum before its rounding to `dtype`.  A row has the same bits
 * whatever T is.
 *   x, residual  : device [T][n] of `dtype`; weight: device fp32 [n]
 *   residual_out : device [T][n] of `dtype` out: s, or NULL.  May be x or residual.
 *   y            : device [T][n] of `ydtype` out: v, or NULL (fp32 for an F32 router)
 *   xq           : device out, T q8 records of v (moe_quantize_q8K's rule, bit for
 *                  bit, of the fp32 v), or NULL; needs n % 32 == 0.  These cannot hold
 *                  a NaN: a block with one has scale 0 and codes 0
 *   x8, x8_scale : device out, e4m3 [T][n] and fp32 [T][ceil(n/128)], both or
 *                  neither: per group of 128 values (the last one may be short)
 *                  amax = max|v|, scale = amax/448, code = e4m3(v * (448/amax)),
 *                  nearest, ties to even.  A group with amax < 2^-119 (the
 *                  inverse would overflow) has scale 0 and codes 0; one that holds
 *                  a NaN has scale NaN and codes NaN.
 * All outputs are written; apart from residual_out none may overlap an input.
 * Limits: T in [0, MOE_MAX_ROWS] (0 is a no-op); n % 16 == 0, 16 <= n <=
 * MOE_MAX_NORM_WIDTH; eps > 0; |s| below 2^56 (squares are summed in fp32).
 * Errors: MOE_ERR_INVALID_ARG for limits, types, no output at all, x8 without
 * x8_scale or the reverse, a NULL input or a buffer that is not 16-byte aligned
 * (x8_scale: 4); MOE_ERR_UNSUPPORTED for a width outside the rules above.
 */
moe_status moe_add_rmsnorm(const void *x, const void *residual, const float *weight, float eps, int T, int n,
                           moe_dtype dtype, void *residual_out, void *y, moe_dtype ydtype, void *xq, void *x8,
                           float *x8_scale, cudaStream_t stream);

/*
 * Per-expert counts and the order by expert of a routing (moe_route's ids, of
 * any number of tokens): the (token, slot) pairs sorted by expert, and within
 * an expert by token, then slot.
 *   ids     : device int32 [T][k].  A pair whose id lies outside [0, E) takes
 *             no part (-1: a padded token; another rank's expert).
 *   counts  : device int32 [E] out: pairs per expert, or NULL
 *   offsets : device int32 [E+1] out: expert e's pairs are the sorted places
 *             [offsets[e], offsets[e+1]), or NULL
 *   rows    : device int32 [T*k] out: the token of each sorted place, -1 in the
 *             places from offsets[E] on, or NULL
 *   pos     : device int32 [T][k] out: the sorted place of each pair, -1 for one
 *             that takes no part, or NULL
 *   ws      : device workspace of moe_expert_order_workspace_bytes(T, k, E)
 *             bytes, 16-byte aligned; needs no preparation (0 bytes: may be
 *             NULL).  Calls that may overlap on the GPU need one each.
 * Limits: T in [0, MOE_MAX_ROWS], 1 <= k <= MOE_MAX_K, T*k <= MOE_MAX_PAIRS,
 * 1 <= E <= MOE_MAX_EXPERTS.  T == 0 writes zero counts and offsets.
 * Errors: MOE_ERR_INVALID_ARG for limits, a NULL ids, a buffer that is not
 * 4-byte aligned or no output; MOE_ERR_WORKSPACE for a missing, short or unaligned ws.
 */
moe_status moe_expert_order(const int32_t *ids, int T, int k, int E, int32_t *counts, int32_t *offsets,
                            int32_t *rows, int32_t *pos, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_expert_order_workspace_bytes(int T, int k, int E);

/*
 * The router's balance loss and its gradient, from the logits and the counts.
 * With p[t][e] the gate probabilities over all E (softmax of the logits, or
 * sigma(l) / sum sigma(l)), c = counts and N = sum c (N/k counted tokens):
 *   loss = alpha * sum_e (E c_e / N) * (k/N * sum_t p[t][e])
 * Even counts give alpha.  The counts carry no gradient:
 *   dloss/dlogits[t][e] = alpha k/N * p[t][e] (f_e - sum_j f_j p[t][j])
 * with f_e = E c_e / N, times (1 - sigma(l[t][e])) for sigmoid gating.
 *   logits    : device [T][E] of `dtype`, finite or -inf.  -inf marks an expert that a
 *               token may not take (p = 0); a row of nothing but -inf adds nothing.
 *               A NaN makes its row's gradient and the loss NaN.
 *   counts    : device int32 [E] >= 0 (moe_expert_order; with expert parallelism
 *               or several micro-batches, of all of them)
 *   valid     : device uint8 [T] or NULL: a token with 0 (padding) adds nothing
 *               and has gradient 0; its logits are not looked at
 *   grad_loss : device fp32 [1] that multiplies the gradient, or NULL (1)
 *   loss      : device fp32 [1] out, or NULL
 *   dlogits   : device [T][E] of `dtype` out, or NULL.  May be logits.
 *   ws        : device workspace of moe_balance_loss_workspace_bytes(T, E) bytes,
 *               16-byte aligned, zero-filled before its first use; every
 *               completed call leaves it ready for the next one.  Calls that
 *               may overlap on the GPU (two captured graphs, too) need one each.
 * N == 0 gives loss 0 and gradient 0.  Sums run in a fixed order.
 * Arithmetic is fp32 (the sum of the rows: fp32 that carries its roundings over,
 * then double).  With u = 2^-24, exp(x) is the machine's and off by (4 + 1.3 |x|) u
 * of itself, x a logit less its row's largest one (sigmoid: also the logit itself),
 * and the inverse of 1 + exp by 2 u; what lies below 2^-126 counts as 0.
 * Limits: T in [0, MOE_MAX_ROWS] (0: loss 0), 1 <= E <= MOE_MAX_EXPERTS,
 * 1 <= k <= min(E, MOE_MAX_K).
 * Errors: MOE_ERR_INVALID_ARG for limits, types, gating, a NULL input, no
 * output, or logits, dlogits that are not 16-byte aligned (counts, loss,
 * grad_loss: 4); MOE_ERR_WORKSPACE for a missing, short or unaligned ws.
 */
moe_status moe_balance_loss(const void *logits, moe_dtype dtype, const int32_t *counts, const uint8_t *valid, int T,
                            int E, int k, moe_gating gating, float alpha, const float *grad_loss, float *loss,
                            void *dlogits, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_balance_loss_workspace_bytes(int T, int E);

/*
 * Products of e4m3 rows with e4m3 matrices that carry a scale for each block
 * of 128 x 128 (rows: for each group of 128 values, as moe_add_rmsnorm makes
 * them), on the tensor cores.  Grouped by expert, or one matrix for all rows:
 *   y[i][n] = sum_b x_scale[r][b] * w_scale[g][n/128][b]
 *             * sum_{j in block b} x8[r][j] * w[g][n][j],   r = rows ? rows[i] : i
 * for the places i of each group g, offsets[g] <= i < offsets[g+1].
 *   x8, x_scale : device e4m3 [X][K], fp32 [X][ceil(K/128)]
 *   rows        : device int32 [M], values in [0, X), or NULL (needs X >= M)
 *   offsets     : device int32 [G+1], rising, in [0, M], or NULL (G == 1, all M)
 *   w, w_scale  : device e4m3 [G][N][K], fp32 [G][ceil(N/128)][ceil(K/128)]
 *   y           : device [M][N] of `ydtype` out.  Rows of no group keep their values.
 *   ws          : device workspace of moe_fp8_matmul_workspace_bytes() bytes
 *                 (the status word, moe_read_device_status), zero-filled before
 *                 its first use.  Calls that overlap on the GPU may share it.
 * Products within a block of 128 are summed by the tensor cores in fp32, the
 * scaled blocks in fp32, in one order for given sizes: equal calls give equal
 * bits.  Other sizes (M, N, K, G) may split K in another way and round differently.
 * Row indexes and offsets outside their ranges are never followed (MOE_DEV_BAD_ROW).
 * Limits: X, M in [0, MOE_MAX_ROWS] (M == 0 is a no-op), 1 <= G <=
 * MOE_MAX_EXPERTS, 1 <= N <= 2^20, K % 16 == 0, 16 <= K <= 2^20, G*N <= 2^30, X*K <= 2^36.
 * Errors: MOE_ERR_INVALID_ARG for limits, types, a NULL buffer, X < M without
 * rows, X == 0, offsets missing with G > 1, or x8, w, y not 16-byte aligned
 * (scales, rows, offsets: 4); MOE_ERR_UNSUPPORTED for a K outside the rule
 * above or more than 2^30 tiles of 128 x 128; MOE_ERR_WORKSPACE for a missing, short or unaligned ws.
 */
moe_status moe_fp8_matmul(const void *x8, const float *x_scale, int X, const int32_t *rows, int M,
                          const int32_t *offsets, int G, const void *w, const float *w_scale, int N, int K,
                          void *y, moe_dtype ydtype, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_fp8_matmul_workspace_bytes(void);

/*
 * The experts of each token and their gating weights, from the logits of any
 * number of tokens (moe_route's choice and weights): the k largest logits of a
 * row in falling order, equal ones by the lower index, and with g = exp(l)
 * (softmax) or sigma(l) (sigmoid)
 *   renormalize : w_e = g_e / sum of g over the chosen
 *   otherwise   : w_e = g_e / sum of g over all E (softmax), g_e (sigmoid)
 *   logits  : device [T][E] of `dtype`.  -inf marks an expert that a token may
 *             not take; where fewer than k are left, the last slots have id -1 and
 *             weight 0.  A NaN counts as larger than any number, so it is chosen
 *             and makes its weights NaN (so does +inf, where weights are ratios).
 *   valid   : device uint8 [T] or NULL: a token with 0 (padding) has ids -1 and
 *             weights 0; its logits are not looked at
 *   ids     : device int32 [T][k] out (moe_expert_order's input)
 *   weights : device fp32 [T][k] out, or NULL
 * Arithmetic is fp32.  The softmax over all E takes the machine's exp, off by
 * (4 + 1.3 |x|) u of itself for x a logit less the row's largest (u = 2^-24);
 * what lies below 2^-126 counts as 0.
 * Limits: T in [0, MOE_MAX_ROWS], 1 <= E <= MOE_MAX_EXPERTS, 1 <= k <= min(E, MOE_MAX_K).
 * Errors: MOE_ERR_INVALID_ARG for limits, types, gating, NULL logits or ids, or
 * logits that are not 16-byte aligned (ids, weights: 4).
 */
moe_status moe_topk(const void *logits, moe_dtype dtype, const uint8_t *valid, int T, int E, int k, moe_gating gating,
                    int renormalize, int32_t *ids, float *weights, cudaStream_t stream);

/*
 * The gradient of moe_topk's weights: dlogits = addend + sum over the slots of
 * dweights dw/dlogits, with the choice held fixed.  With d = dweights, sums over
 * the row's slots:
 *   softmax, renormalised  : w_e (d_e - sum w d) for the chosen, 0 for others
 *   softmax over all E     : w_e (d_e - sum w d), d_e = 0 for others
 *   sigmoid, renormalised  : (1 - sigma(l_e)) w_e (d_e - sum w d) for the chosen
 *   sigmoid                : (1 - w_e) w_e d_e for the chosen
 *   logits   : device [T][E] of `dtype`, as moe_topk had them
 *   ids      : device int32 [T][k]; a slot whose id lies outside [0, E) takes no
 *              part (its dweights are not looked at).  An id that comes twice in
 *              a row counts as two slots.
 *   dweights : device fp32 [T][k] (moe_combine_grad)
 *   addend   : device [T][E] of `dtype` (the balance loss's gradient), or NULL (0)
 *   dlogits  : device [T][E] of `dtype` out.  May be logits or addend.
 * A logit of -inf has weight 0 and gradient 0.  Arithmetic as moe_topk's.
 * Limits as moe_topk's.
 * Errors: MOE_ERR_INVALID_ARG for limits, types, gating, a NULL input or output,
 * or logits, addend, dlogits that are not 16-byte aligned (ids, dweights: 4).
 */
moe_status moe_topk_grad(const void *logits, moe_dtype dtype, const int32_t *ids, const float *dweights, int T, int E,
                         int k, moe_gating gating, int renormalize, const void *addend, void *dlogits,
                         cudaStream_t stream);

/*
 * Token rows to their places in the order by expert (moe_expert_order's pos):
 *   xs[pos[t][s]] = x[t]
 *   x   : device [T][n] of `dtype`
 *   pos : device int32 [T][k]; a pair whose place lies outside [0, M) takes no
 *         part.  No place comes twice.
 *   xs  : device [M][n] of `dtype` out; rows of no pair keep their values.  Must
 *         not overlap x.
 * The gradient is moe_combine_rows without weights.
 * Limits: T, M in [0, MOE_MAX_ROWS], 1 <= k <= MOE_MAX_K, T*k <= MOE_MAX_PAIRS,
 * 1 <= n <= 65536, T*n and M*n <= 2^36.  T == 0 is a no-op.
 * Errors: MOE_ERR_INVALID_ARG for limits, types, a NULL buffer, or rows that
 * are not 16-byte aligned (pos: 4).
 */
moe_status moe_dispatch_rows(const void *x, moe_dtype dtype, const int32_t *pos, int T, int k, int n, int M, void *xs,
                             cudaStream_t stream);

/*
 * Rows in the order by expert back to their tokens:
 *   y[t] = addend[t] + sum_s weights[t][s] o[pos[t][s]]
 * added in fp32 from the addend on, in the order of the slots.
 *   o       : device [M][n] of `dtype`
 *   pos     : device int32 [T][k]; a pair whose place lies outside [0, M) adds nothing
 *   weights : device fp32 [T][k], or NULL (1)
 *   addend  : device [T][n] of `ydtype`, or NULL (0).  May be y.
 *   y       : device [T][n] of `ydtype` out.  Must not overlap o.
 * Limits, errors (weights: 4) as moe_dispatch_rows's; with M == 0 o may be NULL.
 */
moe_status moe_combine_rows(const void *o, moe_dtype dtype, const int32_t *pos, const float *weights, int T, int k,
                            int n, int M, const void *addend, void *y, moe_dtype ydtype, cudaStream_t stream);

/*
 * The gradient of moe_combine_rows:
 *   d_o[pos[t][s]] = weights[t][s] dy[t],   dweights[t][s] = sum_j o[pos[t][s]][j] dy[t][j]
 *   dy       : device [T][n] of `ydtype`
 *   pos      : device int32 [T][k]; a pair whose place lies outside [0, M) has no
 *              row and dweights 0.  No place comes twice.
 *   weights  : device fp32 [T][k], or NULL (1)
 *   o        : device [M][n] of `dtype`; NULL without dweights
 *   d_o      : device [M][n] of `dtype` out, or NULL; rows of no pair keep their
 *              values.  May be o.
 *   dweights : device fp32 [T][k] out, or NULL
 * dweights are fp32 sums in one order for given sizes.  (The addend's gradient is dy.)
 * Limits, errors (weights, dweights: 4) as moe_dispatch_rows's; MOE_ERR_INVALID_ARG
 * also for no output or dweights without o.  With M == 0 o and d_o are not looked at.
 */
moe_status moe_combine_grad(const void *dy, moe_dtype ydtype, const int32_t *pos, const float *weights, int T, int k,
                            int n, int M, const void *o, moe_dtype dtype, void *d_o, float *dweights,
                            cudaStream_t stream);

/*
 * Products of bf16 rows with bf16 matrices on the tensor cores, with bias,
 * activation and residual.  Grouped by expert, or one matrix for all rows: with
 *   v[i][n] = bias[g][n] + sum_k x[r][k] w[g][n][k],   r = rows ? rows[i] : i
 * for the places i of each group g, offsets[g] <= i < offsets[g+1],
 *   y[i] = act(v[i]) + residual[i]
 * for MOE_ACT_NONE to MOE_ACT_SWIGLU, and y[i] = v[i] act'(z[i]) for the gradients
 * (moe_act; the product is then the gradient that comes back through the next
 * matrix, and y is that of v as the forward call had it).
 *   x        : device bf16 [X][K]
 *   rows     : device int32 [M], values in [0, X), or NULL (needs X >= M)
 *   offsets  : device int32 [G+1], rising, in [0, M], or NULL (G == 1, all M)
 *   w        : device bf16 [G][N][K] (MOE_ACT_SWIGLU: [G][2N][K], gate rows, then
 *              up rows), or with transposed != 0 [G][K][N]: a matrix as the forward
 *              call has it takes gradients back
 *   bias     : device fp32 [G][N] ([G][2N]), or NULL; not with the gradients
 *   residual : device [M][N] of `ydtype`, or NULL; not with the gradients.  May be y.
 *   z        : device [M][N] ([M][2N]) of `ydtype`: v, out, or NULL; not with
 *              MOE_ACT_NONE.  The gradients need it, as an input; there it may be y.
 *   y        : device [M][N] ([M][2N] with MOE_ACT_SWIGLU_GRAD) of `ydtype` out.
 *              Rows of no group keep their values (z too).
 *   ws       : device workspace of moe_matmul_workspace_bytes() bytes (the status
 *              word, moe_read_device_status), zero-filled before its first use.
 *              Calls that overlap on the GPU may share it.
 * Sums are fp32, in one order for given sizes: equal calls give equal bits, other
 * sizes may add up in another order.  The tensor cores cut a running sum off below 24
 * bits, towards zero.  For fp32 results it is at most 640 values long (over a matrix of
 * results the error is about 5e-7 of them in the norm, and within 1e-6); for bf16 at
 * most 8192 (about 2^-15 of itself where all terms have one sign, beside the rounding to
 * bf16 by up to 2^-8).  Activations are fp32, of
 * the unrounded v, with sigma by the machine's exp (off by (5 + 1.3 |v|) 2^-24 of itself;
 * what lies below 2^-126, from about v = -87.3 down, counts as 0).
 * Row indexes and offsets outside their ranges are never followed (MOE_DEV_BAD_ROW);
 * the product of such a row is 0.  y and z must not overlap x, w or one another but
 * as stated.
 * Limits: X, M in [0, MOE_MAX_ROWS] (M == 0 is a no-op), 1 <= G <=
 * MOE_MAX_EXPERTS, 1 <= N <= 2^20, 8 <= K <= 2^20, K % 8 == 0; transposed: N % 8 == 0;
 * MOE_ACT_SWIGLU: N % 16 == 0, not transposed; G*N <= 2^30, X*K <= 2^35.
 * Errors: MOE_ERR_INVALID_ARG for limits, types, act, a NULL buffer, X < M without
 * rows, X == 0, offsets missing with G > 1, bias, residual or z where they have no
 * place, z missing, or x, w, y, z, residual not 16-byte aligned (bias, rows,
 * offsets: 4); MOE_ERR_UNSUPPORTED for K or N outside the rules above, or for 2^30 or
 * more tiles of 128 columns (gate and up counted) by 32 places, of which there are
 * ceil(M / 32) a column tile, with offsets floor(M / 32) + min(G, M);
 * MOE_ERR_WORKSPACE for a missing, short or unaligned ws.
 */
moe_status moe_matmul(const void *x, int X, const int32_t *rows, int M, const int32_t *offsets, int G, const void *w,
                      int transposed, const float *bias, moe_act act, const void *residual, void *z, int N, int K,
                      void *y, moe_dtype ydtype, void *ws, size_t ws_bytes, cudaStream_t stream);
size_t moe_matmul_workspace_bytes(void);

/*
 * Reads (and, if clear != 0, zeroes) the device status word at the start of
 * an FFN, layer or product workspace (all keep it in their first 4 bytes).
 * Synchronises `stream`.  *flags receives MOE_DEV_* bits.
 * Returns MOE_ERR_DEVICE_STATUS if any bit was set, MOE_OK otherwise.
 */
moe_status moe_read_device_status(void *ws, int clear, uint32_t *flags, cudaStream_t stream);

/*
 * Test hook: the exact int32 sub-block dots of one row of a packed matrix
 * with one q8 activation record, computed by the same device code the FFN
 * uses (the README's one-row GPU-vs-CPU arbiter idea).  Q4_K: 8 per
 * 256-block; Q2_K: 16; Q8_0 and MXFP4: 1 per 32-block.
 *   packed: device (moe_pack_weights); xq: device, one record of width cols;
 *   isums: device int32 out, cols/256*8, cols/256*16 or cols/32 entries.
 */
moe_status moe_debug_row_dots(const void *packed, moe_qtype qtype, int rows, int cols, int row,
                              const void *xq, int32_t *isums, cudaStream_t stream);

/*
 * Test hook: the bound, in SM clock cycles, on how long a moe_layer_forward
 * launch made after this call waits for another block's exchange words
 * (logits, h, o) before it gives up with MOE_DEV_TIMEOUT; 0 restores the
 * default (8e8 cycles).  A short bound makes the timeout path run without
 * any fault: the launch skips the remaining work, lets its own bulk copies
 * land (those waits keep the long bound) and returns.  Host-side setting of
 * this process, read when a layer launch is made (a captured graph keeps the
 * value it was captured with).  Errors: MOE_ERR_INVALID_ARG for cycles < 0.
 */
moe_status moe_debug_set_exchange_wait(long long cycles);

/*
 * Test hook: makes the waits of moe_fp8_matmul launches made after this call
 * run out (those of more than 16 places; fewer wait for nothing).
 *   hold   : 0 off (the default); 1: each stage's copies wait for one arrival
 *            more, which never comes; 2: each stage's products do
 *   cycles : the bound on waits, in SM clock cycles, taken in units of 65536;
 *            0 restores the default (8e8 cycles)
 * A held launch records MOE_DEV_TIMEOUT, stores nothing, lets its copies and
 * products in flight end (for which it waits up to 8e8 cycles) and returns.  Host-side setting of this process, read when a launch is made
 * (a captured graph keeps the value it was captured with).  Errors:
 * MOE_ERR_INVALID_ARG for another hold or cycles < 0.
 */
moe_status moe_debug_hold_fp8_matmul(int hold, long long cycles);

/*
 * Test hook: the same for moe_matmul launches made after this call (those of more
 * than 32 places or with transposed; fewer may wait for nothing).
 */
moe_status moe_debug_hold_matmul(int hold, long long cycles);

const char *moe_status_str(moe_status s);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */

/*
 * klt.h -- C ABI of the GB300 latent-MoE layer tail library (libklt.so).
 *
 * The tail (Kimi K3 latent MoE, as described in the vLLM pull request "Fuse BF16 shared
 * experts into latent MegaMoE tail", Summary, and DeepGEMM PR 416 "Fuse and publish Kimi
 * K3's BF16 shared expert", Summary) computes, for every token t:
 *
 *   ids, w   = top-k of logits[t] and the softmax of the selected logits   (routing)
 *   zq, zs   = e4m3 quantisation of z[t] per 128 columns, fp32 scale amax/448
 *   r[t]     = sum_j w_j * SwiGLU-expert_{ids_j}(zq)       (routed experts, latent width L)
 *   n[t]     = RMSNorm(r[t]) * gamma                       (fp32 statistics)
 *   out[t]   = bf16( n[t] W_up^T + SwiGLU-shared(x[t]) )   (3584 -> 7168 up-projection
 *                                                           plus the BF16 shared expert,
 *                                                           summed in fp32, rounded once)
 *
 * Routed expert e: h = zq W13_e^T with gate = rows [0, I), up = rows [I, 2I);
 * a = silu(gate) * up quantised per 128 like z; y = aq W2_e^T.  Shared expert:
 * hs = x Ws13^T (gate rows [0, Is), up rows [Is, 2 Is)); s = (silu(g) * u) Ws2^T.
 *
 * Conventions for every entry point:
 *  - every function returns a klt status code (KLT_OK == 0);
 *  - pointers named "device" must be CUDA device pointers on the current device and
 *    16-byte aligned; the library never frees caller memory;
 *  - arguments are checked on the host before anything is launched; a failed check
 *    launches nothing and changes no state;
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).
 */
#ifndef KLT_H_
#define KLT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ status codes */
enum klt_status_code {
  KLT_OK = 0,
  KLT_ERR_INVALID_ARG = 1,     /* null pointer, M < 0, M > max_tokens, bad eps, ...     */
  KLT_ERR_UNSUPPORTED = 2,     /* a width not a multiple of 128, topk > E, E > 256,
                                  routed format unknown, device is not sm_103          */
  KLT_ERR_ALIGN = 3,           /* a pointer is not 16-byte aligned                     */
  KLT_ERR_CUDA = 4,            /* a CUDA runtime call or launch failed                 */
  KLT_ERR_DEVICE_TIMEOUT = 5,  /* a bounded on-device wait ran out (sticky)            */
  KLT_ERR_OOM = 6,             /* device allocation failed in klt_create               */
  KLT_ERR_TOO_LARGE = 7        /* request exceeds the fixed scratch of klt_route_noalloc */
};

/* Routed expert weight formats. */
enum klt_routed_format {
  KLT_FMT_FP8_B128 = 0,  /* e4m3 codes, one fp32 scale per 128 x 128 block            */
  KLT_FMT_NVFP4 = 1,     /* e2m1 codes (two per byte, even K in the low nibble), one
                            e4m3 scale per 16 K-elements, one fp32 scale per matrix    */
  KLT_FMT_MXFP8 = 2,     /* e4m3 codes, one power-of-two scale per 32 K-elements of a row
                            (an UE8M0 byte b: scale 2^(b-127)); the routed activations are
                            quantised the same way (scale 2^(floor(log2 amax) - 8)) and the
                            tensor core applies the scales (block-scaled MMA, no epilogue
                            promotion).  Needs H and L multiples of 256; always runs the
                            token-major engine.                                         */
  KLT_FMT_NVFP4_W4A4 = 3 /* NVFP4 weights as in KLT_FMT_NVFP4, kept packed in device
                            memory (0.5625 bytes per weight), and NVFP4 routed
                            activations: per 16 elements an e4m3 scale s = e4m3(amax / 6)
                            and e2m1 codes of v / s (nearest even, saturating, no tensor
                            scale).  The tensor core applies both operands' e4m3 scales
                            (block-scaled FP4 MMA, scale vector of 4 per 64 K) and the
                            epilogue the weights' fp32 per-matrix scale.  Needs H, L and I
                            multiples of 256; always runs the token-major engine.      */
};

/* klt_create flags. */
enum klt_flags {
  KLT_FLAG_NO_PDL = 1u << 0,  /* launch the kernels with plain stream ordering instead of
                                 programmatic dependent launch                          */
  KLT_FLAG_PHASED = 1u << 1,  /* run the GEMM stages as three launches plus a norm launch
                                 instead of one persistent launch with device-side
                                 dependencies (same results; for comparison)            */
  KLT_FLAG_DETERMINISTIC = 1u << 2 /* combine the routed experts' outputs in a fixed order:
                                 each (token, choice) slot's weighted output is stored and
                                 the norm sums a token's topk slots in choice order, so the
                                 output is bitwise reproducible run to run (by default the
                                 routed L2 units add into an fp32 row as they finish).
                                 Costs max_tokens * topk * L * 4 bytes of workspace and
                                 that traffic per forward.  Not combinable with
                                 KLT_FLAG_PHASED (klt_create: KLT_ERR_UNSUPPORTED).       */
};

/* Layer shape.  H, L, I, Is must be multiples of 128; 1 <= topk <= min(E, 32);
 * 1 <= E <= 256; 1 <= max_tokens and max_tokens * topk <= 2^20; eps > 0. */
typedef struct klt_dims {
  int32_t H;           /* hidden width (7168): shared-expert input and tail output   */
  int32_t L;           /* latent width (3584): routed-expert input and output         */
  int32_t E;           /* routed experts                                              */
  int32_t topk;        /* experts per token                                           */
  int32_t I;           /* routed expert intermediate width                            */
  int32_t Is;          /* shared expert intermediate width                            */
  int32_t routed_fmt;  /* enum klt_routed_format                                      */
  float eps;           /* RMSNorm epsilon                                             */
  int32_t max_tokens;  /* largest M klt_forward accepts; sizes the workspace          */
} klt_dims;

/* Layer weights, all device pointers, row-major.  klt_create copies them into memory the
 * handle owns (re-laid out for the kernels); the caller's buffers are not referenced after
 * klt_create returns.
 *   FP8 routed:   w13 e4m3 [E, 2I, L]; w13_scale f32 [E, 2I/128, L/128];
 *                 w2  e4m3 [E, L, I];  w2_scale  f32 [E, L/128, I/128];
 *                 w13_global, w2_global unused (may be NULL).
 *   NVFP4 routed (KLT_FMT_NVFP4 and KLT_FMT_NVFP4_W4A4):
 *                 w13 packed e2m1 [E, 2I, L/2]; w13_scale e4m3 [E, 2I, L/16];
 *                 w13_global f32 [E]; w2 packed [E, L, I/2]; w2_scale e4m3 [E, L, I/16];
 *                 w2_global f32 [E].
 *   MXFP8 routed: w13 e4m3 [E, 2I, L]; w13_scale uint8 UE8M0 [E, 2I, L/32];
 *                 w2 e4m3 [E, L, I];  w2_scale uint8 UE8M0 [E, L, I/32];
 *                 w13_global, w2_global unused (may be NULL).
 *   Shared/dense: ws13 bf16 [2 Is, H] (gate rows first); ws2 bf16 [H, Is];
 *                 w_up bf16 [H, L]; gamma bf16 [L]. */
typedef struct klt_weights {
  const void* w13;
  const void* w13_scale;
  const float* w13_global;
  const void* w2;
  const void* w2_scale;
  const float* w2_global;
  const void* ws13;
  const void* ws2;
  const void* w_up;
  const void* gamma;
  /* Optional: the step before the tail (both or neither; NULL = klt_forward_hidden is not
   * available on the handle).  w_lat bf16 [L, H] maps the hidden state to the latent
   * input; w_gate bf16 [E, H] gives the router logits. */
  const void* w_lat;
  const void* w_gate;
} klt_weights;

/* Optional routing outputs of klt_forward (every pointer may be NULL; device memory,
 * caller owned).  Pair i = t * topk + j.  Pairs are grouped by expert, pairs of one expert
 * in ascending i; p indexes that order.
 *   ids int32 [M, topk] (descending logit, ties to the lower expert index);
 *   weights f32 [M, topk] (softmax over the selected logits);
 *   cnt int32 [E]; off int32 [E + 1] (exclusive prefix of cnt);
 *   gidx int32 [M * topk] (token of pair p); slot int32 [M * topk] (i of pair p);
 *   pos int32 [M, topk] (p of pair (t, j)). */
typedef struct klt_routing {
  int32_t* ids;
  float* weights;
  int32_t* cnt;
  int32_t* off;
  int32_t* gidx;
  int32_t* slot;
  int32_t* pos;
} klt_routing;

/* Optional stage outputs for testing and profiling (every pointer may be NULL; device
 * memory, caller owned; copied on `stream` after the stage that writes them).
 *   zq e4m3 [M, L], zs f32 [M, L/128]: quantised latent input (MXFP8 layers: zsx below;
 *     NVFP4_W4A4 layers: zq packed e2m1 [M, L/2], even column in the low nibble, and zsx);
 *   aq e4m3 [M * topk, I], as f32 [M * topk, I/128]: quantised routed SwiGLU output,
 *     rows in pair order p (MXFP8 layers: aq only; NVFP4_W4A4 layers: aq packed e2m1
 *     [M * topk, I/2] only);
 *   r f32 [M, L]: routed combine (not formed with KLT_FLAG_DETERMINISTIC, whose norm sums
 *     the per-pair outputs directly; the norm normally zeroes it for the next forward, so
 *     asking for it makes the next forward clear the buffer first); n bf16 [M, L]:
 *     RMSNorm output (gamma applied);
 *   a_s bf16 [M, Is]: shared-expert SwiGLU output;
 *   events: up to 8 cudaEvent_t handles, events[i] recorded after launch i (NULL skips);
 *   stall_after_kblocks: test hook, 0 = off; when > 0 the tile producer of the first
 *     GEMM stops feeding data after that many k-blocks, so its consumers' bounded waits
 *     run out and klt_status reports KLT_ERR_DEVICE_TIMEOUT;
 *   timeout_ms: bound of every on-device wait for this call (0 = the default, 1000 ms);
 *   trace: optional device int64 buffer of 3 * trace_entries * 4 * (SM count) entries; when
 *     set, each GEMM launch g (0..2) records globaltimer stamps (ns) per CTA c and role r
 *     (0 = weight tile copy issued, 1 = work unit published to the MMA issuer and epilogue,
 *     2 = epilogue step done, 3 = task index + 1 of that unit, not a time) at
 *     trace[((g * SMs + c) * 4 + r) * trace_entries + i], first trace_entries
 *     events each; unused entries are left untouched;
 *   force_bn: GEMM engine and token-tile width for this call, for tuning sweeps:
 *     16, 32, 64 or 128 = feature-major engine (128 weight rows x force_bn tokens per
 *     MMA); 256 = token-major engine (128 tokens x 256 features per MMA; needs H and L
 *     multiples of 256 and the fused schedule, else KLT_ERR_UNSUPPORTED); 0 = chosen
 *     from M (feature-major with 16-token tiles up to 16 tokens, token-major above when
 *     available). */
typedef struct klt_debug {
  uint8_t* zq;
  float* zs;
  uint8_t* aq;
  float* as;
  float* r;
  void* n;
  void* a_s;
  void* events[8];
  int32_t stall_after_kblocks;
  int32_t timeout_ms;
  int64_t* trace;
  int32_t trace_entries;
  int32_t force_bn;
  /* klt_forward_hidden only: the latent input bf16 [M, L] and router logits f32 [M, E]
   * it computed from the hidden state */
  void* z;
  float* logits;
  /* MXFP8 layers: the latent input's UE8M0 scale bytes uint8 [M, L/32]; NVFP4_W4A4
   * layers: its e4m3 scale bytes uint8 [M, L/16] (zs is not formed in either) */
  uint8_t* zsx;
} klt_debug;

typedef struct klt_handle klt_handle;

/* Create a tail for one layer on the current device.
 * Defined by: DeepGEMM PR 416 "Fuse and publish Kimi K3's BF16 shared expert", Summary
 * (routed FP8/FP4 experts scheduled with a BF16 shared expert's L1/L2), and the vLLM pull
 * request "Fuse BF16 shared experts into latent MegaMoE tail", Summary (the routed result's
 * RMSNorm and 3584 -> 7168 up-projection before the two branches are added); the weight
 * formats are the readings of those pages' "FP8/FP4" listed with klt_weights.
 * Synchronous.  Copies and re-lays out
 * the weights, allocates the workspace for `d->max_tokens` tokens and encodes the TMA
 * descriptors.  Errors: KLT_ERR_INVALID_ARG (null d/w/out or a null weight pointer),
 * KLT_ERR_UNSUPPORTED (shape rules above; device is not compute capability 10.3),
 * KLT_ERR_ALIGN, KLT_ERR_OOM, KLT_ERR_CUDA.  On error *out is left NULL. */
int klt_create(const klt_dims* d, const klt_weights* w, uint32_t flags, klt_handle** out);

/* Run the tail for M tokens, asynchronously on `stream`.
 * Defined by: the vLLM pull request "Fuse BF16 shared experts into latent MegaMoE tail",
 * Summary (route, routed experts in the 3584-wide latent space, routed RMSNorm, 3584 -> 7168
 * up-projection, shared-expert output added in FP32, BF16 result) and tokenspeed PR 1062
 * "MNNVL CuTe-DSL finalize tail", commit notes (top-k weighted combine as the finalize step;
 * fp32-internal norm, one rounding).
 *   x      device bf16 [M, H]  hidden state (shared-expert input);
 *   z      device bf16 [M, L]  latent state (routed-expert input);
 *   logits device f32  [M, E]  router logits (finite values);
 *   out    device bf16 [M, H]  result.
 * M == 0 launches nothing and returns KLT_OK.  The handle's workspace is reused by every
 * call, so calls on one handle must be ordered on one stream (or synchronised).
 * Errors: KLT_ERR_INVALID_ARG (null handle or pointer, M < 0, M > max_tokens),
 * KLT_ERR_ALIGN, KLT_ERR_CUDA (a launch failed).  Device-side faults of bounded waits are
 * reported later by klt_status. */
int klt_forward(klt_handle* h, const void* x, const void* z, const float* logits, int32_t M,
                void* out, klt_routing* routing_out, klt_debug* dbg, void* stream);

/* Run the step before the tail and then the tail for M tokens, from the hidden state alone,
 * asynchronously on `stream`.
 * Defined by: tokenspeed PR 1062 "MNNVL CuTe-DSL finalize tail", commit notes (the model's
 * latent input projections feeding the latent MoE).  Computes, on the GPU,
 *   z      = bf16( x W_lat^T )     bf16 [M, L]  (fp32 accumulation, one rounding)
 *   logits = x W_gate^T            f32  [M, E]
 * into the handle's workspace and then runs exactly what klt_forward runs on them.
 *   x   device bf16 [M, H];  out device bf16 [M, H].
 * Launches one kernel more than klt_forward (the projection, first).  The handle must have
 * been created with w_lat and w_gate.  Errors: as klt_forward, and KLT_ERR_UNSUPPORTED
 * when the handle has no projection weights. */
int klt_forward_hidden(klt_handle* h, const void* x, int32_t M, void* out,
                       klt_routing* routing_out, klt_debug* dbg, void* stream);

/* Sticky device status of the handle: KLT_OK or KLT_ERR_DEVICE_TIMEOUT.  Reads device
 * memory synchronously, so call it after the forward's stream has been synchronised.  A
 * handle that reported a device error must be destroyed. */
int klt_status(klt_handle* h);

/* Free everything the handle owns (synchronises the device first).  NULL is a no-op. */
int klt_destroy(klt_handle* h);

/* Static description of a status code. */
const char* klt_strerror(int code);

/* Number of kernels one klt_forward launches for the given M and handle at the automatic
 * GEMM configuration (0 for M == 0): the routing launches (one for a feature-major batch of
 * at most 256 (token, choice) pairs with e4m3 activations; otherwise routing, an expert
 * histogram above 1024 pairs, scatter and gather) and then the GEMM launches (one; two for
 * the block-scaled formats; four with KLT_FLAG_PHASED). */
int klt_launch_count(const klt_handle* h, int32_t M);

/* GEMM configuration klt_forward uses for M tokens when klt_debug.force_bn = force_bn
 * (0 = automatic): 16, 32, 64 or 128 = the feature-major engine with that token tile,
 * 256 = the token-major engine (128-token x 256-feature units).  A negative value is the
 * negated status klt_forward would return: -KLT_ERR_UNSUPPORTED when force_bn = 256 is not
 * available for this handle, -KLT_ERR_INVALID_ARG for a NULL handle. */
int klt_gemm_tile(const klt_handle* h, int32_t M, int32_t force_bn);

/* Largest M * topk klt_route_noalloc accepts (its fixed scratch size, about 320 KB). */
#define KLT_NOALLOC_MAX_PAIRS 65536

/* Routing and expert permutation without a handle and without any device allocation.
 * The pages describe no such entry point; it exists for callers that cannot allocate
 * device memory where they route (inside another framework's memory pool, serving loops
 * that fix every allocation at start-up, runtimes without allocator access).
 * Computes the same ids, weights, cnt, off, gidx, slot and pos as klt_forward's routing
 * outputs (same layouts as klt_routing) for `logits` f32 [M, E], all pointers device
 * memory, caller owned, 16-byte aligned, none NULL.  Internal buffers live in one
 * fixed-size device array (KLT_NOALLOC_MAX_PAIRS pairs) that every GPU loading the library
 * holds until exit; calls share it, so calls whose kernels overlap on the GPU race; order
 * them on one stream.  The first call on a device resolves the array's device address
 * and caches it for the life of the process; make that first call before any stream
 * capture.  A device reset (cudaDeviceReset) after that first call is not supported: the
 * library may then load the array at another address while the cache keeps the old one.
 * Asynchronous on `stream`.
 * Errors: KLT_ERR_INVALID_ARG (M < 0, E or topk < 1, NULL pointer), KLT_ERR_UNSUPPORTED
 * (E > 256, topk > E, topk > 32), KLT_ERR_TOO_LARGE (M * topk > KLT_NOALLOC_MAX_PAIRS),
 * KLT_ERR_ALIGN, KLT_ERR_CUDA.  M == 0 launches nothing. */
int klt_route_noalloc(const float* logits, int32_t M, int32_t E, int32_t topk, int32_t* ids,
                      float* weights, int32_t* cnt, int32_t* off, int32_t* gidx,
                      int32_t* slot, int32_t* pos, void* stream);

/* ------------------------------------------------- operators around the tail
 *
 * The steps between layers and the dense FP8 layers beside the mixture-of-experts ones, in
 * the tail's own formats: bf16 (or fp32) activations, and e4m3 codes with one fp32 scale
 * per row and 128 columns (activations) or per 128 x 128 block (weights).  Calls are
 * asynchronous on `stream`, make no host synchronisation and can be captured in CUDA
 * graphs; none of them keeps state between calls, so calls on several streams may overlap
 * as long as their outputs differ.  Strides (ld_*) count elements from one row to the next;
 * columns are contiguous.  Tensors of these calls need the alignment of their element type
 * only, except where a rule is given; rows that start on 16 bytes are faster.  What lies
 * between two rows of an input may be read; between rows of an output nothing is written. */

/* Element types of activations. */
enum klt_dtype {
  KLT_DT_BF16 = 0,
  KLT_DT_F32 = 1,
  KLT_DT_E4M3 = 2 /* e4m3 codes with a scale per row and 128 columns (outputs only)      */
};

/* Quantise x [M, K] (bf16 or fp32) to e4m3 codes q [M, K] and fp32 scales s
 * [M, ceil(K / 128)] (contiguous): per row and 128 columns s = amax / 448 in fp32 (1 where
 * that is 0), codes e4m3(fp32(x / s)), nearest even, saturating; the last group may be
 * short.  The same values as the tail's own latent quantisation.  A group that
 * holds an infinity or a NaN gets a scale that is not finite.
 * Any K from 1 to 2^28; M == 0 launches nothing.  Bytes of q between K and ld_q are left as
 * they are.
 * Errors: KLT_ERR_INVALID_ARG (M < 0, K < 1, null pointer, negative or overlapping output
 * stride), KLT_ERR_UNSUPPORTED (unknown x_dtype, K too large, more than 2^31 groups),
 * KLT_ERR_ALIGN (element alignment), KLT_ERR_CUDA. */
int klt_quantize(const void* x, int32_t x_dtype, int64_t ld_x, int32_t M, int32_t K,
                 uint8_t* q, int64_t ld_q, float* s, void* stream);

/* Largest row klt_block_norm accepts. */
#define KLT_BLOCK_NORM_MAX_H 16384

/* The norms before and after a block, fused with its gate and residual scale: for a row of
 * the residual stream h and of the block's output y,
 *   u  = y / sqrt(mean(y^2) + eps) * gamma_post       (u = y when gamma_post is NULL)
 *   h' = res_scale * h + branch_scale * g * u         (h' = res_scale * h when y is NULL)
 *   n  = h' / sqrt(mean(h'^2) + eps) * gamma_pre      (n = h' when gamma_pre is NULL)
 * with g = gate, or 1 / (1 + e^-gate) with gate_sigmoid, or 1 when gate is NULL.  Everything
 * is fp32 until the outputs, each rounded once; n and its codes come from the unrounded h'.
 * So one call leaves a block and enters the next one; y == NULL enters the first block. */
typedef struct klt_block_norm_args {
  int32_t M, H;           /* rows; columns, 1 <= H <= KLT_BLOCK_NORM_MAX_H               */
  int32_t h_dtype;        /* of h and h_out: KLT_DT_BF16 or KLT_DT_F32                    */
  int32_t y_dtype;        /* KLT_DT_BF16 or KLT_DT_F32                                    */
  int32_t gate_dtype;     /* KLT_DT_BF16 or KLT_DT_F32                                    */
  int32_t gate_sigmoid;   /* non-zero: g = sigmoid(gate)                                  */
  float eps, res_scale, branch_scale;
  const void* h;          /* [M, H] residual stream                                       */
  const void* y;          /* [M, H] block output, or NULL                                 */
  const void* gate;       /* element (m, c) at m * gate_row + c * gate_col, or NULL: strides
                             (0, 1) one gate per channel, (1, 0) one per token            */
  const void* gamma_post; /* bf16 [H] or NULL                                             */
  const void* gamma_pre;  /* bf16 [H] or NULL                                             */
  void* h_out;            /* h' [M, H], or NULL; may be h itself with the same stride     */
  void* n;                /* bf16 [M, H], or NULL; may be y (bf16) with the same stride   */
  uint8_t* q;             /* e4m3 codes of n [M, H], or NULL: n = t / rms with t = h' gamma_pre;
                             codes e4m3(fp32(t / d)) with d = fp32(amax of t / 448) per row
                             and 128 columns, both unrounded, so the row's 1 / rms enters
                             the scale alone                                              */
  float* s;               /* scales of q [M, ceil(H / 128)], with q: fp32(d / rms) (1, with
                             codes of 0, where that is 0).  klt_quantize of the same n differs
                             by the scale's last bit and by codes next to a tie           */
  int64_t ld_h, ld_y, gate_row, gate_col, ld_h_out, ld_n, ld_q;
} klt_block_norm_args;

/* Run klt_block_norm_args on `stream`.  M == 0 launches nothing.  Outputs overlap each
 * other or the inputs only as the fields above allow.
 * Errors: KLT_ERR_INVALID_ARG (null args or h, M < 0, H < 1, eps negative or NaN, no output
 * at all, q without s or s without q, gate or gamma_post without y, negative stride, output
 * rows that overlap), KLT_ERR_UNSUPPORTED (H too large, unknown dtype), KLT_ERR_ALIGN
 * (element alignment), KLT_ERR_CUDA. */
int klt_block_norm(const klt_block_norm_args* a, void* stream);

/* A linear layer with FP8 weights, y = x W^T:  out[m, o] = sum over k of
 * (xq[m, k] xs[m, k / 128]) (wq[o, k] ws[o / 128, k / 128]); products of 128 columns are
 * summed by the tensor core in fp32, multiplied by the fp32 product of their two scales (which
 * is to stay in the normal range), added up in fp32, and rounded once. */
enum klt_linear_act {
  KLT_ACT_NONE = 0,
  KLT_ACT_SWIGLU = 1 /* out[m, i] = silu(y[m, i]) * y[m, N/2 + i]: the gate rows of W come
                        first, as in the expert weights; N a multiple of 256              */
};
typedef struct klt_linear_dims {
  int32_t N;         /* rows of W (outputs; for SwiGLU twice the outputs), >= 1           */
  int32_t K;         /* columns of W, >= 1                                                */
  int32_t act;       /* enum klt_linear_act                                               */
  int32_t out_dtype; /* KLT_DT_BF16; KLT_DT_F32 (KLT_ACT_NONE only); KLT_DT_E4M3
                        (KLT_ACT_SWIGLU only): codes and scales as klt_quantize of the
                        unrounded fp32 result                                             */
} klt_linear_dims;

typedef struct klt_linear klt_linear;

/* Test and tuning hooks of klt_linear_forward (NULL or zeros = none). */
typedef struct klt_linear_debug {
  int32_t stall_after_kblocks; /* > 0: every copy producer stops after that many k-blocks, so
                                  the waits on its data run out (klt_linear_status)       */
  int32_t timeout_ms;          /* bound of every on-device wait (0 = 1000 ms)             */
  int32_t force_tile;          /* token tile: 16, 32, 64, 128 = feature-major kernel, 256 =
                                  token-major kernel, 0 = chosen from the sizes           */
  int32_t force_split;         /* parts that K is split into: 1, 2, 4, 8 (tile 256: 1, 2),
                                  at most K / 128 rounded up; 0 = chosen                  */
} klt_linear_debug;

/* Create a linear layer on the current device.  w: e4m3 [N, K] row-major; w_scale: fp32
 * [ceil(N / 128), ceil(K / 128)]; both device memory, copied (re-laid out) into memory the
 * handle owns; the caller's buffers are not referenced after the call returns.
 * Synchronous, on the legacy default stream, and not during a stream's capture.
 * Errors: KLT_ERR_INVALID_ARG (null pointer), KLT_ERR_UNSUPPORTED (shape or format rules
 * above; N or K above 2^20; device is not compute capability 10.3), KLT_ERR_ALIGN (w_scale not
 * 4-byte aligned), KLT_ERR_OOM, KLT_ERR_CUDA.  On error *out is left NULL. */
int klt_linear_create(const klt_linear_dims* d, const void* w, const float* w_scale,
                      klt_linear** out);

/* out = act(x W^T) for M tokens.  xq: e4m3 [M, K], 16-byte aligned, ld_xq a multiple of 16;
 * xs: fp32 [M, ceil(K / 128)] contiguous; out: [M, N] (SwiGLU: [M, N/2]) of out_dtype;
 * out_s: fp32 [M, N / 256] for KLT_DT_E4M3, else ignored.  M == 0 launches nothing.  The
 * handle has no workspace: calls on several streams may overlap.  One launch.
 * Errors: KLT_ERR_INVALID_ARG (null handle or pointer, M < 0 or M > 2^22, a stride shorter
 * than a row, another device current than at creation, bad debug value), KLT_ERR_UNSUPPORTED
 * (M * ceil(K / 128) above 2^31 - 1; debug: a tile and split that do not go together or
 * more than 65535 token tiles), KLT_ERR_ALIGN (xq or ld_xq not 16-byte, out, xs or out_s not
 * element aligned), KLT_ERR_CUDA.  Expired device waits: klt_linear_status. */
int klt_linear_forward(klt_linear* h, const uint8_t* xq, int64_t ld_xq, const float* xs,
                       int32_t M, void* out, int64_t ld_out, float* out_s,
                       const klt_linear_debug* dbg, void* stream);

/* Kernel configuration klt_linear_forward chooses for M tokens: the token tile (as
 * force_tile) plus 1000 times the K split, or the negated status code. */
int klt_linear_tile(const klt_linear* h, int32_t M);

/* Sticky device status, as klt_status: KLT_OK or KLT_ERR_DEVICE_TIMEOUT, read
 * synchronously; call it after the forward's stream has been synchronised. */
int klt_linear_status(klt_linear* h);

/* Free everything the handle owns (synchronises the device first).  NULL is a no-op. */
int klt_linear_destroy(klt_linear* h);

#ifdef __cplusplus
}
#endif

#endif /* KLT_H_ */

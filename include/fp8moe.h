/*
 * fp8moe.h - C ABI of a GB300 (sm_103a) routed Mixture-of-Experts FFN layer
 * whose expert weights are blockwise FP8.
 *
 * The layer (one decoder MoE block's routed experts) computes, for T tokens:
 *   1. router logits in f32 inputs (dragon.c, "Precision": router f32),
 *      top-k by logit with ties to the lower expert index (Trochilus, "What
 *      makes it different", the lowest row wins a tie), weights = softmax over
 *      the k selected logits (softmax, top-k, renormalise);
 *   2. a histogram / exclusive scan / stable scatter of the T*k (token,
 *      expert) pairs by expert (Trochilus, "Acknowledgements": pairs sorted by
 *      a counting sort);
 *   3. per expert, SwiGLU: h = silu(W13[e, :I] x) * (W13[e, I:] x), with the
 *      gate rows before the up rows (DeepSeek-V4.1-Flash post, "Repack experts
 *      for the disk": gate | up | down);
 *   4. y = W2[e] h;
 *   5. out[t] = bf16( sum over r = 0..k-1, in router rank order, of
 *      w[t, r] * y[t, r] ) (WARP BACKENDS.md, "Coherent memory": partials
 *      reduced in original router order), with no float atomics.
 * Weights are e4m3 codes with one f32 scale per 128x128 block, stored with
 * the weights (dragon.c, "Precision"); a weight's value is its code's value
 * times its block's scale.
 *
 * Conventions (every call):
 *   - Return value: MOE_OK (0) or a negative MOE_ERR_* code; nothing throws.
 *   - Tensor arguments are raw pointers; "device" pointers must be CUDA
 *     device (or managed) memory of the context's device.  The caller owns
 *     every tensor; the context owns only its workspace.
 *   - All integer sizes are int64_t; all index arithmetic inside is 64-bit.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the host is not synchronised, except where stated.
 *   - One context serves one stream at a time: calls on one context must not
 *     overlap on the GPU.
 */
#ifndef FP8MOE_H
#define FP8MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_ARG (-1)            /* NULL pointer, bad enum, T < 0          */
#define MOE_ERR_SHAPE (-2)          /* H or I not a multiple of 128, k out of  */
                                    /* [1, min(E, max_top_k)], T > max_tokens  */
#define MOE_ERR_ALIGN (-3)          /* a pointer breaks its stated alignment   */
#define MOE_ERR_CUDA (-4)           /* a CUDA runtime/driver call failed       */
#define MOE_ERR_DEVICE_TIMEOUT (-5) /* a bounded device-side wait gave up      */
#define MOE_ERR_NOMEM (-6)          /* workspace allocation failed             */
#define MOE_ERR_UNSUPPORTED (-7)    /* device is not compute capability 10.3   */
#define MOE_ERR_NONFINITE (-8)      /* a router logit was NaN or infinite      */
#define MOE_ERR_DEVICE (-9)         /* a device-side consistency check failed  */

typedef struct moe_ctx moe_ctx; /* opaque; owned by the library */

typedef struct moe_config {
  int64_t max_tokens; /* largest T a forward may be called with (> 0)            */
  int64_t hidden;     /* H: model width, multiple of 128, <= 65536              */
  int64_t n_experts;  /* E: routed experts, 1..1024                             */
  int64_t inter;      /* I: expert FFN width, multiple of 128, <= 65536         */
  int32_t max_top_k;  /* largest k a forward may use, 1..min(E, 32)             */
  int32_t device;     /* CUDA device ordinal the context lives on              */
} moe_config;

/*
 * moe_init - validate `cfg` and allocate a context with a device workspace
 * sized for max_tokens * max_top_k (token, expert) pairs.
 *   out : receives the new context (host pointer to a host pointer).
 * Errors: MOE_ERR_ARG (NULL), MOE_ERR_SHAPE (cfg out of range; checked before
 * any CUDA call), MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_NOMEM.  On error
 * *out is set to NULL and nothing is leaked.
 */
int moe_init(moe_ctx **out, const moe_config *cfg);

/*
 * moe_layer_forward - run the layer on T tokens (steps 1-5 above).
 *   hidden      : device, bf16 [T, H] row-major, 16-byte aligned.
 *   router_w    : device, f32 [E, H] row-major, 16-byte aligned.
 *   router_bias : device, f32 [E], or NULL for none.  When present it is added
 *                 to the logits before selection and softmax.
 *   w13         : device, e4m3 [E, 2I, H] row-major (rows [0,I) gate,
 *                 [I,2I) up), 16-byte aligned.
 *   s13         : device, f32 [E, 2I/128, H/128] block scales, 4-byte aligned.
 *   w2          : device, e4m3 [E, H, I] row-major, 16-byte aligned.
 *   s2          : device, f32 [E, H/128, I/128] block scales, 4-byte aligned.
 *   top_k       : k, in [1, min(E, max_top_k)].
 *   out         : device, bf16 [T, H], 16-byte aligned; must not overlap any
 *                 input.
 *   stream      : cudaStream_t or NULL.
 * T = 0 is a no-op.  Routing is exact: indices, counts and the permutation
 * equal those of exact arithmetic on the inputs (f32 logits carry a rigorous
 * error bound; tokens whose order the bound cannot certify are recomputed
 * from exact products with every rounding error carried).  Device-side failures (a bounded wait that gave up, a non-finite
 * logit) are recorded in the context and reported by moe_status.
 */
int moe_layer_forward(moe_ctx *ctx, const void *hidden, int64_t T, const float *router_w,
                      const float *router_bias, const uint8_t *w13, const float *s13,
                      const uint8_t *w2, const float *s2, int32_t top_k, void *out,
                      void *stream);

/*
 * moe_layer_forward_host - moe_layer_forward with the activations in HOST
 * memory: copies hidden_host (bf16 [T, H]) to the device, runs the layer, and
 * copies the result into out_host (bf16 [T, H]).  Weights stay device
 * pointers as in moe_layer_forward.  Host buffers should be pinned
 * (cudaHostAlloc / cudaHostRegister) for asynchronous copies.  The call
 * returns after the result is in out_host (it synchronises `stream`).
 */
int moe_layer_forward_host(moe_ctx *ctx, const void *hidden_host, int64_t T,
                           const float *router_w, const float *router_bias, const uint8_t *w13,
                           const float *s13, const uint8_t *w2, const float *s2, int32_t top_k,
                           void *out_host, void *stream);

/*
 * moe_layer_forward_nvfp4 - the same layer (steps 1-5 above) with FP4 expert
 * weights in the NVFP4 format of the Qwen post's experts ("Why this model, of
 * all models"; "The engine", piece 1: half a byte per weight plus one e4m3
 * scale per 16 weights; piece 4: the e2m1 -> f16x2 hardware conversion).  A
 * weight's value is e2m1(code) * e4m3(group scale) * global scale.  The
 * router, hidden, out, top_k and stream arguments are those of
 * moe_layer_forward.
 *   w13  : device, u8 [E, 2I, H/2]: e2m1 codes of W13 (rows [0,I) gate,
 *          [I,2I) up), two per byte along H, element 2j in the low nibble;
 *          16-byte aligned.
 *   sf13 : device, u8 [E, 2I, H/16]: e4m3 scale of each 16 consecutive
 *          weights of a row; 2-byte aligned.
 *   g13  : device, f32 [E]: global scale of each expert's W13; 4-byte aligned.
 *   w2, sf2, g2 : the same for W2 [E, H, I] (codes [E, H, I/2], scales
 *          [E, H, I/16], globals [E]).
 * The expert kernels are grouped GEMVs (any T; built for small batches).
 * Errors as for moe_layer_forward; sf13 / sf2 NULL is MOE_ERR_ARG.
 */
int moe_layer_forward_nvfp4(moe_ctx *ctx, const void *hidden, int64_t T, const float *router_w,
                            const float *router_bias, const uint8_t *w13, const uint8_t *sf13,
                            const float *g13, const uint8_t *w2, const uint8_t *sf2,
                            const float *g2, int32_t top_k, void *out, void *stream);

/*
 * moe_get_routing - copy the routing of the last forward into caller device
 * buffers (any may be NULL to skip it).  Sizes for that forward's T and k,
 * P = T*k:
 *   idx     int32 [T, k]  experts of each token in rank order
 *   wts     f32   [T, k]  renormalised weights, same order
 *   counts  int32 [E]     pairs routed to each expert
 *   offsets int32 [E+1]   exclusive scan of counts
 *   perm    int32 [P]     position -> pair id p = t*k + r, ascending p within
 *                         each expert segment
 *   inv     int32 [P]     pair id -> position
 * Enqueued on `stream`.
 */
int moe_get_routing(moe_ctx *ctx, int32_t *idx, float *wts, int32_t *counts, int32_t *offsets,
                    int32_t *perm, int32_t *inv, void *stream);

/*
 * moe_status - synchronise the context's last stream and return MOE_OK or
 * the first device-side error recorded since the previous call (the flag is
 * cleared).
 */
int moe_status(moe_ctx *ctx);

/* moe_free - release the context and its workspace; NULL is a no-op. */
void moe_free(moe_ctx *ctx);

/* moe_strerror - static description of a return code. */
const char *moe_strerror(int code);

/*
 * Path selection.  MOE_PATH_AUTO picks the tensor-core decode path for
 * T <= 64 and the tensor-core grouped-GEMM path above (both need H % 256 == 0;
 * otherwise the grouped-GEMV path runs); the other values force one path (all
 * compute the same layer).
 *   MOE_PATH_GEMV   e4m3 weights dequantised in registers, mma.sync f16
 *                   (activations as f16 hi/lo pairs);
 *   MOE_PATH_GEMM   tcgen05 grouped GEMM, tiles of 128 positions;
 *   MOE_PATH_TCGEMV tcgen05 decode FFN: gate/up and down in one launch, tiles
 *                   of 16 positions (the weight rows are the MMA's N operand).
 */
#define MOE_PATH_AUTO 0
#define MOE_PATH_GEMV 1
#define MOE_PATH_GEMM 2
#define MOE_PATH_TCGEMV 3
int moe_set_path(moe_ctx *ctx, int path);
/* moe_resolve_path - the MOE_PATH_* (not AUTO) a forward of T tokens would
 * take on this context; MOE_ERR_ARG for a NULL context or T < 0. */
int moe_resolve_path(moe_ctx *ctx, int64_t T);

/*
 * Kernel timing.  moe_set_timing(ctx, mask) records CUDA events around each
 * kernel whose bit (1 << MOE_K_*) is set in `mask`, on the forward's stream
 * (mask 0 turns timing off; every call resets the totals).  moe_kernel_time
 * returns the summed device time (ms) and the number of timed launches of one
 * kernel (it synchronises).  moe_launch_count returns how many kernels the
 * context has launched since moe_init, timed or not.
 */
#define MOE_K_ROUTER_LOGITS 0
#define MOE_K_ROUTER_SELECT 1
#define MOE_K_PERMUTE 2
#define MOE_K_GATE_UP 3 /* grouped GEMV or GEMM for W13 with SwiGLU */
#define MOE_K_DOWN 4    /* grouped GEMV or GEMM for W2            */
#define MOE_K_COMBINE 5
#define MOE_K_ACT_QUANT 6
#define MOE_K_ROUTE 7   /* small batches: logits, selection and sort in one kernel */
#define MOE_K_COUNT 8
int moe_set_timing(moe_ctx *ctx, int mask);
int moe_kernel_time(moe_ctx *ctx, int kernel, double *total_ms, int64_t *launches);
int64_t moe_launch_count(moe_ctx *ctx);
const char *moe_kernel_name(int kernel);

/*
 * moe_debug_copy - copy a workspace buffer of the last forward into a caller
 * device buffer, for tests: "logits" f32 [T,E], "h" f32 [P,I] (GEMV path,
 * position order), "y" f32 [P,H] (position order; GEMV and GEMM paths),
 * "y_terms" f32 [3,P,H] (tensor-core decode path: y of a position is the sum
 * of its three rows, one per h term), "x16" f16 [T,H].  Copies
 * min(capacity, size) bytes on `stream` and stores the buffer's full size in
 * *nbytes (may be NULL).
 */
int moe_debug_copy(moe_ctx *ctx, const char *name, void *dst, int64_t capacity, int64_t *nbytes,
                   void *stream);

/*
 * Experts larger than device memory (DeepSeek-V4.1-Flash post, "Bytes per
 * token decide everything" and "Making it faster", v4: a cache in front of
 * the slow tier and the next layer's experts guessed from its router and
 * prefetched into the gap; Qwen post, "Where the time actually goes":
 * speculative copies one layer early).  The expert weights (e4m3 codes) stay
 * in host memory; `n_slots` experts at a time are held in device memory
 * (slabs of one expert's W13 and W2 codes) and streamed in over NVLink-C2C;
 * the layer's own kernels read expert e's codes from the slab a table names.
 * The f32 block scales (1/16384 of the codes) stay resident and are passed
 * as device pointers.
 *
 * moe_cache_init - create a cache for context `ctx`.
 *   w13_host : host, e4m3 [E, 2I, H] (layout of moe_layer_forward's w13).
 *   w2_host  : host, e4m3 [E, H, I].
 *   n_slots  : experts held in device memory, 1..E (3*I*H bytes of device
 *              memory each).
 * The host ranges are page-locked (cudaHostRegister) for the life of the
 * cache unless the caller already registered them; they must stay valid and
 * unchanged until moe_cache_free.
 * Errors: MOE_ERR_ARG, MOE_ERR_SHAPE (n_slots out of range), MOE_ERR_NOMEM,
 * MOE_ERR_CUDA.
 */
typedef struct moe_expert_cache moe_expert_cache;
int moe_cache_init(moe_expert_cache **out, moe_ctx *ctx, const uint8_t *w13_host,
                   const uint8_t *w2_host, int64_t n_slots);

/*
 * moe_cache_forward - moe_layer_forward with the cache's experts: routes on
 * `stream`, waits for the active-expert list (a host synchronisation of
 * `stream`), brings the missing experts into least recently used slots
 * (copies on `stream`), waits for earlier prefetches, then enqueues the
 * expert kernels and the combine.  Results are bit-identical to
 * moe_layer_forward with the same weights in device memory.  Consecutive
 * forwards of one cache must use one stream.  MOE_ERR_NOMEM if the batch
 * needs more experts than there are slots.
 */
int moe_cache_forward(moe_expert_cache *c, const void *hidden, int64_t T, const float *router_w,
                      const float *router_bias, const float *s13, const float *s2, int32_t top_k,
                      void *out, void *stream);

/*
 * moe_cache_prefetch - start bringing `experts` (host array of n expert
 * ids, best guess first) into the cache on the cache's own copy stream,
 * into slots that the last forward does not use; stops when no such slot is
 * left.  Returns the number of copies started (>= 0) or an error.  The next
 * moe_cache_forward waits for them.
 */
int moe_cache_prefetch(moe_expert_cache *c, const int32_t *experts, int64_t n);

/*
 * moe_cache_guess - the experts a router would pick for `hidden`: routes
 * hidden (device bf16 [T, H], T <= 64) with router_w / router_bias (device,
 * f32 [E, H] / [E] or NULL) on the cache's own stream, and writes to
 * experts_out (host, n_guess ints) the chosen experts ordered by the number
 * of tokens choosing them, then by their best rank, then by id.  Used with
 * the NEXT layer's router on this layer's input to guess what to prefetch.
 * Returns the number written (<= n_guess) or an error.
 */
int moe_cache_guess(moe_expert_cache *c, const void *hidden, int64_t T, const float *router_w,
                    const float *router_bias, int32_t top_k, int32_t n_guess, int32_t *experts_out);

/* moe_cache_stats - counters since moe_cache_init, out[0 .. n-1] (host). */
#define MOE_CACHE_HITS 0          /* active experts found in the cache        */
#define MOE_CACHE_MISSES 1        /* active experts copied in by a forward    */
#define MOE_CACHE_PREFETCHED 2    /* experts copied in by moe_cache_prefetch  */
#define MOE_CACHE_PREFETCH_USED 3 /* prefetched experts a forward then used   */
#define MOE_CACHE_EVICTIONS 4
#define MOE_CACHE_BYTES_COPIED 5  /* host -> device bytes of expert codes     */
#define MOE_CACHE_STATS 6
int moe_cache_stats(const moe_expert_cache *c, int64_t *out, int32_t n);

/* moe_cache_resident - slot of every expert, -1 if not cached (host int[E]). */
int moe_cache_resident(const moe_expert_cache *c, int32_t *slot_of_expert);

/* moe_cache_free - wait for the device and release everything; NULL is a
 * no-op. */
void moe_cache_free(moe_expert_cache *c);

/*
 * Shortcut-connected MoE (dragon.c, "Shortcut-connected MoE": the MoE is
 * computed on sub-block-0's normed hidden state and its output is added at
 * the END of sub-block-1, "a designed overlap window"; §10: "thread the MoE
 * against sub-block-1's attention").  The MoE forward and sub-block-1's
 * attention run on two streams; the two calls below make that overlap work.
 *
 * moe_set_sm_budget - let the layer's persistent kernels (one CTA per SM)
 * use at most n_sms SMs, leaving the rest to work on other streams; n_sms
 * <= 0 restores all SMs.  Takes effect from the next forward.
 */
int moe_set_sm_budget(moe_ctx *ctx, int32_t n_sms);

/*
 * moe_decode_attention - softmax attention of one new token per sequence
 * against its key/value cache:
 *   out[b, h] = softmax(q[b, h] . K[b, :, c]^T / sqrt(d)) V[b, :, c],
 *   c = h / (n_heads / n_kv_heads).
 *   q        : device bf16 [B, n_heads, d];
 *   k_cache, v_cache : device bf16 [B, S, n_kv_heads, d];
 *   out      : device bf16 [B, n_heads, d];
 *   workspace: device, at least moe_attention_workspace_bytes(B, S,
 *              n_heads, d) bytes (f32 partial results; caller-owned).
 * d must be 128; n_heads / n_kv_heads one of 1, 2, 4, 8 (MOE_ERR_SHAPE
 * otherwise); pointers 16-byte aligned.  f32 arithmetic, bf16 output.  No
 * counterpart in the pages beyond its role: sub-block-1's attention, the
 * work the MoE overlaps.
 */
int64_t moe_attention_workspace_bytes(int64_t B, int64_t S, int32_t n_heads, int32_t head_dim);
int moe_decode_attention(const void *q, const void *k_cache, const void *v_cache, int64_t B,
                         int64_t S, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, void *out,
                         void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Attention over a paged key/value cache: the serving form of the attention
 * beside the MoE (dragon.c, "Shortcut-connected MoE").  Many sequences of
 * different lengths share one cache of fixed-size pages; a decode step norms
 * and rotates the new token's query and key heads, puts its key and value
 * rows into the cache (bf16, or quantised to e4m3) and attends to the
 * sequence's pages.  No counterpart in the pages beyond the role.
 *
 * The cache is the caller's memory, described by moe_paged_kv.  The row of
 * page p, key/value head c and slot s starts at element
 *   p * page_stride + c * head_stride + s * slot_stride
 * of k and of v (head_dim elements, contiguous), its scale at element
 *   p * scale_page_stride + c * scale_head_stride + s * scale_slot_stride
 * of k_scale and of v_scale.  Any order of the three is allowed, and a slice
 * of a larger allocation too.
 *   MOE_KV_BF16 : rows of bf16; the scales are not used (may be NULL).
 *   MOE_KV_E4M3 : rows of e4m3 codes, value = code * the row's f32 scale
 *                 (scales are >= 0).
 * Alignment: k and v 16 bytes, and the three row strides multiples of 16
 * bytes; scales 4 bytes.  A stride is at most 2^40 elements, and the last row
 * and scale lie within 2^62 bytes of the first (MOE_ERR_SHAPE).
 */
#define MOE_KV_BF16 0
#define MOE_KV_E4M3 1
typedef struct moe_paged_kv {
  void *k, *v;                 /* device */
  float *k_scale, *v_scale;    /* device; MOE_KV_E4M3 only */
  int64_t n_pages;             /* >= 1 */
  int64_t page_stride, head_stride, slot_stride;                   /* elements */
  int64_t scale_page_stride, scale_head_stride, scale_slot_stride; /* elements */
  int32_t page_size;           /* tokens per page, any number >= 1 */
  int32_t format;              /* MOE_KV_* */
} moe_paged_kv;

typedef struct moe_attn moe_attn; /* opaque; owned by the library */

typedef struct moe_attn_config {
  int32_t n_heads;     /* query heads, a multiple of n_kv_heads, <= 1024     */
  int32_t n_kv_heads;  /* key/value heads, >= 1; query head h reads key/value */
                       /* head h / (n_heads / n_kv_heads)                    */
  int32_t head_dim;    /* d: 64, 128 or 256                                  */
  int32_t rope_dim;    /* R: leading elements of a head that are rotated;    */
                       /* 0 for none, else a multiple of 16, <= head_dim     */
  int32_t interleaved; /* rotated pairs: 0 (i, i + R/2), 1 (2i, 2i + 1)      */
  int32_t max_sms;     /* SMs moe_attn_decode and _prefill may fill; 0: all  */
  int32_t device;      /* CUDA device ordinal the context lives on           */
  const double *rope_freqs; /* host, f64 [R/2]: radians per position, finite; */
                            /* read during moe_attn_init only; NULL if R = 0  */
} moe_attn_config;

/*
 * moe_attn_init - validate `cfg` and allocate a context: the frequencies as
 * 64-bit fractions of a turn and moe_attn_decode's workspace, whose size does
 * not depend on the batch or the lengths.
 * Errors: MOE_ERR_ARG (NULL, a frequency that is not finite), MOE_ERR_SHAPE
 * (both before any CUDA call), MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA,
 * MOE_ERR_NOMEM.  On error *out is set to NULL and nothing is leaked.
 */
int moe_attn_init(moe_attn **out, const moe_attn_config *cfg);

/* moe_attn_free - release the context; NULL is a no-op. */
void moe_attn_free(moe_attn *a);

/*
 * moe_attn_status - synchronise the context's last stream and return MOE_OK,
 * or MOE_ERR_DEVICE if a call since the previous moe_attn_status met a slot,
 * page or length outside the cache or the page table (the flag is cleared), or
 * MOE_ERR_DEVICE_TIMEOUT if a wait of moe_attn_prefill gave up.
 * Such a slot is neither written nor read, rows of such a page count as
 * zeros, and such a length is cut to the page table.
 */
int moe_attn_status(moe_attn *a);

/*
 * moe_attn_norm_rope - norm and rotate the query and key heads of T tokens.
 * Per head row x of d elements, in f32:
 *   y = x / sqrt(mean(x^2) + eps) * weight        (skipped if weight is NULL;
 *       right where x^2 is beyond f32 too, for a root of 2^-126 and more)
 *   rotate pair i < R/2 of y by the angle position * rope_freqs[i]
 * and one rounding to bf16.  Angles are taken modulo a turn to 2^-33 of one at
 * every int32 position, for frequencies of either sign up to 1 radian, and what is
 * left beside the nearest quarter turn is rounded to f32 (2^-28 of a turn at most).
 *   q, k       : device bf16; row h of token t at t * q_stride + h * d (elements),
 *                strides multiples of 8, pointers 16-byte aligned.  Slices of
 *                a fused projection's rows are fine.
 *   positions  : device int32 [T]; may be NULL if R = 0.
 *   q_weight, k_weight : device f32 [d], 16-byte aligned, or NULL.
 *   eps        : >= 0 and finite.
 *   q_out, k_out : like q and k; may be q and k themselves (same stride),
 *                must not overlap them otherwise.
 */
int moe_attn_norm_rope(moe_attn *a, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const int32_t *positions, int64_t T, const float *q_weight,
                       const float *k_weight, float eps, void *q_out, int64_t q_out_stride,
                       void *k_out, int64_t k_out_stride, void *stream);

/*
 * moe_attn_append - moe_attn_norm_rope whose key rows, and the value rows as
 * they are, go into the cache.
 *   v     : device bf16 [T, n_kv_heads, d] rows like k.
 *   slots : device int64 [T]: page * page_size + slot of each token's place,
 *           negative to store nothing for that token.  Two tokens of a call
 *           must not share a slot.
 * Storing a row as e4m3: e is the smallest integer >= -126 with max|v| <=
 * 448 * 2^e over the row's finite values (0 if they are all zero), scale =
 * 2^e, code = e4m3(v / 2^e) rounded to nearest even; a NaN or an infinity
 * becomes the NaN code.  The f32 value is rounded once, to the cache's type.
 */
int moe_attn_append(moe_attn *a, const moe_paged_kv *kv, const void *q, int64_t q_stride,
                    const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                    const int32_t *positions, const int64_t *slots, int64_t T,
                    const float *q_weight, const float *k_weight, float eps, void *q_out,
                    int64_t q_out_stride, void *stream);

/*
 * moe_attn_write - put key and value rows into the cache as they are
 * (arguments and storing as for moe_attn_append).
 */
int moe_attn_write(moe_attn *a, const moe_paged_kv *kv, const void *k, int64_t k_stride,
                   const void *v, int64_t v_stride, const int64_t *slots, int64_t T, void *stream);

/*
 * moe_attn_read - read key and value rows back from the cache as bf16 rows
 * [T, n_kv_heads, d] (strides as for k); a negative slot gives a row of zeros.
 */
int moe_attn_read(moe_attn *a, const moe_paged_kv *kv, const int64_t *slots, int64_t T, void *k_out,
                  int64_t k_out_stride, void *v_out, int64_t v_out_stride, void *stream);

/*
 * moe_attn_decode - attention of one new token per sequence over its pages.
 * With p = seq_lens[b] - 1 the new token's position and c = h / (n_heads /
 * n_kv_heads):
 *   s_j = scale * q[b, h] . K[b, j, c]
 *   s_j = softcap * tanh(s_j / softcap)              if softcap > 0
 *   s_j = s_j + slopes[h] * (j - p)                  if slopes is given
 * for the visible positions: j <= p, j >= starts[b] if given, and j > p -
 * window if window > 0;
 *   out[b, h] = softmax(s) V,  lse[b, h] = log(sum_j exp(s_j)).
 * Position j is slot j % page_size of page page_table[b, j / page_size].
 * A sequence with no visible position gives out = 0 and lse = -infinity.
 * Sums and softmax statistics are f32.  For their products with the values, weights
 * are rounded to 16 bits (bf16 cache), or weights times the value's scale to 22 bits
 * and to 2^-48 of the head's largest (e4m3 cache); out is rounded to bf16.  With an
 * e4m3 cache, elements of q below 2^-28 of their head's largest are rounded to 2^-39
 * of it.
 *   q          : device bf16 [B, n_heads, d], token stride q_stride (elements,
 *                a multiple of 8), 16-byte aligned.
 *   page_table : device int32 [B, max_pages], row stride table_stride.
 *   seq_lens   : device int32 [B], at most max_pages * page_size (which is at
 *                most 2^31 - 64) tokens each, counting the new token.
 *   starts     : device int32 [B] or NULL.
 *   slopes     : device f32 [n_heads] or NULL.
 *   out        : device bf16 [B, n_heads, d] contiguous, 16-byte aligned.
 *   lse        : device f32 [B, n_heads] or NULL.
 * B <= 2^20; B * n_kv_heads * g * ceil(max_pages * page_size / 16) up to 2^29 is
 * taken (what is more may be refused with MOE_ERR_SHAPE), g = ceil(n_heads /
 * n_kv_heads / 16), or / 8 with d = 256.  B = 0 is a no-op.
 * How the work is split, and with it the order of the sums, follows from B, the
 * heads, the format, max_pages * page_size, the lengths and max_sms: the same call
 * gives the same bits.  The calls on one context share its workspace: they must
 * not overlap on the GPU.
 */
int moe_attn_decode(moe_attn *a, const moe_paged_kv *kv, const void *q, int64_t q_stride,
                    const int32_t *page_table, int64_t table_stride, int64_t max_pages,
                    const int32_t *seq_lens, const int32_t *starts, int64_t B, float scale,
                    float softcap, const float *slopes, int32_t window, void *out, float *lse,
                    void *stream);

/*
 * moe_attn_decode_clusters - how moe_attn_decode splits a call of B sequences with
 * page tables of max_pages columns: the clusters of CTAs that share each sequence
 * and group of heads (few sequences whose tables are not long), or 0 where the
 * tiles of all sequences are cut evenly over the device.  Negative: MOE_ERR_*, as
 * for the call.
 */
int moe_attn_decode_clusters(const moe_attn *a, const moe_paged_kv *kv, int64_t B, int64_t max_pages);

/*
 * moe_attn_prefill - attention of whole prompts, or of chunks of them whose
 * earlier keys are given too, packed one after another.  Sequence b has the query
 * rows [q_starts[b], q_starts[b + 1]) and the key and value rows [k_starts[b],
 * k_starts[b + 1]); its last query is its last key's token.  With Lq and Lk rows,
 * query i of the sequence at position p = i + Lk - Lq, and c = h / (n_heads /
 * n_kv_heads):
 *   s_j = scale * q[i, h] . K[j, c]
 *   s_j = softcap * tanh(s_j / softcap)              if softcap > 0
 *   s_j = s_j + slopes[h] * (j - p)                  if slopes is given
 * for the visible keys j of the sequence: j <= p if causal, and j > p - window if
 * window > 0;
 *   out[i, h] = softmax(s) V,  lse[i, h] = log(sum_j exp(s_j)).
 * A query with no visible key gives out = 0 and lse = -infinity.  Rows outside the
 * sequences are not read as keys or values of any, and out and lse are left as they
 * are there.  What hidden keys and values hold does not matter, NaN included; but a row
 * that meets infinities or NaN, hidden ones in blocks that it reads or visible ones, and
 * one whose scores rise by more than 88 within a block, is computed a second time, a
 * hundred times as slowly.
 * Sums and softmax statistics are f32; for their product with the values, weights
 * are rounded to bf16 (2^-8 of each at most, as the output is), or keep 16 bits if
 * the caller chooses (moe_attn_prefill_bits); out is rounded to bf16.
 * A cap of at most 128 makes a score off by 2^-19 of the cap at most, one above by 2^-20
 * of the score.
 *   q       : device bf16 [Tq, n_heads, d] rows as for moe_attn_norm_rope (a slice of
 *             a fused projection's rows is fine), Tq <= 2^31 - 1.
 *   k, v    : device bf16 [Tk, n_kv_heads, d] rows like q, Tk <= 2^31 - 1.
 *   q_starts, k_starts : device int32 [B + 1], non-decreasing, within [0, Tq] and
 *             [0, Tk].  Others are cut to these ranges, never followed, and
 *             moe_attn_status reports them (the outputs mean nothing then).
 *   causal  : 0 or 1.
 *   slopes  : device f32 [n_heads] or NULL.
 *   out     : device bf16 rows like q; must not overlap q, k or v.
 *   lse     : device f32 [Tq, n_heads] contiguous, or NULL.
 * B <= 2^20.  Where few tiles of queries would leave SMs idle, clusters of up to 16
 * CTAs share a tile's keys.  The order of the sums follows from the sizes, the
 * lengths, the options and max_sms alone: the same call gives the same bits.  No
 * workspace is used but the context's error flag.
 */
int moe_attn_prefill(moe_attn *a, const void *q, int64_t q_stride, int64_t Tq, const void *k, int64_t k_stride,
                     const void *v, int64_t v_stride, int64_t Tk, const int32_t *q_starts,
                     const int32_t *k_starts, int64_t B, int32_t causal, float scale, float softcap,
                     const float *slopes, int32_t window, void *out, int64_t out_stride, float *lse,
                     void *stream);

/*
 * moe_attn_prefill_bits - the bits that the weights of later moe_attn_prefill calls
 * keep for their product with the values: 8 (the default: 2^-8 of each weight is lost
 * at most) or 16 (2^-15), which takes 1.1 to 1.5 times as long.  Others: MOE_ERR_SHAPE.
 */
int moe_attn_prefill_bits(moe_attn *a, int32_t bits);

/*
 * Projections around the attention and the MoE, in the experts' weight format
 * (dragon.c, "Precision": e4m3 codes with one f32 scale per 128x128 block, the
 * dense branches too): the hidden states' norm with the residual's addition and an
 * e4m3 output, and the product of such rows with such weights.  Unlike the routed
 * experts, whose activations are exact, a projection's activations are one e4m3
 * term with a f32 scale per row and 128 columns.
 */
typedef struct moe_proj moe_proj; /* opaque; owned by the library */

/*
 * moe_proj_init - a context of `device` (its error flag is all it owns); max_sms:
 * the SMs a call may fill, 0 for all (a limit is one of CTAs too: each of the call's may
 * be on an SM of its own).  Errors: MOE_ERR_ARG (out NULL),
 * MOE_ERR_SHAPE (negative; both before any CUDA call), MOE_ERR_UNSUPPORTED,
 * MOE_ERR_CUDA, MOE_ERR_NOMEM.  On error *out is set to NULL and nothing is leaked.
 * Calls on one context may overlap on the GPU.
 */
int moe_proj_init(moe_proj **out, int32_t device, int32_t max_sms);

/* moe_proj_free - release the context; NULL is a no-op. */
void moe_proj_free(moe_proj *p);

/*
 * moe_proj_status - synchronise the context's last stream and return MOE_OK, or
 * MOE_ERR_DEVICE_TIMEOUT if a wait of a call since the previous moe_proj_status
 * gave up (the flag is cleared).
 */
int moe_proj_status(moe_proj *p);

/*
 * moe_proj_norm - residual addition, RMS norm and quantisation of T rows of H
 * columns.  Per row, in f32:
 *   r' = bf16(x + residual)                     (x itself if residual is NULL)
 *   y  = r' / sqrt(mean(r'^2) + eps) * weight   (r' itself if weight is NULL; right
 *        where r'^2 is beyond f32 too)
 *   residual_out = r'; out = bf16(y); and per block of 128 columns (the last one may
 *   be shorter) scale = max(max|y| / 448, 2^-126) over its finite values (1 if they
 *   are all zero), code = e4m3(y / scale) rounded to nearest even (the quotient to
 *   f32); a NaN or an infinity becomes the NaN code.
 *   x, residual   : device bf16; row t at t * stride (elements, a multiple of 8, at
 *                   least H), 16-byte aligned.  residual may be NULL.
 *   T, H          : T >= 0; H a multiple of 8, 8..16384.
 *   weight        : device f32 [H], 16-byte aligned, or NULL.
 *   eps           : >= 0 and finite.
 *   residual_out  : like x; NULL if and only if residual is.  May be residual or x
 *                   (same stride).
 *   out           : like x, or NULL.  May be x (same stride).
 *   codes         : device u8, row t at t * codes_stride (a multiple of 8, at least
 *                   H), 8-byte aligned, or NULL.
 *   scales        : device f32; that of row t and block b at t * scale_row_stride +
 *                   b * scale_block_stride (elements, positive).  NULL if and only
 *                   if codes is.
 * One of out, codes and residual_out at least is given; outputs must not overlap
 * each other or the inputs otherwise.
 */
int moe_proj_norm(moe_proj *p, const void *x, int64_t x_stride, const void *residual,
                  int64_t residual_stride, int64_t T, int64_t H, const float *weight, float eps,
                  void *residual_out, int64_t residual_out_stride, void *out, int64_t out_stride,
                  uint8_t *codes, int64_t codes_stride, float *scales, int64_t scale_row_stride,
                  int64_t scale_block_stride, void *stream);

/*
 * moe_proj_matmul - product of e4m3 rows with e4m3 weights:
 *   out[m, n] = bf16( sum over blocks b of 128 of K of
 *       a_scale[m, b] * w_scale[n / 128, b] * sum over k in b of a[m, k] * w[n, k] )
 * Sums are f32, rounded once at the end.  The product of a block's two scales is
 * formed first, in f32: scales as moe_proj_norm and the experts' format have them
 * stay well within, but one below 2^-126 keeps fewer bits, and one beyond f32 gives
 * infinities or NaN, whatever the result would be.
 *   a       : device u8 e4m3 codes, row m at m * a_stride, 16-byte aligned, a_stride
 *             a multiple of 16 and at least K.
 *   a_scale : device f32, as moe_proj_norm writes them.
 *   w       : device u8 e4m3 codes, row n at n * w_stride; alignment as for a.
 *   w_scale : device f32 [ceil(N / 128), ceil(K / 128)] contiguous, 4-byte aligned.
 *   out     : device bf16, row m at m * out_stride (a multiple of 8, at least N),
 *             16-byte aligned; must not overlap the inputs.
 * M, N, K: any from 0 up to 2^31 - 256 (K = 0 gives zeros); M or N = 0 is a no-op.
 * The order of the sums follows from the sizes and max_sms alone.
 */
int moe_proj_matmul(moe_proj *p, const uint8_t *a, int64_t a_stride, const float *a_scale,
                    int64_t scale_row_stride, int64_t scale_block_stride, int64_t M, const uint8_t *w,
                    int64_t w_stride, const float *w_scale, int64_t N, int64_t K, void *out,
                    int64_t out_stride, void *stream);

/*
 * moe_selftest_wait_timeout - exercise the bounded device-side waits.  Every
 * wait inside the layer's kernels (mbarriers of TMA copies and tensor-core
 * work, cross-CTA counters) gives up after a time limit and records
 * MOE_ERR_DEVICE_TIMEOUT instead of hanging the GPU.  This call enqueues one
 * CTA that holds tensor memory as those kernels do and waits, with the same
 * helpers, on an mbarrier that nothing arrives on and on a counter in the
 * context's workspace that nothing increments, `limit_ns` each; both waits
 * give up, the CTA frees its tensor memory and returns.
 *   limit_ns : 1 .. 1e9 nanoseconds per wait.
 *   which    : device int32 or NULL; receives the waits that gave up (bit 0
 *              the mbarrier, bit 1 the counter: 3 when both did).
 *   stream   : cudaStream_t or NULL.
 * Afterwards moe_status reports MOE_ERR_DEVICE_TIMEOUT once (and clears it);
 * the context stays usable.  No counterpart in the pages: it tests the
 * failure handling of this library.
 */
int moe_selftest_wait_timeout(moe_ctx *ctx, int64_t limit_ns, int32_t *which, void *stream);

/*
 * moe_route_noalloc - the routing step alone (steps 1 and 2 above) for callers
 * that may not allocate device memory once running: applications that hand
 * all device memory to their own allocator at start-up, or inference loops
 * with a fixed memory budget, where a cudaMalloc could fail or stall the
 * device.  It allocates nothing and needs no context: its temporary buffers
 * live in one statically sized device array of this library (about 269 KB,
 * held on every GPU that loads the library until the process exits).
 * There is no counterpart in the pages; it computes the same routing as
 * moe_layer_forward followed by moe_get_routing.
 *   hidden      : device, bf16 [T, H], 16-byte aligned; T <= 64.
 *   H           : multiple of 128, <= 65536.
 *   router_w    : device, f32 [E, H], 16-byte aligned; 1 <= E <= 1024.
 *   router_bias : device, f32 [E], or NULL.
 *   top_k       : 1..min(E, 32).
 *   idx, wts    : device outputs, int32 / f32 [T, k], rank order.
 *   counts      : device output, int32 [E].
 *   offsets     : device output, int32 [E+1].
 *   perm, inv   : device outputs, int32 [T*k].
 *   stream      : cudaStream_t or NULL.
 * Sizes beyond these limits return MOE_ERR_SHAPE; T = 0 is a no-op.  The
 * first call on a device looks up the array's device address (a host-side
 * query, done once per device, with that device current): make that first
 * call outside any stream capture.  Every call shares the one array and
 * clears the part that must start at zero; calls whose work overlaps on the
 * GPU (other streams, other host threads) race on it and must be serialised
 * by the caller.  Device-side errors (non-finite logits) are not reported.
 */
int moe_route_noalloc(const void *hidden, int64_t T, int64_t H, const float *router_w,
                      const float *router_bias, int64_t E, int32_t top_k, int32_t *idx, float *wts,
                      int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *inv, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOE_H */

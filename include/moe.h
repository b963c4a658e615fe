/*
 * moe.h — C ABI of a dropless mixture-of-experts layer (forward and backward) for AMD
 * Instinct MI355X (gfx950).  Library: libmoe.so.
 *
 * Pages the operations are defined on (titles as published; headings translated in []):
 *   [Prime] "Prime Mega MoE: tanításra is jó a DeepSeek MoE kernele" (neuraldaily.news)
 *   [JAX]   "Az NVIDIA szerint tízszer gyorsabb lett a dropless MoE tanítása JAX-ban" (aihirek.info)
 *   [TE]    "NVIDIA מציגה דרך יעילה לאמן מודלי MoE בביולוגיה" (sitech.ge)
 *   [Mega]  the DeepGEMM "Mega MoE" announcement on itsolotime.com
 *
 * Notation: T tokens, d model dim, f expert FFN dim, E experts, k slots per token.  A pair
 * p = t*k + j is slot j of token t.  A = T*k is the maximum number of routed pairs; buffers are
 * sized by it, never by E x capacity (dropless: [JAX] "A dropless MoE minden tokent
 * feldolgoz" [dropless MoE processes every token]).
 *
 * Layouts (all row-major, contiguous, device memory unless stated):
 *   x, dx, y, dy   bf16 [T, d]              (fp8: x is e4m3 [T, d] with x_scale fp32 [T, d/128])
 *   W1, dW1        bf16 [E, d, 2f]          columns [0,f) are the gate, [f,2f) the up projection
 *                                           (fp8: e4m3 with W1_scale fp32 [E, d/128, 2f/128])
 *   W2, dW2        bf16 [E, f, d]           (fp8: e4m3 with W2_scale fp32 [E, f/128, d/128])
 *   logits, d_logits  fp32 [T, E]
 *   topk_ids       int32 [T, k]  slot j = j-th largest logit, ties to the lower id; -1 = the
 *                                slot is not routed here (pre-routed input only)
 *   topk_w, d_topk_w  fp32 [T, k]
 *   counts         int32 [E]     routed pairs per expert
 *   offsets        int32 [E+1]   exclusive prefix sum of counts; offsets[E] = routed pairs
 *   perm           int32 [T*k]   sorted position -> pair p (entries >= offsets[E] unused)
 *   inv_perm       int32 [T*k]   pair p -> sorted position, -1 for a slot that is not routed
 * The sorted order is expert-major, then ascending pair index within an expert (a stable
 * counting sort), which makes it unique and bit-reproducible.
 *
 * Conventions for every call:
 *   - Ownership: the caller allocates every buffer (including `ws` workspace and the `saved`
 *     forward->backward context).  The library allocates nothing and keeps no state between
 *     calls; calls are re-entrant.  The one exception is moe_route_noalloc, which takes no
 *     workspace and uses a fixed device array of the library instead (see there).
 *   - Streams: `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue work
 *     on it and return; nothing synchronises the host and no count leaves the device.
 *   - Validation: arguments are checked on the host only.  Device contents are preconditions:
 *     inputs finite, expert ids in [-1, E), a token's valid ids distinct.  Ids outside
 *     [0, E) are treated as "not routed here".
 *   - Errors: a negative MOE_ERR_* code is returned and nothing is enqueued; MOE_ERR_HIP means
 *     a launch failed (moe_status_string() then names the HIP error).
 *   - Shapes (MOE_ERR_SHAPE otherwise): T >= 0, 1 <= E <= 1024, 1 <= k <= min(E, 64),
 *     d and f positive multiples of 128 (MOE_FP8_E4M3, MOE_MXFP8: of 256) and at most 65536,
 *     T*k < 2^31 (MOE_MXFP8: T*k + 127*E rounded up to 128 < 2^31).
 *     moe_norm_*, moe_grad_norm, moe_adamw_step, moe_score_*, moe_bias_update and moe_fp8_* take sizes of
 *     their own (see there); MOE_F32 is an element type of theirs and no dtype of the layer.
 *   - fp8 (MOE_FP8_E4M3): codes are OCP e4m3 (bias 7, max 448, no infinities); a block's value
 *     is code * scale with its fp32 scale ([Prime] "Mit csinált a Prime Intellect?": blockwise
 *     FP8 is one of the kernel's data types).  Outputs and gradients stay bf16/fp32.
 *   - MXFP8 (MOE_MXFP8): x, W1, W2 are passed in bf16 (the 16-bit master copies) and the
 *     library quantises them on every call to OCP MXFP8 (e4m3 codes, one E8M0 exponent per 32
 *     values along each GEMM's K; [JAX] "Csoportosított mátrixszorzás és összevont
 *     adatmozgatás": group-aware MXFP8 quantisation feeding an MXFP8 grouped GEMM; [TE]
 *     "צמצום הזיכרון ותקורות הכימות": one scale per 32 values).  The exponent of a block is the
 *     smallest power of two that brings its maximum magnitude within 448 (no clipping); elements
 *     round to nearest even.  The data-gradient GEMMs use weights quantised along their own K;
 *     moe_forward produces both quantisations in one pass over each weight matrix and keeps
 *     the backward's in `saved`.  Weight gradients run in MXFP8 too, quantised along their K,
 *     the token axis (see moe_backward).  d and f must be multiples of 256.
 *   - Alignment (MOE_ERR_ALIGN otherwise): tensors 16-byte aligned, ws and saved 256-byte
 *     aligned (every torch/hipMalloc allocation is).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_BF16 = 0, MOE_FP8_E4M3 = 1, MOE_MXFP8 = 2, MOE_F32 = 3 } moe_dtype;

typedef struct {
  int64_t T, d, f, E, k;
  int32_t dtype; /* moe_dtype */
  int32_t reserved; /* must be 0 */
} moe_dims;

enum {
  MOE_OK = 0,
  MOE_ERR_NULL = -1,      /* a required pointer is NULL */
  MOE_ERR_SHAPE = -2,     /* dims outside the supported range */
  MOE_ERR_DTYPE = -3,     /* dtype not supported by this call */
  MOE_ERR_WORKSPACE = -4, /* ws_bytes smaller than moe_workspace_bytes() */
  MOE_ERR_HIP = -5,       /* a HIP launch failed */
  MOE_ERR_ALIGN = -6      /* a device buffer is not 16-byte aligned (ws and saved: 256) */
};

enum { MOE_WS_ROUTE = 0, MOE_WS_FORWARD = 1, MOE_WS_BACKWARD = 2, MOE_WS_ROUTER = 3 };

/* Workspace bytes needed by moe_route/moe_plan (which = MOE_WS_ROUTE), moe_forward
 * (MOE_WS_FORWARD), moe_backward (MOE_WS_BACKWARD) or moe_router_backward (MOE_WS_ROUTER).
 * Host only. */
int moe_workspace_bytes(const moe_dims* dims, int which, size_t* out);

/* Bytes of the `saved` context moe_forward writes and moe_backward reads (the GEMM1 output
 * H = [gate | up] and the scaled SwiGLU activations).  Host only. */
int moe_saved_bytes(const moe_dims* dims, size_t* out);

/* Top-k routing plus the expert plan.  Per token: the k largest logits (descending, ties to
 * the lower expert id) and topk_w = softmax over those k logits in fp32 ([JAX] "A dropless MoE
 * minden tokent feldolgoz": a learned router activates only the top-K experts per token).
 * Then counts, offsets, perm and inv_perm as for moe_plan. */
int moe_route(const moe_dims* dims, const float* logits, int32_t* topk_ids, float* topk_w,
              int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm,
              void* ws, size_t ws_bytes, void* stream);

/* moe_route without a workspace argument, for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).  Same outputs,
 * bit for bit.  The plan's tables live in a fixed 4 MiB device array inside the library, one per
 * GPU, held until the process ends; every shape this header accepts fits it (MOE_ERR_WORKSPACE
 * otherwise).  The call allocates nothing.  All calls on one GPU share that array, so calls that
 * overlap in time on one GPU (different streams, or different host threads) race and must be
 * serialised by the caller; calls on one stream are ordered and safe.  The first call on a GPU
 * looks up the array's device address (MOE_ERR_HIP if that fails). */
int moe_route_noalloc(const moe_dims* dims, const float* logits, int32_t* topk_ids, float* topk_w,
                      int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm, void* stream);

/* Expert plan for already-routed pairs: per-expert counts, their exclusive prefix sum and the
 * stable counting sort of pairs by expert (ragged per-expert groups: [JAX] "Az egyenetlen
 * terhelés lassítja a tanítást" [uneven load slows training]; per-expert counts as split
 * sizes: [TE] "מומחים מקובצים במקום לולאת Python" [grouped experts instead of a Python loop]).
 * Integer only, bit-exact and deterministic.  Ids -1 are skipped (inv_perm = -1). */
int moe_plan(const moe_dims* dims, const int32_t* topk_ids, int32_t* counts, int32_t* offsets,
             int32_t* perm, int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);

/* Forward: y[t] = sum_j w[t,j] * (silu(x_t W1[e] gate) * (x_t W1[e] up)) W2[e], e = ids[t,j],
 * over routed slots ([Mega] "Mega MoE คืออะไร?" [what is Mega MoE?]: dispatch, two linear layers,
 * SwiGLU, combine; [TE] "צמצום הזיכרון ותקורות הכימות": GroupedLinear -> ScaledSwiGLU ->
 * GroupedLinear).  The token gather is fused into the first grouped GEMM's operand loads, the
 * routing weight into its SwiGLU epilogue, and the combine sums a token's k per-pair outputs in
 * fp32 in slot order with one bf16 rounding.  Each expert is computed at its real row count
 * ([JAX] "Csoportosított mátrixszorzás és összevont adatmozgatás" [grouped GEMM and fused data
 * movement]).  `saved` (moe_saved_bytes) receives what moe_backward needs.  For
 * dtype = MOE_FP8_E4M3 the *_scale arguments are required when T > 0 (MOE_ERR_NULL); for bf16
 * they must be NULL (MOE_ERR_DTYPE).  fp8: both grouped GEMMs run on e4m3 operands with fp32
 * accumulation and per-128-K scale promotion; the scaled SwiGLU output feeding the second one
 * is requantised to e4m3 with one scale (its absolute maximum / 448) per row per 128 columns
 * ([TE] "צמצום הזיכרון ותקורות הכימות" [reducing memory and quantisation overheads]). */
int moe_forward(const moe_dims* dims, const void* x, const float* x_scale,
                const void* W1, const float* W1_scale, const void* W2, const float* W2_scale,
                const float* topk_w, const int32_t* offsets, const int32_t* perm,
                const int32_t* inv_perm, void* y, void* saved, void* ws, size_t ws_bytes,
                void* stream);

/* The bf16 moe_forward with the dispatch gather, both grouped GEMMs and the scaled SwiGLU in one
 * persistent launch fed by a device work queue, followed by the combine ([Mega] "Mega MoE
 * คืออะไร?" [what is Mega MoE?]: dispatch, the two linear layers and SwiGLU fused into one
 * kernel).  Same arguments, results and `saved` contents as moe_forward with dtype MOE_BF16 and
 * NULL scales, so moe_backward accepts its `saved`; y, H and As are bitwise equal to
 * moe_forward's.  A work item is a row tile (256 sorted rows of one expert): its block runs the
 * up product over all of f, then the down product over all of d for the same rows, so the work
 * is coarser than moe_forward's per-tile launches (slower when the row tiles are few against the
 * compute units).  Blocks take items with atomic adds on counters in `ws` and never wait for
 * one another; `ws` needs moe_workspace_bytes(MOE_WS_FORWARD).  dtype other than MOE_BF16:
 * MOE_ERR_DTYPE.  Other errors as moe_forward. */
int moe_forward_fused(const moe_dims* dims, const void* x, const void* W1, const void* W2,
                      const float* topk_w, const int32_t* offsets, const int32_t* perm,
                      const int32_t* inv_perm, void* y, void* saved, void* ws, size_t ws_bytes,
                      void* stream);

/* Backward of moe_forward for L = sum(dy * y) ([Prime] "Mit csinált a Prime Intellect?" [what
 * did Prime Intellect do?]: a backward pass for the fused MoE kernel).  Writes dx (bf16),
 * dW1 and dW2 (bf16; an expert with no routed pair gets exactly zero), d_topk_w (fp32, 0 on
 * unrouted slots) and, if d_logits is not NULL, d_logits[t, ids[t,j]] =
 * w[t,j] * (d_topk_w[t,j] - sum_i w[t,i] d_topk_w[t,i]) and 0 elsewhere (the softmax over the
 * kept logits; topk_ids is then required).  `saved` must come from moe_forward on the same
 * inputs.  Every reduction has a fixed order, so results are bitwise reproducible.
 * fp8 (MOE_FP8_E4M3): dy is quantised like the forward activations (1x128 blocks) for the two
 * data-gradient GEMMs and dH is requantised the same way between them.  The weight gradients
 * dW2 = As^T dy and dW1 = x^T dH run as bf16 GEMMs with fp32 accumulation on the bf16 dy, the
 * layer's own bf16 As and dH, and x dequantised once to bf16 (code * scale in fp32, one
 * rounding): their K is the token axis, which the 1x128 blocks of the inputs do not follow.
 * MXFP8 (MOE_MXFP8): the weight gradients run as MXFP8 GEMMs whose K is the expert's rows; both
 * operands are quantised in blocks of 32 consecutive sorted rows that never straddle two experts
 * ([JAX] "Csoportosított mátrixszorzás és összevont adatmozgatás": group-aware quantisation). */
int moe_backward(const moe_dims* dims, const void* dy, const void* x, const float* x_scale,
                 const void* W1, const float* W1_scale, const void* W2, const float* W2_scale,
                 const int32_t* topk_ids, const float* topk_w, const int32_t* offsets,
                 const int32_t* perm, const int32_t* inv_perm, const void* saved, void* dx,
                 void* dW1, void* dW2, float* d_topk_w, float* d_logits, void* ws,
                 size_t ws_bytes, void* stream);

/* Router scores (the gate in front of moe_route): logits[T, E] = x[T, d] . Wg[d, E] with bf16 x and
 * gate weight Wg (row-major [d, E]), fp32 accumulation and fp32 output ([JAX] "A dropless MoE
 * minden tokent feldolgoz": a learned router scores the experts and keeps the top K).  Feeding
 * these logits to moe_route gives the layer's routing.  dtype MOE_BF16 or MOE_MXFP8 (x is bf16 in
 * both; MOE_FP8_E4M3: MOE_ERR_DTYPE).  x, Wg and logits 16-byte aligned; T = 0 does nothing. */
int moe_router_logits(const moe_dims* dims, const void* x, const void* Wg, float* logits, void* stream);

/* Backward through moe_router_logits for the layer's d_logits [T, E] (fp32, as moe_backward writes
 * it).  dWg = x^T . d_logits (bf16 [d, E], fp32 accumulation) when dWg is not NULL: the token axis
 * is cut into slices whose fp32 partial sums live in `ws` (moe_workspace_bytes(MOE_WS_ROUTER)) and
 * are added in slice order, so the result is bitwise reproducible; an empty layer (T = 0) writes
 * zeros.  When dx is not NULL, the part of the input gradient that flows through the logits is
 * added to it in place: dx[t] = bf16(dx[t] + sum_e d_logits[t, e] Wg[:, e]), the sum in fp32 and
 * one rounding (pass moe_backward's dx to get the whole input gradient of the routed layer).
 * d_logits enters the MFMA rounded to bf16.  Same dtype, alignment and workspace rules as the
 * other calls (ws 256-byte aligned). */
int moe_router_backward(const moe_dims* dims, const void* x, const void* Wg, const float* d_logits,
                        void* dx, void* dWg, void* ws, size_t ws_bytes, void* stream);

/* Dispatch on its own (bf16): for every slot with pos = inv_perm[t*k+j] >= 0, xp[pos] = x[t]
 * (so xp[pos] = x[perm[pos] / k] for pos < offsets[E]); rows of xp at or past offsets[E] are left
 * untouched.  Token-major: each row of x is read once and written to its k positions.  xp is
 * bf16 [T*k, d].  ([JAX] "Csoportosított mátrixszorzás és összevont adatmozgatás": dispatch
 * sends tokens to their experts.)  The forward pass does not call it (its GEMM gathers rows
 * directly); it exists for callers that want expert-sorted activations. */
int moe_permute(const moe_dims* dims, const void* x, const int32_t* inv_perm, void* xp, void* stream);

/* Combine on its own (bf16): y[t] = sum over j = 0..k-1 with inv_perm[t*k+j] >= 0 of
 * op[t*k+j], summed in fp32 in ascending j and rounded once to bf16 (combine gathers the
 * results back and restores token order: [JAX] "Az egyenetlen terhelés lassítja a
 * tanítást").  op is bf16 [T*k, d] in pair (slot) order. */
int moe_combine(const moe_dims* dims, const void* op, const int32_t* inv_perm, void* y,
                void* stream);

/* Load-balancing loss of the gate, with per-expert counts ([JAX] "Az egyenetlen terhelés lassítja a
 * tanítást" [uneven load slows training]).  The tokens come in S groups (sequences, or one group
 * for the whole batch): group g holds tokens group_offsets[g] .. group_offsets[g+1]-1 (int32
 * [S+1], never decreasing, within [0, T]; NULL with S = 1: all T tokens); tokens before the first
 * or behind the last group belong to none.  A token counts if it lies in a group, its token_mask
 * byte is not 0 (uint8 [T]; NULL: every token) and it has a logit that is not -inf.  With
 * p = softmax(logits) over all E, over the counted tokens:
 *   counts[g, e] = slots of g's tokens with topk_ids = e,  P[g, e] = sum of p[t, e],  N_g = tokens
 *   losses[0] = 1/G sum_{g: N_g > 0} E / (k N_g^2) sum_e counts[g, e] P[g, e],  G = such groups
 *   losses[1] = 1/N sum_t lse_t^2,  lse_t = log sum_e exp(logits[t, e]),  N = sum_g N_g
 * (both 0 when nothing counts).  losses[0] is 1 for an even load, losses[1] the router's z-loss.
 * Outputs: counts int32 [S, E]; group_tokens int32 [S+2]: N_g, then N, then G; losses fp32 [2];
 * lse fp32 [T], -inf for a token that does not count.  Nothing is read of the logits and ids of a
 * token that is masked or lies in no group.  A logit of -inf is an expert that cannot be chosen (p = 0);
 * a token with a NaN or +inf counts, whatever its other logits are, and makes its lse and the losses
 * NaN.  Sums run in a fixed order (bitwise reproducible): in fp32 over up to 512 tokens of a group that
 * follow each other (T / 65536 where T is above 2^25), in 64 bits over those sums.  dims: T, E
 * and k are used.  S: 1 .. 65535 (MOE_ERR_SHAPE).  ws: moe_balance_workspace_bytes.  logits, topk_ids,
 * counts and lse 16-byte aligned, the other arrays to their type. */
int moe_balance_workspace_bytes(const moe_dims* dims, int64_t S, size_t* out);
int moe_balance_forward(const moe_dims* dims, const float* logits, const int32_t* topk_ids,
                        const uint8_t* token_mask, const int32_t* group_offsets, int64_t S, int32_t* counts,
                        int32_t* group_tokens, float* losses, float* lse, void* ws, size_t ws_bytes,
                        void* stream);

/* Gradient of d_losses[0] * losses[0] + d_losses[1] * losses[1] (d_losses: fp32 [2] on the device)
 * with respect to the logits, added to d_logits_in (fp32 [T, E]; NULL: zeros) and written to
 * d_logits, which may be d_logits_in itself (pass moe_backward's d_logits as both):
 *   d_logits = d_logits_in + p (d_losses[0] E / (k N_g^2 G) (counts[g, e] - sum_i counts[g, i] p_i)
 *                               + 2 d_losses[1] lse / N)
 * The counts carry no gradient.  Rows of tokens that do not count are those of d_logits_in (their logits are
 * read and not used).  p is a row's exponentials over their sum, so it keeps its bits at any size of lse.
 * logits, topk routing and groups as in the forward call, with its lse, counts and group_tokens
 * (counts and group_tokens may have been summed over other GPUs' tokens in between, for the loss of
 * the joint batch: N_g, N and the counts summed, G the number of joint groups). */
int moe_balance_backward(const moe_dims* dims, const float* logits, const float* lse,
                         const int32_t* group_offsets, int64_t S, const int32_t* counts,
                         const int32_t* group_tokens, const float* d_losses, const float* d_logits_in,
                         float* d_logits, void* stream);

/* RMS norms before and after a block, fused with the block's gate and the scaled residual ([TE]: the
 * expert layer is the feed-forward part of a transformer block).  For each of T rows of d values,
 * with rms(v) = sqrt(mean(v^2) + eps):
 *   n     = w_post * y / rms(y)                     (n = y when w_post is NULL)
 *   h_out = res_scale * h + out_scale * gate * n    (gate 1 for MOE_GATE_NONE)
 *   x     = w_pre * h_out / rms(h_out)
 * h: the residual stream before the block, y: the block's output (bf16, moe_forward's y), h_out: the
 * stream behind it, x: the next block's input (bf16).  Without y (NULL, with h_out, w_post and gate
 * NULL too) only the norm before a block is taken: x = w_pre * h / rms(h).  Without w_pre and x
 * (both NULL) only the part behind the block.  x comes from h_out before its rounding.  h_out may be
 * h itself; otherwise outputs overlap no input.  Sums and statistics are fp32, each output is
 * rounded once. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2, MOE_GATE_FULL = 3 } moe_gate;

typedef struct {
  int64_t T, d;        /* rows, values in a row: a multiple of 8, 8 .. 16384; T*d < 2^40, T < 2^31 */
  int32_t h_dtype;     /* MOE_BF16 or MOE_F32: h, h_out, dh_out, dh */
  int32_t w_dtype;     /* MOE_BF16 or MOE_F32: w_post, w_pre, gate and their gradients */
  int32_t gate;        /* moe_gate: NONE, CHANNEL [d], TOKEN [T], FULL [T, d] */
  int32_t reserved;    /* must be 0 */
  float eps;           /* > 0 and finite */
  float res_scale, out_scale; /* finite; used when y is given */
} moe_norm_desc;

int moe_norm_workspace_bytes(const moe_norm_desc* desc, size_t* out);
int moe_norm_forward(const moe_norm_desc* desc, const void* y, const void* h, const void* w_post,
                     const void* gate, const void* w_pre, void* h_out, void* x, void* stream);

/* Backward of moe_norm_forward.  dh_out: gradient of h_out from its other uses (the residual stream
 * above; NULL: zeros), dx: gradient of x (bf16, moe_backward's dx), h_out as the forward wrote it
 * (h itself when there was no y).  With D the whole gradient of h_out:
 *   dh = res_scale * D (D when there is no y)    dy = out_scale * gate * D through the norm of y
 *   dw_pre, dw_post [d], dgate (the gate's shape): summed over what the weight or gate is shared by
 * Any output may be NULL (not wanted).  dh may be dh_out itself; otherwise outputs overlap no input.
 * The sums over tokens are fp32 in a fixed order (bitwise reproducible).  h_out and dx go with w_pre: all three or
 * none (MOE_ERR_NULL; MOE_ERR_SHAPE if dx or h_out come without w_pre), and one of y and w_pre is
 * needed (MOE_ERR_NULL).  T = 0 writes zeros to dw_pre, dw_post and a channel gate's dgate.
 * ws: moe_norm_workspace_bytes. */
int moe_norm_backward(const moe_norm_desc* desc, const void* y, const void* h_out, const void* w_post,
                      const void* gate, const void* w_pre, const void* dh_out, const void* dx, void* dh,
                      void* dy, void* dw_post, void* dgate, void* dw_pre, void* ws, size_t ws_bytes,
                      void* stream);

/* One tensor of the lists below: n values, contiguous.  p: the parameter (p_dtype), g its gradient
 * (g_dtype), each MOE_BF16 or MOE_F32.  master: an fp32 copy of a bf16 parameter that the update runs
 * on (p is then its rounding), or NULL.  state = MOE_STATE_F32: m and v fp32 [n], scales NULL.
 * state = MOE_STATE_8BIT: m and v hold e4m3 codes [n] of m and of sqrt(v) (never negative), with one fp32 scale for each
 * 256 values (m_scale, v_scale: [(n + 255) / 256]; value = code * scale, scale = the block's largest
 * magnitude / 448, or 1 for a block of zeros).  All bytes 0 is the state before the first step.
 * ([TE] "צמצום הזיכרון ותקורות הכימות" [reducing memory and quantisation overheads]) */
typedef enum { MOE_STATE_F32 = 0, MOE_STATE_8BIT = 1 } moe_state;

typedef struct {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t n;              /* 0 .. 2^40 */
  int32_t p_dtype, g_dtype, state;
  float weight_decay;     /* >= 0 and finite */
} moe_tensor;

/* L2 norm of the gradients of n_tensors tensors together (g, n and g_dtype are read; the other
 * members may be NULL), norm = sqrt(sum g^2) (fp32 [1] on the device, sums in 64 bits in a fixed
 * order), and the factor that clips it, scale = min(1, max_norm / (norm + 1e-6)) (fp32 [1], or NULL
 * if not wanted), NaN when the norm is not finite.  The scale is what moe_adamw_step takes as
 * d_grad_scale.  `tensors` is a host array.  ws: moe_grad_norm_workspace_bytes. */
int moe_grad_norm_workspace_bytes(const moe_tensor* tensors, int64_t n_tensors, size_t* out);
int moe_grad_norm(const moe_tensor* tensors, int64_t n_tensors, float max_norm, float* norm, float* scale,
                  void* ws, size_t ws_bytes, void* stream);

/* One AdamW step on n_tensors tensors (a host array; one launch for each 64 of them, or for each 54
 * if some have 8-bit states):
 *   g' = s g,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   w  = (1 - lr weight_decay) w - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32 on the master copy where there is one, else on p.  s = *d_grad_scale, or 1.  If
 * *d_grad_scale is not finite the whole step is skipped: nothing changes.  8-bit states are
 * rounded stochastically (a code up with the probability of the remainder; a nonzero sqrt(v) never
 * becomes zero), and so is a bf16 parameter without a master copy if `stochastic` is 1 (to nearest
 * if 0); the random bits are a function of seed, step, the tensor's place in the list and the
 * value's index, so a step is bitwise reproducible.  A gradient that is not finite makes its weight
 * NaN and leaves nothing of the 8-bit states of its 256 values (one whose square passes fp32's range
 * leaves nothing of their sqrt(v)); the scale of moe_grad_norm skips such a step, or brings it into range.
 * lr and step may live on the device (d_lr, d_step) for a captured graph whose replays move on; they are
 * read when the step runs.  The tensors overlap nowhere. */
typedef struct {
  double lr;              /* >= 0 and finite; unused with d_lr */
  double beta1, beta2;    /* in [0, 1) */
  double eps;             /* at least 2^-126 and finite in fp32 */
  int64_t step;           /* 1 for the first step; unused with d_step */
  uint64_t seed;
  int32_t stochastic;     /* 0 or 1 */
  int32_t reserved;       /* must be 0 */
  const float* d_lr;          /* fp32 [1] or NULL */
  const int64_t* d_step;      /* int64 [1] (at least 1) or NULL */
  const float* d_grad_scale;  /* fp32 [1] or NULL */
} moe_adamw;

int moe_adamw_step(const moe_adamw* hyper, const moe_tensor* tensors, int64_t n_tensors, void* stream);

/* Routing by scores, plus the expert plan: the gate's choice where moe_route's softmax over the k
 * largest logits is not what a model was trained with ([JAX] "A dropless MoE minden tokent feldolgoz": a
 * learned router scores the experts and keeps the top K).  With l a token's logits (fp32 [T, E]):
 *   s = softmax(l) over all E, or sigmoid(l) of each         c = s + bias (fp32 [E]; NULL: zeros)
 *   the E experts lie in `groups` groups of E / groups neighbours; a group's value is the sum of its
 *   group_best (1 or 2) largest c; the group_topk groups of the largest value stay
 *   ids = the k largest c among the experts that stay, descending
 *   w_j = scale * s[ids_j] / sum_i s[ids_i] (renormalise = 1), or scale * s[ids_j]
 * The bias moves the choice alone, never a weight.  Equal values go to the lower id (group, expert).  The
 * choice is the one that c in 64 bits gives; weights are computed in fp32, to 2^-18 of their value (from
 * a score below fp32's normal range: to 2^-148 times the larger of 1 and scale).
 * An expert whose logit or bias is -inf cannot be chosen: where fewer than k can, the slots behind them
 * have id -1 and weight 0 (a group in which none can be chosen never stays, and one with a single such
 * expert has its c for a value).  A token whose token_mask byte is 0 (uint8 [T]; NULL: none) has ids -1
 * and weights 0, whatever its logits are.  A token with a NaN among its logits or the bias, or a +inf
 * logit where the score is a softmax, has ids -1 and weights NaN.
 * counts, offsets, perm and inv_perm as moe_plan writes them; ws: moe_score_workspace_bytes.  T, E, k as
 * for moe_route; 1 <= groups <= 64 divides E, 1 <= group_topk <= groups, k <= group_topk * E / groups.
 * logits 16-byte aligned, the other arrays to their type. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

typedef struct {
  int64_t T, E, k;
  int32_t score;        /* moe_score */
  int32_t renormalise;  /* 0 or 1 */
  int32_t groups, group_topk, group_best;
  float scale;          /* finite */
  int32_t reserved;     /* must be 0 */
} moe_score_desc;

int moe_score_workspace_bytes(const moe_score_desc* desc, size_t* out);
int moe_score_route(const moe_score_desc* desc, const float* logits, const float* bias, const uint8_t* token_mask,
                    int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm,
                    int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);

/* Gradient of moe_score_route's weights: d_logits (fp32 [T, E], written whole) for d_topk_w (fp32 [T, k],
 * moe_backward's; call that one with d_logits NULL).  The choice carries no gradient.  With g = scale *
 * d_topk_w over the slots whose id is in [0, E), S their scores' sum and q = s / S:
 *   sigmoid              d_logits[ids_j] = g_j s_j (1 - s_j), and 0 elsewhere
 *   sigmoid, renormalise d_logits[ids_j] = (g_j - sum_i g_i q_i) q_j (1 - s_j), and 0 elsewhere
 *   softmax, renormalise d_logits[ids_j] = (g_j - sum_i g_i q_i) q_j, and 0 elsewhere
 *   softmax              d_logits[e] = s_e (sum_{j: ids_j = e} g_j - sum_i g_i s[ids_i]) for every e
 * The subtractions are made in 64 bits, of 64-bit scores of the chosen experts, so a confident token's
 * gradient keeps fp32's digits (the other experts' scores are fp32 exponentials, to |logit - max| + 2 units of
 * 2^-24) until it falls below 2^-48 of the g.
 * A token without such a slot has a row of zeros, whatever its logits are.  desc: T, E, k, score,
 * renormalise and scale are used (the others checked).  logits and d_logits 16-byte aligned, the other
 * arrays to their type; d_logits overlaps no input. */
int moe_score_backward(const moe_score_desc* desc, const float* logits, const int32_t* topk_ids,
                       const float* d_topk_w, float* d_logits, void* stream);

/* The bias moved against uneven loads ([JAX] "Az egyenetlen terhelés lassítja a tanítást" [uneven load
 * slows training]): bias_out[e] = bias[e] + rate * sign(mean(counts) - counts[e]), the sign from whole
 * numbers.  counts int32 [E] as moe_score_route writes them (they may have been summed over GPUs);
 * bias_out may be bias.  1 <= E <= 1024, rate finite.  Arrays aligned to their type. */
int moe_bias_update(int64_t E, const int32_t* counts, float rate, const float* bias, float* bias_out, void* stream);

/* Blockwise e4m3 quantisation, the layer's fp8 format (MOE_FP8_E4M3) on its own.  src: [rows, cols] of
 * src_dtype (MOE_BF16 or MOE_F32), `ld` values from one row to the next.  With m = max(largest magnitude
 * of a block, 448 * 2^-126): scale = m / 448 and code = e4m3(value * (448 / m)), each quotient and product
 * rounded to fp32, the code to nearest even; a block of zeros has the scale 1.  A NaN gets the code of NaN; an
 * infinity makes its block's scale infinite.  (moe_forward and moe_backward make the same codes of what they
 * quantise themselves, but for a NaN, -448 there, and without the least m.)
 *   MOE_BLOCK_ROWS    128 values of a row (moe_forward's x):  codes [rows, cols], scales [rows, ceil(cols/128)]
 *   MOE_BLOCK_TOKENS  128 rows of a column, transposed: codes [cols, R16] with R16 = rows rounded up to 16
 *                     (codes behind the last row are 0), scales [cols, ceil(rows/128)]: an operand of a
 *                     product over the rows, such as a weight gradient's
 *   MOE_BLOCK_TILES   128 x 128 (weights):  codes [rows, cols], scales [ceil(rows/128), ceil(cols/128)]
 * The last block of a row, column or matrix is a partial one.  rows >= 0, cols a positive multiple of 16,
 * both at most 2^24, rows * cols < 2^34; cols <= ld <= 2^31, ld a multiple of 8.  src and codes 16-byte aligned. */
typedef enum { MOE_BLOCK_ROWS = 0, MOE_BLOCK_TOKENS = 1, MOE_BLOCK_TILES = 2 } moe_block_form;

int moe_fp8_quantize(const void* src, int32_t src_dtype, int64_t rows, int64_t cols, int64_t ld, int32_t form,
                     void* codes, float* scales, void* stream);

/* Matrix product of blockwise e4m3 operands: C[M, N] = A . B (+ C_in), with A [M, K] codes and A_scale fp32
 * [M, ceil(K/128)] (MOE_BLOCK_ROWS), and B by b_form:
 *   MOE_B_KN       B [K, N], B_scale [ceil(K/128), ceil(N/128)]   a weight as the layer stores it: x . W
 *   MOE_B_NK       B [N, K], B_scale [ceil(N/128), ceil(K/128)]   the same weight's rows: dy . W^T, or a weight
 *                                                                 that is stored [out, in]
 *   MOE_B_NK_ROWS  B [N, K], B_scale [N, ceil(K/128)]             two quantised activations: with both as
 *                                                                 MOE_BLOCK_TOKENS writes them, x^T . dy
 * Products of codes are summed over each block of 128 along K, each block's sum times its two scales is
 * added in fp32, then C_in (c_dtype, C's layout; NULL: none; may be C itself), and C (bf16 or
 * fp32) is rounded once.  For an fp32 C the block's sums are fp32; for a bf16 C they come from the fp8 matrix
 * instruction, which drops what lies more than 13 bits below the largest of eight products (along K) before it
 * adds them: 1.5e-5 of the result's norm on normal data, and at most 7 * 2^-13 of the sum of all terms'
 * magnitudes, which is more than C's own rounding where terms cancel (an fp32 C keeps them).  The product of two
 * scales that meet has to be a normal fp32 number, and A's scale times a block's sum finite.  Sums run in a fixed
 * order (bitwise reproducible), which M, N, K, b_form and c_dtype decide.  lda, ldb, ldc: codes or values
 * from one row to the next; what lies between two rows is not touched.
 * M of any size, 0 .. 2^30; N and K positive multiples of 16 up to 2^24, M * N < 2^36; lda, ldb
 * multiples of 16, ldc of 8, at least the row's length; lda and ldb at most 2^28, ldc 2^31.  ws:
 * moe_fp8_matmul_workspace_bytes (256-byte aligned; may be NULL where that is 0).  A, B, C and C_in 16-byte aligned. */
typedef enum { MOE_B_KN = 0, MOE_B_NK = 1, MOE_B_NK_ROWS = 2 } moe_b_form;

typedef struct {
  int64_t M, N, K;
  int64_t lda, ldb, ldc;
  int32_t b_form;   /* moe_b_form */
  int32_t c_dtype;  /* MOE_BF16 or MOE_F32 */
  int32_t reserved; /* must be 0 */
} moe_matmul_desc;

int moe_fp8_matmul_workspace_bytes(const moe_matmul_desc* desc, size_t* out);
int moe_fp8_matmul(const moe_matmul_desc* desc, const void* A, const float* A_scale, const void* B,
                   const float* B_scale, const void* C_in, void* C, void* ws, size_t ws_bytes, void* stream);

/* Optional profiling hook (process-wide; none by default).  When set, each call invokes
 * hook(stage, 1, stream, user) on the calling thread right before it enqueues a stage's kernel
 * and hook(stage, 0, stream, user) right after, so a profiler can record stream events around
 * every kernel.  `stage` is a static string naming the kernel ("gemm_up", "combine", ...).
 * Pass NULL to remove the hook.  Setting it while another thread is inside a call races. */
typedef void (*moe_stage_hook)(const char* stage, int begin, void* stream, void* user);
int moe_set_stage_hook(moe_stage_hook hook, void* user);

/* MXFP8 quantisation on its own (the same kernels the MOE_MXFP8 path runs).  src is bf16
 * [batch, rows, cols] (row-major).  block_axis = 1: each block is 32 consecutive values of a row
 * (cols % 32 == 0), exps is [batch, rows, cols/32]; block_axis = 0: each block is 32
 * consecutive rows of one column (rows % 32 == 0, cols % 8 == 0), exps is [batch, rows/32,
 * cols].  codes (e4m3) has src's shape; exps are E8M0 bytes (2^(E-127)).  Rules as for
 * MOE_MXFP8 above.  Tensors 16-byte aligned.  ([JAX] "Csoportosított mátrixszorzás és
 * összevont adatmozgatás": group-aware MXFP8 quantisation.) */
int moe_mxfp8_quantize(const void* src, int64_t batch, int64_t rows, int64_t cols, int block_axis, void* codes,
                       void* exps, void* stream);

/* The MOE_MXFP8 path's weight quantiser on its own: one read of bf16 src [batch, rows, cols]
 * (row-major; rows % 32 == 0, cols % 256 == 0) writes both orientations of each matrix.
 * col_codes / col_exps: blocks of 32 consecutive rows of one column, exponents [batch, rows/32,
 * cols] (as block_axis = 0 above).  row_codes / row_words: blocks of 32 consecutive values of a
 * row, with the exponents as 32-bit words by 128-column step, [batch, cols/128, rows] words:
 * word (t, r) holds the E8M0 bytes of blocks 4t .. 4t+3 of row r (byte j for block 4t + j), the
 * layout the MXFP8 GEMMs read.  Codes have src's shape.  src and the codes 16-byte aligned,
 * col_exps 8-byte aligned, row_words 4-byte aligned.  ([JAX] "Csoportosított mátrixszorzás és
 * összevont adatmozgatás": MXFP8 blocks along each product's K; a weight matrix is the K operand
 * of the forward along its rows and of the data gradient along its columns.) */
int moe_mxfp8_quantize_weights(const void* src, int64_t batch, int64_t rows, int64_t cols, void* col_codes,
                               void* col_exps, void* row_codes, void* row_words, void* stream);

/* Static string for a status code (for MOE_ERR_HIP: the last HIP error on this thread). */
const char* moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */

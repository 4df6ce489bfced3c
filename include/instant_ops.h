/*
 * instant_ops.h - C ABI of the operators around the linear layer y = x . w^T of instant.h:
 * its forward with bias, activation and residual, its exact backward from activations kept
 * in 8 bits, and the RMS norm that produces its input. They are stateless (no handle): the
 * low-rank path of instant.h compresses what a layer keeps between calibrations, these serve
 * the steps whose backward is exact, and the parts of a layer around the product. Behind them
 * stand the operators at a language model's two ends, tokens to rows and logits to log
 * probabilities, with their gradients, and a step's last act before the optimizer: the norm over
 * all gradients, and clipping.
 *
 * Shapes and layouts (all row-major, contiguous, M = rows = tokens of all samples):
 *   x     [M, K]    the layer's input            w    [N, K]   weight (y = x . w^T)
 *   bias  [N]                                    res  [M, N]   residual added after the activation
 *   y, z  [M, N]    output, pre-activation       gy, gz, gx, gw, gb  gradients of y, z, x, w, bias
 *
 * A checkpoint in 8 bits of a matrix [M, C] is
 *   q      int8  [M, C]
 *   scale  uint8 [M, ceil(C / 32)]   one biased power-of-two exponent per 32 channels of a row
 * and stands for q * 2^(scale - 127). The exponent is the smallest of 1 .. 248 with
 * max |value| <= 127 * 2^(scale - 127), and q the nearest integer (ties to even), so an element
 * is off by at most half a step, 2^(scale - 128) <= max |group| / 127. |q| <= 127 takes 7 bits:
 * every value a checkpoint stands for is finite and exact in bfloat16. At the ends of float's
 * range: a group whose largest is above 127 * 2^121 (the last 1/128 of the largest binade) has
 * scale 248, and elements above that are kept as it, at most a step (2^121 < max |group| / 127)
 * off; a group whose largest is below 63.5 * 2^-126 has scale 1, and half a step is 2^-127 there.
 * A group that holds a NaN or an infinity has scale 255 and stands for NaN throughout, so a fault
 * is not hidden.
 *
 * Conventions (where they differ from instant.h it is said so)
 *   - Pointers are device pointers of the current device, aligned to 16 bytes (scale and rstd:
 *     to their element). The library never allocates device memory: what a call needs beyond
 *     its arguments is the caller's workspace (the *_workspace_bytes functions; 256-byte
 *     aligned; nothing in it need be initialised, nothing is kept in it). Two calls that may
 *     run at the same time need a workspace each.
 *   - Calls are asynchronous on `stream`, can be captured into a HIP graph, and give the same
 *     bits every time for the same arguments (no float atomics).
 *   - dtype (instant_dtype) is the type of x, w, bias, res, y, z, gy, gz, gx, gw, gb and of the
 *     norm's tensors. Sums, statistics and the activation are float32; each output is rounded
 *     once.
 *   - K, N and C must be multiples of 8, at most 2^18. 0 <= M <= 2^26; with M = 0 nothing is
 *     read, and gradients that sum over rows are written as zeros.
 *   - Outputs must not overlap inputs, except where said.
 *   - Errors are detected on the host, before anything is enqueued: E_ARG (null or misaligned
 *     pointer, bad enum, negative size), E_SHAPE (a size the operator does not take, or a
 *     workspace that is too small), E_HIP (a launch failed).
 */
#ifndef INSTANT_OPS_H_
#define INSTANT_OPS_H_

#include "instant.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation functions.
 *   RELU      max(z, 0)                 (slope 0 at z = 0)
 *   GELU      z Phi(z), Phi the normal distribution function
 *   GELU_TANH z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   SILU      z / (1 + exp(-z)) */
typedef enum {
  INSTANT_ACT_NONE = 0,
  INSTANT_ACT_RELU = 1,
  INSTANT_ACT_GELU = 2,
  INSTANT_ACT_GELU_TANH = 3,
  INSTANT_ACT_SILU = 4
} instant_act;

/* The layout of a checkpoint in 8 bits: channels that share a scale. */
#define INSTANT_CKPT_GROUP 32

/* Packs x [M, C] into q [M, C] and scale [M, ceil(C / 32)]. */
instant_status instant_ckpt_pack(const void* x, int32_t M, int32_t C, int32_t dtype, void* q, void* scale,
                                 void* stream);

/* Writes the values a checkpoint stands for to x [M, C] (exact in both dtypes). */
instant_status instant_ckpt_unpack(const void* q, const void* scale, int32_t M, int32_t C, int32_t dtype, void* x,
                                   void* stream);

/* Bytes of workspace that are enough for each of instant_linear_fwd, instant_act_bwd and
 * instant_linear_bwd (x in full or as a checkpoint) with these sizes (0 if the sizes are not
 * accepted; at least 256 otherwise): partial sums of a split contraction, and for gw from a
 * checkpoint up to 256 MB of x's values at a time. */
size_t instant_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype);

/* What each of the three calls needs alone, the backward with x as a checkpoint (x_ckpt != 0) or
 * in full (x_ckpt 0), for both gradients or for one of them (0: nothing, the workspace may be
 * NULL; also where the sizes are not accepted, which the call itself reports). */
size_t instant_linear_fwd_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype);
size_t instant_linear_bwd_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t x_ckpt);
size_t instant_linear_gx_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype);
size_t instant_linear_gw_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t x_ckpt);
size_t instant_act_bwd_workspace_bytes(int32_t M, int32_t N, int32_t dtype);

/* y = act(x w^T + bias) + res. bias and res may be NULL; res may be y itself. The
 * pre-activation x w^T + bias is also written where asked for: z [M, N], or the checkpoint zq,
 * zscale of the unrounded pre-activation (all NULL: not kept; z and zq exclude each other). */
instant_status instant_linear_fwd(const void* x, const void* w, const void* bias, const void* res, int32_t M,
                                  int32_t N, int32_t K, int32_t dtype, int32_t act, void* y, void* z, void* zq,
                                  void* zscale, void* workspace, size_t workspace_bytes, void* stream);

/* gz = gy * act'(z) [M, N] and gb = sum over rows of gz [N] (summed before gz is rounded), with
 * z given in full or as a checkpoint zq, zscale (exactly one; for INSTANT_ACT_NONE neither).
 * gz or gb may be NULL (not both); gz may be gy itself. The residual's gradient is gy. */
instant_status instant_act_bwd(const void* gy, const void* z, const void* zq, const void* zscale, int32_t M,
                               int32_t N, int32_t dtype, int32_t act, void* gz, void* gb, void* workspace,
                               size_t workspace_bytes, void* stream);

/* gx = gz w [M, K] and gw = gz^T x [N, K] (overwritten), with x given in full or as a checkpoint
 * xq, xscale. gx or gw may be NULL (not both); w is read only for gx, x only for gw (what is not
 * read may be NULL). */
instant_status instant_linear_bwd(const void* gz, const void* w, const void* x, const void* xq, const void* xscale,
                                  int32_t M, int32_t N, int32_t K, int32_t dtype, void* gx, void* gw,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* RMS norm with the residual's addition, over rows of C <= 65536 channels:
 *   h = x + res (rounded to dtype; h = x and not written when res is NULL)
 *   rstd = (mean(h^2) + eps)^(-1/2) [M] float32        y = h * rstd * g, g [C]
 * y [M, C] and the checkpoint yq, yscale of the rounded y are each written where given (one of
 * the two at least); rstd may be NULL. h may be x or res itself; h must be NULL exactly when res
 * is. eps >= 0. */
instant_status instant_rmsnorm_fwd(const void* x, const void* res, const void* g, int32_t M, int32_t C, int32_t dtype,
                                   float eps, void* h, void* y, void* yq, void* yscale, float* rstd, void* stream);

/* Bytes of workspace for instant_rmsnorm_bwd (0 if the sizes are not accepted). */
size_t instant_rmsnorm_workspace_bytes(int32_t M, int32_t C);

/* The norm's gradients: with u = gy * g,
 *   gx = rstd (u - h rstd^2 mean(u h)) + gh [M, C]     gg = sum over rows of gy h rstd [C]
 * gh, the gradient that reaches h past the norm, may be NULL. x and res have the same gradient
 * gx. gx may be gy or gh itself. gg may be NULL. */
instant_status instant_rmsnorm_bwd(const void* gy, const void* h, const void* g, const float* rstd, const void* gh,
                                   int32_t M, int32_t C, int32_t dtype, void* gx, void* gg, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ---- The ends of a training step. Differences from the conventions above:
 *   - Tokens and targets are integers of token_bytes bytes (4 or 8), aligned to their size.
 *   - A vocabulary is 1 <= V <= 2^18; logits have rows of any width, so V need not be a multiple
 *     of 8, and they and their gradient are aligned to an element only.
 *   - What integers hold is not known on the host. One outside 0 .. V - 1 (and not the ignored or
 *     padding one) reads nothing out of range: its row of y, its log probability and its row of gz
 *     are NaN, so the fault is not hidden; the table's gradient has no place for it. */

/* y = scale * table[tokens] [M, C], for table [V, C] (rounded once; exact for scale 1). */
instant_status instant_embed_fwd(const void* tokens, int32_t token_bytes, int32_t M, const void* table, int32_t V,
                                 int32_t C, int32_t dtype, float scale, void* y, void* stream);

/* Bytes of workspace for instant_embed_bwd (0: nothing, or sizes that are not accepted). */
size_t instant_embed_workspace_bytes(int32_t M, int32_t V, int32_t C);

/* The table's gradient: gtable[v] = scale * sum of the rows of gy [M, C] whose token is v, added in
 * float32; rows without a token are zeros. The tokens alone fix the order of the additions, so the bits
 * are the same every time. It is not row after row: the rows, grouped by token (a token's in their order),
 * are added in eights, those in tiles of 64 and those by eighths of a run, and where a run is cut depends
 * on how many rows other tokens have before it. Rows whose token is `padding` (-1: none) take no part.
 * accumulate != 0: the sums are added to what gtable holds (and rounded
 * once), rows without a token stay as they are. gtable may not share memory with gy (E_ARG). M <= 2^22,
 * M * C <= 2^36. */
instant_status instant_embed_bwd(const void* gy, const void* tokens, int32_t token_bytes, int32_t M, int32_t V,
                                 int32_t C, int32_t dtype, float scale, int64_t padding, int32_t accumulate,
                                 void* gtable, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace for instant_logprobs_fwd (0: nothing, or sizes that are not accepted): few
 * long rows are split. */
size_t instant_logprobs_workspace_bytes(int32_t M, int32_t V, int32_t dtype, int32_t k);

/* Log probabilities from logits [M, W], of whose columns the first V <= W <= 2^18 count. Each of
 *   logp     float [M]     log of the probability of targets[m]; 0 where that is `ignore`
 *   lse      float [M]     log sum exp(logits)
 *   entropy  float [M]     -sum p log p
 *   stats    float [M, 2]  the largest logit and the log of sum exp(logits - it), for the gradient
 *   top_logp float [M, k], top_index int64 [M, k]   the k <= 32, k <= V likeliest in order, equal
 *                          ones by their place (-0 is 0), and their log probabilities
 * may be NULL; targets may be NULL with logp (and must be given with it), and both top_* are given
 * exactly when k > 0.
 * A logit of -inf has probability 0 (log probability -inf). A row of nothing else has probability 0
 * throughout: lse -inf, entropy 0, log probabilities -inf, alternatives 0 .. k - 1. A NaN or +inf
 * makes its row's results NaN; among the alternatives a NaN ranks with -inf. */
instant_status instant_logprobs_fwd(const void* logits, const void* targets, int32_t token_bytes, int32_t M,
                                    int32_t W, int32_t V, int32_t dtype, int64_t ignore, int32_t k, float* logp,
                                    float* lse, float* entropy, float* stats, float* top_logp, int64_t* top_index,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* The logits' gradient gz [M, W] for gradients g_logp, g_lse, g_entropy [M] (each may be NULL, not
 * all) of logp, lse and entropy, with stats and (for g_entropy) entropy from the forward pass:
 *   gz_j = g_logp (1[j = t] - p_j) + g_lse p_j - g_entropy p_j (log p_j + entropy),   j < V
 * and 0 in the columns behind V. g_logp needs targets, and takes no part where they are `ignore`.
 * A row whose gradients are all 0 gets zeros, whatever it holds (with g_logp, unless its target is outside
 * the vocabulary: NaN). gz may be logits itself,
 * but not share memory with it otherwise (E_ARG). */
instant_status instant_logprobs_bwd(const void* logits, const void* targets, int32_t token_bytes, int32_t M,
                                    int32_t W, int32_t V, int32_t dtype, int64_t ignore, const float* stats,
                                    const float* entropy, const float* g_logp, const float* g_lse,
                                    const float* g_entropy, void* gz, void* stream);

/* The Euclidean norm over n tensors, norm[0] = (sum of all squares)^(1/2) float32, summed in
 * float64. grads, count and dtype are host arrays, read before the call returns: device pointers
 * (aligned to an element; NULL where count is 0), elements (0 <= count <= 2^40) and instant_dtype.
 * 0 <= n <= 2^20. A tensor that is listed twice counts twice. */
size_t instant_grad_norm_workspace_bytes(int32_t n);
instant_status instant_grad_norm(const void* const* grads, const int64_t* count, const int32_t* dtype, int32_t n,
                                 float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* The same norm, and out[i] = c * grads[i] with c = 1 if norm + 1e-6 <= max_norm, else
 * max_norm / (norm + 1e-6) (max_norm >= 0, infinity allowed). Each product is rounded once to
 * out_dtype[i]. out[i] may be grads[i] itself in the same type; no other overlap of an output with
 * an output or a gradient is accepted (E_ARG). A NaN norm makes everything NaN, an infinite one
 * gives c = 0 (unless max_norm is infinite). */
instant_status instant_clip_grads(const void* const* grads, const int64_t* count, const int32_t* dtype,
                                  void* const* out, const int32_t* out_dtype, int32_t n, float max_norm, float* norm,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INSTANT_OPS_H_ */

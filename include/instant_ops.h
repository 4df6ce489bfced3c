/*
 * instant_ops.h - C ABI of the operators around the linear layer y = x . w^T of instant.h:
 * its forward with bias, activation and residual, its exact backward from activations kept
 * in 8 bits, and the RMS norm that produces its input. They are stateless (no handle): the
 * low-rank path of instant.h compresses what a layer keeps between calibrations, these serve
 * the steps whose backward is exact, and the parts of a layer around the product.
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

#ifdef __cplusplus
}
#endif

#endif /* INSTANT_OPS_H_ */

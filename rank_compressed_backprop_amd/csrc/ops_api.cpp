// C entry points of the operators around the linear layer and at a training step's ends
// (include/instant_ops.h): argument checks and workspace use; every step is a stream-ordered launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "instant_ops.h"
#include "ops.hpp"

#define INSTANT_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace instant;

static_assert(INSTANT_CKPT_GROUP == CK_GROUP && INSTANT_ACT_RELU == ACT_RELU && INSTANT_ACT_GELU == ACT_GELU &&
                  INSTANT_ACT_GELU_TANH == ACT_GELU_TANH && INSTANT_ACT_SILU == ACT_SILU,
              "the header's constants");

inline hipStream_t S(void* stream) { return (hipStream_t)stream; }
inline instant_status hip_ok(hipError_t e) { return e == hipSuccess ? INSTANT_OK : INSTANT_E_HIP; }
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <class... P> bool off16(P... p) { return (... || (((uintptr_t)p) % 16)); }
bool dtype_ok(int32_t d) { return d == INSTANT_FP32 || d == INSTANT_BF16; }
bool act_ok(int32_t a) { return a >= INSTANT_ACT_NONE && a <= INSTANT_ACT_SILU; }

// The largest sizes: block counts and row counts rounded up to tiles stay within 32 bits.
constexpr int32_t MAX_ROWS = 1 << 26, MAX_WIDTH = 1 << 18;

// rows >= 0 and widths that are positive multiples of 8 (E_ARG: not positive at all)
instant_status sizes(int32_t M, std::initializer_list<int32_t> widths) {
  if (M < 0) return INSTANT_E_ARG;
  for (int32_t c : widths)
    if (c < 1) return INSTANT_E_ARG;
  if (M > MAX_ROWS) return INSTANT_E_SHAPE;
  for (int32_t c : widths)
    if (c % 8 || c > MAX_WIDTH) return INSTANT_E_SHAPE;
  return INSTANT_OK;
}

size_t linear_fwd_bytes(bool bf, int M, int N, int K) { return 4 * linear_part_floats(bf, Prod::Fwd, M, N, K, false); }
size_t linear_gx_bytes(bool bf, int M, int N, int K) { return 4 * linear_part_floats(bf, Prod::Gx, M, N, K, false); }
size_t linear_gw_bytes(bool bf, int M, int N, int K, bool x_ckpt) {
  return 4 * linear_part_floats(bf, Prod::Gw, M, N, K, x_ckpt);
}
size_t linear_bwd_bytes(bool bf, int M, int N, int K, bool x_ckpt) {
  return std::max(linear_gx_bytes(bf, M, N, K), linear_gw_bytes(bf, M, N, K, x_ckpt));
}

// A workspace that a call needs `need` bytes of (none: it may be null).
instant_status workspace_ok(const void* ws, size_t have, size_t need) {
  if (!need) return INSTANT_OK;
  if (!ws || ((uintptr_t)ws) % 256) return INSTANT_E_ARG;
  return have < need ? INSTANT_E_SHAPE : INSTANT_OK;
}

}  // namespace

#define TRY(s)                           \
  do {                                   \
    const instant_status s_ = (s);       \
    if (s_ != INSTANT_OK) return s_;     \
  } while (0)

INSTANT_API instant_status instant_ckpt_pack(const void* x, int32_t M, int32_t C, int32_t dtype, void* q, void* scale,
                                             void* stream) {
  TRY(sizes(M, {C}));
  if (!dtype_ok(dtype) || off16(x, q)) return INSTANT_E_ARG;
  if (M == 0) return INSTANT_OK;
  if (!x || !q || !scale) return INSTANT_E_ARG;
  return hip_ok(launch_ckpt_pack(dtype == INSTANT_BF16, x, M, C, Ckpt{(int8_t*)q, (uint8_t*)scale}, S(stream)));
}

INSTANT_API instant_status instant_ckpt_unpack(const void* q, const void* scale, int32_t M, int32_t C, int32_t dtype,
                                               void* x, void* stream) {
  TRY(sizes(M, {C}));
  if (!dtype_ok(dtype) || off16(x, q)) return INSTANT_E_ARG;
  if (M == 0) return INSTANT_OK;
  if (!x || !q || !scale) return INSTANT_E_ARG;
  return hip_ok(launch_ckpt_unpack(dtype == INSTANT_BF16, Ckpt{(int8_t*)q, (uint8_t*)scale}, M, C, x, S(stream)));
}

INSTANT_API size_t instant_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype) {
  if (sizes(M, {N, K}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  const bool bf = dtype == INSTANT_BF16;
  return align256(std::max({(size_t)256, linear_fwd_bytes(bf, M, N, K), linear_bwd_bytes(bf, M, N, K, true),
                            linear_bwd_bytes(bf, M, N, K, false), 4 * act_bwd_part_floats(M, N)}));
}

INSTANT_API size_t instant_linear_fwd_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype) {
  if (sizes(M, {N, K}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  return linear_fwd_bytes(dtype == INSTANT_BF16, M, N, K);
}

INSTANT_API size_t instant_linear_bwd_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t x_ckpt) {
  if (sizes(M, {N, K}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  return linear_bwd_bytes(dtype == INSTANT_BF16, M, N, K, x_ckpt != 0);
}

INSTANT_API size_t instant_linear_gx_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype) {
  if (sizes(M, {N, K}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  return linear_gx_bytes(dtype == INSTANT_BF16, M, N, K);
}

INSTANT_API size_t instant_linear_gw_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t x_ckpt) {
  if (sizes(M, {N, K}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  return linear_gw_bytes(dtype == INSTANT_BF16, M, N, K, x_ckpt != 0);
}

INSTANT_API size_t instant_act_bwd_workspace_bytes(int32_t M, int32_t N, int32_t dtype) {
  if (sizes(M, {N}) != INSTANT_OK || !dtype_ok(dtype)) return 0;
  return 4 * act_bwd_part_floats(M, N);
}

INSTANT_API instant_status instant_linear_fwd(const void* x, const void* w, const void* bias, const void* res,
                                              int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t act, void* y,
                                              void* z, void* zq, void* zscale, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  TRY(sizes(M, {N, K}));
  if (!dtype_ok(dtype) || !act_ok(act) || off16(x, w, bias, res, y, z, zq)) return INSTANT_E_ARG;
  if ((zq == nullptr) != (zscale == nullptr) || (z && zq)) return INSTANT_E_ARG;
  if (M == 0) return INSTANT_OK;
  if (!x || !w || !y) return INSTANT_E_ARG;
  const bool bf = dtype == INSTANT_BF16;
  TRY(workspace_ok(workspace, workspace_bytes, linear_fwd_bytes(bf, M, N, K)));
  const Epi ep{bias, res, y, z, Ckpt{(int8_t*)zq, (uint8_t*)zscale}, act};
  return hip_ok(launch_linear_fwd(bf, x, w, M, N, K, ep, (float*)workspace, S(stream)));
}

INSTANT_API instant_status instant_act_bwd(const void* gy, const void* z, const void* zq, const void* zscale,
                                           int32_t M, int32_t N, int32_t dtype, int32_t act, void* gz, void* gb,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  TRY(sizes(M, {N}));
  if (!dtype_ok(dtype) || !act_ok(act) || off16(gy, z, zq, gz, gb)) return INSTANT_E_ARG;
  if ((zq == nullptr) != (zscale == nullptr) || (z && zq)) return INSTANT_E_ARG;
  if ((M > 0 && !gz && !gb) || (act == INSTANT_ACT_NONE && (z || zq))) return INSTANT_E_ARG;
  if (M > 0 && (!gy || (act != INSTANT_ACT_NONE && !z && !zq))) return INSTANT_E_ARG;
  TRY(workspace_ok(workspace, workspace_bytes, gb ? 4 * act_bwd_part_floats(M, N) : 0));
  return hip_ok(launch_act_bwd(dtype == INSTANT_BF16, gy, z, Ckpt{(int8_t*)zq, (uint8_t*)zscale}, M, N, act, gz, gb,
                               (float*)workspace, S(stream)));
}

INSTANT_API instant_status instant_linear_bwd(const void* gz, const void* w, const void* x, const void* xq,
                                              const void* xscale, int32_t M, int32_t N, int32_t K, int32_t dtype,
                                              void* gx, void* gw, void* workspace, size_t workspace_bytes,
                                              void* stream) {
  TRY(sizes(M, {N, K}));
  if (!dtype_ok(dtype) || off16(gz, w, x, xq, gx, gw)) return INSTANT_E_ARG;
  if ((xq == nullptr) != (xscale == nullptr) || (x && xq) || (M > 0 && !gx && !gw)) return INSTANT_E_ARG;
  if (M > 0 && (!gz || (gx && !w) || (gw && !x && !xq))) return INSTANT_E_ARG;
  const bool bf = dtype == INSTANT_BF16;
  TRY(workspace_ok(workspace, workspace_bytes,
                   std::max(gx ? linear_gx_bytes(bf, M, N, K) : 0,
                            gw ? linear_gw_bytes(bf, M, N, K, xq != nullptr) : 0)));
  hipError_t e = hipSuccess;
  if (gx && M > 0) e = launch_linear_gx(bf, gz, w, M, N, K, gx, (float*)workspace, S(stream));
  if (e == hipSuccess && gw)
    e = launch_linear_gw(bf, gz, x, Ckpt{(int8_t*)xq, (uint8_t*)xscale}, M, N, K, gw, (float*)workspace, S(stream));
  return hip_ok(e);
}

INSTANT_API instant_status instant_rmsnorm_fwd(const void* x, const void* res, const void* g, int32_t M, int32_t C,
                                               int32_t dtype, float eps, void* h, void* y, void* yq, void* yscale,
                                               float* rstd, void* stream) {
  TRY(sizes(M, {C}));
  if (!dtype_ok(dtype) || !(eps >= 0.0f) || std::isinf(eps) || off16(x, res, g, h, y, yq) || ((uintptr_t)rstd) % 4)
    return INSTANT_E_ARG;
  if ((yq == nullptr) != (yscale == nullptr)) return INSTANT_E_ARG;
  if (C > NORM_MAX_C) return INSTANT_E_SHAPE;
  if (M == 0) return INSTANT_OK;
  if ((res == nullptr) != (h == nullptr) || (!y && !yq)) return INSTANT_E_ARG;
  if (!x || !g) return INSTANT_E_ARG;
  return hip_ok(launch_rmsnorm_fwd(dtype == INSTANT_BF16, x, res, g, M, C, eps, h, y,
                                   Ckpt{(int8_t*)yq, (uint8_t*)yscale}, rstd, S(stream)));
}

INSTANT_API size_t instant_rmsnorm_workspace_bytes(int32_t M, int32_t C) {
  if (sizes(M, {C}) != INSTANT_OK || C > NORM_MAX_C) return 0;
  return align256(std::max<size_t>(256, 4 * rmsnorm_part_floats(M, C)));
}

INSTANT_API instant_status instant_rmsnorm_bwd(const void* gy, const void* h, const void* g, const float* rstd,
                                               const void* gh, int32_t M, int32_t C, int32_t dtype, void* gx, void* gg,
                                               void* workspace, size_t workspace_bytes, void* stream) {
  TRY(sizes(M, {C}));
  if (!dtype_ok(dtype) || off16(gy, h, g, gh, gx, gg) || ((uintptr_t)rstd) % 4) return INSTANT_E_ARG;
  if (C > NORM_MAX_C) return INSTANT_E_SHAPE;
  if (M > 0 && (!gy || !h || !g || !rstd || !gx)) return INSTANT_E_ARG;
  if (M == 0 && !gg) return INSTANT_OK;
  TRY(workspace_ok(workspace, workspace_bytes, gg ? 4 * rmsnorm_part_floats(M, C) : 0));
  return hip_ok(launch_rmsnorm_bwd(dtype == INSTANT_BF16, gy, h, g, rstd, gh, M, C, gx, gg, (float*)workspace,
                                   S(stream)));
}

namespace {

bool tokens_ok(const void* t, int32_t bytes) { return (bytes == 4 || bytes == 8) && ((uintptr_t)t) % bytes == 0; }

// 1 <= V <= W <= MAX_WIDTH, of any residue
instant_status vocab(int32_t M, int32_t W, int32_t V) {
  if (M < 0 || V < 1 || W < V) return INSTANT_E_ARG;
  return M > MAX_ROWS || W > MAX_WIDTH ? INSTANT_E_SHAPE : INSTANT_OK;
}

// logits may start at any element, as rows cut out of a matrix of odd width do
bool logits_ok(const void* z, int32_t dtype) { return ((uintptr_t)z) % (dtype == INSTANT_BF16 ? 2 : 4) == 0; }

template <class... P> bool off4(P... p) { return (... || (((uintptr_t)p) % 4)); }

// whether [a, a + na) and [b, b + nb), in elements of dtype, share memory
bool overlap(const void* a, int64_t na, const void* b, int64_t nb, int32_t dtype) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b, e = dtype == INSTANT_BF16 ? 2 : 4;
  return x < y + (uintptr_t)nb * e && y < x + (uintptr_t)na * e;
}

instant_status embed_sizes(int32_t M, int32_t V, int32_t C) {
  TRY(sizes(M, {C}));
  if (V < 1) return INSTANT_E_ARG;
  return V > MAX_WIDTH ? INSTANT_E_SHAPE : INSTANT_OK;
}

instant_status embed_bwd_sizes(int32_t M, int32_t V, int32_t C) {
  TRY(embed_sizes(M, V, C));
  return M > EMBED_MAX_M || (int64_t)M * C > (int64_t)1 << 36 ? INSTANT_E_SHAPE : INSTANT_OK;
}

constexpr int32_t MAX_TENSORS = 1 << 20;

instant_status tensors(const void* const* p, const int64_t* count, const int32_t* dtype, int32_t n) {
  if (n < 0 || (n > 0 && (!p || !count || !dtype))) return INSTANT_E_ARG;
  if (n > MAX_TENSORS) return INSTANT_E_SHAPE;
  for (int32_t i = 0; i < n; ++i) {
    if (count[i] < 0 || !dtype_ok(dtype[i])) return INSTANT_E_ARG;
    if (count[i] > (int64_t)1 << 40) return INSTANT_E_SHAPE;
    if (count[i] && (!p[i] || ((uintptr_t)p[i]) % (dtype[i] == INSTANT_BF16 ? 2 : 4))) return INSTANT_E_ARG;
  }
  return INSTANT_OK;
}

// Whether an output of clip_grads shares memory with another tensor of the call (other than an
// output with its own gradient, of the same type in the same place). Two intervals that overlap
// are found by a sweep over the starts; gradients may share memory with each other.
bool outputs_overlap(const void* const* g, void* const* out, const int64_t* count, const int32_t* dtype,
                     const int32_t* out_dtype, int32_t n) {
  struct Span {
    uintptr_t a, b;
    bool out;
  };
  std::vector<Span> v;
  v.reserve(2 * (size_t)n);
  for (int32_t i = 0; i < n; ++i) {
    if (!count[i]) continue;
    const uintptr_t a = (uintptr_t)g[i], o = (uintptr_t)out[i];
    v.push_back({o, o + (uintptr_t)count[i] * (out_dtype[i] == INSTANT_BF16 ? 2 : 4), true});
    if (a != o || dtype[i] != out_dtype[i])
      v.push_back({a, a + (uintptr_t)count[i] * (dtype[i] == INSTANT_BF16 ? 2 : 4), false});
  }
  std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t any = 0, outs = 0;  // the furthest ends so far
  for (const Span& s : v) {
    if (s.a < (s.out ? any : outs)) return true;
    any = std::max(any, s.b);
    if (s.out) outs = std::max(outs, s.b);
  }
  return false;
}

}  // namespace

INSTANT_API instant_status instant_embed_fwd(const void* tokens, int32_t token_bytes, int32_t M, const void* table,
                                             int32_t V, int32_t C, int32_t dtype, float scale, void* y, void* stream) {
  TRY(embed_sizes(M, V, C));
  if (!dtype_ok(dtype) || !tokens_ok(tokens, token_bytes) || off16(table, y) || !std::isfinite(scale))
    return INSTANT_E_ARG;
  if (M == 0) return INSTANT_OK;
  if (!tokens || !table || !y) return INSTANT_E_ARG;
  return hip_ok(
      launch_embed_fwd(dtype == INSTANT_BF16, tokens, token_bytes == 8, M, table, V, C, scale, y, S(stream)));
}

INSTANT_API size_t instant_embed_workspace_bytes(int32_t M, int32_t V, int32_t C) {
  if (embed_bwd_sizes(M, V, C) != INSTANT_OK) return 0;
  return embed_bwd_bytes(M, C);
}

INSTANT_API instant_status instant_embed_bwd(const void* gy, const void* tokens, int32_t token_bytes, int32_t M,
                                             int32_t V, int32_t C, int32_t dtype, float scale, int64_t padding,
                                             int32_t accumulate, void* gtable, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  TRY(embed_bwd_sizes(M, V, C));
  if (!dtype_ok(dtype) || !tokens_ok(tokens, token_bytes) || off16(gy, gtable) || !std::isfinite(scale) || !gtable ||
      padding < -1)
    return INSTANT_E_ARG;
  if (M > 0 && (!gy || !tokens || overlap(gy, (int64_t)M * C, gtable, (int64_t)V * C, dtype))) return INSTANT_E_ARG;
  TRY(workspace_ok(workspace, workspace_bytes, embed_bwd_bytes(M, C)));
  return hip_ok(launch_embed_bwd(dtype == INSTANT_BF16, gy, tokens, token_bytes == 8, M, V, C, scale, padding,
                                 accumulate != 0, gtable, workspace, S(stream)));
}

INSTANT_API size_t instant_logprobs_workspace_bytes(int32_t M, int32_t V, int32_t dtype, int32_t k) {
  if (vocab(M, V, V) != INSTANT_OK || !dtype_ok(dtype) || k < 0 || k > LOGPROBS_MAX_TOP || k > V) return 0;
  return logprobs_fwd_bytes(dtype == INSTANT_BF16, M, V, k);
}

INSTANT_API instant_status instant_logprobs_fwd(const void* logits, const void* targets, int32_t token_bytes,
                                                int32_t M, int32_t W, int32_t V, int32_t dtype, int64_t ignore,
                                                int32_t k, float* logp, float* lse, float* entropy, float* stats,
                                                float* top_logp, int64_t* top_index, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  TRY(vocab(M, W, V));
  if (!dtype_ok(dtype) || !tokens_ok(targets, token_bytes) || !logits_ok(logits, dtype) ||
      off4(logp, lse, entropy, stats, top_logp) || ((uintptr_t)top_index) % 8)
    return INSTANT_E_ARG;
  if (k < 0) return INSTANT_E_ARG;
  if (k > LOGPROBS_MAX_TOP || k > V) return INSTANT_E_SHAPE;
  if (M == 0) return INSTANT_OK;
  if (!logits || (targets == nullptr) != (logp == nullptr)) return INSTANT_E_ARG;
  if ((k > 0) != (top_logp != nullptr) || (k > 0) != (top_index != nullptr)) return INSTANT_E_ARG;
  if (!logp && !lse && !entropy && !stats && !k) return INSTANT_E_ARG;
  const bool bf = dtype == INSTANT_BF16;
  TRY(workspace_ok(workspace, workspace_bytes, logprobs_fwd_bytes(bf, M, V, k)));
  return hip_ok(launch_logprobs_fwd(bf, logits, targets, token_bytes == 8, M, W, V, ignore, k, logp, lse, entropy,
                                    stats, top_logp, top_index, workspace, S(stream)));
}

INSTANT_API instant_status instant_logprobs_bwd(const void* logits, const void* targets, int32_t token_bytes,
                                                int32_t M, int32_t W, int32_t V, int32_t dtype, int64_t ignore,
                                                const float* stats, const float* entropy, const float* g_logp,
                                                const float* g_lse, const float* g_entropy, void* gz, void* stream) {
  TRY(vocab(M, W, V));
  if (!dtype_ok(dtype) || !tokens_ok(targets, token_bytes) || !logits_ok(logits, dtype) || !logits_ok(gz, dtype) ||
      off4(stats, entropy, g_logp, g_lse, g_entropy))
    return INSTANT_E_ARG;
  if (M == 0) return INSTANT_OK;
  if (!logits || !stats || !gz || (!g_logp && !g_lse && !g_entropy)) return INSTANT_E_ARG;
  if ((g_logp && !targets) || (g_entropy && !entropy)) return INSTANT_E_ARG;
  if (gz != logits && overlap(gz, (int64_t)M * W, logits, (int64_t)M * W, dtype)) return INSTANT_E_ARG;
  return hip_ok(launch_logprobs_bwd(dtype == INSTANT_BF16, logits, targets, token_bytes == 8, M, W, V, ignore, stats,
                                    entropy, g_logp, g_lse, g_entropy, gz, S(stream)));
}

INSTANT_API size_t instant_grad_norm_workspace_bytes(int32_t n) {
  return n < 0 || n > MAX_TENSORS ? 0 : grad_norm_bytes(n);
}

INSTANT_API instant_status instant_grad_norm(const void* const* grads, const int64_t* count, const int32_t* dtype,
                                             int32_t n, float* norm, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  TRY(tensors(grads, count, dtype, n));
  if (!norm || off4(norm)) return INSTANT_E_ARG;
  TRY(workspace_ok(workspace, workspace_bytes, grad_norm_bytes(n)));
  return hip_ok(launch_grad_norm(grads, count, dtype, n, norm, workspace, S(stream)));
}

INSTANT_API instant_status instant_clip_grads(const void* const* grads, const int64_t* count, const int32_t* dtype,
                                              void* const* out, const int32_t* out_dtype, int32_t n, float max_norm,
                                              float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  TRY(tensors(grads, count, dtype, n));
  TRY(tensors(out, count, out_dtype, n));
  if (!norm || off4(norm) || !(max_norm >= 0.0f)) return INSTANT_E_ARG;
  TRY(workspace_ok(workspace, workspace_bytes, grad_norm_bytes(n)));
  try {
    if (outputs_overlap(grads, out, count, dtype, out_dtype, n)) return INSTANT_E_ARG;
  } catch (const std::bad_alloc&) {
    return INSTANT_E_HIP;
  }
  return hip_ok(launch_clip_grads(grads, count, dtype, out, out_dtype, n, max_norm, norm, workspace, S(stream)));
}

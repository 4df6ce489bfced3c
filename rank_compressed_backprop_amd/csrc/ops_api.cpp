// C entry points of the operators around the linear layer (include/instant_ops.h): argument
// checks and workspace use; every step is a stream-ordered launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

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

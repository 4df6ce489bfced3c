// Shared by the operators around the linear layer (include/instant_ops.h): the 8-bit
// checkpoint format, activations and their slopes, the GEMM epilogue, host launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"

namespace instant {

constexpr int CK_GROUP = 32;  // channels that share a scale
__host__ __device__ inline int ck_groups(int C) { return (C + CK_GROUP - 1) / CK_GROUP; }

constexpr int ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4;

// A matrix as a checkpoint in 8 bits, or (q null) none.
struct Ckpt {
  int8_t* q;
  uint8_t* scale;
};

// f(0) .. f(N - 1) with constant arguments: register arrays are indexed by constants whatever
// the size of the body
template <int... I, class F> __device__ __forceinline__ void each(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void each(F&& f) {
  each(std::make_integer_sequence<int, N>{}, f);
}

// ---- the checkpoint format on the device

// Magnitude bits of a float. As unsigned integers they order finite numbers, infinity and NaN
// by size, so a group's largest also finds a NaN or infinity in it.
__device__ __forceinline__ unsigned mag_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// The biased exponent of a group's scale from the magnitude bits of its largest element: the
// smallest power of two s with amax <= 127 s. 127 = 1.984375 * 2^6, so an amax with mantissa
// field above 0x7e0000 needs one exponent more: the addition carries exactly then. At most 248:
// 64 steps of the next would be 2^128, no float.
constexpr unsigned CK_MAX_SCALE = 248;
__device__ __forceinline__ unsigned ck_scale_byte(unsigned amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)((amax + 0x01ffffu) >> 23) - 6;
  return (unsigned)(b < 1 ? 1 : b > (int)CK_MAX_SCALE ? (int)CK_MAX_SCALE : b);
}
// 2^(byte - 127); the float of byte 255 is infinity, and such a group's q is 0: 0 * inf = NaN.
__device__ __forceinline__ float ck_scale(unsigned byte) { return __builtin_bit_cast(float, byte << 23); }
// its inverse (byte <= 248 for finite groups, so the exponent field stays normal)
__device__ __forceinline__ float ck_inv_scale(unsigned byte) { return __builtin_bit_cast(float, (254u - byte) << 23); }

// Eight values to int8 (nearest, ties to even): packed low to high. The product with the scale's
// inverse is exact, and adding 1.5 * 2^23 (where a float's step is 1) rounds it to the nearest
// integer, whose low byte is the float's: one operation a value, and the packing. Only at the
// largest scale can that be 128 steps (from above 127.5, at the end of float's range): those
// become 127, in a branch of their own, as the others need no limit.
__device__ __forceinline__ uint2 ck_quant8(const float v[8], unsigned byte) {
  const float inv = ck_inv_scale(byte == 255u ? 254u : byte);
  unsigned t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = __builtin_bit_cast(unsigned, fmaf(v[j], inv, 12582912.0f));
  if (byte == CK_MAX_SCALE) {  // (as integers the floats' bits differ by the steps)
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = min(max(t[j], 0x4b400000u - 127u), 0x4b400000u + 127u);
  }
  unsigned r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const unsigned lo = __builtin_amdgcn_perm(t[4 * h + 1], t[4 * h], 0x0c0c0400u);
    const unsigned hi = __builtin_amdgcn_perm(t[4 * h + 3], t[4 * h + 2], 0x04000c0cu);
    r[h] = byte == 255u ? 0u : lo | hi;
  }
  return uint2{r[0], r[1]};
}

__device__ __forceinline__ void ck_dequant8(uint2 q, unsigned byte, float v[8]) {
  const float s = ck_scale(byte);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = h ? (int)q.y : (int)q.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * h + j] = (float)((w << (24 - 8 * j)) >> 24) * s;
  }
}

// The largest magnitude of 32 channels held 8 a lane by the four lanes that differ in lane-id
// bits X1 and X2 (every one of them must be active).
template <int X1, int X2>
__device__ __forceinline__ unsigned ck_group_amax(const float v[8], bool in) {
  unsigned a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned m = mag_bits(v[j]);
    a = m > a ? m : a;
  }
  if (!in) a = 0;
  unsigned o = __shfl_xor(a, X1);
  a = o > a ? o : a;
  o = __shfl_xor(a, X2);
  return o > a ? o : a;
}

// ---- activations (float32). FAST takes the hardware's exp and reciprocal (1 ulp each) and is
// used for bfloat16 outputs, whose own rounding is up to 2^-8 of the value.

template <bool FAST> __device__ __forceinline__ float ex(float v) {
  return FAST ? __builtin_amdgcn_exp2f(v * 1.44269504088896341f) : expf(v);
}
template <bool FAST> __device__ __forceinline__ float inv1(float v) {
  return FAST ? __builtin_amdgcn_rcpf(v) : 1.0f / v;
}

// Phi(z), the normal distribution function; `e` receives exp(-z^2 / 2). FAST: Phi(-x) =
// t (c1 + t (c2 + ...)) exp(-x^2 / 2) with t = 1 / (1 + p x), x >= 0, p and the six coefficients
// fitted to the least largest error up to x = 13.2, where the exponential leaves float's normal
// range: evaluated in float32 it is within 2.6e-7, and within 2.1e-5 of the value, so that GELU is
// rounded once in its tail too. (A fit of the absolute error alone is off by 0.4% of the value at
// z = -6 and by 3% at -12.)
template <bool FAST> __device__ __forceinline__ float phi(float z, float& e) {
  e = ex<FAST>(-0.5f * z * z);
  if constexpr (!FAST) {
    return 0.5f * erfcf(-z * 0.70710678118654752f);
  } else {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.2972787f, fabsf(z), 1.0f));
    float p = fmaf(-0.08200984f, t, 0.23852773f);
    p = fmaf(p, t, -0.040558513f);
    p = fmaf(p, t, 0.15472628f);
    p = fmaf(p, t, 0.1101131f);
    p = fmaf(p, t, 0.11920107f);
    const float low = p * t * e;  // Phi(-|z|)
    return z < 0.0f ? low : 1.0f - low;
  }
}

constexpr float GT_C = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float GT_A = 0.044715f;

template <int ACT, bool FAST> __device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays
  if constexpr (ACT == ACT_GELU) {
    float e;
    return z * phi<FAST>(z, e);
  }
  if constexpr (ACT == ACT_GELU_TANH) {  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
    const float u2 = z * fmaf(2.0f * GT_C * GT_A, z * z, 2.0f * GT_C);
    return z * inv1<FAST>(1.0f + ex<FAST>(-u2));
  }
  if constexpr (ACT == ACT_SILU) return z * inv1<FAST>(1.0f + ex<FAST>(-z));
  return z;
}

template <int ACT, bool FAST> __device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);  // a NaN stays
  if constexpr (ACT == ACT_GELU) {
    float e;
    const float p = phi<FAST>(z, e);
    return e == 0.0f ? p : fmaf(z * 0.39894228040143268f, e, p);  // (an infinite z: no inf * 0)
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    const float z2 = z * z;
    const float s = inv1<FAST>(1.0f + ex<FAST>(-2.0f * GT_C * z * fmaf(GT_A, z2, 1.0f)));
    const float r = s * (1.0f - s);  // 0 where the slope has settled (there z2 may overflow)
    return r == 0.0f ? s : fmaf(z * r, 2.0f * GT_C * fmaf(3.0f * GT_A, z2, 1.0f), s);
  }
  if constexpr (ACT == ACT_SILU) {
    const float s = inv1<FAST>(1.0f + ex<FAST>(-z));
    const float r = s * (1.0f - s);
    return r == 0.0f ? s : fmaf(z, r, s);
  }
  return 1.0f;
}

template <bool FAST, int NB> __device__ __forceinline__ void act_fwd_all(int act, float (&v)[NB][8]) {
#define INSTANT_ACT(A)                                                                     \
  case A:                                                                                  \
    _Pragma("unroll") for (int k = 0; k < NB; ++k)                                         \
        _Pragma("unroll") for (int j = 0; j < 8; ++j) v[k][j] = act_fwd<A, FAST>(v[k][j]); \
    break;
  switch (act) {
    INSTANT_ACT(ACT_RELU)
    INSTANT_ACT(ACT_GELU)
    INSTANT_ACT(ACT_GELU_TANH)
    INSTANT_ACT(ACT_SILU)
  }
#undef INSTANT_ACT
}

// ---- vectors of 8 elements

template <class T> __device__ __forceinline__ void load8(const T* p, float v[8]) {
  const typename MM<T>::vec8 r = *reinterpret_cast<const typename MM<T>::vec8*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)r[j];
}

// ---- the forward's epilogue: y = act(z + bias) + res, with z or its checkpoint kept
struct Epi {
  const void* bias;  // [N] or null
  const void* res;   // [M][N] or null
  void* y;           // [M][N]
  void* z;           // [M][N] or null
  Ckpt zc;           // or q null
  int act;
};

template <class T> __device__ __forceinline__ void load_bias(const Epi& ep, int n, int N, float b[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = 0.0f;
  if (ep.bias && n < N) load8((const T*)ep.bias + n, b);
}

// The eight consecutive columns n .. n+7 (n % 8 == 0) of rows m, m + step, ... (NB of them, each
// `in` the output or not; `all` when the compiler may take every lane's as in, which a whole tile
// of the output says): their bias (zeros without one), their residuals r (anything without) and
// their sums v, which are used up. The four lanes that differ in lane-id bits X1, X2 hold the
// 32-column group of n and must all call.
template <class T, int NB, int X1, int X2>
__device__ __forceinline__ void epilogue(const Epi& ep, const float bias[8], const typename MM<T>::vec8 (&r)[NB],
                                         float (&v)[NB][8], int m, int step, int n, int N, const bool (&in)[NB],
                                         bool all) {
  constexpr bool FAST = sizeof(T) == 2;
  const size_t at = (size_t)m * N + n, down = (size_t)step * N;
  auto store = [&](T* p) {
    if (all) {
#pragma unroll
      for (int k = 0; k < NB; ++k) store_row<T, 8>(p + k * down, v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (in[k]) store_row<T, 8>(p + k * down, v[k]);
    }
  };
  if (ep.bias) {
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] += bias[j];
  }
  if (ep.zc.q) {
    const size_t G = ck_groups(N), g = (size_t)m * G + n / CK_GROUP;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const unsigned byte = ck_scale_byte(ck_group_amax<X1, X2>(v[k], in[k]));
      if (in[k]) {
        *reinterpret_cast<uint2*>(ep.zc.q + at + k * down) = ck_quant8(v[k], byte);
        if (n % CK_GROUP == 0) ep.zc.scale[g + k * step * G] = (uint8_t)byte;
      }
    }
  } else if (ep.z) {
    store((T*)ep.z + at);
  }
  act_fwd_all<FAST, NB>(ep.act, v);
  if (ep.res) {
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] += (float)r[k][j];
  }
  store((T*)ep.y + at);
}

// One row of it.
template <class T, int X1, int X2>
__device__ __forceinline__ void epilogue8(const Epi& ep, float (&v)[8], int m, int n, int N, bool in) {
  float bias[8], w[1][8];
  typename MM<T>::vec8 r[1];
  r[0] = zero_vec8<T>();
  load_bias<T>(ep, n, N, bias);
  if (in && ep.res) r[0] = *reinterpret_cast<const typename MM<T>::vec8*>((const T*)ep.res + (size_t)m * N + n);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[0][j] = v[j];
  const bool ok[1] = {in};
  epilogue<T, 1, X1, X2>(ep, bias, r, w, m, 0, n, N, ok, false);
}

// ---- host launchers (each returns the launch status; pointers are device pointers)

hipError_t launch_ckpt_pack(bool bf16_io, const void* x, int M, int C, Ckpt c, hipStream_t st);
hipError_t launch_ckpt_unpack(bool bf16_io, Ckpt c, int M, int C, void* x, hipStream_t st);

// The three products of a layer with x [M][K], w [N][K], gz [M][N].
enum class Prod { Fwd, Gx, Gw };
// Floats of workspace one product needs (gw: with x as a checkpoint or in full).
size_t linear_part_floats(bool bf16_io, Prod p, int M, int N, int K, bool x_ckpt);
// Fwd: ep given. Gx: out [M][K]. Gw: out [N][K], x in full or (xc.q) as a checkpoint.
hipError_t launch_linear_fwd(bool bf16_io, const void* x, const void* w, int M, int N, int K, const Epi& ep,
                             float* part, hipStream_t st);
hipError_t launch_linear_gx(bool bf16_io, const void* gz, const void* w, int M, int N, int K, void* gx, float* part,
                            hipStream_t st);
hipError_t launch_linear_gw(bool bf16_io, const void* gz, const void* x, Ckpt xc, int M, int N, int K, void* gw,
                            float* part, hipStream_t st);

size_t act_bwd_part_floats(int M, int N);
hipError_t launch_act_bwd(bool bf16_io, const void* gy, const void* z, Ckpt zc, int M, int N, int act, void* gz,
                          void* gb, float* part, hipStream_t st);

// out[c] = sum over the S rows of part [S][N], in a fixed order (S = 0: zeros).
hipError_t launch_column_sum(bool bf16_io, const float* part, int S, int N, void* out, hipStream_t st);

constexpr int NORM_MAX_C = 65536;
hipError_t launch_rmsnorm_fwd(bool bf16_io, const void* x, const void* res, const void* g, int M, int C, float eps,
                              void* h, void* y, Ckpt yc, float* rstd, hipStream_t st);
size_t rmsnorm_part_floats(int M, int C);
hipError_t launch_rmsnorm_bwd(bool bf16_io, const void* gy, const void* h, const void* g, const float* rstd,
                              const void* gh, int M, int C, void* gx, void* gg, float* part, hipStream_t st);

}  // namespace instant

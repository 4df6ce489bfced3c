// Activation checkpoints in 8 bits (format: include/instant_ops.h), and the elementwise half of
// a layer's backward that reads them: gz = gy * act'(z) with the bias gradient.
#include <algorithm>

#include "ops.hpp"

namespace instant {

// A thread takes 8 channels, four neighbouring lanes a group of 32; u = 4 * groups units a row.
// FLAT (C % 32 == 0): the groups are contiguous in memory and need no row.
template <class T, bool FLAT>
__global__ __launch_bounds__(256) void ckpt_pack_kernel(const T* __restrict__ x, int C, size_t units, Ckpt c) {
  const int u = ck_groups(C) * 4;
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < units; e += (size_t)gridDim.x * 256) {
    size_t at = e * 8;
    bool in = true;
    if constexpr (!FLAT) {
      const size_t m = e / u;
      const int n = (int)(e % u) * 8;
      in = n < C;
      at = m * C + n;
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (in) load8(x + at, v);
    const unsigned byte = ck_scale_byte(ck_group_amax<1, 2>(v, in));
    if (in) *reinterpret_cast<uint2*>(c.q + at) = ck_quant8(v, byte);
    if (e % 4 == 0) c.scale[e / 4] = (uint8_t)byte;
  }
}

template <class T, bool FLAT>
__global__ __launch_bounds__(256) void ckpt_unpack_kernel(Ckpt c, int C, size_t units, T* __restrict__ x) {
  const int u = ck_groups(C) * 4;
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < units; e += (size_t)gridDim.x * 256) {
    size_t at = e * 8;
    if constexpr (!FLAT) {
      const size_t m = e / u;
      const int n = (int)(e % u) * 8;
      if (n >= C) continue;
      at = m * C + n;
    }
    float v[8];
    ck_dequant8(*reinterpret_cast<const uint2*>(c.q + at), c.scale[e / 4], v);
    store_row<T, 8>(x + at, v);
  }
}

namespace {
unsigned stream_grid(size_t units) { return (unsigned)std::min<size_t>((units + 255) / 256, 16384); }
}  // namespace

hipError_t launch_ckpt_pack(bool bf16_io, const void* x, int M, int C, Ckpt c, hipStream_t st) {
  const size_t units = (size_t)M * ck_groups(C) * 4;
#define PACK(T, F) \
  hipLaunchKernelGGL((ckpt_pack_kernel<T, F>), dim3(stream_grid(units)), dim3(256), 0, st, (const T*)x, C, units, c)
  if (C % CK_GROUP == 0) {
    if (bf16_io) PACK(bf16, true);
    else PACK(float, true);
  } else {
    if (bf16_io) PACK(bf16, false);
    else PACK(float, false);
  }
#undef PACK
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack(bool bf16_io, Ckpt c, int M, int C, void* x, hipStream_t st) {
  const size_t units = (size_t)M * ck_groups(C) * 4;
#define UNPACK(T, F) \
  hipLaunchKernelGGL((ckpt_unpack_kernel<T, F>), dim3(stream_grid(units)), dim3(256), 0, st, c, C, units, (T*)x)
  if (C % CK_GROUP == 0) {
    if (bf16_io) UNPACK(bf16, true);
    else UNPACK(float, true);
  } else {
    if (bf16_io) UNPACK(bf16, false);
    else UNPACK(float, false);
  }
#undef UNPACK
  return hipGetLastError();
}

// ---- gz = gy * act'(z), gb = sum_m gz
//
// A block takes 256 columns (32 threads of 8) of a strip of rows (8 threads deep); the strip's
// column sums are reduced over the 8 in LDS and left as part[strip][N], which the column sum adds
// in a fixed order. Up to 128 rows there is one strip, and its sums are gb (a second launch costs
// the host 4 us, a thread's 16 rows less). gz is summed before its rounding.
//
// gz is rounded to the I/O type, like the gradient an unfused activation would hand on: in bfloat16
// it is the operand that the matrix cores take in both products. Held in float32 it would need two
// bfloat16 operands (twice the products: 2400 of 2540 us of 16384 x 4096 -> 11008) and twice its
// bytes. It costs g_x and g_w one rounding of up to 2^-8 more: 2.3e-3 off 64 bits (root mean square)
// where the output's own rounding leaves 1.7e-3. In float32 there is nothing to choose.

namespace {
constexpr int AB_COLS = 256, AB_DEEP = 8;

int act_strips(int M, int N) {
  if (M <= 128) return 1;
  const int cb = (N + AB_COLS - 1) / AB_COLS;
  int strips = std::min(256, std::max(1, 2048 / cb));
  return std::max(1, std::min(strips, (M + AB_DEEP - 1) / AB_DEEP));
}
}  // namespace

template <class T, int ACT, bool Q8>
__global__ __launch_bounds__(256) void act_bwd_kernel(const T* gy, const T* z, Ckpt zc, int M, int N, T* gz,
                                                      T* __restrict__ gb, float* __restrict__ part) {
  constexpr bool FAST = sizeof(T) == 2;
  __shared__ float sums[AB_DEEP][AB_COLS + 4];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = blockIdx.x * AB_COLS + 8 * cx;
  const int strips = gridDim.y, s = blockIdx.y;
  const int r0 = (int)((long)M * s / strips), r1 = (int)((long)M * (s + 1) / strips);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  if (n < N) {
    for (int m = r0 + ry; m < r1; m += AB_DEEP) {
      const size_t at = (size_t)m * N + n;
      float g[8];
      load8(gy + at, g);
      if constexpr (ACT != ACT_NONE) {
        float v[8];
        if constexpr (Q8) {
          ck_dequant8(*reinterpret_cast<const uint2*>(zc.q + at), zc.scale[(size_t)m * ck_groups(N) + n / CK_GROUP],
                      v);
        } else {
          load8(z + at, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= act_slope<ACT, FAST>(v[j]);
      }
      if (gz) store_row<T, 8>(gz + at, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
    }
  }
  if (!gb) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[ry][8 * cx + j] = sum[j];
  __syncthreads();
  const int c = blockIdx.x * AB_COLS + threadIdx.x;
  if (c < N) {
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < AB_DEEP; ++r) v += sums[r][threadIdx.x];
    if (strips == 1) gb[c] = from_f32<T>(v);
    else part[(size_t)s * N + c] = v;
  }
}

// out[c] = sum over S rows of part [S][N]: 32 columns a block, the rows dealt to 32 threads each
// (many loads in flight: the sum is bound by latency), whose sums are added in order. S = 0
// writes zeros.
template <class T>
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part, int S, int N,
                                                          T* __restrict__ out) {
  __shared__ float sums[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float v = 0.0f;
  if (c < N) {
#pragma unroll 4
    for (int s = ry; s < S; s += 32) v += part[(size_t)s * N + c];
  }
  sums[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && c < N) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += sums[r][cx];
    out[c] = from_f32<T>(t);
  }
}

hipError_t launch_column_sum(bool bf16_io, const float* part, int S, int N, void* out, hipStream_t st) {
  const dim3 grid((N + 31) / 32);
  if (bf16_io)
    hipLaunchKernelGGL(column_sum_kernel<bf16>, grid, dim3(1024), 0, st, part, S, N, (bf16*)out);
  else
    hipLaunchKernelGGL(column_sum_kernel<float>, grid, dim3(1024), 0, st, part, S, N, (float*)out);
  return hipGetLastError();
}

size_t act_bwd_part_floats(int M, int N) { const int S = M ? act_strips(M, N) : 0;
  return S > 1 ? (size_t)S * N : 0; }

hipError_t launch_act_bwd(bool bf16_io, const void* gy, const void* z, Ckpt zc, int M, int N, int act, void* gz,
                          void* gb, float* part, hipStream_t st) {
  const int S = M ? act_strips(M, N) : 0;
  if (M) {
    const dim3 grid((N + AB_COLS - 1) / AB_COLS, S);
#define ACTB(T, A, Q)                                                                                             \
  hipLaunchKernelGGL((act_bwd_kernel<T, A, Q>), grid, dim3(256), 0, st, (const T*)gy, (const T*)z, zc, M, N, (T*)gz, \
                     (T*)gb, part)
#define ACTB_Q(T, A)      \
  case A:                 \
    if (zc.q) ACTB(T, A, true); \
    else ACTB(T, A, false);     \
    break;
#define ACTB_T(T)                                         \
  switch (act) {                                          \
    case ACT_NONE: ACTB(T, ACT_NONE, false); break;       \
    ACTB_Q(T, ACT_RELU)                                   \
    ACTB_Q(T, ACT_GELU)                                   \
    ACTB_Q(T, ACT_GELU_TANH)                              \
    ACTB_Q(T, ACT_SILU)                                   \
  }
    if (bf16_io) { ACTB_T(bf16) }
    else { ACTB_T(float) }
#undef ACTB_T
#undef ACTB_Q
#undef ACTB
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return gb && S != 1 ? launch_column_sum(bf16_io, part, S, N, gb, st) : hipSuccess;
}

}  // namespace instant

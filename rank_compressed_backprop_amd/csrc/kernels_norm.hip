// RMS norm with the residual's addition and an output in 8 bits, and its gradients
// (include/instant_ops.h):
//   h = x + r;  rstd = (mean h^2 + eps)^-1/2;  y = h rstd g
//   gx = rstd (u - h rstd^2 mean(u h)) + gh, u = gy g;  gg = sum_m gy h rstd
//
// Both are one pass over memory: a row stays in its threads' registers between its statistic
// and its outputs (the gradients' rows of more than 16384 channels are read a second time: with
// their sums and two operands they do not fit). A row of up to 2048 channels belongs to one wave
// (no barrier), a longer one to a block. The checkpoint is taken from the rounded y, so it is what packing y would give.
#include <algorithm>

#include "ops.hpp"

namespace instant {

namespace {

// Sum over the TPR threads of a row (every thread receives it; a fixed order).
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (TPR > WAVE) {
    constexpr int W = TPR / WAVE;
    __syncthreads();  // the last sum's readers are done
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += lds[i];
  }
  return v;
}

template <class T> using vec8_t = typename MM<T>::vec8;

}  // namespace

// TPR threads a row (64: four rows a block of 256; else the block), NV units of 8 channels a
// thread: unit i * TPR + t.
template <class T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_fwd_kernel(const T* x, const T* res,
                                                                          const T* __restrict__ g, int M, int C,
                                                                          float eps, T* h, T* __restrict__ y, Ckpt yc,
                                                                          float* __restrict__ rstd_out) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float lds[TPR > WAVE ? TPR / WAVE : 1];
  const int t = threadIdx.x % TPR;
  for (int m = blockIdx.x * RPB + threadIdx.x / TPR; m < M; m += gridDim.x * RPB) {
    const size_t row = (size_t)m * C;
    vec8_t<T> v[NV];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = 8 * (i * TPR + t);
      v[i] = zero_vec8<T>();
      if (n < C) v[i] = *reinterpret_cast<const vec8_t<T>*>(x + row + n);
    }
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = 8 * (i * TPR + t);
        if (n < C) {
          const vec8_t<T> r = *reinterpret_cast<const vec8_t<T>*>(res + row + n);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = from_f32<T>((float)v[i][j] + (float)r[j]);
          *reinterpret_cast<vec8_t<T>*>(h + row + n) = v[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf((float)v[i][j], (float)v[i][j], ss);
    ss = row_sum<TPR>(ss, lds);
    const float rstd = 1.0f / sqrtf(ss / (float)C + eps);
    if (rstd_out && t == 0) rstd_out[m] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = 8 * (i * TPR + t);
      const bool in = n < C;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      if (in) {
        float w[8];
        load8(g + n, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (float)from_f32<T>((float)v[i][j] * rstd * w[j]);
        if (y) store_row<T, 8>(y + row + n, o);
      }
      if (yc.q) {
        const unsigned byte = ck_scale_byte(ck_group_amax<1, 2>(o, in));
        if (in) {
          *reinterpret_cast<uint2*>(yc.q + row + n) = ck_quant8(o, byte);
          if (n % CK_GROUP == 0) yc.scale[(size_t)m * ck_groups(C) + n / CK_GROUP] = (uint8_t)byte;
        }
      }
    }
  }
}

// Rows are dealt to the blocks in turn; a thread keeps its channels' gg sums over its rows, and
// every row slot leaves one partial row: part [slots][C], added in slot order by the column sum.
// HOLD: the row's gy and h stay in registers; else they are read again (long rows).
template <class T, int TPR, int NV, bool HOLD>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_bwd_kernel(
    const T* gy, const T* __restrict__ h, const T* __restrict__ g, const float* __restrict__ rstd, const T* gh, int M,
    int C, T* gx, float* __restrict__ part) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float lds[TPR > WAVE ? TPR / WAVE : 1];
  const int t = threadIdx.x % TPR;
  const int slot = blockIdx.x * RPB + threadIdx.x / TPR, slots = gridDim.x * RPB;
  float gg[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) gg[i][j] = 0.0f;
  vec8_t<T> w[HOLD ? NV : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = 8 * (i * TPR + t);
      w[i] = zero_vec8<T>();
      if (n < C) w[i] = *reinterpret_cast<const vec8_t<T>*>(g + n);
    }
  }
  // the trip count is the block's (a block-wide row sum has barriers; with TPR = 64 it has none)
  for (int m = slot; m < M; m += slots) {
    const size_t row = (size_t)m * C;
    const float rs = rstd[m];
    vec8_t<T> a[HOLD ? NV : 1], b[HOLD ? NV : 1];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = 8 * (i * TPR + t);
      const int k = HOLD ? i : 0;
      a[k] = b[k] = zero_vec8<T>();
      if (!HOLD) w[0] = zero_vec8<T>();
      if (n < C) {
        a[k] = *reinterpret_cast<const vec8_t<T>*>(gy + row + n);
        b[k] = *reinterpret_cast<const vec8_t<T>*>(h + row + n);
        if (!HOLD) w[0] = *reinterpret_cast<const vec8_t<T>*>(g + n);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = (float)a[k][j] * (float)b[k][j];
        dot = fmaf(q, (float)w[k][j], dot);
        gg[i][j] = fmaf(q, rs, gg[i][j]);
      }
    }
    dot = row_sum<TPR>(dot, lds);
    const float c = dot / (float)C * rs * rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = 8 * (i * TPR + t);
      if (n >= C) continue;
      const int k = HOLD ? i : 0;
      if constexpr (!HOLD) {
        a[0] = *reinterpret_cast<const vec8_t<T>*>(gy + row + n);
        b[0] = *reinterpret_cast<const vec8_t<T>*>(h + row + n);
        w[0] = *reinterpret_cast<const vec8_t<T>*>(g + n);
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rs * ((float)a[k][j] * (float)w[k][j] - (float)b[k][j] * c);
      if (gh) {
        float e[8];
        load8(gh + row + n, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += e[j];
      }
      store_row<T, 8>(gx + row + n, o);
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int n = 8 * (i * TPR + t);
    if (n < C) store_row<float, 8>(part + (size_t)slot * C + n, gg[i]);
  }
}

namespace {

// threads a row, units of 8 channels a thread
struct Shape {
  int tpr, nv;
};
Shape shape_of(int C) {
  const int u = ck_groups(C) * 4;
  const int tpr = u <= 4 * 64 ? 64 : u <= 8 * 256 ? 256 : 1024;
  int nv = 1;
  while (tpr * nv < u) nv *= 2;
  return Shape{tpr, nv};
}

int bwd_slots(int M, int C) {
  const Shape s = shape_of(C);
  const int rpb = s.tpr < 256 ? 256 / s.tpr : 1;
  return std::min((M + rpb - 1) / rpb, s.tpr < 256 ? 256 : 512) * rpb;
}

}  // namespace

// (tpr, nv) pairs that shape_of gives: 64 x 1, 2, 4; 256 x 2, 4, 8; 1024 x 4, 8
#define NORM_SHAPES(CALL)                       \
  if (s.tpr == 64) {                            \
    if (s.nv == 1) CALL(64, 1)                  \
    else if (s.nv == 2) CALL(64, 2)             \
    else CALL(64, 4)                            \
  } else if (s.tpr == 256) {                    \
    if (s.nv == 2) CALL(256, 2)                 \
    else if (s.nv == 4) CALL(256, 4)            \
    else CALL(256, 8)                           \
  } else {                                      \
    if (s.nv == 4) CALL(1024, 4)                \
    else CALL(1024, 8)                          \
  }

template <class T>
static hipError_t norm_fwd(const void* x, const void* res, const void* g, int M, int C, float eps, void* h, void* y,
                           Ckpt yc, float* rstd, hipStream_t st) {
  const Shape s = shape_of(C);
  const int rpb = s.tpr < 256 ? 256 / s.tpr : 1;
  // (a block for every row, up to what a launch takes)
  const dim3 grid(std::min((M + rpb - 1) / rpb, 1 << 20)), block(s.tpr < 256 ? 256 : s.tpr);
#define FWD(TPR, NV)                                                                                            \
  hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, TPR, NV>), grid, block, 0, st, (const T*)x, (const T*)res, (const T*)g, \
                     M, C, eps, (T*)h, (T*)y, yc, rstd);
  NORM_SHAPES(FWD)
#undef FWD
  return hipGetLastError();
}

template <class T>
static hipError_t norm_bwd(const void* gy, const void* h, const void* g, const float* rstd, const void* gh, int M,
                           int C, void* gx, float* part, hipStream_t st) {
  const Shape s = shape_of(C);
  const int rpb = s.tpr < 256 ? 256 / s.tpr : 1;
  const dim3 grid(bwd_slots(M, C) / rpb), block(s.tpr < 256 ? 256 : s.tpr);
#define BWD(TPR, NV)                                                                                             \
  hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, TPR, NV, (TPR < 1024)>), grid, block, 0, st, (const T*)gy, (const T*)h, \
                     (const T*)g, rstd, (const T*)gh, M, C, (T*)gx, part);
  NORM_SHAPES(BWD)
#undef BWD
  return hipGetLastError();
}

hipError_t launch_rmsnorm_fwd(bool bf16_io, const void* x, const void* res, const void* g, int M, int C, float eps,
                              void* h, void* y, Ckpt yc, float* rstd, hipStream_t st) {
  return bf16_io ? norm_fwd<bf16>(x, res, g, M, C, eps, h, y, yc, rstd, st)
                 : norm_fwd<float>(x, res, g, M, C, eps, h, y, yc, rstd, st);
}

size_t rmsnorm_part_floats(int M, int C) { return M ? (size_t)bwd_slots(M, C) * C : 0; }

hipError_t launch_rmsnorm_bwd(bool bf16_io, const void* gy, const void* h, const void* g, const float* rstd,
                              const void* gh, int M, int C, void* gx, void* gg, float* part, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (M) {
    float* p = gg ? part : nullptr;
    e = bf16_io ? norm_bwd<bf16>(gy, h, g, rstd, gh, M, C, gx, p, st)
                : norm_bwd<float>(gy, h, g, rstd, gh, M, C, gx, p, st);
  }
  if (e == hipSuccess && gg) e = launch_column_sum(bf16_io, part, M ? bwd_slots(M, C) : 0, C, gg, st);
  return e;
}

}  // namespace instant

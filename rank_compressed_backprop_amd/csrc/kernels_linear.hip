// The three products of a linear layer (include/instant_ops.h) on the tile kernel (tile_kernel.hpp):
// the choice of its tile and split, and the sum of the partials where the contraction is split.
#include <algorithm>

#include "launch.hpp"
#include "ops.hpp"
#include "tile.hpp"

namespace instant {

// out = epilogue(sum_{z < S} part[z][m][n]), slices in order (the same bits every time); a thread
// takes 8 columns, four neighbouring threads a group of 32.
template <class T>
__global__ __launch_bounds__(256) void part_sum_kernel(const float* __restrict__ part, int S, int M, int N, Epi ep) {
  const int u = ck_groups(N) * 4;
  const size_t all = (size_t)M * u, slice = (size_t)M * N;
  // all is a multiple of 4, and so is the stride: the lanes of a group stay together
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < all; e += (size_t)gridDim.x * 256) {
    const int m = (int)(e / u), n = (int)(e % u) * 8;
    const bool in = n < N;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (in) {
      const float* p = part + (size_t)m * N + n;
      load8(p, v);
#pragma unroll 4
      for (int z = 1; z < S; ++z) {
        float w[8];
        load8(p + z * slice, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += w[j];
      }
    }
    epilogue8<T, 1, 2>(ep, v, m, n, N, in);
  }
}

namespace {

template <class T>
hipError_t sum_parts(const Plan& p, const float* part, int M, int N, const Epi& ep, hipStream_t st) {
  const size_t units = (size_t)M * ck_groups(N) * 4;
  hipLaunchKernelGGL((part_sum_kernel<T>), dim3((unsigned)std::min<size_t>((units + 255) / 256, 4096)), dim3(256), 0,
                     st, part, p.S, M, N, ep);
  return hipGetLastError();
}

template <class T>
hipError_t run(TileLaunch launch, const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
               float* part, hipStream_t st) {
  const Plan p = plan(sizeof(T) == 2, M, N, K, ep.act != ACT_NONE || ep.zc.q);
  if (p.part && !part) return hipErrorInvalidValue;
  const hipError_t e = launch(p, A, lda, M, B, ldb, N, K, ep, part, st);
  return e == hipSuccess && p.part ? sum_parts<T>(p, part, M, N, ep, st) : e;
}

Epi plain_out(void* out) { return Epi{nullptr, nullptr, out, nullptr, Ckpt{nullptr, nullptr}, ACT_NONE}; }

// A checkpoint of x is unpacked for gw, `chunk` rows at a time: up to 256 MB of copy. (Unpacking
// costs 3% of the product it precedes at 16384 x 4096; dequantising inside the product would
// repeat it for every 256 columns of gz.) More than one chunk adds up in the partials.
constexpr size_t UNPACKED_BYTES = (size_t)256 << 20;
int chunk_rows(bool bf16_io, int M, int K) {
  const size_t rows = UNPACKED_BYTES / ((size_t)K * (bf16_io ? 2 : 4)) / 64 * 64;
  return (int)std::min<size_t>(M, std::max<size_t>(rows, 64));
}
size_t unpacked_floats(bool bf16_io, int rows, int K) {
  return ((size_t)rows * K * (bf16_io ? 2 : 4) + 255) / 256 * 64;
}

template <class T>
hipError_t run_gw8(TileLaunch launch, const T* gz, Ckpt x, int M, int N, int K, const Epi& ep, float* ws,
                   hipStream_t st) {
  constexpr bool BF = sizeof(T) == 2;
  const int rows = chunk_rows(BF, M, K);
  float* part = ws + unpacked_floats(BF, rows, K);
  if (rows == M) {
    const hipError_t e = launch_ckpt_unpack(BF, x, M, K, ws, st);
    return e == hipSuccess ? run<T>(launch, gz, N, N, ws, K, K, M, ep, part, st) : e;
  }
  Plan p = plan(BF, N, K, rows, false);
  const int S = p.S;
  p.part = true;
  for (int m = 0; m < M; m += rows) {
    const int r = std::min(rows, M - m);
    const Ckpt c{x.q + (size_t)m * K, x.scale + (size_t)m * ck_groups(K)};
    hipError_t e = launch_ckpt_unpack(BF, c, r, K, ws, st);
    p.add = m > 0;
    p.S = std::min(S, (r + (BF ? 63 : 31)) / (BF ? 64 : 32));  // every slice of a short last chunk has a stage
    if (e == hipSuccess) e = launch(p, gz + (size_t)m * N, N, N, ws, K, K, r, ep, part, st);
    if (e != hipSuccess) return e;
  }
  p.S = S;
  return sum_parts<T>(p, part, N, K, ep, st);
}

}  // namespace

size_t linear_part_floats(bool bf16_io, Prod p, int M, int N, int K, bool x_ckpt) {
  const int a = p == Prod::Gw ? N : M, b = p == Prod::Fwd ? N : K;
  int k = p == Prod::Fwd ? K : p == Prod::Gx ? N : M;
  if (!a || !k) return 0;
  size_t n = 0;
  bool chunks = false;
  if (p == Prod::Gw && x_ckpt) {
    k = chunk_rows(bf16_io, M, K);
    chunks = k < M;
    n = unpacked_floats(bf16_io, k, K);
  }
  int S = plan(bf16_io, a, b, k, false).S;
  if (p == Prod::Fwd) S = std::max(S, plan(bf16_io, a, b, k, true).S);  // whatever its epilogue
  return n + (S > 1 || chunks ? (size_t)S * a * b : 0);
}

hipError_t launch_linear_fwd(bool bf16_io, const void* x, const void* w, int M, int N, int K, const Epi& ep,
                             float* part, hipStream_t st) {
  return bf16_io ? run<bf16>(launch_tile_bf16_fwd, x, K, M, w, K, N, K, ep, part, st)
                 : run<float>(launch_tile_fp32_fwd, x, K, M, w, K, N, K, ep, part, st);
}

hipError_t launch_linear_gx(bool bf16_io, const void* gz, const void* w, int M, int N, int K, void* gx, float* part,
                            hipStream_t st) {
  return bf16_io ? run<bf16>(launch_tile_bf16_gx, gz, N, M, w, K, K, N, plain_out(gx), part, st)
                 : run<float>(launch_tile_fp32_gx, gz, N, M, w, K, K, N, plain_out(gx), part, st);
}

hipError_t launch_linear_gw(bool bf16_io, const void* gz, const void* x, Ckpt xc, int M, int N, int K, void* gw,
                            float* part, hipStream_t st) {
  if (M == 0) return launch_zero(gw, (size_t)N * K * (bf16_io ? 2 : 4), st);
  const Epi ep = plain_out(gw);
  const TileLaunch launch = bf16_io ? launch_tile_bf16_gw : launch_tile_fp32_gw;
  if (xc.q)
    return bf16_io ? run_gw8<bf16>(launch, (const bf16*)gz, xc, M, N, K, ep, part, st)
                   : run_gw8<float>(launch, (const float*)gz, xc, M, N, K, ep, part, st);
  return bf16_io ? run<bf16>(launch, gz, N, N, x, K, K, M, ep, part, st)
                 : run<float>(launch, gz, N, N, x, K, K, M, ep, part, st);
}

}  // namespace instant

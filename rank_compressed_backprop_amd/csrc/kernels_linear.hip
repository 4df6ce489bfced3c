// The three products of a linear layer y = act(x w^T + b) + r (include/instant_ops.h):
//   fwd  y  [M][N]: A = x  [M][K] (k contiguous), B = w [N][K] (k contiguous)
//   gx   gx [M][K]: A = gz [M][N] (k contiguous), B = w [N][K] (k-major: the contraction is N)
//   gw   gw [N][K]: A = gz [M][N] (k-major: the contraction is M), B = x [M][K] (k-major), or
//                   B = a checkpoint of x in 8 bits, dequantised as it is staged
//
// tile32_kernel serves every case in float32 arithmetic: stages of 16 k are converted to
// float32 on their way into LDS, stored k-major ([k][row], so a lane's matrix-core operand is
// one 4-byte read and neither layout needs a transpose there), and multiplied with
// v_mfma_f32_16x16x4_f32. 128 x 128 block tiles, four waves of 64 x 64.
//
// Orientation: the MFMA computes D[n][m] (the B operand takes the first slot). A lane receives
// D rows 4 q + v (q = lane / 16, v < 4) of column m = lane % 16. With operand row i of tile hh
// (0, 1) of a 32-column pair standing for column 8 (i / 4) + 4 hh + i % 4, those rows of the
// two tiles are the columns 8 q .. 8 q + 7: a lane owns 8 consecutive outputs of a row, and
// the four lanes of equal lane % 16 own a group of 32, which shares a checkpoint's scale.
//
// Split K: with grid.z = S > 1 every slice leaves float32 partials [S][rows][cols]; a second
// launch adds them in slice order (the same bits every time) and applies the epilogue.
#include <algorithm>

#include "ops.hpp"
#include "tile16.hpp"

namespace instant {

namespace {

constexpr int T32 = 128;      // block tile edge
constexpr int K32 = 16;       // k per stage
constexpr int LD32 = 144;     // floats a k row in LDS: the four k rows of an operand read use
                              // different halves of the banks

enum { SRC_ROWK, SRC_KMAJ, SRC_KMAJ_Q8 };  // operand stored [row][k], [k][row], or the latter in 8 bits

struct Operand {
  const void* p;
  const uint8_t* scale;  // SRC_KMAJ_Q8
  int ld;                // elements between stored rows
  int rows;              // extent across the output
};

// This thread's 8 elements of a stage: SRC_ROWK: row r, k = k8 .. k8 + 7; else k row, 8 rows.
template <class T, int SRC>
__device__ __forceinline__ void fetch8(const Operand& op, int row0, int k0, int K, int tid, float v[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if constexpr (SRC == SRC_ROWK) {
    const int r = row0 + (tid & 127), k = k0 + 8 * (tid >> 7);
    if (r < op.rows && k < K) load8((const T*)op.p + (size_t)r * op.ld + k, v);
  } else {
    const int r = row0 + 8 * (tid & 15), k = k0 + (tid >> 4);
    if (r < op.rows && k < K) {
      const size_t at = (size_t)k * op.ld + r;
      if constexpr (SRC == SRC_KMAJ) {
        load8((const T*)op.p + at, v);
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>((const int8_t*)op.p + at);
        ck_dequant8(q, op.scale[(size_t)k * ck_groups(op.ld) + r / CK_GROUP], v);
      }
    }
  }
}

template <int SRC> __device__ __forceinline__ void put8(float (*tile)[LD32], int tid, const float v[8]) {
  if constexpr (SRC == SRC_ROWK) {
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[8 * (tid >> 7) + j][tid & 127] = v[j];
  } else {
    float* d = &tile[tid >> 4][8 * (tid & 15)];
    *reinterpret_cast<f32x4*>(d) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(d + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

}  // namespace

// C[a][b] = sum_k A(a, k) B(b, k) over k slice blockIdx.z. Grid (tiles, 1, S); a.rows, b.rows
// the output's extents, b.rows % 8 == 0. PART: float32 partials, else the epilogue.
template <class T, int ASRC, int BSRC, bool PART>
__global__ __launch_bounds__(256) void tile32_kernel(Operand a, Operand b, int K, Epi ep, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) float sa[2][K32][LD32];
  __shared__ __attribute__((aligned(16))) float sb[2][K32][LD32];
  const int tid = threadIdx.x, lane = tid & (WAVE - 1), wave = tid / WAVE;
  const int mt_all = (a.rows + T32 - 1) / T32, nt_all = (b.rows + T32 - 1) / T32;
  const int t = xcd_unit(blockIdx.x, mt_all * nt_all);
  const int m0 = (t % mt_all) * T32, n0 = (t / mt_all) * T32;
  const int nst = (K + K32 - 1) / K32, S = gridDim.z, z = blockIdx.z;
  const int s0 = (int)((long)nst * z / S), s1 = (int)((long)nst * (z + 1) / S);
  const int wm = wave >> 1, wn = wave & 1, q4 = lane >> 4, l16 = lane & 15;

  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = zero4();

  float va[8], vb[8];
  if (s0 < s1) {
    fetch8<T, ASRC>(a, m0, s0 * K32, K, tid, va);
    fetch8<T, BSRC>(b, n0, s0 * K32, K, tid, vb);
  }
  for (int s = s0; s < s1; ++s) {
    const int cur = (s - s0) & 1;
    put8<ASRC>(sa[cur], tid, va);
    put8<BSRC>(sb[cur], tid, vb);
    if (s + 1 < s1) {  // in flight while this stage is multiplied
      fetch8<T, ASRC>(a, m0, (s + 1) * K32, K, tid, va);
      fetch8<T, BSRC>(b, n0, (s + 1) * K32, K, tid, vb);
    }
    // one barrier a stage: a wave that is ahead writes the other buffer, whose readers
    // passed this barrier's predecessor only after they had read it
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K32; k += 4) {
      float fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[i] = sa[cur][k + q4][64 * wm + 16 * i + l16];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        fb[j] = sb[cur][k + q4][64 * wn + 32 * (j >> 1) + 8 * (l16 >> 2) + 4 * (j & 1) + (l16 & 3)];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 64 * wm + 16 * i + l16;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int n = n0 + 64 * wn + 32 * p + 8 * q4;
      const bool in = m < a.rows && n < b.rows;
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = acc[i][2 * p][j];
        v[4 + j] = acc[i][2 * p + 1][j];
      }
      if constexpr (PART) {
        if (in) store_row<float, 8>(part + ((size_t)z * a.rows + m) * b.rows + n, v);
      } else {
        epilogue8<T, 16, 32>(ep, v, m, n, b.rows, in);
      }
    }
  }
}

// out = epilogue(sum_{z < S} part[z][m][n]), slices in order; a thread takes 8 columns, four
// neighbouring threads a group of 32.
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

// K slices of an output of a x b over K: until the tiles' blocks fill the chip twice, as long
// as a slice keeps 8 stages.
int slices32(int a, int b, int K) {
  const long tiles = (long)((a + T32 - 1) / T32) * ((b + T32 - 1) / T32);
  const int nst = (K + K32 - 1) / K32;
  int S = 1;
  while (tiles * S < 512 && S < 32 && nst / (2 * S) >= 8) S *= 2;
  return S;
}

template <class T>
hipError_t sum_parts(const float* part, int S, int M, int N, const Epi& ep, hipStream_t st) {
  const size_t units = (size_t)M * ck_groups(N) * 4;
  hipLaunchKernelGGL((part_sum_kernel<T>), dim3((unsigned)std::min<size_t>((units + 255) / 256, 4096)), dim3(256), 0,
                     st, part, S, M, N, ep);
  return hipGetLastError();
}

template <class T, int ASRC, int BSRC>
hipError_t run32(const Operand& a, const Operand& b, int K, const Epi& ep, float* part, hipStream_t st) {
  const int S = slices32(a.rows, b.rows, K);
  const unsigned tiles = (unsigned)(((a.rows + T32 - 1) / T32) * ((b.rows + T32 - 1) / T32));
  if (S == 1) {
    hipLaunchKernelGGL((tile32_kernel<T, ASRC, BSRC, false>), dim3(tiles), dim3(256), 0, st, a, b, K, ep, part);
    return hipGetLastError();
  }
  if (!part) return hipErrorInvalidValue;
  hipLaunchKernelGGL((tile32_kernel<T, ASRC, BSRC, true>), dim3(tiles, 1, S), dim3(256), 0, st, a, b, K, ep, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return sum_parts<T>(part, S, a.rows, b.rows, ep, st);
}

// float32 words of the bfloat16 copy that a checkpoint of x is unpacked to for gw; 0 where that
// would take more than 1 GB (the float32-arithmetic kernel then reads the checkpoint itself)
size_t gw_unpacked_floats(int M, int K) {
  const size_t n = ((size_t)M * K / 2 + 63) / 64 * 64;
  return n > ((size_t)1 << 28) ? 0 : n;
}

Epi plain_out(void* out) { return Epi{nullptr, nullptr, out, nullptr, Ckpt{nullptr, nullptr}, ACT_NONE}; }

}  // namespace

namespace {

template <class L>
hipError_t run16(L launch, const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
                 float* part, hipStream_t st) {
  const int S = plan16(M, N, K).S;
  if (S > 1 && !part) return hipErrorInvalidValue;
  const hipError_t e = launch(A, lda, M, B, ldb, N, K, ep, part, st);
  return e == hipSuccess && S > 1 ? sum_parts<bf16>(part, S, M, N, ep, st) : e;
}

}  // namespace

// A product's time by what its blocks cost: a compute unit runs `fit` blocks of a shape at once;
// a block takes at least `lone` us a stage (the latency of its requests), k of them together at
// least k * `each` (the matrix cores and the operands' way to them), and `ends` for its start and
// its epilogue. Split K pays for a second launch and the partials' way to memory and back. The
// figures are fitted to the times of 39 products of 1 to 16384 rows by 10 tile shapes and ring
// depths by 10 splits on gfx950 (13% rms); the shape chosen is within 5% of the best one measured
// in 31 of the 39, at worst 18% off (4.6 against 3.9 us). Examples, best against a fixed 256 x
// 256 tile: 8 x 11008 over 4096 15.0 against 73 us, 768 x 768 over 16384 39.6 against 309 us,
// 512 x 4096 over 1024 8.8 against 31 us.
Plan16 plan16(int M, int N, int K) {
  struct Shape {
    int wm, wn, ns, fit;
    float lone, each, ends;
  };
  static constexpr Shape shapes[] = {
      {8, 8, 2, 1, 1.24f, 1.24f, 8.1f}, {8, 6, 2, 1, 0.91f, 0.87f, 6.3f}, {4, 4, 2, 2, 0.56f, 0.43f, 2.4f},
      {4, 4, 4, 1, 0.42f, 0.25f, 3.5f}, {2, 4, 3, 2, 0.30f, 0.27f, 2.0f}, {2, 4, 2, 3, 0.47f, 0.28f, 1.6f},
      {2, 2, 2, 4, 0.42f, 0.17f, 1.1f}, {2, 2, 4, 2, 0.13f, 0.18f, 1.45f}};
  static constexpr int slices[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int nst = (K + 63) / 64;
  Plan16 best{0, 0, 0, 1};
  float least = 0.0f;
  for (const Shape& s : shapes) {
    const long tiles = (((long)M + 32 * s.wm - 1) / (32 * s.wm)) * (((long)N + 32 * s.wn - 1) / (32 * s.wn));
    for (int S : slices) {
      if (S > 1 && (tiles * S > 2048 || nst < 2 * S)) break;
      const long n = (tiles * S + 255) / 256;  // blocks of the busiest compute unit
      const int nq = (nst + S - 1) / S;
      auto group = [&](int k) { return nq * std::max(s.lone, k * s.each) + s.ends * (0.5f + 0.5f * k); };
      const int rest = (int)(n % s.fit);
      float t = (float)(n / s.fit) * group(s.fit) + (rest ? group(rest) : 0.0f);
      if (S > 1) t += 4.0f + (float)S * M * N * 8.0f / 7.4e6f;
      if (!best.wm || t < least) {
        best = Plan16{s.wm, s.wn, s.ns, S};
        least = t;
      }
    }
  }
  return best;
}

size_t linear_part_floats(bool bf16_io, Prod p, int M, int N, int K) {
  const int a = p == Prod::Gw ? N : M, b = p == Prod::Fwd ? N : K, k = p == Prod::Fwd ? K : p == Prod::Gx ? N : M;
  if (!a || !k) return 0;
  int S = bf16_io ? plan16(a, b, k).S : slices32(a, b, k);
  if (bf16_io && p == Prod::Gw && !gw_unpacked_floats(M, K)) S = std::max(S, slices32(a, b, k));
  return (S > 1 ? (size_t)S * a * b : 0) + (bf16_io && p == Prod::Gw ? gw_unpacked_floats(M, K) : 0);
}

hipError_t launch_linear_fwd(bool bf16_io, const void* x, const void* w, int M, int N, int K, const Epi& ep,
                             float* part, hipStream_t st) {
  if (bf16_io) return run16(launch_tile16_fwd, x, K, M, w, K, N, K, ep, part, st);
  const Operand a{x, nullptr, K, M}, b{w, nullptr, K, N};
  return run32<float, SRC_ROWK, SRC_ROWK>(a, b, K, ep, part, st);
}

hipError_t launch_linear_gx(bool bf16_io, const void* gz, const void* w, int M, int N, int K, void* gx, float* part,
                            hipStream_t st) {
  if (bf16_io) return run16(launch_tile16_gx, gz, N, M, w, K, K, N, plain_out(gx), part, st);
  const Operand a{gz, nullptr, N, M}, b{w, nullptr, K, K};
  return run32<float, SRC_ROWK, SRC_KMAJ>(a, b, N, plain_out(gx), part, st);
}

hipError_t launch_linear_gw(bool bf16_io, const void* gz, const void* x, Ckpt xc, int M, int N, int K, void* gw,
                            float* part, hipStream_t st) {
  const Epi ep = plain_out(gw);
  if (bf16_io && M > 0 && (!xc.q || gw_unpacked_floats(M, K))) {  // (no rows: zeros, from the kernel below)
    if (xc.q) {
      const hipError_t e = launch_ckpt_unpack(true, xc, M, K, part, st);
      if (e != hipSuccess) return e;
      x = part;
      part += gw_unpacked_floats(M, K);
    }
    return run16(launch_tile16_gw, gz, N, N, x, K, K, M, ep, part, st);
  }
  const Operand a{gz, nullptr, N, N}, b{xc.q ? (const void*)xc.q : x, xc.scale, K, K};
  if (bf16_io && xc.q) return run32<bf16, SRC_KMAJ, SRC_KMAJ_Q8>(a, b, M, ep, part, st);
  if (bf16_io) return run32<bf16, SRC_KMAJ, SRC_KMAJ>(a, b, M, ep, part, st);
  if (xc.q) return run32<float, SRC_KMAJ, SRC_KMAJ_Q8>(a, b, M, ep, part, st);
  return run32<float, SRC_KMAJ, SRC_KMAJ>(a, b, M, ep, part, st);
}

}  // namespace instant

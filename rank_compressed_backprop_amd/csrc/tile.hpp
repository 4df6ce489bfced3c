// Host interface of the tile kernel (tile_kernel.hpp), and the order of its blocks.
#pragma once

#include "ops.hpp"
#include "plan.hpp"

namespace instant {

// C(m, n) = sum_k A(m, k) B(n, k) for an M x N output (N % 8 == 0), K >= 1:
//   fwd: A [M][lda], B [N][ldb], K % 8 == 0     gx: A [M][lda], B [K][ldb], K % 8 == 0
//   gw : A [K][lda], B [K][ldb], M % 8 == 0
// Every slice needs a stage of its own: p.S at most the stages of K (128 bytes of k each).
// The epilogue is applied, or (part) float32 partials [S][M][N] go to part.
typedef hipError_t (*TileLaunch)(const Plan& p, const void* A, int lda, int M, const void* B, int ldb, int N, int K,
                                 const Epi& ep, float* part, hipStream_t st);
hipError_t launch_tile_bf16_fwd(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                                hipStream_t);
hipError_t launch_tile_bf16_gx(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                               hipStream_t);
hipError_t launch_tile_bf16_gw(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                               hipStream_t);
hipError_t launch_tile_fp32_fwd(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                                hipStream_t);
hipError_t launch_tile_fp32_gx(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                               hipStream_t);
hipError_t launch_tile_fp32_gw(const Plan&, const void*, int, int, const void*, int, int, int, const Epi&, float*,
                               hipStream_t);

// Tile (tm, tn) of unit t: bands of 8 tile rows, down the band first, so the blocks that run
// together on an XCD (32, consecutive units) share about 8 + 4 operand panels in its L2.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& tm, int& tn) {
  const int band = t / (8 * nt), left = mt - 8 * band, h = left < 8 ? left : 8;
  const int u = t - band * 8 * nt;
  tm = 8 * band + u % h;
  tn = u / h;
}

}  // namespace instant

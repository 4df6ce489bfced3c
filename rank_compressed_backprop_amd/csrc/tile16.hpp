// Host interface of the bfloat16 tile kernel (tile16_kernel.hpp), and the order of its blocks.
#pragma once

#include "ops.hpp"

namespace instant {

// Tile (wm, wn: 16-row tiles of a wave; a block is 32 wm x 32 wn), stages held in LDS and K
// slices of a product.
struct Plan16 {
  int wm, wn, ns, S;
};
Plan16 plan16(int M, int N, int K);

// C(m, n) = sum_k A(m, k) B(n, k) for an M x N output (N % 8 == 0), K >= 1:
//   fwd: A [M][lda], B [N][ldb], K % 8 == 0     gx: A [M][lda], B [K][ldb], K % 8 == 0
//   gw : A [K][lda], B [K][ldb], M % 8 == 0
// With one slice (plan16) the epilogue is applied, else float32 partials [S][M][N] go to part.
hipError_t launch_tile16_fwd(const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
                             float* part, hipStream_t st);
hipError_t launch_tile16_gx(const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
                            float* part, hipStream_t st);
hipError_t launch_tile16_gw(const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
                            float* part, hipStream_t st);

// Tile (tm, tn) of unit t: bands of 8 tile rows, down the band first, so the blocks that run
// together on an XCD (32, consecutive units) share about 8 + 4 operand panels in its L2.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& tm, int& tn) {
  const int band = t / (8 * nt), left = mt - 8 * band, h = left < 8 ? left : 8;
  const int u = t - band * 8 * nt;
  tm = 8 * band + u % h;
  tn = u / h;
}

}  // namespace instant

// The float32 tile kernel (tile_kernel.hpp) for y = x w^T: both operands with k contiguous.
#include "tile_kernel.hpp"

namespace instant {

hipError_t launch_tile_fp32_fwd(const Plan& p, const void* A, int lda, int M, const void* B, int ldb, int N, int K,
                              const Epi& ep, float* part, hipStream_t st) {
  return launch_planned<float, false, false>(p, A, lda, M, B, ldb, N, K, ep, part, st);
}

}  // namespace instant

// The bfloat16 tile kernel (tile16_kernel.hpp) for gx = gz w: A with k contiguous, B k-major.
#include "tile16_kernel.hpp"

namespace instant {

hipError_t launch_tile16_gx(const void* A, int lda, int M, const void* B, int ldb, int N, int K, const Epi& ep,
                             float* part, hipStream_t st) {
  return launch16<false, true>(A, lda, M, B, ldb, N, K, ep, part, st);
}

}  // namespace instant

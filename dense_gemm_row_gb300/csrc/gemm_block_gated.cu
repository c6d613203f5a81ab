// gemm_block_gated.cu -- the 256-row tile kernel of the gated layer with block-scaled
// e4m3 operands (gemm_block_tile.cuh).
#include "gemm_block_tile.cuh"

namespace dgr {

cudaError_t launch_block_gated(const DeviceInfo &dev, int M, int N, int K, const void *A,
                               int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                               cudaStream_t stream) {
  return launch_block_form<256, true>(dev, M, N, K, A, lda, B, ldb, epi, stream);
}

}  // namespace dgr

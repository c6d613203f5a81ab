// gemm_block.cu -- the 256-row tile kernel of the block-scaled e4m3 product
// (gemm_block_tile.cuh).
#include "gemm_block_tile.cuh"

namespace dgr {

cudaError_t launch_block_fwd(const DeviceInfo &dev, int tile_n, int M, int N, int K, const void *A,
                             int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                             cudaStream_t stream) {
  return tile_n == 256
             ? launch_block_form<256, false>(dev, M, N, K, A, lda, B, ldb, epi, stream)
             : launch_block_form<128, false>(dev, M, N, K, A, lda, B, ldb, epi, stream);
}

}  // namespace dgr

// gemm_block_split.cu -- the few-rows kernel of the block-scaled e4m3 product, plain and
// gated (gemm_epi_split.cuh).
#include "gemm_epi_split.cuh"

namespace dgr {

cudaError_t launch_block_split(const DeviceInfo &dev, int mp, int M, int N, int K, const void *A,
                               int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                               cudaStream_t stream) {
  return epi.gated ? launch_split<true, false, true, true>(dev, mp, true, M, N, K, A, lda, B, ldb,
                                                           epi, nullptr, stream)
                   : launch_split<true, false, false, true>(dev, mp, true, M, N, K, A, lda, B, ldb,
                                                            epi, nullptr, stream);
}

}  // namespace dgr

// gemm_epi_grad.cu -- the 256-row tile kernel with the gradient epilogue
// (gemm_epi_tile.cuh).
#include "gemm_epi_tile.cuh"

namespace dgr {

cudaError_t launch_epi_grad(const DeviceInfo &dev, int tile_n, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, float *part, cudaStream_t stream) {
  return tile_n == 256 ? launch_epi_tile<false, 256, true>(dev, a_t, b_t, M, N, K, A, lda, B, ldb,
                                                           epi, part, stream)
                       : launch_epi_tile<false, 128, true>(dev, a_t, b_t, M, N, K, A, lda, B, ldb,
                                                           epi, part, stream);
}

}  // namespace dgr

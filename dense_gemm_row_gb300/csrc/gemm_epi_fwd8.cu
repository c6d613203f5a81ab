// gemm_epi_fwd8.cu -- the 256-row tile kernel for e4m3 operands, forward
// epilogue (gemm_epi_tile.cuh).
#include "gemm_epi_tile.cuh"

namespace dgr {

cudaError_t launch_epi_fwd8(const DeviceInfo &dev, int tile_n, int M, int N, int K, const void *A,
                            int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                            cudaStream_t stream) {
  return tile_n == 256 ? launch_epi_tile<true, 256, false>(dev, false, true, M, N, K, A, lda, B,
                                                           ldb, epi, nullptr, stream)
                       : launch_epi_tile<true, 128, false>(dev, false, true, M, N, K, A, lda, B,
                                                           ldb, epi, nullptr, stream);
}

}  // namespace dgr

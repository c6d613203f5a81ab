// gemm_gated_fwd.cu -- the 256-row tile kernel of the gated layer, 16-bit operands
// (gemm_epi_tile.cuh).
#include "gemm_epi_tile.cuh"

namespace dgr {

cudaError_t launch_gated_fwd(const DeviceInfo &dev, bool a_t, bool b_t, int M, int N, int K,
                             const void *A, int64_t lda, const void *B, int64_t ldb,
                             const EpiCall &epi, cudaStream_t stream) {
  return launch_epi_tile<false, 256, false, true>(dev, a_t, b_t, M, N, K, A, lda, B, ldb, epi,
                                                  nullptr, stream);
}

}  // namespace dgr

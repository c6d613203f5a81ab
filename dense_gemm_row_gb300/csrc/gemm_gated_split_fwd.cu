// gemm_gated_split_fwd.cu -- the few-rows kernel of the gated layer, 16-bit operands
// (gemm_epi_split.cuh).
#include "gemm_epi_split.cuh"

namespace dgr {

cudaError_t launch_gated_split_fwd(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                                  const void *A, int64_t lda, const void *B, int64_t ldb,
                                  const EpiCall &epi, float *part, cudaStream_t stream) {
  return launch_split<false, false, true>(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, part, stream);
}

}  // namespace dgr

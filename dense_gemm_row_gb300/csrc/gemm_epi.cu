// gemm_epi.cu -- dispatch of the product with a fused epilogue, and its form
// without an inner dimension (K == 0).
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "epi.cuh"
#include "launch.h"

namespace dgr {

// The tile kernel's instantiations (gemm_epi_fwd.cu, gemm_epi_fwd8.cu, gemm_epi_grad.cu).
cudaError_t launch_epi_fwd(const DeviceInfo &dev, int tile_n, bool a_t, bool b_t, int M, int N,
                           int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                           const EpiCall &epi, cudaStream_t stream);
cudaError_t launch_epi_fwd8(const DeviceInfo &dev, int tile_n, int M, int N, int K, const void *A,
                            int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                            cudaStream_t stream);
cudaError_t launch_epi_grad(const DeviceInfo &dev, int tile_n, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, float *part, cudaStream_t stream);
// The few-rows kernel's (gemm_epi_split_fwd.cu, _fwd8.cu, _grad.cu); mp: rows per token tile.
cudaError_t launch_split_fwd(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                             const void *A, int64_t lda, const void *B, int64_t ldb,
                             const EpiCall &epi, float *part, cudaStream_t stream);
cudaError_t launch_split_fwd8(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                              const void *A, int64_t lda, const void *B, int64_t ldb,
                              const EpiCall &epi, float *part, cudaStream_t stream);
cudaError_t launch_split_grad(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                              const void *A, int64_t lda, const void *B, int64_t ldb,
                              const EpiCall &epi, float *part, cudaStream_t stream);

namespace {

// K == 0: the product is zero. z = bias, or a gradient of zeros.
template <bool kBf16>
__global__ void epi_empty_kernel(int M, int N, const EpiCall c) {
  const int64_t total = static_cast<int64_t>(M) * N;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / N, j = i - r * N;
    float d = 0.f;
    if (!c.grad) {
      const float z = c.bias ? from16<kBf16>(c.bias[j]) : 0.f;
      if (c.Z) c.Z[r * c.ldz + j] = to16<kBf16>(z);
      with_act(c.act, [&](auto a) { d = act_value<decltype(a)::value>(z); });
      if (c.R) d += from16<kBf16>(c.R[r * c.ldr + j]);
    }
    c.D[r * c.ldd + j] = to16<kBf16>(d);
  }
}

cudaError_t launch_empty(int M, int N, const EpiCall &epi, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(M) * N + 255) / 256, 4096);
  auto kern = epi.bf16 ? epi_empty_kernel<true> : epi_empty_kernel<false>;
  kern<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(M, N, epi);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && epi.dbias != nullptr)
    e = launch_col_sums(epi.bf16, nullptr, 0, N, N, epi.dbias, stream);
  return e;
}

// Rows per token tile of the few-rows kernel, or 0 for the 256-row tiles.
int split_rows(const DeviceInfo &dev, bool a_t, int M, int N, int K) {
  (void)dev, (void)N, (void)K;
  if (a_t || M > 256) return 0;  // its token tiles are K-major
  return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
}

}  // namespace

cudaError_t launch_gemm_epi(const DeviceInfo &dev, bool e4m3, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, cudaStream_t stream) {
  if (K == 0) return launch_empty(M, N, epi, stream);
  const int mp = split_rows(dev, a_t, M, N, K);
  const int tile_n = 256;
  if (!epi.grad) {
    if (e4m3)
      return mp ? launch_split_fwd8(dev, mp, true, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
                : launch_epi_fwd8(dev, tile_n, M, N, K, A, lda, B, ldb, epi, stream);
    return mp ? launch_split_fwd(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
              : launch_epi_fwd(dev, tile_n, a_t, b_t, M, N, K, A, lda, B, ldb, epi, stream);
  }
  // Gradient: partial column sums, one row per token tile or per 32 rows of D.
  const int parts = static_cast<int>((static_cast<int64_t>(M) + (mp ? mp : 32) - 1) / (mp ? mp : 32));
  void *part = nullptr;
  if (epi.dbias != nullptr) {
    cudaMemPool_t pool;
    cudaError_t e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    e = cudaMallocFromPoolAsync(&part, static_cast<size_t>(parts) * N * 4, pool, stream);
    if (e != cudaSuccess) return e;
  }
  float *sums = static_cast<float *>(part);
  cudaError_t e = mp ? launch_split_grad(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, sums, stream)
                     : launch_epi_grad(dev, tile_n, a_t, b_t, M, N, K, A, lda, B, ldb, epi, sums,
                                       stream);
  if (part != nullptr) {
    if (e == cudaSuccess)
      e = launch_col_sums(epi.bf16, sums, parts, N, N, epi.dbias, stream);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace dgr

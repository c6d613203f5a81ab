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

// Which kernel takes a problem. Measured on GB300 (bf16 and e4m3, 32 to 2048 rows,
// N 1024 to 16384, K 512 to 8192; KB = k-blocks of 128 bytes, GPU time in us):
//   256 x 256 tiles   5.2 + waves * KB * 0.28
//   256 x 128 tiles   4.2 + waves * KB * 0.165 (dearer per output, fewer idle SMs)
//   few-rows kernel   up to 64 rows always: 64 x 4096 x 4096 9.9 against 15.2,
//                     64 x 1024 x 512 4.5 against 5.2; up to 128 where D's rows
//                     are not whole 16-byte units, which the tiles' epilogue
//                     writes 2 bytes at a time: 100 x 1023 x 513 6.4 against 7.7;
//                     above, where the 256 x 128 tiles would fill the GPU `idle`
//                     >= 2 times over and leave a long k range to one pair each:
//                     KB >= 16 and KB * idle >= 128 (128 x 1024 x 4096 7.6 against
//                     14.5, 256 x 4096 x 4096 15.1 against 15.8; not
//                     256 x 1024 x 512, 8.4 against 5.6, nor 300 x 95 x 93, 8.1
//                     against 6.4).
struct EpiPlan {
  int split_rows;  // rows per token tile of the few-rows kernel, or 0
  int tile_n;      // columns per tile otherwise
};
EpiPlan plan_epi(const DeviceInfo &dev, bool a_t, int M, int N, int KB, bool ragged) {
  const int64_t pairs = std::max(dev.sm_count / 2, 1);
  const int64_t rows = (static_cast<int64_t>(M) + 255) / 256;
  const int64_t t256 = rows * ((static_cast<int64_t>(N) + 255) / 256);
  const int64_t t128 = rows * ((static_cast<int64_t>(N) + 127) / 128);
  const int64_t idle = pairs / t128;
  EpiPlan plan{0, 256};
  // The few-rows kernel's token tiles are K-major.
  if (!a_t && (M <= (ragged ? 128 : 64) || (idle >= 2 && KB >= 16 && KB * idle >= 128)))
    plan.split_rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const double w256 = static_cast<double>((t256 + pairs - 1) / pairs);
  const double w128 = static_cast<double>((t128 + pairs - 1) / pairs);
  if (4.2 + w128 * KB * 0.165 < 5.2 + w256 * KB * 0.28) plan.tile_n = 128;
  return plan;
}

}  // namespace

cudaError_t launch_gemm_epi(const DeviceInfo &dev, bool e4m3, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, cudaStream_t stream) {
  if (K == 0) return launch_empty(M, N, epi, stream);
  const bool ragged = N % 8 != 0 || epi.ldd % 8 != 0 || reinterpret_cast<uintptr_t>(epi.D) % 16 != 0;
  const EpiPlan plan = plan_epi(dev, a_t, M, N, (K - 1) / (e4m3 ? 128 : 64) + 1, ragged);
  const int mp = plan.split_rows, tile_n = plan.tile_n;
  if (!epi.grad) {
    if (e4m3)
      return mp ? launch_split_fwd8(dev, mp, true, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
                : launch_epi_fwd8(dev, tile_n, M, N, K, A, lda, B, ldb, epi, stream);
    return mp ? launch_split_fwd(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
              : launch_epi_fwd(dev, tile_n, a_t, b_t, M, N, K, A, lda, B, ldb, epi, stream);
  }
  // Gradient: partial column sums, one row per token tile or per 32 rows of D. A
  // single token tile's kernel writes dbias itself.
  if (mp && M <= mp)
    return launch_split_grad(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream);
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

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
// The gated layer's and its gradient's (gemm_gated_*.cu).
cudaError_t launch_gated_fwd(const DeviceInfo &dev, bool a_t, bool b_t, int M, int N, int K,
                             const void *A, int64_t lda, const void *B, int64_t ldb,
                             const EpiCall &epi, cudaStream_t stream);
cudaError_t launch_gated_grad(const DeviceInfo &dev, int tile_n, bool a_t, bool b_t, int M, int N,
                              int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                              const EpiCall &epi, float *part, cudaStream_t stream);
cudaError_t launch_gated_split_fwd(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                                   const void *A, int64_t lda, const void *B, int64_t ldb,
                                   const EpiCall &epi, float *part, cudaStream_t stream);
cudaError_t launch_gated_split_grad(const DeviceInfo &dev, int mp, bool b_t, int M, int N, int K,
                                    const void *A, int64_t lda, const void *B, int64_t ldb,
                                    const EpiCall &epi, float *part, cudaStream_t stream);
// The block-scaled e4m3 product's (gemm_block*.cu).
cudaError_t launch_block_fwd(const DeviceInfo &dev, int tile_n, int M, int N, int K, const void *A,
                             int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                             cudaStream_t stream);
cudaError_t launch_block_gated(const DeviceInfo &dev, int M, int N, int K, const void *A,
                               int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                               cudaStream_t stream);
cudaError_t launch_block_split(const DeviceInfo &dev, int mp, int M, int N, int K, const void *A,
                               int64_t lda, const void *B, int64_t ldb, const EpiCall &epi,
                               cudaStream_t stream);

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
      if (c.gated) {
        const float z2 = c.bias2 ? from16<kBf16>(c.bias2[j]) : 0.f;
        if (c.Z2) c.Z2[r * c.ldz2 + j] = to16<kBf16>(z2);
        d *= z2;
      }
      if (c.R) d += from16<kBf16>(c.R[r * c.ldr + j]);
    }
    c.D[r * c.ldd + j] = to16<kBf16>(d);
    if (c.D2) c.D2[r * c.ldd2 + j] = to16<kBf16>(d);
  }
}

cudaError_t launch_empty(int M, int N, const EpiCall &epi, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(M) * N + 255) / 256, 4096);
  auto kern = epi.bf16 ? epi_empty_kernel<true> : epi_empty_kernel<false>;
  kern<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(M, N, epi);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && (epi.dbias != nullptr || epi.dbias2 != nullptr))
    e = launch_col_sums(epi.bf16, nullptr, 0, N, N, epi.dbias, stream, 0, epi.dbias2);
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
EpiPlan plan_epi(const DeviceInfo &dev, bool a_t, int M, int64_t N, int KB, bool ragged) {
  const int64_t pairs = std::max(dev.sm_count / 2, 1);
  const int64_t rows = (static_cast<int64_t>(M) + 255) / 256;
  const int64_t t256 = rows * ((N + 255) / 256);
  const int64_t t128 = rows * ((N + 127) / 128);
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

// Times of the kernels (us), fitted to measurements: a start, and for each wave of tiles
// a part per k-block and one for its epilogue.
struct WaveCost {
  double start, per_kb, per_wave;
  double of(int64_t waves, int64_t kb) const {
    return start + static_cast<double>(waves) * (static_cast<double>(kb) * per_kb + per_wave);
  }
};
// Waves and k-blocks per CTA of the few-rows kernel, whose launcher cuts k likewise. (76
// clusters of 4 CTAs take two waves on 152 SMs that have two CTAs each: clusters leave a
// few places free.)
double split_cost(const DeviceInfo &dev, int64_t tiles, int KB, const WaveCost &cost) {
  const int64_t slots = 2LL * dev.sm_count;
  int cl = 1;
  while (cl < 8 && tiles * cl * 2 <= slots && cl * 2 <= KB) cl *= 2;
  const int64_t places = cl > 1 ? slots - slots / 16 : slots;
  return cost.of((tiles * cl + places - 1) / places, (KB + cl - 1) / cl);
}
double tile_cost(const DeviceInfo &dev, int M, int N, int width, int KB, const WaveCost &cost) {
  const int64_t pairs = std::max(dev.sm_count / 2, 1);
  const int64_t tiles = (static_cast<int64_t>(M) + 255) / 256 *
                        ((static_cast<int64_t>(N) + width - 1) / width);
  return cost.of((tiles + pairs - 1) / pairs, KB);
}
// The cheapest of 256-row tiles (`best`: their time) and token tiles of the few-rows
// kernel of 16, 32 and 64 rows; cols: columns of D of one of its tiles.
int plan_split(const DeviceInfo &dev, int M, int N, int cols, int KB, double best,
               const WaveCost (&cost)[3]) {
  const int64_t blocks = (static_cast<int64_t>(N) + cols - 1) / cols;
  int rows = 0;
  for (int i = 0; i < 3; ++i) {
    const int64_t tiles = blocks * ((static_cast<int64_t>(M) + (16 << i) - 1) / (16 << i));
    const double t = split_cost(dev, tiles, KB, cost[i]);
    if (t < best) best = t, rows = 16 << i;
    if (M <= (16 << i)) break;
  }
  return rows;
}

// The gated layer and its gradient. Over 150 problems each of 24 to 1500 rows, N 512 to
// 8192, K 512 to 4096 (bf16, B stored N x K, without biases, sums or stored projections) the
// choice is 2.2 % and 1.3 % slower than the best kernel on average, at most 29 % and 18 %,
// where the other products' rule is 19 % and 14 % slower on average; 128-row token tiles
// hardly ever win. For instance 300 x 1000 x 520, gradient: tiles 10.1, 32 rows 8.2; 128 x
// 4096 x 4096: tiles 22.9, 64 rows 14.5; 1000 x 2048 x 512: tiles 8.7, 64 rows 14.9.
EpiPlan plan_gated(const DeviceInfo &dev, bool a_t, bool grad, int M, int N, int KB) {
  static constexpr WaveCost kForward[3] = {{1.5, 0.17, 3.0}, {1.5, 0.192, 3.4}, {1.4, 0.245, 4.6}};
  static constexpr WaveCost kGradient[3] = {{0, 0.18, 4.4}, {0, 0.2, 5.4}, {0, 0.273, 7.3}};
  static constexpr WaveCost kTile = {4.5, 0.266, 1.3};
  static constexpr WaveCost kWide = {3.3, 0.278, 6.4}, kNarrow = {3.3, 0.137, 3.0};
  EpiPlan plan{0, 256};
  if (grad) plan.tile_n = plan_epi(dev, true, M, N, KB, false).tile_n;
  if (a_t) return plan;  // the few-rows kernel's token tiles are K-major
  const bool wide = plan.tile_n == 256;
  const double tiles = grad ? tile_cost(dev, M, N, plan.tile_n, KB, wide ? kWide : kNarrow)
                            : tile_cost(dev, M, N, 128, KB, kTile);
  plan.split_rows = plan_split(dev, M, N, grad ? 128 : 64, KB, tiles, grad ? kGradient : kForward);
  return plan;
}

// The block-scaled e4m3 product, plain and gated: 200 problems each of 16 to 1500 rows, N
// 512 to 16384, K 512 to 16384 (bf16 results, no bias or residual), 1.8 % and 1.9 % slower
// than the best on average, at most 32 % and 38 %. For instance 100 x
// 4096 x 4096: 256-row tiles 12.6 us, token tiles of 64 rows 10.4, of 32 10.7, of 16 12.5;
// 100 x 512 x 4096: 12.3, 7.3, 6.2, 5.4; 1024 x 4096 x 1024: tiles of 256 columns 9.5, of
// 128 11.0.
EpiPlan plan_block(const DeviceInfo &dev, bool gated, int M, int N, int KB) {
  static constexpr WaveCost kPlain[3] = {{0.8, 0.26, 3.3}, {0, 0.353, 4.5}, {-2.7, 0.564, 7.5}};
  static constexpr WaveCost kGated[3] = {{1.1, 0.257, 2.8}, {1.0, 0.349, 3.4}, {-0.1, 0.569, 5.0}};
  EpiPlan plan{0, 256};
  double best;
  if (gated) {
    best = tile_cost(dev, M, N, 128, KB, {3.2, 0.389, 3.2});
  } else {
    best = tile_cost(dev, M, N, 256, KB, {3.5, 0.388, 2.5});
    const double narrow = tile_cost(dev, M, N, 128, KB, {3.5, 0.238, 1.4});
    if (narrow < best) best = narrow, plan.tile_n = 128;
  }
  plan.split_rows = plan_split(dev, M, N, gated ? 64 : 128, KB, best, gated ? kGated : kPlain);
  return plan;
}

}  // namespace

cudaError_t launch_gemm_epi(const DeviceInfo &dev, bool e4m3, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, cudaStream_t stream) {
  if (K == 0) return launch_empty(M, N, epi, stream);
  const bool ragged = N % 8 != 0 || epi.ldd % 8 != 0 || reinterpret_cast<uintptr_t>(epi.D) % 16 != 0;
  if (epi.block) {
    const EpiPlan plan = plan_block(dev, epi.gated, M, N, (K - 1) / 128 + 1);
    if (plan.split_rows)
      return launch_block_split(dev, plan.split_rows, M, N, K, A, lda, B, ldb, epi, stream);
    return epi.gated ? launch_block_gated(dev, M, N, K, A, lda, B, ldb, epi, stream)
                     : launch_block_fwd(dev, plan.tile_n, M, N, K, A, lda, B, ldb, epi, stream);
  }
  const int KB = (K - 1) / (e4m3 ? 128 : 64) + 1;
  const EpiPlan plan = epi.gated ? plan_gated(dev, a_t, epi.grad, M, N, KB)
                                 : plan_epi(dev, a_t, M, N, KB, ragged);
  const int mp = plan.split_rows, tile_n = plan.tile_n;
  if (epi.gated && !epi.grad)
    return mp ? launch_gated_split_fwd(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
              : launch_gated_fwd(dev, a_t, b_t, M, N, K, A, lda, B, ldb, epi, stream);
  if (!epi.grad) {
    if (e4m3)
      return mp ? launch_split_fwd8(dev, mp, true, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
                : launch_epi_fwd8(dev, tile_n, M, N, K, A, lda, B, ldb, epi, stream);
    return mp ? launch_split_fwd(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream)
              : launch_epi_fwd(dev, tile_n, a_t, b_t, M, N, K, A, lda, B, ldb, epi, stream);
  }
  // Gradient: partial column sums, one row per token tile or per 32 rows of D. A
  // single token tile's kernel writes dbias itself.
  auto split = epi.gated ? launch_gated_split_grad : launch_split_grad;
  auto tiles = epi.gated ? launch_gated_grad : launch_epi_grad;
  if (mp && M <= mp)
    return split(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, nullptr, stream);
  const int parts = static_cast<int>((static_cast<int64_t>(M) + (mp ? mp : 32) - 1) / (mp ? mp : 32));
  void *part = nullptr;
  if (epi.dbias != nullptr || epi.dbias2 != nullptr) {
    cudaMemPool_t pool;
    cudaError_t e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    e = cudaMallocFromPoolAsync(&part, static_cast<size_t>(epi.gated ? 2 : 1) * parts * N * 4, pool,
                                stream);
    if (e != cudaSuccess) return e;
  }
  float *sums = static_cast<float *>(part);
  cudaError_t e = mp ? split(dev, mp, b_t, M, N, K, A, lda, B, ldb, epi, sums, stream)
                     : tiles(dev, tile_n, a_t, b_t, M, N, K, A, lda, B, ldb, epi, sums, stream);
  if (part != nullptr) {
    if (e == cudaSuccess)
      e = launch_col_sums(epi.bf16, sums, parts, N, N, epi.dbias, stream,
                          static_cast<int64_t>(parts) * N, epi.dbias2);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace dgr

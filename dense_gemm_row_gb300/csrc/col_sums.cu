// col_sums.cu -- the last step of a column sum: adds the rows of an fp32
// partial-sum matrix and rounds once to 16 bits (bias and gain gradients).
//
// Every producer writes one partial row per block of rows it owns, so the sums
// need no atomics and are the same bits on every run: row slot y of a block
// adds partial rows y, y + 32, ... in order, then the 32 slots are added in
// slot order. Latency is what it costs (a few hundred partial rows at most), so
// a thread's loads are issued together.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

constexpr int kSlots = 32;

// A second sum of the same shape: its partial rows and its result.
struct Second {
  int64_t apart;
  uint16_t *out;
};
struct NoSecond {};

template <bool kBf16, typename Two>
__global__ void __launch_bounds__(32 * kSlots)
    col_sums_kernel(const float *part, int parts, int n, int64_t ld, uint16_t *out, Two two) {
  __shared__ float red[kSlots][32];
  grid_dependency_wait();
  if constexpr (std::is_same_v<Two, Second>)
    if (blockIdx.y != 0) part += two.apart, out = two.out;
  const int j = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (j < n) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += kSlots) s += part[static_cast<int64_t>(p) * ld + j];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && j < n) {
    float t = 0.f;
#pragma unroll
    for (int y = 0; y < kSlots; ++y) t += red[y][threadIdx.x];
    out[j] = to16<kBf16>(t);
  }
}

}  // namespace

cudaError_t launch_col_sums(bool bf16, const float *part, int parts, int n, int64_t ld,
                            uint16_t *out, cudaStream_t stream, int64_t apart, uint16_t *out2) {
  if (out == nullptr) part += apart, out = out2, out2 = nullptr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n - 1) / 32 + 1), out2 ? 2 : 1, 1);
  cfg.blockDim = dim3(32, kSlots, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launch = [&](auto two) {
    using Two = decltype(two);
    return cudaLaunchKernelEx(&cfg,
                              bf16 ? col_sums_kernel<true, Two> : col_sums_kernel<false, Two>,
                              part, parts, n, ld, out, two);
  };
  return out2 ? launch(Second{apart, out2}) : launch(NoSecond());
}

}  // namespace dgr

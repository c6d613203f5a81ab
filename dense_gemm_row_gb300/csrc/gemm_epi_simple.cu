// gemm_epi_simple.cu -- the product with a fused epilogue, one thread per
// output element: the simplest form that is right for every size and type.
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

constexpr int kT = 16;  // tile edge

template <bool kBf16, bool kE4m3>
__device__ __forceinline__ float load_elem(const void *p, int64_t i) {
  if constexpr (kE4m3) {
    __nv_fp8_e4m3 v;
    v.__x = static_cast<const uint8_t *>(p)[i];
    return static_cast<float>(v);
  } else {
    return from16<kBf16>(static_cast<const uint16_t *>(p)[i]);
  }
}

// Element (i, k) of op(A) is at i * a_i + k * a_k, (k, j) of op(B) at k * b_k + j * b_j.
template <bool kBf16, bool kE4m3>
__global__ void __launch_bounds__(kT *kT)
    epi_simple_kernel(int M, int N, int K, const void *A, int64_t a_i, int64_t a_k, const void *B,
                      int64_t b_k, int64_t b_j, EpiCall c, float *part) {
  __shared__ float as[kT][kT + 1], bs[kT][kT + 1];
  grid_dependency_wait();
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int j = blockIdx.x * kT + tx;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.y) * kT; i0 < M;
       i0 += static_cast<int64_t>(gridDim.y) * kT) {
    const int64_t i = i0 + ty;
    float acc = 0.f;
    for (int k0 = 0; k0 < K; k0 += kT) {
      as[ty][tx] = i < M && k0 + tx < K
                       ? load_elem<kBf16, kE4m3>(A, i * a_i + (k0 + tx) * a_k) : 0.f;
      bs[ty][tx] = k0 + ty < K && j < N
                       ? load_elem<kBf16, kE4m3>(B, (k0 + ty) * b_k + j * b_j) : 0.f;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kT; ++k) acc = fmaf(as[ty][k], bs[k][tx], acc);
      __syncthreads();
    }
    float out = 0.f;
    if (i < M && j < N) {
      float z = c.alpha * acc;
      if (c.scale_a) z *= c.scale_a[i];
      if (c.scale_b) z *= c.scale_b[j];
      if (c.bias) z += from16<kBf16>(c.bias[j]);
      const float r = c.R ? from16<kBf16>(c.R[i * c.ldr + j]) : 0.f;
      with_act(c.act, [&](auto a) {
        out = c.grad ? z * act_slope<decltype(a)::value>(r) : act_value<decltype(a)::value>(z);
      });
      if (!c.grad && c.R) out += r;
      if (c.Z) c.Z[i * c.ldz + j] = to16<kBf16>(z);
      c.D[i * c.ldd + j] = to16<kBf16>(out);
    }
    if (part) {  // column sums of this block of rows
      as[ty][tx] = out;
      __syncthreads();
      if (ty == 0 && j < N) {
        float t = 0.f;
        for (int y = 0; y < kT; ++y) t += as[y][tx];
        part[(i0 / kT) * N + j] = t;
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_gemm_epi(const DeviceInfo &dev, bool e4m3, bool a_t, bool b_t, int M, int N,
                            int K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const EpiCall &epi, cudaStream_t stream) {
  const int tiles_m = (M + kT - 1) / kT, tiles_n = (N + kT - 1) / kT;
  float *part = nullptr;
  if (epi.dbias != nullptr) {
    cudaMemPool_t pool;
    cudaError_t e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    void *p = nullptr;
    e = cudaMallocFromPoolAsync(&p, static_cast<size_t>(tiles_m) * N * 4, pool, stream);
    if (e != cudaSuccess) return e;
    part = static_cast<float *>(p);
  }
  auto kern = epi.bf16 ? (e4m3 ? epi_simple_kernel<true, true> : epi_simple_kernel<true, false>)
                       : (e4m3 ? epi_simple_kernel<false, true> : epi_simple_kernel<false, false>);
  const dim3 grid(static_cast<unsigned>(tiles_n),
                  static_cast<unsigned>(tiles_m < 65535 ? tiles_m : 65535));
  kern<<<grid, dim3(kT, kT), 0, stream>>>(M, N, K, A, a_t ? 1 : lda, a_t ? lda : 1, B,
                                          b_t ? 1 : ldb, b_t ? ldb : 1, epi, part);
  cudaError_t e = cudaGetLastError();
  if (part != nullptr) {
    if (e == cudaSuccess) e = launch_col_sums(epi.bf16, part, tiles_m, N, N, epi.dbias, stream);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace dgr

// act_grad.cu -- the gradient at a linear layer's pre-activation when the
// output's gradient is already in memory:
//
//     dZ_ij = dD_ij act'(Z_ij),    dbias_j = sum_i dZ_ij
//
// Bound by memory (2 matrices in, 1 out, nothing used twice) and, for the gelus,
// nearly as much by instructions: about 20 per value with the slopes on packed
// pairs. At 8192 x 4096 (floor 29.7 us): relu 34.4, silu 34.8, gelu_tanh 35.8,
// gelu 38.1 us, 3 us of each the addition of the partial sums. A block owns 256
// columns of a chunk of rows: 32 threads x 8 columns (512 contiguous bytes of a
// row) times 8 rows at a time. Each thread keeps the fp32 sums of its 8 columns
// over its rows (of the unrounded products), the block adds its 8 row slots in
// shared memory in slot order, and writes one partial row; col_sums adds them.
// The chunk count is what fills the GPU once, so the partial rows are about 1 %
// of the traffic at 8192 x 4096.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

constexpr int kCols = 256;  // columns per block
constexpr int kSlots = 8;   // rows at a time
constexpr int kBlocksPerSm = 3;
constexpr int64_t kMaxChunk = 1 << 30;  // rows; its round-up stays in 32 bits
// Row groups loaded together, with a second such set in flight (2-byte loads: one,
// for the registers). Measured at 8192 x 4096, gelu: 1 / 2 / 3 groups 40.1 / 38.1 /
// 48.4 us; 3 blocks per SM against 4: 38.1, 39.7 us.
template <bool kVec>
constexpr int kAheadOf = kVec ? 2 : 1;

// Column of element e of lane x within the block's 256 columns: contiguous
// 8-element groups (kVec), or strided by 32 for matrices whose rows cannot be
// read in 16-byte units.
template <bool kVec>
__device__ __forceinline__ int col_of(int x, int e) {
  return kVec ? 8 * x + e : x + 32 * e;
}

// A thread's 8 values of one row, packed.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int x, int left) {
  uint4 w = make_uint4(0, 0, 0, 0);
  if constexpr (kVec) {
    if (8 * x < left) w = __ldcs(reinterpret_cast<const uint4 *>(p + 8 * x));
  } else {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x + 32 * e < left ? __ldcs(p + x + 32 * e) : 0;
    w = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                   v[6] | (v[7] << 16));
  }
  return w;
}

template <bool kBf16, bool kVec, int kAct>
__device__ __forceinline__ void act_grad_body(int M, int N, const uint16_t *dD, int64_t ldd,
                                              const uint16_t *Z, int64_t ldz, uint16_t *dZ,
                                              int64_t lddz, float *part, int chunk,
                                              float (&red)[kSlots][kCols]) {
  constexpr int kAhead = kAheadOf<kVec>;
  const int x = threadIdx.x, y = threadIdx.y;
  const int c0 = blockIdx.x * kCols, left = N - c0;
  const int64_t r0 = blockIdx.y * static_cast<int64_t>(chunk);
  const int64_t r1 = r0 + chunk < M ? r0 + chunk : M;
  F2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = f2(0.f);
  struct Rows {
    uint4 d[kAhead], z[kAhead];
  };
  auto load = [&](int64_t r, Rows &v) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t row = r + i * kSlots;
      v.d[i] = v.z[i] = make_uint4(0, 0, 0, 0);
      if (row < r1) {
        v.d[i] = load8<kVec>(dD + row * ldd + c0, x, left);
        if constexpr (kAct != kActNone) v.z[i] = load8<kVec>(Z + row * ldz + c0, x, left);
      }
    }
  };
  auto work = [&](int64_t r, const Rows &v) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t row = r + i * kSlots;
      if (row >= r1) break;
      const uint32_t dw[4] = {v.d[i].x, v.d[i].y, v.d[i].z, v.d[i].w};
      const uint32_t zw[4] = {v.z[i].x, v.z[i].y, v.z[i].z, v.z[i].w};
      uint32_t g[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        unpack16<kBf16>(dw[e], a, b);
        F2 out = f2(a, b);
        if constexpr (kAct != kActNone) {
          float za, zb;
          unpack16<kBf16>(zw[e], za, zb);
          out = mul2(out, act_slope2<kAct>(za, zb));
        }
        sum[e] = add2(sum[e], out);
        split(out, a, b);
        g[e] = pack16<kBf16>(a, b);
      }
      if (dZ != nullptr) {
        uint16_t *out = dZ + row * lddz + c0;
        if constexpr (kVec) {
          if (8 * x < left)
            __stcs(reinterpret_cast<uint4 *>(out + 8 * x), make_uint4(g[0], g[1], g[2], g[3]));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (x + 32 * e < left)
              out[x + 32 * e] = static_cast<uint16_t>(g[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  };
  // The loads of the next kAhead rows are in flight while these are worked on (a
  // store could alias them, so the compiler would not move them up). Two sets of
  // registers in turn: copying one into the other would wait for its loads.
  constexpr int kStep = kSlots * kAhead;
  Rows even, odd;
  int64_t r = r0 + y;
  load(r, even);
  while (r < r1) {
    load(r + kStep, odd);
    work(r, even);
    r += kStep;
    if (r >= r1) break;
    load(r + kStep, even);
    work(r, odd);
    r += kStep;
  }
  if (part == nullptr) return;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    split(sum[e], red[y][col_of<kVec>(x, 2 * e)], red[y][col_of<kVec>(x, 2 * e + 1)]);
  __syncthreads();
  const int c = y * 32 + x;
  if (c < left) {
    float t = 0.f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) t += red[s][c];
    part[blockIdx.y * static_cast<int64_t>(N) + c0 + c] = t;
  }
}

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(32 * kSlots, kBlocksPerSm)
    act_grad_kernel(int M, int N, int act, const uint16_t *dD, int64_t ldd, const uint16_t *Z,
                    int64_t ldz, uint16_t *dZ, int64_t lddz, float *part, int chunk) {
  __shared__ float red[kSlots][kCols];
  grid_dependency_wait();
  grid_launch_dependents();
  with_act(act, [&](auto a) {
    act_grad_body<kBf16, kVec, decltype(a)::value>(M, N, dD, ldd, Z, ldz, dZ, lddz, part, chunk,
                                                 red);
  });
}

bool vec_ok(const void *p, int64_t ld) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
}

}  // namespace

cudaError_t launch_act_grad(const DeviceInfo &dev, bool bf16, int M, int N, int act,
                            const uint16_t *dD, int64_t ldd, const uint16_t *Z, int64_t ldz,
                            uint16_t *dZ, int64_t lddz, uint16_t *dbias, cudaStream_t stream) {
  if (M == 0) return launch_col_sums(bf16, nullptr, 0, N, N, dbias, stream);
  // As many row chunks as fill the GPU once (kBlocksPerSm blocks per SM).
  const int strips = (N - 1) / kCols + 1;  // sizes up to 2^31 - 1
  const int64_t want =
      std::max<int64_t>(1, static_cast<int64_t>(dev.sm_count) * kBlocksPerSm / strips);
  const int64_t even = (M - 1) / want + 1;
  const int chunk =
      static_cast<int>(std::min<int64_t>((even - 1) / kSlots * kSlots + kSlots, kMaxChunk));
  const int chunks = (M - 1) / chunk + 1;
  float *part = nullptr;
  if (dbias != nullptr) {
    cudaMemPool_t pool;
    cudaError_t e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    void *p = nullptr;
    e = cudaMallocFromPoolAsync(&p, static_cast<size_t>(chunks) * N * 4, pool, stream);
    if (e != cudaSuccess) return e;
    part = static_cast<float *>(p);
  }
  const bool vec = N % 8 == 0 && vec_ok(dD, ldd) && vec_ok(Z, ldz) && vec_ok(dZ, lddz);
  auto kern = bf16 ? (vec ? act_grad_kernel<true, true> : act_grad_kernel<true, false>)
                   : (vec ? act_grad_kernel<false, true> : act_grad_kernel<false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(strips), static_cast<unsigned>(chunks), 1);
  cfg.blockDim = dim3(32, kSlots, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e =
      cudaLaunchKernelEx(&cfg, kern, M, N, act, dD, ldd, Z, ldz, dZ, lddz, part, chunk);
  if (e == cudaSuccess && part != nullptr)
    e = launch_col_sums(bf16, part, chunks, N, N, dbias, stream);
  if (part != nullptr) {
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace dgr

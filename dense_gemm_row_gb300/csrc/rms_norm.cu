// rms_norm.cu -- root-mean-square norm with the residual's addition, and its
// gradient. Per row of n columns, in fp32:
//
//     h = x + r,   s = (mean_j h_j^2 + eps)^(-1/2),   y_j = h_j s w_j
//
// h is written rounded to 16 bits (the residual stream), y rounded to 16 bits
// or as e4m3 values q with one scale per row: scale = max_j |y_j| / 448,
// q = y / scale rounded to nearest even (448 is e4m3's largest value; a row of
// zeros has scale 0 and q = 0). The statistic and y use the unrounded h.
//
// Gradient, with n_j = h_j s and g_j = dy_j w_j:
//
//     dx_j = s (g_j - n_j mean_k(g_k n_k)) + dh_j,    dw_j = sum_i dy_ij n_ij
//
// Both are bound by memory: every value is read once, kept in registers and
// written once. A row belongs to one block, or (short rows) to one warp of a
// block; threads hold 8 consecutive values per 16-byte load. The largest |h w|
// is reduced together with the sum of squares, so the 8-bit form has one block
// reduction too: max |y| = s max |h w| up to rounding.
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

constexpr float kE4m3Max = 448.f;
// A row whose largest |y| is below this counts as zeros (scale 0): 448 / |y|
// must not overflow.
constexpr float kE4m3Least = 1e-30f;

// 1 / scale of a row, and its scale; NaN and infinity stay visible in both the
// scale and the values (0 * inf and NaN).
__device__ __forceinline__ void e4m3_scale(float most, float &scale, float &inv) {
  const bool zeros = most < kE4m3Least;
  scale = zeros ? 0.f : most / kE4m3Max;
  inv = zeros ? 0.f : kE4m3Max / most;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// V values of a row from column c (V = 8: one 16-byte load).
template <bool kBf16, int V>
__device__ __forceinline__ void load_row(const uint16_t *p, int c, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p + c));
    unpack16<kBf16>(w.x, v[0], v[1]);
    unpack16<kBf16>(w.y, v[2], v[3]);
    unpack16<kBf16>(w.z, v[4], v[5]);
    unpack16<kBf16>(w.w, v[6], v[7]);
  } else {
    v[0] = from16<kBf16>(__ldcs(p + c));
  }
}
template <bool kBf16, int V>
__device__ __forceinline__ void store_row(uint16_t *p, int c, const float (&v)[V]) {
  if constexpr (V == 8) {
    __stcs(reinterpret_cast<uint4 *>(p + c),
           make_uint4(pack16<kBf16>(v[0], v[1]), pack16<kBf16>(v[2], v[3]),
                      pack16<kBf16>(v[4], v[5]), pack16<kBf16>(v[6], v[7])));
  } else {
    p[c] = to16<kBf16>(v[0]);
  }
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *p, int c, const float (&v)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint2 *>(p + c) =
        make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16),
                   e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
  } else {
    p[c] = static_cast<uint8_t>(e4m3x2(v[0], 0.f));
  }
}

// The sum of a and the largest of m over the T threads of a row (a whole block
// in warps, or one warp), in one fixed order. red: one slot pair per warp.
template <int T>
__device__ __forceinline__ void row_reduce(float &a, float &m, float2 *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, m);
    __syncthreads();
    a = 0.f;
    m = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) {
      const float2 v = red[i];
      a += v.x;
      m = max_nan(m, v.y);
    }
  }
}

// T threads per row, V values per load, at most NV loads per thread and array:
// rows of up to T * V * NV columns. Blocks of max(T, 128) threads.
template <bool kBf16, int T, int V, int NV>
__global__ void __launch_bounds__(T < 128 ? 128 : T) rms_norm_kernel(const RmsCall c) {
  __shared__ float2 red[T / 32];
  constexpr int kRows = T < 128 ? 128 / T : 1;
  const int row = static_cast<int>(blockIdx.x) * kRows + static_cast<int>(threadIdx.x) / T;
  const int t = static_cast<int>(threadIdx.x) % T;
  grid_dependency_wait();
  grid_launch_dependents();
  if (kRows > 1 && row >= c.rows) return;  // whole warps; no block barrier follows
  const int64_t r = row;
  const uint16_t *X = c.X + r * c.ldx, *R = c.R ? c.R + r * c.ldr : nullptr;
  float h[NV][V], w[NV][V];
  float sum = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * T + t) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) h[i][e] = 0.f, w[i][e] = 1.f;
    if (col < c.cols) {
      load_row<kBf16, V>(X, col, h[i]);
      if (R) {
        float x[V];
        load_row<kBf16, V>(R, col, x);
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] += x[e];
      }
      if (c.W) {
        if constexpr (V == 8) {
          const uint4 q = __ldg(reinterpret_cast<const uint4 *>(c.W + col));
          unpack16<kBf16>(q.x, w[i][0], w[i][1]);
          unpack16<kBf16>(q.y, w[i][2], w[i][3]);
          unpack16<kBf16>(q.z, w[i][4], w[i][5]);
          unpack16<kBf16>(q.w, w[i][6], w[i][7]);
        } else {
          w[i][0] = from16<kBf16>(__ldg(c.W + col));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * T + t) * V;
    if (c.H && col < c.cols) store_row<kBf16, V>(c.H + r * c.ldh, col, h[i]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sum = fmaf(h[i][e], h[i][e], sum);
      w[i][e] *= h[i][e];
      top = max_nan(top, fabsf(w[i][e]));
    }
  }
  row_reduce<T>(sum, top, red);
  const float s = rsqrtf(sum / static_cast<float>(c.cols) + c.eps);
  if (t == 0 && c.rstd) c.rstd[r] = s;
  if (c.scale) {
    float scale, inv;
    e4m3_scale(top * s, scale, inv);
    if (t == 0) c.scale[r] = scale;
    uint8_t *Y = static_cast<uint8_t *>(c.Y) + r * c.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) w[i][e] = w[i][e] * s * inv;
      if (col < c.cols) store_e4m3<V>(Y, col, w[i]);
    }
  } else {
    uint16_t *Y = static_cast<uint16_t *>(c.Y) + r * c.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) w[i][e] *= s;
      if (col < c.cols) store_row<kBf16, V>(Y, col, w[i]);
    }
  }
}

// Rows of any length: each block walks its row twice (the second pass reads it
// from L2).
template <bool kBf16>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const RmsCall c) {
  __shared__ float2 red[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint16_t *X = c.X + r * c.ldx, *R = c.R ? c.R + r * c.ldr : nullptr;
  float sum = 0.f, top = 0.f;
  for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
    float h = from16<kBf16>(X[j]);
    if (R) h += from16<kBf16>(R[j]);
    sum = fmaf(h, h, sum);
    top = max_nan(top, fabsf(c.W ? h * from16<kBf16>(c.W[j]) : h));
  }
  row_reduce<1024>(sum, top, red);
  const float s = rsqrtf(sum / static_cast<float>(c.cols) + c.eps);
  if (threadIdx.x == 0 && c.rstd) c.rstd[r] = s;
  float scale, inv;
  e4m3_scale(top * s, scale, inv);
  if (threadIdx.x == 0 && c.scale) c.scale[r] = scale;
  for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
    float h = from16<kBf16>(X[j]);
    if (R) h += from16<kBf16>(R[j]);
    const float y = (c.W ? h * from16<kBf16>(c.W[j]) : h) * s;
    if (c.H) c.H[r * c.ldh + j] = to16<kBf16>(h);
    if (c.scale) {
      static_cast<uint8_t *>(c.Y)[r * c.ldy + j] = static_cast<uint8_t>(e4m3x2(y * inv, 0.f));
    } else {
      static_cast<uint16_t *>(c.Y)[r * c.ldy + j] = to16<kBf16>(y);
    }
  }
}

// ------------------------------------------------------------------ gradient

// Blocks walk rows blockIdx.x, + gridDim.x, ...; each thread keeps the sums of
// dw for its columns over the block's rows and writes them once, as one partial
// row per block (and per warp, where a warp has its own row).
template <bool kBf16, int T, int V, int NV>
__global__ void __launch_bounds__(T < 128 ? 128 : T)
    rms_norm_grad_kernel(const RmsGradCall c, float *part) {
  __shared__ float2 red[2][T / 32];
  constexpr int kRows = T < 128 ? 128 / T : 1;
  const int t = static_cast<int>(threadIdx.x) % T;
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
  grid_dependency_wait();
  grid_launch_dependents();
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * T + t) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) w[i][e] = 1.f, dw[i][e] = 0.f;
    if (c.W && col < c.cols) load_row<kBf16, V>(c.W, col, w[i]);
  }
  const float inv_n = 1.f / static_cast<float>(c.cols);
  int flip = 0;
  for (int64_t r = slot; r < c.rows; r += static_cast<int64_t>(gridDim.x) * kRows) {
    const uint16_t *dY = c.dY + r * c.lddy, *H = c.H + r * c.ldh;
    const float s = c.rstd[r];
    float g[NV][V], n[NV][V], b[NV][V];
    float dot = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = n[i][e] = b[i][e] = 0.f;
      if (col < c.cols) {
        load_row<kBf16, V>(dY, col, g[i]);
        load_row<kBf16, V>(H, col, n[i]);
        if (c.dH) load_row<kBf16, V>(c.dH + r * c.lddh, col, b[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        n[i][e] *= s;
        dw[i][e] = fmaf(g[i][e], n[i][e], dw[i][e]);
        g[i][e] *= w[i][e];
        dot = fmaf(g[i][e], n[i][e], dot);
      }
    }
    // Two sets of slots in turn: a warp may write the next row's while another
    // still reads this row's.
    row_reduce<T>(dot, unused, red[flip]);
    flip ^= 1;
    const float mean = dot * inv_n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * T + t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = fmaf(s, g[i][e] - n[i][e] * mean, b[i][e]);
      if (col < c.cols) store_row<kBf16, V>(c.dX + r * c.lddx, col, g[i]);
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * T + t) * V;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (col + e < c.cols) part[slot * c.cols + col + e] = dw[i][e];
  }
}

// Rows of any length: one block per group of rows; the partial sums of dw live
// in the block's partial row in global memory.
template <bool kBf16>
__global__ void __launch_bounds__(1024)
    rms_norm_grad_long_kernel(const RmsGradCall c, float *part) {
  __shared__ float2 red[2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const float inv_n = 1.f / static_cast<float>(c.cols);
  float *mine = part ? part + blockIdx.x * static_cast<int64_t>(c.cols) : nullptr;
  int flip = 0;
  bool first = true;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const uint16_t *dY = c.dY + r * c.lddy, *H = c.H + r * c.ldh;
    const float s = c.rstd[r];
    float dot = 0.f, unused = 0.f;
    for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
      const float d = from16<kBf16>(dY[j]), n = from16<kBf16>(H[j]) * s;
      dot = fmaf(c.W ? d * from16<kBf16>(c.W[j]) : d, n, dot);
      if (mine) mine[j] = first ? d * n : fmaf(d, n, mine[j]);  // this thread's own element
    }
    row_reduce<1024>(dot, unused, red[flip]);
    flip ^= 1;
    const float mean = dot * inv_n;
    for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
      const float d = from16<kBf16>(dY[j]), n = from16<kBf16>(H[j]) * s;
      const float g = c.W ? d * from16<kBf16>(c.W[j]) : d;
      const float b = c.dH ? from16<kBf16>(c.dH[r * c.lddh + j]) : 0.f;
      c.dX[r * c.lddx + j] = to16<kBf16>(fmaf(s, g - n * mean, b));
    }
    first = false;
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, cudaStream_t stream,
                       A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

bool vec_ok(const void *p, int64_t ld, int units) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % units == 0);
}

template <bool kBf16, int V>
cudaError_t launch_norm(const RmsCall &c, cudaStream_t stream) {
  const int units = (c.cols + V - 1) / V;  // loads per row and array
  const unsigned rows = static_cast<unsigned>(c.rows);
  if (units <= 32) return launch_pdl(rms_norm_kernel<kBf16, 32, V, 1>, (rows + 3) / 4, 128, stream, c);
  if (units <= 128) return launch_pdl(rms_norm_kernel<kBf16, 32, V, 4>, (rows + 3) / 4, 128, stream, c);
  if (units <= 256) return launch_pdl(rms_norm_kernel<kBf16, 128, V, 2>, rows, 128, stream, c);
  if (units <= 512) return launch_pdl(rms_norm_kernel<kBf16, 256, V, 2>, rows, 256, stream, c);
  if (units <= 1024) return launch_pdl(rms_norm_kernel<kBf16, 512, V, 2>, rows, 512, stream, c);
  if (units <= 2048) return launch_pdl(rms_norm_kernel<kBf16, 1024, V, 2>, rows, 1024, stream, c);
  if (V == 1 && units <= 8192)
    return launch_pdl(rms_norm_kernel<kBf16, 1024, V, 8 / V>, rows, 1024, stream, c);
  return launch_pdl(rms_norm_long_kernel<kBf16>, rows, 1024, stream, c);
}

template <bool kBf16, int T, int V, int NV>
cudaError_t launch_grad_form(const DeviceInfo &dev, const RmsGradCall &c, cudaStream_t stream) {
  constexpr int kThreads = T < 128 ? 128 : T;
  constexpr int kRows = kThreads / T;
  // One wave: as many blocks as are resident at once, or one per row.
  auto kern = rms_norm_grad_kernel<kBf16, T, V, NV>;
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, 0);
  if (e != cudaSuccess) return e;
  const int64_t blocks = std::min<int64_t>(static_cast<int64_t>(std::max(per_sm, 1)) * dev.sm_count,
                                           (static_cast<int64_t>(c.rows) + kRows - 1) / kRows);
  const int64_t parts = blocks * kRows;
  void *part = nullptr;
  if (c.dW != nullptr) {
    cudaMemPool_t pool;
    e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    e = cudaMallocFromPoolAsync(&part, static_cast<size_t>(parts) * c.cols * 4, pool, stream);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kern, static_cast<unsigned>(blocks), kThreads, stream, c,
                 static_cast<float *>(part));
  if (part != nullptr) {
    if (e == cudaSuccess)
      e = launch_col_sums(c.bf16, static_cast<const float *>(part), static_cast<int>(parts),
                          c.cols, c.cols, c.dW, stream);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

template <bool kBf16>
cudaError_t launch_grad_long(const DeviceInfo &dev, const RmsGradCall &c, cudaStream_t stream) {
  const int blocks = std::min(c.rows, 2 * dev.sm_count);
  void *part = nullptr;
  cudaError_t e = cudaSuccess;
  if (c.dW != nullptr) {
    cudaMemPool_t pool;
    e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    e = cudaMallocFromPoolAsync(&part, static_cast<size_t>(blocks) * c.cols * 4, pool, stream);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(rms_norm_grad_long_kernel<kBf16>, static_cast<unsigned>(blocks), 1024, stream, c,
                 static_cast<float *>(part));
  if (part != nullptr) {
    if (e == cudaSuccess)
      e = launch_col_sums(c.bf16, static_cast<const float *>(part), blocks, c.cols, c.cols, c.dW,
                          stream);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

template <bool kBf16, int V>
cudaError_t launch_grad(const DeviceInfo &dev, const RmsGradCall &c, cudaStream_t stream) {
  const int units = (c.cols + V - 1) / V;
  if (units <= 32) return launch_grad_form<kBf16, 32, V, 1>(dev, c, stream);
  if (units <= 128) return launch_grad_form<kBf16, 128, V, 1>(dev, c, stream);
  if (units <= 256) return launch_grad_form<kBf16, 256, V, 1>(dev, c, stream);
  if (units <= 512) return launch_grad_form<kBf16, 512, V, 1>(dev, c, stream);
  if (units <= 1024) return launch_grad_form<kBf16, 1024, V, 1>(dev, c, stream);
  if (V == 1 && units <= 8192) return launch_grad_form<kBf16, 1024, V, 8 / V>(dev, c, stream);
  return launch_grad_long<kBf16>(dev, c, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const DeviceInfo &dev, const RmsCall &c, cudaStream_t stream) {
  (void)dev;
  // 16-byte loads need 16-byte aligned rows (8-byte ones for the e4m3 output)
  // and whole groups of 8 columns.
  const bool vec = c.cols % 8 == 0 && vec_ok(c.X, c.ldx, 8) && vec_ok(c.R, c.ldr, 8) &&
                   vec_ok(c.H, c.ldh, 8) && vec_ok(c.Y, c.ldy, 8) && vec_ok(c.W, 8, 8);
  if (c.bf16) return vec ? launch_norm<true, 8>(c, stream) : launch_norm<true, 1>(c, stream);
  return vec ? launch_norm<false, 8>(c, stream) : launch_norm<false, 1>(c, stream);
}

cudaError_t launch_rms_norm_grad(const DeviceInfo &dev, const RmsGradCall &c,
                                 cudaStream_t stream) {
  if (c.rows == 0)
    return c.dW ? launch_col_sums(c.bf16, nullptr, 0, c.cols, c.cols, c.dW, stream) : cudaSuccess;
  const bool vec = c.cols % 8 == 0 && vec_ok(c.dY, c.lddy, 8) && vec_ok(c.H, c.ldh, 8) &&
                   vec_ok(c.dH, c.lddh, 8) && vec_ok(c.dX, c.lddx, 8) && vec_ok(c.W, 8, 8);
  if (c.bf16)
    return vec ? launch_grad<true, 8>(dev, c, stream) : launch_grad<true, 1>(dev, c, stream);
  return vec ? launch_grad<false, 8>(dev, c, stream) : launch_grad<false, 1>(dev, c, stream);
}

}  // namespace dgr

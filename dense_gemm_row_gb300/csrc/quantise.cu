// quantise.cu -- a 16-bit matrix as e4m3 values with a scale for each block of 128
// columns of a row, or of 128 rows x 128 columns:
//
//     scale = max |x| / 448,   y = x / scale rounded to nearest even
//
// (448 is e4m3's largest value; a block below 1e-30 has scale 0 and zeros.) Bound by
// memory: 2 bytes in, 1 out, each value held in registers between the two.
//
// A row's block of 128 belongs to 16 threads with 8 values each: one 16-byte load, one
// 8-byte store. Rows that are not in whole 16-byte units (or 8-byte units of Y) go
// value by value, 8 consecutive ones per thread, so that a line is fetched once.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

constexpr int kBlock = 128;
constexpr int kLanes = 16;  // threads per row of a block

struct QuantArgs {
  int rows, cols, col_blocks;
  const uint16_t *X;
  int64_t ldx;
  uint8_t *Y;
  int64_t ldy;
  float *scale;
  int64_t lds;
  bool x_vec, y_vec;  // rows in whole 16-byte units / 8-byte units
};

// 8 values from column `col` of a row, packed; zeros past the last column.
__device__ __forceinline__ uint4 load8(const QuantArgs &q, int64_t row, int col) {
  const uint16_t *p = q.X + row * q.ldx + col;
  const int n = q.cols - col;
  if (q.x_vec && n >= 8) return __ldcs(reinterpret_cast<const uint4 *>(p));
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = e < n ? p[e] : 0;
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                    h[6] | (h[7] << 16));
}
// The largest magnitude of 8 packed values, as bits: those of |x| order like |x|, NaN last.
__device__ __forceinline__ uint32_t top8(const uint4 &v) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}
template <bool kBf16>
__device__ __forceinline__ float top_value(uint32_t pair) {
  return from16<kBf16>(max(pair & 0xffffu, pair >> 16));
}
template <bool kBf16>
__device__ __forceinline__ void store8(const QuantArgs &q, int64_t row, int col, const uint4 &v,
                                       float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    split(mul2(unpack2<kBf16>(w[e]), f2(inv)), lo, hi);
    b[e] = e4m3x2(lo, hi);
  }
  const uint32_t lo = b[0] | (b[1] << 16), hi = b[2] | (b[3] << 16);
  uint8_t *p = q.Y + row * q.ldy + col;
  const int n = q.cols - col;
  if (q.y_vec && n >= 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
}

// Blocks of 1 x 128: a group of 16 threads takes kAhead of them together.
constexpr int kRowThreads = 256, kAhead = 4;

template <bool kBf16>
__global__ void __launch_bounds__(kRowThreads) quantise_rows_kernel(const QuantArgs q) {
  const int lane = threadIdx.x & (kLanes - 1);
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t total = static_cast<int64_t>(q.rows) * q.col_blocks;
  const int64_t first =
      (blockIdx.x * static_cast<int64_t>(kRowThreads / kLanes)) * kAhead + threadIdx.x / kLanes;
  uint4 v[kAhead];
  int64_t row[kAhead];
  int cb[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t at = first + i * (kRowThreads / kLanes);
    row[i] = at / q.col_blocks;
    cb[i] = static_cast<int>(at - row[i] * q.col_blocks);
    v[i] = make_uint4(0, 0, 0, 0);
    if (at < total) v[i] = load8(q, row[i], cb[i] * kBlock + 8 * lane);
  }
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    uint32_t top = top8(v[i]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (first + i * (kRowThreads / kLanes) >= total) continue;
    const float most = top_value<kBf16>(top);
    if (lane == 0) q.scale[row[i] * q.lds + cb[i]] = e4m3_scale(most);
    store8<kBf16>(q, row[i], cb[i] * kBlock + 8 * lane, v[i], e4m3_inverse(most));
  }
}

// Blocks of 128 x 128: one block of threads each, 8 rows per thread.
constexpr int kTileThreads = 256, kTileRows = kBlock / (kTileThreads / kLanes);

template <bool kBf16>
__global__ void __launch_bounds__(kTileThreads) quantise_tiles_kernel(const QuantArgs q) {
  __shared__ uint32_t tops[kTileThreads / 32];
  const int lane = threadIdx.x & (kLanes - 1);
  grid_dependency_wait();
  grid_launch_dependents();
  const int rb = static_cast<int>(blockIdx.x / q.col_blocks);
  const int cb = static_cast<int>(blockIdx.x) - rb * q.col_blocks;
  const int64_t row0 = static_cast<int64_t>(rb) * kBlock + threadIdx.x / kLanes;
  const int col = cb * kBlock + 8 * lane;
  uint4 v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    const int64_t row = row0 + i * (kTileThreads / kLanes);
    v[i] = row < q.rows ? load8(q, row, col) : make_uint4(0, 0, 0, 0);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) top = __vmaxu2(top, top8(v[i]));
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) top = max(top, tops[i]);
  const float most = from16<kBf16>(top);
  if (threadIdx.x == 0) q.scale[rb * q.lds + cb] = e4m3_scale(most);
  const float inv = e4m3_inverse(most);
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    const int64_t row = row0 + i * (kTileThreads / kLanes);
    if (row < q.rows) store8<kBf16>(q, row, col, v[i], inv);
  }
}

}  // namespace

cudaError_t launch_quantise(bool bf16, int rows, int cols, int block_rows, const uint16_t *X,
                            int64_t ldx, uint8_t *Y, int64_t ldy, float *scale, int64_t lds,
                            cudaStream_t stream) {
  QuantArgs q;
  q.rows = rows, q.cols = cols;
  q.col_blocks = (cols - 1) / kBlock + 1;
  q.X = X, q.ldx = ldx;
  q.Y = Y, q.ldy = ldy;
  q.scale = scale, q.lds = lds;
  q.x_vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
  q.y_vec = reinterpret_cast<uintptr_t>(Y) % 8 == 0 && ldy % 8 == 0;
  const bool one = block_rows == 1;
  const int64_t per_block = one ? kRowThreads / kLanes * kAhead : 1;
  const int64_t blocks =
      (static_cast<int64_t>(one ? rows : (rows - 1) / kBlock + 1) * q.col_blocks + per_block - 1) /
      per_block;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(one ? kRowThreads : kTileThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = one ? (bf16 ? quantise_rows_kernel<true> : quantise_rows_kernel<false>)
                  : (bf16 ? quantise_tiles_kernel<true> : quantise_tiles_kernel<false>);
  return cudaLaunchKernelEx(&cfg, kern, q);
}

}  // namespace dgr

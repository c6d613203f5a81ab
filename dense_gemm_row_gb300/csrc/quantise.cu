// quantise.cu -- a 16-bit matrix as e4m3 values with a scale for each block of 128
// columns of a row, or of 128 rows x 128 columns:
//
//     scale = max |x| / 448,   y = x / scale rounded to nearest even
//
// (448 is e4m3's largest value; a block below 1e-30 has scale 0 and zeros.) Bound by
// memory: 2 bytes in, 1 out, each value held in registers between the two.
//
// A row's block of 128 belongs to 16 threads with 8 values each: one 16-byte load, one
// 8-byte store. Rows that are not in whole 16-byte units go value by value, 8 consecutive
// ones per thread, so that a line is fetched once. (One aligned load per thread, with the
// rest from its neighbour by shuffles, took as long for many rows and longer for few:
// 1001 x 4095 in blocks of 128 rows 6.6 us against 5.4.)
// bf16 8192 x 8192: 30 us in short runs in either blocks (6.8 TB/s, the copy rate), 31.6
// repeated; 8192 x 8191 55 us, f16 1001 x 4095 in blocks of 128 rows 4.8.
#include <algorithm>
#include <cstdint>
#include <type_traits>

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
  bool y_vec;  // Y's rows in whole 8-byte units
};

// 8 values, packed, of which n exist; zeros past the last column. kAligned: rows in whole
// 16-byte units, kInner: all values of the thread's block exist.
template <bool kAligned, bool kInner>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int n) {
  if constexpr (kAligned && kInner) {
    return __ldcs(reinterpret_cast<const uint4 *>(p));
  } else {
    if (kAligned && n >= 8) return __ldcs(reinterpret_cast<const uint4 *>(p));
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = kInner || e < n ? p[e] : 0;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                      h[6] | (h[7] << 16));
  }
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
// x / scale of 8 values, in e4m3: the product with the scale's inverse, which is within
// 2^-22 of the quotient, as the scale itself is of max / 448. (The rounded quotient by
// the stored scale, one more multiply-add pair, took 8 % longer and is no nearer to the
// exact one.)
template <bool kBf16, bool kInner>
__device__ __forceinline__ void store8(uint8_t *p, int n, bool vec, const uint4 &v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    split(mul2(unpack2<kBf16>(w[e]), f2(inv)), lo, hi);
    b[e] = e4m3x2(lo, hi);
  }
  const uint32_t lo = b[0] | (b[1] << 16), hi = b[2] | (b[3] << 16);
  if (kInner || (vec && n >= 8)) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
}

// A block of threads takes 128 columns of kThreads / 16 * kRows rows, kRows per thread;
// kTile: those 128 rows are one block. (Rows walked along, a group of 16 threads on
// four blocks of 1 x 128 in turn, took 41.8 us for 8192 x 8192.)
template <bool kBf16, bool kAligned, bool kTile, bool kInner, int kThreads, int kRows>
__device__ __forceinline__ void quantise_block(const QuantArgs &q, int rb, int cb,
                                               uint32_t (&tops)[kThreads / 32]) {
  constexpr int kStep = kThreads / kLanes;
  static_assert(!kTile || kStep * kRows == kBlock, "a block's rows");
  static_assert(kTile || kRows <= kLanes, "a lane per row");
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t row0 = static_cast<int64_t>(rb) * (kStep * kRows) + threadIdx.x / kLanes;
  const int col = cb * kBlock + 8 * lane, n = q.cols - col;
  auto live = [&](int i) { return kInner || row0 + i * kStep < q.rows; };
  uint4 v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint16_t *x = q.X + (row0 + i * kStep) * q.ldx + col;
    v[i] = live(i) ? load8<kAligned, kInner>(x, n) : make_uint4(0, 0, 0, 0);
  }
  float most;
  if constexpr (kTile) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) top = __vmaxu2(top, top8(v[i]));
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, tops[i]);
    most = from16<kBf16>(top);
    if (threadIdx.x == 0) q.scale[rb * q.lds + cb] = e4m3_scale(most);
  } else {
    // The lanes of a row exchange halves of their rows' maxima until two lanes are left
    // with one row, whose divisions they make: 2 per thread instead of 2 per row.
    uint32_t top[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) top[i] = top8(v[i]);
#pragma unroll
    for (int k = kRows / 2, o = kLanes / 2; o > 0; o >>= 1, k /= 2) {
      const bool up = (lane & o) != 0;
      if (k > 0) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const uint32_t give = up ? top[i] : top[i + k], keep = up ? top[i + k] : top[i];
          top[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
      } else {
        top[0] = __vmaxu2(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
      }
    }
    constexpr int kSame = kLanes / kRows;  // lanes left with one row
    most = top_value<kBf16>(top[0]);
    const int64_t row = row0 + lane / kSame * kStep;
    if (lane % kSame == 0 && (kInner || row < q.rows))
      q.scale[row * q.lds + cb] = e4m3_scale(most);
  }
  const float inv = e4m3_inverse(most);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    constexpr int kSame = kTile ? 1 : kLanes / kRows;
    const float by = kTile ? inv : __shfl_sync(0xffffffffu, inv, i * kSame, kLanes);
    uint8_t *y = q.Y + (row0 + i * kStep) * q.ldy + col;
    if (live(i)) store8<kBf16, kInner>(y, n, q.y_vec, v[i], by);
  }
}

template <bool kBf16, bool kAligned, bool kTile, int kThreads, int kRows>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantArgs q) {
  constexpr int kBlockRows = kThreads / kLanes * kRows;
  __shared__ uint32_t tops[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int rb = static_cast<int>(blockIdx.x / static_cast<uint32_t>(q.col_blocks));
  const int cb = static_cast<int>(blockIdx.x) - rb * q.col_blocks;
  // Blocks inside the matrix need no checks (8192 x 8192 32.5 -> 30.0 us, in blocks of 128
  // rows 35 -> 30). Where there are few, a second body's code does not pay.
  if (kRows == 8 && q.y_vec && rb < q.rows / kBlockRows && cb < q.cols / kBlock) {
    quantise_block<kBf16, kAligned, kTile, true, kThreads, kRows>(q, rb, cb, tops);
  } else {
    quantise_block<kBf16, kAligned, kTile, false, kThreads, kRows>(q, rb, cb, tops);
  }
}

}  // namespace

cudaError_t launch_quantise(const DeviceInfo &dev, bool bf16, int rows, int cols, int block_rows,
                            const uint16_t *X, int64_t ldx, uint8_t *Y, int64_t ldy, float *scale,
                            int64_t lds, cudaStream_t stream) {
  QuantArgs q;
  q.rows = rows, q.cols = cols;
  q.col_blocks = (cols - 1) / kBlock + 1;
  q.X = X, q.ldx = ldx;
  q.Y = Y, q.ldy = ldy;
  q.scale = scale, q.lds = lds;
  const bool x_vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
  q.y_vec = reinterpret_cast<uintptr_t>(Y) % 8 == 0 && ldy % 8 == 0;
  // Few blocks of threads: fewer rows per thread, or more threads per block of values
  // (1001 x 4096 in blocks of 128 rows, with the checks that these had then: 3.9 us with
  // 256 threads, 3.6 with 512, 4.2 with 1024; 1001 x 4095: 5.4, 5.4, 6.1).
  const bool tile = block_rows == kBlock;
  const int64_t tiles = (static_cast<int64_t>(rows - 1) / kBlock + 1) * q.col_blocks;
  const bool few = tiles < 4LL * dev.sm_count;
  const int64_t blocks = few && !tile ? (static_cast<int64_t>(rows - 1) / 16 + 1) * q.col_blocks
                                      : tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(few && tile ? 512 : 256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto pick = [&](auto bf, auto al) {
    constexpr bool kBf16 = decltype(bf)::value, kAligned = decltype(al)::value;
    return tile ? (few ? quantise_kernel<kBf16, kAligned, true, 512, 4>
                       : quantise_kernel<kBf16, kAligned, true, 256, 8>)
                : (few ? quantise_kernel<kBf16, kAligned, false, 256, 1>
                       : quantise_kernel<kBf16, kAligned, false, 256, 8>);
  };
  const std::true_type yes;
  const std::false_type no;
  auto kern = bf16 ? (x_vec ? pick(yes, yes) : pick(yes, no))
                   : (x_vec ? pick(no, yes) : pick(no, no));
  return cudaLaunchKernelEx(&cfg, kern, q);
}

}  // namespace dgr

// norm.cuh -- the norms with the residual's addition, and their gradients, shared by
// the translation units that instantiate them: rms_norm.cu (root mean square) and
// layer_norm.cu (kLayer). Per row of n columns, in fp32, with h = x + r:
//
//     rms     s = (mean_j h_j^2 + eps)^(-1/2),          y_j = h_j s w_j
//     layer   s = (mean_j (h_j - m)^2 + eps)^(-1/2),    y_j = (h_j - m) s w_j + b_j
//             with m = mean_j h_j
//
// h is written rounded to 16 bits (the residual stream), y rounded to 16 bits
// or (rms) as e4m3 values q with one scale per row: scale = max_j |y_j| / 448,
// q = y / scale rounded to nearest even (448 is e4m3's largest value; a row of
// zeros has scale 0 and q = 0). The statistics and y use the unrounded h. The layer
// norm sums the squares about the mean, in a second reduction: their sum less n m^2
// would lose the variance of rows whose mean is large beside it. Its m is a quotient: the
// product with a rounded 1 / n is off where the sum is exact, and a row of 1000 values of
// 60000 gave y = -0.78, not 0.
//
// Gradient, with n_j = h_j s (layer: (h_j - m) s) and g_j = dy_j w_j:
//
//     dx_j = s (g_j - n_j mean_k(g_k n_k)) + dh_j,    dw_j = sum_i dy_ij n_ij
//     layer: - s mean_k(g_k) too,                     db_j = sum_i dy_ij
//
// Both are bound by memory: every value is read once and written once. A row
// belongs to one block, or to one warp of a block; while few rows are to be done
// a thread holds its values in registers and a block ends with its row, with many
// rows blocks walk over them with the next rows' copies in flight. The largest
// |h w| is reduced together with the sum of squares, so the 8-bit form has one
// block reduction too: max |y| = s max |h w| up to rounding.
//
// Layer norm, bf16: 16384 x 4096 with a residual 86.0 us (6.2 TB/s), 1 x 4096 2.6 us;
// gradient 8192 x 8192 with dh 91.8 us (5.8 TB/s), 32768 x 1024 47.3, f16 333 x 1001 7.0.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace dgr {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// How a row of `cols` values is walked: `head` values up to the first 16-byte
// boundary of its first matrix, `units` whole 16-byte units of 8 values, and
// fewer than 8 values of tail. Head and tail are one extra value for 16 threads
// each row (thread t < 8: head, 8 <= t < 16: tail), so that no load waits for
// another and nothing outside the row is touched.
struct RowWalk {
  int head, units;
  int extra;  // this thread's extra column, or -1
};
__device__ __forceinline__ int row_offset(const void *row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7);
}
__device__ __forceinline__ RowWalk row_walk(const void *row, int cols, int t) {
  RowWalk k;
  k.head = min((8 - row_offset(row)) & 7, cols);
  k.units = (cols - k.head) >> 3;
  const int tail0 = k.head + 8 * k.units;
  k.extra = t < k.head ? t : (t >= 8 && t - 8 < cols - tail0) ? tail0 + t - 8 : -1;
  return k;
}
// Unit u, packed (zeros past the last, or without a matrix). `same`: the matrix
// has the first one's alignment; others go element by element.
__device__ __forceinline__ uint4 load_unit(const uint16_t *row, const RowWalk &k, int u,
                                           bool same) {
  if (row == nullptr || u >= k.units) return make_uint4(0, 0, 0, 0);
  const uint16_t *p = row + k.head + 8 * u;
  if (same) return __ldcs(reinterpret_cast<const uint4 *>(p));
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = p[e];
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                    h[6] | (h[7] << 16));
}
__device__ __forceinline__ uint32_t load_extra(const uint16_t *row, const RowWalk &k) {
  return row != nullptr && k.extra >= 0 ? row[k.extra] : 0u;
}
__device__ __forceinline__ void store_unit(uint16_t *row, const RowWalk &k, int u, bool same,
                                           const uint4 &w) {
  if (u >= k.units) return;
  uint16_t *p = row + k.head + 8 * u;
  if (same) {
    __stcs(reinterpret_cast<uint4 *>(p), w);
    return;
  }
  const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
}
template <bool kBf16>
__device__ __forceinline__ void unit_values(const uint4 &w, float (&v)[8]) {
  unpack16<kBf16>(w.x, v[0], v[1]);
  unpack16<kBf16>(w.y, v[2], v[3]);
  unpack16<kBf16>(w.z, v[4], v[5]);
  unpack16<kBf16>(w.w, v[6], v[7]);
}
template <bool kBf16>
__device__ __forceinline__ uint4 unit_pack(const float (&v)[8]) {
  return make_uint4(pack16<kBf16>(v[0], v[1]), pack16<kBf16>(v[2], v[3]),
                    pack16<kBf16>(v[4], v[5]), pack16<kBf16>(v[6], v[7]));
}

// The sum of a and the largest of m over the T threads of a row (a whole block
// in warps, one warp or half of one), in one fixed order. red: one slot pair per
// warp.
template <int T>
__device__ __forceinline__ void row_reduce(float &a, float &m, float2 *red) {
#pragma unroll
  for (int o = T < 32 ? T / 2 : 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if (T < 32) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  // m >= 0 or NaN, whose bits order like its values (NaN last).
  if (T >= 32) m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
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

// The sum of a over the T threads of a row, in one fixed order.
template <int T>
__device__ __forceinline__ float row_sum(float a, float *red) {
#pragma unroll
  for (int o = T < 32 ? T / 2 : 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; i += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(red + i);
      a += v.x;
      a += v.y;
    }
  }
  return a;
}

// The sums of a and of b (layer norm's gradient). red: one slot pair per warp.
template <int T>
__device__ __forceinline__ void row_sums(float &a, float &b, float2 *red) {
#pragma unroll
  for (int o = T < 32 ? T / 2 : 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) {
      const float2 v = red[i];
      a += v.x;
      b += v.y;
    }
  }
}

// sum / n, rounded to nearest, from the rounded inv_n = 1 / n: the product is corrected by
// its remainder, which the fused multiply-add leaves exact (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990). Sums below 2^-100,
// whose remainder is subnormal, may be a unit off. (The division itself, once per row:
// layer norm 16384 x 8192 102.6 us, this 100.3, the product alone 99.7.)
__device__ __forceinline__ float quotient(float sum, float n, float inv_n) {
  const float q = sum * inv_n;
  return fabsf(q) <= kFltMax ? fmaf(fmaf(-q, n, sum), inv_n, q) : q;
}

// Writes a row's units of 8 8-bit values where they lie `head` bytes off Y's 8-byte
// boundaries: the aligned 8 bytes number a are the last `head` values of unit
// a - 1 and the first 8 - head of unit a. unit(u): unit u, behind a barrier.
// (16384 rows of 7777 values 265 -> 204 us against byte stores, of 4095 102 -> 91;
// in the one-row form of shorter rows the byte stores are the faster ones, 26
// against 29 us at 1001.)
template <typename Unit>
__device__ __forceinline__ void store_shifted(uint8_t *Y, const RowWalk &k, int t, int threads,
                                              Unit &&unit) {
  const int sh = 8 * k.head;
  for (int a = t; a <= k.units; a += threads) {
    const uint64_t below = a > 0 ? unit(a - 1) : 0, above = a < k.units ? unit(a) : 0;
    const uint64_t w = (below >> (64 - sh)) | (above << sh);
    if (a > 0 && a < k.units) {
      *reinterpret_cast<uint64_t *>(Y + 8 * a) = w;
    } else {
      const int e0 = a == 0 ? k.head : 0, e1 = a == 0 ? 8 : k.head;
      for (int e = e0; e < e1; ++e) Y[8 * a + e] = static_cast<uint8_t>(w >> (8 * e));
    }
  }
}

// The gain's packed values, widened again for every row: hoisted out of the row
// loop, the widened ones would take twice the registers and spill.
__device__ __forceinline__ uint4 per_row(uint4 w) {
  asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
  return w;
}

// T threads per row, at most NV units per thread and array: rows of up to T * NV
// units. Blocks of max(T, 128) threads.
template <bool kLayer, bool kBf16, int T, int NV>
__global__ void __launch_bounds__(T < 128 ? 128 : T) norm_kernel(const NormCall c) {
  __shared__ __align__(16) float2 red[T < 32 ? 1 : T / 32];
  __shared__ uint64_t packed[kLayer || T < 256 ? 1 : T * NV];  // a row's 8-bit values
  constexpr int kRows = T < 128 ? 128 / T : 1;
  const int row = static_cast<int>(blockIdx.x) * kRows + static_cast<int>(threadIdx.x) / T;
  const int t = static_cast<int>(threadIdx.x) % T;
  grid_dependency_wait();
  grid_launch_dependents();
  if (T == 32 && row >= c.rows) return;  // whole warps; no block barrier follows
  // Half warps past the last row take part in their warp's reductions.
  const bool live = T >= 32 || row < c.rows;
  const int64_t r = live ? row : c.rows - 1;
  const uint16_t *X = c.X + r * c.ldx, *R = c.R ? c.R + r * c.ldr : nullptr;
  uint16_t *H = c.H ? c.H + r * c.ldh : nullptr;
  const int cols = c.cols, off = row_offset(X);
  RowWalk k = row_walk(X, cols, t);
  if (!live) k.units = 0, k.extra = -1;
  const bool same_r = row_offset(R) == off, same_w = row_offset(c.W) == off;
  uint4 x[NV], q[NV], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = load_unit(X, k, i * T + t, true);
    q[i] = load_unit(R, k, i * T + t, same_r);
  }
  const uint32_t xe = load_extra(X, k), qe = load_extra(R, k), we = load_extra(c.W, k);
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = load_unit(c.W, k, i * T + t, same_w);
  if constexpr (kLayer) {
    const bool same_b = row_offset(c.B) == off;
    uint4 b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i] = load_unit(c.B, k, i * T + t, same_b);
    const float be = from16<kBf16>(load_extra(c.B, k));
    F2 h[NV][4], sums = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      const uint32_t qw[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i][e] = unpack2<kBf16>(xw[e]);
        if (R) h[i][e] = add2(h[i][e], unpack2<kBf16>(qw[e]));
        sums = add2(sums, h[i][e]);
      }
      if (H)
        store_unit(H, k, i * T + t, row_offset(H) == off,
                   make_uint4(pack2<kBf16>(h[i][0]), pack2<kBf16>(h[i][1]),
                              pack2<kBf16>(h[i][2]), pack2<kBf16>(h[i][3])));
    }
    float he = from16<kBf16>(xe);
    if (R) he += from16<kBf16>(qe);
    if (H && k.extra >= 0) H[k.extra] = to16<kBf16>(he);
    const float inv_n = 1.f / static_cast<float>(cols);
    float *slots = reinterpret_cast<float *>(red);
    float m, m1;
    split(sums, m, m1);
    m = quotient(row_sum<T>(m + m1 + (k.extra >= 0 ? he : 0.f), slots), static_cast<float>(cols),
                 inv_n);
    const F2 minus = f2(-m);
    F2 squares = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i][e] = add2(h[i][e], minus);
        if (i * T + t < k.units) squares = fma2(h[i][e], h[i][e], squares);
      }
    }
    he -= m;
    float sq, sq1;
    split(squares, sq, sq1);
    sq += sq1;
    if (k.extra >= 0) sq = fmaf(he, he, sq);
    sq = row_sum<T>(sq, slots + (T > 32 ? T / 32 : 0));
    const float s = rsqrtf(sq * inv_n + c.eps);
    if (t == 0 && live) {
      if (c.mean) c.mean[r] = m;
      if (c.rstd) c.rstd[r] = s;
    }
    uint16_t *Y = static_cast<uint16_t *>(c.Y) + r * c.ldy;
    const bool same = row_offset(Y) == off;
    const F2 s2 = f2(s);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      const uint32_t bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const F2 n = mul2(h[i][e], s2);
        y[e] = pack2<kBf16>(c.W ? fma2(n, unpack2<kBf16>(ww[e]), unpack2<kBf16>(bw[e]))
                                : add2(n, unpack2<kBf16>(bw[e])));
      }
      store_unit(Y, k, i * T + t, same, make_uint4(y[0], y[1], y[2], y[3]));
    }
    if (k.extra >= 0)
      Y[k.extra] = to16<kBf16>(fmaf(he * s, c.W ? from16<kBf16>(we) : 1.f, be));
    return;
  }
  float h[NV][8], g[NV][8];
  float sum = 0.f, top = 0.f;
  auto add = [&](float &hv, float rv, float &gv) {
    if (R) hv += rv;
    gv = c.W ? gv * hv : hv;
    sum = fmaf(hv, hv, sum);
    if (c.scale) top = max_nan(top, fabsf(gv));
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[8];
    unit_values<kBf16>(x[i], h[i]);
    unit_values<kBf16>(q[i], a);
    unit_values<kBf16>(w[i], g[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) add(h[i][e], a[e], g[i][e]);
    if (H) store_unit(H, k, i * T + t, row_offset(H) == off, unit_pack<kBf16>(h[i]));
  }
  float he = from16<kBf16>(xe), ge = from16<kBf16>(we);
  add(he, from16<kBf16>(qe), ge);
  if (H && k.extra >= 0) H[k.extra] = to16<kBf16>(he);
  row_reduce<T>(sum, top, red);
  const float s = rsqrtf(sum / static_cast<float>(cols) + c.eps);
  if (t == 0 && live && c.rstd) c.rstd[r] = s;
  if (c.scale) {
    const float inv = e4m3_inverse(top * s);
    if (t == 0 && live) c.scale[r] = e4m3_scale(top * s);
    uint8_t *Y = static_cast<uint8_t *>(c.Y) + r * c.ldy;
    const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(Y) & 7);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * T + t;
#pragma unroll
      for (int e = 0; e < 8; ++e) g[i][e] = g[i][e] * s * inv;
      const uint32_t lo = e4m3x2(g[i][0], g[i][1]) | (e4m3x2(g[i][2], g[i][3]) << 16);
      const uint32_t hi = e4m3x2(g[i][4], g[i][5]) | (e4m3x2(g[i][6], g[i][7]) << 16);
      const uint64_t w = static_cast<uint64_t>(hi) << 32 | lo;
      if (u >= k.units) continue;
      uint8_t *p = Y + k.head + 8 * u;
      if (((lead + k.head) & 7) == 0) {
        *reinterpret_cast<uint64_t *>(p) = w;
      } else if (T >= 256 && lead == 0) {
        packed[u] = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = static_cast<uint8_t>(w >> (8 * e));
      }
    }
    if (T >= 256 && lead == 0 && k.head != 0 && k.units > 0) {
      __syncthreads();
      store_shifted(Y, k, t, T, [&](int u) { return packed[u]; });
    }
    if (k.extra >= 0) Y[k.extra] = static_cast<uint8_t>(e4m3x2(ge * s * inv, 0.f));
  } else {
    uint16_t *Y = static_cast<uint16_t *>(c.Y) + r * c.ldy;
    const bool same = row_offset(Y) == off;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[i][e] *= s;
      store_unit(Y, k, i * T + t, same, unit_pack<kBf16>(g[i]));
    }
    if (k.extra >= 0) Y[k.extra] = to16<kBf16>(ge * s);
  }
}

// A lane's extra value of a coming row, copied to shared memory asynchronously like
// the units: a plain load in flight shares a scoreboard with the shared-memory loads
// and stalls them (16384 x 5279 88 -> 69 us). The copy takes the aligned pair of
// values that the extra one is in; past the row's end nothing is read, before its
// start the end of the previous row (`first`: there is none).
__device__ __forceinline__ void copy_extra(uint32_t dst, const uint16_t *row, const RowWalk &k,
                                           int cols, bool first) {
  if (k.extra < 0) return;
  const uint16_t *p = row + k.extra;
  const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) >> 1) & 1u;
  if (first && odd && k.extra == 0) {
    asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(dst + 2), "h"(*p) : "memory");
  } else {
    cp_async_4(dst, p - odd, !odd && k.extra + 1 == cols ? 2u : 4u);
  }
}
// Where in its four bytes the extra value is.
__device__ __forceinline__ uint32_t extra_at(const void *row, const RowWalk &k) {
  return static_cast<uint32_t>((reinterpret_cast<uintptr_t>(row) >> 1) + (k.extra & 1)) & 1u;
}

// Many rows: blocks walk rows blockIdx.x, + gridDim.x, ... (T = 32: one warp per
// row, the block's warps on rows of their own), and every thread copies its own
// units of the next rows into shared memory, `stages` rows deep, so that memory is
// busy during the reductions and the stores and no thread waits for another's
// copies. X and R must be aligned alike; the stride between a block's rows is a
// multiple of 8 rows, so that all have the same alignment and a thread the same
// columns of W in each.
//
// 512 threads per SM with 4 units of 8 values each: what a row costs a thread beside
// its values (the reduction, the scale, addresses) is as much as some 20 values, and
// 1024 threads with 2 units took 94 us, not 63, at 16384 x 6144 and 135, not 76, with
// 8-bit output.
constexpr int kNormThreads = 512, kNormUnits = 4;

template <bool kLayer, bool kBf16, bool kOut8, int T>
__global__ void __launch_bounds__(T > 32 ? T : kNormThreads, T > 32 ? kNormThreads / T : 1)
    norm_ring_kernel(const NormCall c, int stages) {
  static_assert(!(kLayer && kOut8), "layer norm has 16-bit output");
  constexpr int NV = kNormUnits;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float2 red[2][T / 32];
  constexpr uint32_t kSlab = NV * T * 16;  // one matrix's row, unit u at 16 u
  const int t = static_cast<int>(threadIdx.x) % T, group = static_cast<int>(threadIdx.x) / T;
  const int groups = T > 32 ? 1 : static_cast<int>(blockDim.x) / T;
  auto sync = [] {
    if constexpr (T > 32) {
      __syncthreads();
    } else {
      __syncwarp();
    }
  };
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int rows = slot < c.rows ? static_cast<int>((c.rows - slot + step - 1) / step) : 0;
  if (rows == 0) return;  // a whole group
  const int mats = c.R ? 2 : 1;
  const uint16_t *X = c.X + slot * c.ldx, *R = c.R ? c.R + slot * c.ldr : nullptr;
  uint16_t *H = c.H ? c.H + slot * c.ldh : nullptr;
  constexpr int kSize = kOut8 ? 1 : 2;
  uint8_t *out = static_cast<uint8_t *>(c.Y) + slot * c.ldy * kSize;
  float *rstd = c.rstd ? c.rstd + slot : nullptr, *scales = kOut8 ? c.scale + slot : nullptr;
  const int64_t step_x = step * c.ldx, step_r = step * c.ldr, step_h = step * c.ldh;
  const int64_t step_y = step * c.ldy * kSize;
  const int off = row_offset(X);
  const RowWalk k = row_walk(X, c.cols, t);
  const bool ragged = c.cols != 8 * k.units;  // rows with a head or a tail
  const float inv_n = 1.f / static_cast<float>(c.cols);
  uint8_t *mine = ring + static_cast<uint32_t>(group * stages * mats) * kSlab;
  // The extra values: 16 lanes' words per row and matrix, behind the units.
  uint8_t *side = ring + static_cast<uint32_t>(groups * stages * mats) * kSlab +
                  static_cast<uint32_t>(group * stages * mats) * 64u + t * 4;
  const uint32_t side_at = 2 * extra_at(X, k);
  const uint16_t *fx = X, *fr = R;
  const int first_unit = k.head + 8 * t;
  int filled = 0;
  auto fill = [&](int stage) {
    if (filled < rows) {
      const uint32_t dst = smem_u32(mine) + static_cast<uint32_t>(stage * mats) * kSlab + t * 16;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * T + t >= k.units) continue;
        cp_async_16(dst + i * T * 16, fx + first_unit + i * T * 8, 16);
        if (fr) cp_async_16(dst + kSlab + i * T * 16, fr + first_unit + i * T * 8, 16);
      }
      if (ragged) {
        const uint32_t to = smem_u32(side) + static_cast<uint32_t>(stage * mats) * 64u;
        const bool top_row = slot == 0 && filled == 0;
        copy_extra(to, fx, k, c.cols, top_row);
        if (fr) copy_extra(to + 64, fr, k, c.cols, top_row);
      }
      fx += step_x;
      if (fr) fr += step_r;
      ++filled;
    }
    cp_async_commit();
  };
  for (int n = 0; n < stages; ++n) fill(n);
  const uint32_t one = kBf16 ? 0x3f803f80u : 0x3c003c00u;  // no gain: ones
  uint4 w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    w[i] = c.W ? load_unit(c.W, k, i * T + t, row_offset(c.W) == off)
               : make_uint4(one, one, one, one);
  const float we = c.W ? from16<kBf16>(load_extra(c.W, k)) : 1.f;
  uint4 b[kLayer ? NV : 1];
  float be = 0.f;
  float *mean = nullptr;
  if constexpr (kLayer) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      b[i] = load_unit(c.B, k, i * T + t, row_offset(c.B) == off);
    be = from16<kBf16>(load_extra(c.B, k));
    mean = c.mean ? c.mean + slot : nullptr;
  }
  int stage = 0;
  for (int n = 0; n < rows; ++n) {
    const bool same_h = row_offset(H) == off;
    switch (stages) {  // all but the newest stages - 1 rows are there
      case 2: cp_async_wait<1>(); break;
      case 3: cp_async_wait<2>(); break;
      default: cp_async_wait<3>(); break;
    }
    uint8_t *row = mine + static_cast<uint32_t>(stage * mats) * kSlab;
    float he = 0.f, ge = 0.f;
    if (ragged && k.extra >= 0) {
      const uint8_t *from = side + static_cast<uint32_t>(stage * mats) * 64u + side_at;
      he = from16<kBf16>(*reinterpret_cast<const uint16_t *>(from));
      if (R) he += from16<kBf16>(*reinterpret_cast<const uint16_t *>(from + 64));
      ge = he * we;
    }
    F2 g[NV][4], sums = f2(0.f);  // layer: h, then h - m
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * T + t;
      if (u >= k.units) continue;
      const uint4 x = *reinterpret_cast<const uint4 *>(row + 16 * u), wi = per_row(w[i]);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, ww[4] = {wi.x, wi.y, wi.z, wi.w};
      F2 h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = unpack2<kBf16>(xw[q]);
      if (R) {
        const uint4 b = *reinterpret_cast<const uint4 *>(row + kSlab + 16 * u);
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = add2(h[q], unpack2<kBf16>(bw[q]));
      }
      if (H)
        store_unit(H, k, u, same_h, make_uint4(pack2<kBf16>(h[0]), pack2<kBf16>(h[1]),
                                               pack2<kBf16>(h[2]), pack2<kBf16>(h[3])));
      if constexpr (kLayer) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sums = add2(sums, h[q]);
          g[i][q] = h[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sums = fma2(h[q], h[q], sums);
          g[i][q] = mul2(h[q], unpack2<kBf16>(ww[q]));
          if constexpr (kOut8) {
            float a, b;
            split(g[i][q], a, b);
            top = max_nan(top, max_nan(fabsf(a), fabsf(b)));
          }
        }
      }
    }
    float sum, sum1;
    split(sums, sum, sum1);
    sum += sum1;
    if constexpr (kLayer) {
      if (ragged && k.extra >= 0) {
        sum += he;
        if (H) H[k.extra] = to16<kBf16>(he);
      }
      const float m = quotient(row_sum<T>(sum, reinterpret_cast<float *>(red[n & 1])),
                               static_cast<float>(c.cols), inv_n);
      const F2 minus = f2(-m);
      sums = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * T + t >= k.units) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          g[i][q] = add2(g[i][q], minus);
          sums = fma2(g[i][q], g[i][q], sums);
        }
      }
      split(sums, sum, sum1);
      sum += sum1;
      he -= m;
      if (ragged && k.extra >= 0) sum = fmaf(he, he, sum);
      ge = he * we;
      if (t == 0 && mean) mean[0] = m;
      sum = row_sum<T>(sum, reinterpret_cast<float *>(red[n & 1]) + (T > 32 ? T / 32 : 0));
    } else if (ragged && k.extra >= 0) {
      sum = fmaf(he, he, sum);
      if (kOut8) top = max_nan(top, fabsf(ge));
      if (H) H[k.extra] = to16<kBf16>(he);
    }
    if constexpr (kOut8) {
      row_reduce<T>(sum, top, red[n & 1]);
    } else if constexpr (!kLayer) {
      sum = row_sum<T>(sum, reinterpret_cast<float *>(red[n & 1]));
    }
    const float s = rsqrtf(sum * inv_n + c.eps);
    if (t == 0 && rstd) rstd[0] = s;
    const F2 s2 = f2(s);
    if constexpr (kOut8) {
      const float inv = e4m3_inverse(top * s);
      if (t == 0) scales[0] = e4m3_scale(top * s);
      uint8_t *Y = out;
      const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(Y) & 7);
      const bool whole = ((lead + k.head) & 7) == 0, shifted = !whole && lead == 0 && k.units > 0;
      const F2 inv2 = f2(inv);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = i * T + t;
        if (u >= k.units) continue;
        uint32_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y0, y1;
          split(mul2(mul2(g[i][q], s2), inv2), y0, y1);
          b[q] = e4m3x2(y0, y1);
        }
        const uint64_t v =
            static_cast<uint64_t>(b[2] | (b[3] << 16)) << 32 | (b[0] | (b[1] << 16));
        uint8_t *p = Y + k.head + 8 * u;
        if (whole) {
          *reinterpret_cast<uint64_t *>(p) = v;
        } else if (shifted) {
          *reinterpret_cast<uint64_t *>(row + 16 * u) = v;  // in place of X's unit
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = static_cast<uint8_t>(v >> (8 * e));
        }
      }
      if (k.extra >= 0) Y[k.extra] = static_cast<uint8_t>(e4m3x2(ge * s * inv, 0.f));
      if (shifted) {
        sync();
        store_shifted(Y, k, t, T, [&](int u) {
          return *reinterpret_cast<const uint64_t *>(row + 16 * u);
        });
        sync();  // before the next row is copied over the units
      }
    } else {
      uint16_t *Y = reinterpret_cast<uint16_t *>(out);
      const bool same_y = row_offset(Y) == off;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int u = i * T + t;
        if (u >= k.units) continue;
        if constexpr (kLayer) {
          const uint4 wi = per_row(w[i]), bi = per_row(b[i]);
          const uint32_t ww[4] = {wi.x, wi.y, wi.z, wi.w}, bw[4] = {bi.x, bi.y, bi.z, bi.w};
          uint32_t y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            y[q] = pack2<kBf16>(
                fma2(mul2(g[i][q], s2), unpack2<kBf16>(ww[q]), unpack2<kBf16>(bw[q])));
          store_unit(Y, k, u, same_y, make_uint4(y[0], y[1], y[2], y[3]));
        } else {
          store_unit(Y, k, u, same_y,
                     make_uint4(pack2<kBf16>(mul2(g[i][0], s2)), pack2<kBf16>(mul2(g[i][1], s2)),
                                pack2<kBf16>(mul2(g[i][2], s2)), pack2<kBf16>(mul2(g[i][3], s2))));
        }
      }
      if (k.extra >= 0) Y[k.extra] = to16<kBf16>(kLayer ? fmaf(ge, s, be) : ge * s);
    }
    fill(stage);
    if (++stage == stages) stage = 0;
    if (H) H += step_h;
    out += step_y;
    if (rstd) rstd += step;
    if (kLayer && mean) mean += step;
    if (kOut8) scales += step;
  }
}

// Sums of rows of any length. A thread's values, 1024 columns apart, are added 8 at a
// time, and those sums with compensation: `low` collects what each addition to `sum` rounds
// off (the two-sum of D. Knuth, "The Art of Computer Programming" 2, 4.2.2). Added in one
// chain, whose error grows with the row, 2^26 values of 1 + 2^-10 had a mean of 1 + 2^-12.
// (bf16 8192 x 20000 with a residual 372 us, in one chain with fewer loads in flight 472;
// without 321, 298; layer norm's gradient 820, 1197.)
struct LongSum {
  float sum = 0.f, low = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = sum + v, w = t - sum;
    low += (sum - (t - w)) + (v - w);
    sum = t;
  }
  // (An infinite sum has no remainder.)
  __device__ __forceinline__ float value() const { return fabsf(sum) <= kFltMax ? sum + low : sum; }
};
// column(j) for each of the thread's columns, eight() after every 8 of them.
template <typename Column, typename Eight>
__device__ __forceinline__ void walk_long(int cols, Column &&column, Eight &&eight) {
  for (int64_t j0 = threadIdx.x; j0 < cols; j0 += 8 * 1024) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j0 + i * 1024 < cols) column(j0 + i * 1024);
    eight();
  }
}

// Rows of any length: each block walks its row twice (the second pass reads it
// from L2).
template <bool kLayer, bool kBf16>
__global__ void __launch_bounds__(1024, kLayer ? 2 : 1) norm_long_kernel(const NormCall c) {
  __shared__ __align__(16) float2 red[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint16_t *X = c.X + r * c.ldx, *R = c.R ? c.R + r * c.ldr : nullptr;
  if constexpr (kLayer) {
    float *slots = reinterpret_cast<float *>(red);
    const float inv_n = 1.f / static_cast<float>(c.cols);
    auto value = [&](int64_t j) {
      const float h = from16<kBf16>(X[j]);
      return R ? h + from16<kBf16>(R[j]) : h;
    };
    LongSum sums, squares;
    float part = 0.f;
    walk_long(c.cols, [&](int64_t j) { part += value(j); }, [&] { sums.add(part), part = 0.f; });
    const float m =
        quotient(row_sum<1024>(sums.value(), slots), static_cast<float>(c.cols), inv_n);
    walk_long(
        c.cols,
        [&](int64_t j) {
          const float d = value(j) - m;
          part = fmaf(d, d, part);
        },
        [&] { squares.add(part), part = 0.f; });
    const float s = rsqrtf(row_sum<1024>(squares.value(), slots + 32) * inv_n + c.eps);
    if (threadIdx.x == 0) {
      if (c.mean) c.mean[r] = m;
      if (c.rstd) c.rstd[r] = s;
    }
    for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
      const float h = value(j);
      if (c.H) c.H[r * c.ldh + j] = to16<kBf16>(h);
      static_cast<uint16_t *>(c.Y)[r * c.ldy + j] =
          to16<kBf16>(fmaf((h - m) * s, c.W ? from16<kBf16>(c.W[j]) : 1.f,
                           c.B ? from16<kBf16>(c.B[j]) : 0.f));
    }
    return;
  }
  LongSum squares;
  float part = 0.f, top = 0.f;
  walk_long(
      c.cols,
      [&](int64_t j) {
        float h = from16<kBf16>(X[j]);
        if (R) h += from16<kBf16>(R[j]);
        part = fmaf(h, h, part);
        top = max_nan(top, fabsf(c.W ? h * from16<kBf16>(c.W[j]) : h));
      },
      [&] { squares.add(part), part = 0.f; });
  float sum = squares.value();
  row_reduce<1024>(sum, top, red);
  const float s = rsqrtf(sum / static_cast<float>(c.cols) + c.eps);
  if (threadIdx.x == 0 && c.rstd) c.rstd[r] = s;
  const float inv = e4m3_inverse(top * s);
  if (threadIdx.x == 0 && c.scale) c.scale[r] = e4m3_scale(top * s);
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
// row per block. The launcher makes
// the stride between a block's rows a multiple of 8 rows, so that all of them
// have the same alignment and a thread the same columns in each.
template <bool kLayer, bool kBf16, int NV>
struct GradSums {
  uint4 w[NV];
  uint32_t we;
  F2 dw[NV][4], db[kLayer ? NV : 1][4];
  float dwe, dbe;

  template <int T>
  __device__ __forceinline__ void begin(const NormGradCall &c, const RowWalk &k, int off, int t) {
    dwe = dbe = 0.f;
    const uint32_t one = kBf16 ? 0x3f803f80u : 0x3c003c00u;  // no gain: ones
    we = c.W ? load_extra(c.W, k) : one & 0xffffu;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        dw[i][q] = f2(0.f);
        if constexpr (kLayer) db[i][q] = f2(0.f);
      }
      w[i] = c.W ? load_unit(c.W, k, i * T + t, row_offset(c.W) == off)
                 : make_uint4(one, one, one, one);
    }
  }
  // Sums number `which` (0: dw, 1: db) of unit i's pair q, and of the extra column.
  __device__ __forceinline__ F2 pair(int which, int i, int q) const {
    if constexpr (kLayer) return which ? db[i][q] : dw[i][q];
    return dw[i][q];
  }
  __device__ __forceinline__ float last(int which) const { return kLayer && which ? dbe : dwe; }

  template <int T>
  __device__ __forceinline__ void end(int which, float *out, const RowWalk &k, int t) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * T + t >= k.units) continue;
      float *p = out + k.head + 8 * (i * T + t);
#pragma unroll
      for (int q = 0; q < 4; ++q) split(pair(which, i, q), p[2 * q], p[2 * q + 1]);
    }
    if (k.extra >= 0) out[k.extra] = last(which);
  }
};

// One row by T threads. get(a, i): packed unit i of this thread of matrix a (0:
// dY, 1: H, 2: dH), called for units inside the row; extra[a]: its extra value.
// Units are read twice, before and after the reduction, instead of being held in
// registers over it. between() runs behind the reduction. X: the row of dX; back:
// whether there is a dH; inv_n: 1 / cols.
//
// With t = dy s: dw += t h and sum(g n) = sum(t w h), so that
// dx = s (dy w - h (s mean(g n))) + dh takes three operations per value, on packed
// pairs. (No s^2, which overflows for s above 1.8e19 where dx need not.) The layer
// norm's h is h - m throughout, and dy w loses mean(g), whose sum is reduced with
// the other one.
template <bool kLayer, bool kBf16, int T, int NV, typename Get, typename Between>
__device__ __forceinline__ void grad_row(uint16_t *X, const RowWalk &k, bool same, bool past,
                                         int t, GradSums<kLayer, kBf16, NV> &sums, float s,
                                         float m, float inv_n, const uint32_t (&extra)[3],
                                         float *red, Get &&get, Between &&between) {
  const F2 s2 = f2(s), minus = f2(-m);
  F2 dots = f2(0.f), levels = f2(0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * T + t < k.units) {
      const uint4 y = get(0, i), h = get(1, i), w = per_row(sums.w[i]);
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w}, hw[4] = {h.x, h.y, h.z, h.w};
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const F2 ts = mul2(unpack2<kBf16>(yw[q]), s2);
        F2 hv = unpack2<kBf16>(hw[q]);
        if constexpr (kLayer) {
          hv = add2(hv, minus);
          sums.db[i][q] = add2(sums.db[i][q], unpack2<kBf16>(yw[q]));
          levels = fma2(unpack2<kBf16>(yw[q]), unpack2<kBf16>(ww[q]), levels);
        }
        sums.dw[i][q] = fma2(ts, hv, sums.dw[i][q]);
        dots = fma2(mul2(ts, unpack2<kBf16>(ww[q])), hv, dots);
      }
    }
  }
  float dot, dot1;
  split(dots, dot, dot1);
  dot += dot1;
  const float ye = from16<kBf16>(extra[0]);
  const float he = kLayer ? from16<kBf16>(extra[1]) - m : from16<kBf16>(extra[1]);
  const float we = from16<kBf16>(sums.we);
  float level = 0.f;
  if constexpr (kLayer) {
    float level1;
    split(levels, level, level1);
    level += level1;
  }
  if (k.extra >= 0) {
    sums.dwe = fmaf(ye * s, he, sums.dwe);
    dot = fmaf(ye * s * we, he, dot);
    if constexpr (kLayer) {
      sums.dbe += ye;
      level = fmaf(ye, we, level);
    }
  }
  if constexpr (kLayer) {
    row_sums<T>(dot, level, reinterpret_cast<float2 *>(red));
    level *= -inv_n;
  } else {
    dot = row_sum<T>(dot, red);
  }
  between();
  const float back = -s * (dot * inv_n);
  const F2 back2 = f2(back), level2 = f2(level);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * T + t < k.units) {
      const uint4 y = get(0, i), h = get(1, i), w = per_row(sums.w[i]);
      const uint4 b = past ? get(2, i) : make_uint4(0, 0, 0, 0);
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w}, hw[4] = {h.x, h.y, h.z, h.w};
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, bw[4] = {b.x, b.y, b.z, b.w};
      uint32_t out[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (kLayer) {
          out[q] = pack2<kBf16>(
              fma2(fma2(add2(unpack2<kBf16>(hw[q]), minus), back2,
                        fma2(unpack2<kBf16>(yw[q]), unpack2<kBf16>(ww[q]), level2)),
                   s2, unpack2<kBf16>(bw[q])));
        } else {
          out[q] = pack2<kBf16>(
              fma2(fma2(unpack2<kBf16>(hw[q]), back2,
                        mul2(unpack2<kBf16>(yw[q]), unpack2<kBf16>(ww[q]))),
                   s2, unpack2<kBf16>(bw[q])));
        }
      }
      store_unit(X, k, i * T + t, same, make_uint4(out[0], out[1], out[2], out[3]));
    }
  }
  if (k.extra >= 0) {
    const float g = kLayer ? fmaf(ye, we, level) : ye * we;
    X[k.extra] = to16<kBf16>(fmaf(fmaf(he, back, g), s, from16<kBf16>(extra[2])));
  }
}

// Short rows of matrices that are aligned differently: one warp per row, straight
// from global memory; the warps in residence hide each other's latency.
template <int NV>
constexpr int kGradWarpBlocks = NV == 1 ? 6 : 4;  // per SM

template <bool kLayer, bool kBf16, int NV>
__global__ void __launch_bounds__(128, kGradWarpBlocks<NV>)
    norm_grad_warp_kernel(const NormGradCall c, float *part) {
  const int t = static_cast<int>(threadIdx.x) & 31;
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  grid_dependency_wait();
  grid_launch_dependents();
  const int off = row_offset(c.dY + slot * c.lddy);
  const RowWalk k = row_walk(c.dY + slot * c.lddy, c.cols, t);
  GradSums<kLayer, kBf16, NV> sums;
  sums.template begin<32>(c, k, off, t);
  for (int64_t r = slot; r < c.rows; r += static_cast<int64_t>(gridDim.x) * 4) {
    const uint16_t *rows[3] = {c.dY + r * c.lddy, c.H + r * c.ldh,
                               c.dH ? c.dH + r * c.lddh : nullptr};
    uint4 v[3][NV];
    uint32_t extra[3];
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      const bool same = row_offset(rows[a]) == off;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[a][i] = load_unit(rows[a], k, i * 32 + t, same);
      extra[a] = load_extra(rows[a], k);
    }
    uint16_t *X = c.dX + r * c.lddx;
    grad_row<kLayer, kBf16, 32, NV>(X, k, row_offset(X) == off, c.dH != nullptr, t, sums,
                                    c.rstd[r], kLayer ? c.mean[r] : 0.f,
                                    1.f / static_cast<float>(c.cols), extra, nullptr,
                                    [&](int a, int i) { return v[a][i]; }, [] {});
  }
  if (part == nullptr) return;
  // The block's warps add their sums in warp order (their rows may be aligned
  // differently, so a column sits in different lanes).
  __shared__ float mine[4][64 * NV * 4 + 8];
#pragma unroll
  for (int which = 0; which < (kLayer ? 2 : 1); ++which) {
    if (which) __syncthreads();
    sums.template end<32>(which, mine[threadIdx.x >> 5], k, t);
    __syncthreads();
    for (int j = threadIdx.x; j < c.cols; j += 128)
      part[(which * static_cast<int64_t>(gridDim.x) + blockIdx.x) * c.cols + j] =
          ((mine[0][j] + mine[1][j]) + mine[2][j]) + mine[3][j];
  }
}

// Longer rows: one block per row, rows brought by bulk copies into a ring of
// `stages` rows of shared memory (the whole units of dY, H and dH, which must be
// aligned alike, and dX with them), so stages - 1 rows are always in flight
// whatever the threads do, and the values cost no registers between the two
// passes over them. (Prefetching the next row into registers reached 96 us at
// 8192 x 8192, and 143 us once the extra columns' loads shared their
// scoreboards.) What bounds it beside memory is instructions: packed pairs, no
// division for the ring's indexes and no 64-bit products per row.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

constexpr int kMaxGradStages = 4;

// Wide rows take 512 threads per SM with 4 units each, as in the forward pass, for
// what a row costs a thread beside its values (8192 rows: 5280 columns 62 -> 56 us,
// 8192 86.4 -> 84.9, 10240 124 -> 105, 16384 205 -> 182, against 1024 with 2 units).
template <bool kLayer, bool kBf16, int T, int NV>
__global__ void __launch_bounds__(T, (NV > 2 ? 512 : 1024) / T)
    norm_grad_kernel(const NormGradCall c, float *part, int stages, uint32_t *err_word) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxGradStages];
  __shared__ __align__(16) float red[2][(kLayer ? 2 : 1) * T / 32];
  __shared__ int abort_flag;
  volatile int *abort = &abort_flag;
  const int t = static_cast<int>(threadIdx.x);
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  // Pointers to this block's first row, advanced by a fixed number of elements.
  const int64_t slot = blockIdx.x;
  const int rows = static_cast<int>((c.rows - slot + gridDim.x - 1) / gridDim.x);
  const uint16_t *Y = c.dY + slot * c.lddy, *H = c.H + slot * c.ldh;
  const uint16_t *B = c.dH ? c.dH + slot * c.lddh : nullptr;
  uint16_t *X = c.dX + slot * c.lddx;
  const float *rstd = c.rstd + slot;
  const int64_t step_y = gridDim.x * c.lddy, step_h = gridDim.x * c.ldh;
  const int64_t step_b = gridDim.x * c.lddh, step_x = gridDim.x * c.lddx;
  const RowWalk k = row_walk(Y, c.cols, t);
  const bool ragged = c.cols != 8 * k.units;  // rows with a head or a tail
  const uint32_t bytes = static_cast<uint32_t>(k.units) * 16u;
  const uint32_t slab = (static_cast<uint32_t>(c.cols) / 8u) * 16u;  // one matrix's row
  // The next row to copy (thread 0), and its stage.
  const uint16_t *fy = Y + k.head, *fh = H + k.head, *fb = B ? B + k.head : nullptr;
  int filled = 0, fstage = 0;
  auto fill = [&] {
    if (filled == rows || bytes == 0) return;
    const uint32_t bar = smem_u32(&full[fstage]);
    const uint32_t dst = smem_u32(ring) + static_cast<uint32_t>(fstage) * 3u * slab;
    mbar_arrive_expect_tx(bar, fb ? 3u * bytes : 2u * bytes);
    bulk_load(dst, fy, bytes, bar);
    bulk_load(dst + slab, fh, bytes, bar);
    if (fb) bulk_load(dst + 2 * slab, fb, bytes, bar);
    fy += step_y, fh += step_h;
    if (fb) fb += step_b;
    ++filled;
    if (++fstage == stages) fstage = 0;
  };
  if (t == 0)
    for (int n = 0; n < stages - 1; ++n) fill();
  GradSums<kLayer, kBf16, NV> sums;
  sums.template begin<T>(c, k, row_offset(Y), t);
  uint32_t stage = 0, phase = 0;
  const float inv_n = 1.f / static_cast<float>(c.cols);
  float s = *rstd;
  const float *mean = kLayer ? c.mean + slot : nullptr;
  float m = kLayer ? *mean : 0.f;
  uint32_t extra[3] = {0, 0, 0};
  for (int n = 0; n < rows; ++n) {
    if (ragged) {
      extra[0] = load_extra(Y, k);
      extra[1] = load_extra(H, k);
      extra[2] = load_extra(B, k);
    }
    float s2 = 0.f, m2 = 0.f;
    if (n + 1 < rows) {
      s2 = rstd[gridDim.x];
      if constexpr (kLayer) m2 = mean[gridDim.x];
    }
    if (bytes != 0)
      mbar_wait_bounded(smem_u32(&full[stage]), phase, abort, err_word, kWaitFull);
    const uint8_t *row = ring + stage * 3u * slab + t * 16;
    grad_row<kLayer, kBf16, T, NV>(
        X, k, true, B != nullptr, t, sums, s, m, inv_n, extra, red[n & 1],
        [&](int a, int i) {
          return *reinterpret_cast<const uint4 *>(row + a * slab + i * T * 16);
        },
        [&] {
          // Behind the reduction's barrier every thread has left the previous
          // row, whose stage takes the row stages - 1 ahead.
          if (t == 0) fill();
        });
    s = s2, m = m2;
    Y += step_y, H += step_h, X += step_x, rstd += gridDim.x;
    if constexpr (kLayer) mean += gridDim.x;
    if (B) B += step_b;
    if (++stage == static_cast<uint32_t>(stages)) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // After a wait that gave up: never leave with a copy still writing.
  if (t == 0 && *abort && bytes != 0) {
    volatile int never = 0;
    for (int i = rows > stages ? rows - stages : 0; i < rows; ++i)
      mbar_wait_bounded(smem_u32(&full[i % stages]), static_cast<uint32_t>(i / stages) & 1u, &never,
                        err_word, kWaitDrain);
  }
  if (part == nullptr) return;
  // The block's partial row goes out in whole lines: through shared memory (the
  // ring is free), value e of unit u at e * pitch + u, with a pitch that spreads
  // the 32 consecutive columns a warp reads back over the banks. Written from
  // the threads directly, 8 columns apart per lane, it took longer than a row.
  float *sums8 = reinterpret_cast<float *>(ring);
  const int pitch = (k.units + 27) / 32 * 32 + 4;  // 4 modulo 32, at least units
#pragma unroll
  for (int which = 0; which < (kLayer ? 2 : 1); ++which) {
    float *out = part + (which * static_cast<int64_t>(gridDim.x) + slot) * c.cols;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * T + t;
      if (u >= k.units) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        split(sums.pair(which, i, q), sums8[2 * q * pitch + u], sums8[(2 * q + 1) * pitch + u]);
    }
    if (k.extra >= 0) out[k.extra] = sums.last(which);
    __syncthreads();
    for (int j = t; j < 8 * k.units; j += T)
      out[k.head + j] = sums8[(j & 7) * pitch + (j >> 3)];
  }
}

// Rows of up to 2048 columns whose matrices are aligned alike: one warp per row.
// Every lane copies its own units of the warp's next rows into shared memory
// (asynchronous 16-byte copies), so that no row waits for a block's barrier, no
// lane for another's copies, and the next rows are in flight whatever the warp
// does. (Bulk copies instead, three of 512 bytes per row, took 25 us against 19
// at 32768 x 256.) The block's warps add their sums of dw at the end: one partial
// row per block. Memory bounds it: 32768 x 1024 with dh 47.5 us, 5.7 TB/s.
template <int NV>
constexpr int kGradRowStages = NV == 8 ? 2 : 8 / NV;
// At most: 192 KB of rows per SM. (The layer norm keeps two sums per value: 8 warps
// where 16 would spill.)
template <bool kLayer, int NV>
constexpr int kGradRowWarps = NV == 8 || (kLayer && NV == 4) ? 8 : 16;

// Where column j of a warp's sums is kept: lanes 8 columns apart hit all banks.
__device__ __forceinline__ int sums_at(int j) { return j + (j >> 5); }

template <bool kLayer, bool kBf16, int NV>
__global__ void __launch_bounds__(32 * kGradRowWarps<kLayer, NV>, 1)
    norm_grad_rows_kernel(const NormGradCall c, float *part) {
  constexpr int kStages = kGradRowStages<NV>;
  constexpr uint32_t kSlab = NV * 512;  // one matrix's row
  extern __shared__ __align__(128) uint8_t ring[];
  const int t = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int warps = static_cast<int>(blockDim.x) >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * warps + warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
  const int rows = slot < c.rows ? static_cast<int>((c.rows - slot + step - 1) / step) : 0;
  const uint16_t *Y = c.dY + slot * c.lddy, *H = c.H + slot * c.ldh;
  const uint16_t *B = c.dH ? c.dH + slot * c.lddh : nullptr;
  uint16_t *X = c.dX + slot * c.lddx;
  const float *rstd = c.rstd + slot;
  const int64_t step_y = step * c.lddy, step_h = step * c.ldh;
  const int64_t step_b = step * c.lddh, step_x = step * c.lddx;
  const RowWalk k = row_walk(Y, c.cols, t);
  uint8_t *mine = ring + static_cast<uint32_t>(warp) * kStages * 3 * kSlab + t * 16;
  // The warp's next row to copy: this lane's units, rstd and extra values.
  const uint16_t *fy = Y + k.head + 8 * t, *fh = H + k.head + 8 * t;
  const uint16_t *fb = B ? B + k.head + 8 * t : nullptr;
  int filled = 0;
  auto fill = [&](uint32_t stage) {
    if (filled < rows) {
      const uint32_t dst = smem_u32(mine) + stage * 3 * kSlab;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * 32 + t >= k.units) continue;
        cp_async_16(dst + i * 512, fy + i * 256, 16);
        cp_async_16(dst + kSlab + i * 512, fh + i * 256, 16);
        if (fb) cp_async_16(dst + 2 * kSlab + i * 512, fb + i * 256, 16);
      }
      fy += step_y, fh += step_h;
      if (fb) fb += step_b;
      ++filled;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < kStages; ++n) fill(n);
  GradSums<kLayer, kBf16, NV> sums;
  sums.template begin<32>(c, k, row_offset(Y), t);
  uint32_t stage = 0;
  const float inv_n = 1.f / static_cast<float>(c.cols);
  float s = 0.f, m = 0.f;
  const float *mean = kLayer ? c.mean + slot : nullptr;
  uint32_t extra[3] = {0, 0, 0};
  if (rows > 0) {
    s = *rstd;
    if constexpr (kLayer) m = *mean;
    extra[0] = load_extra(Y, k), extra[1] = load_extra(H, k), extra[2] = load_extra(B, k);
  }
  for (int n = 0; n < rows; ++n) {
    Y += step_y, H += step_h, rstd += step;
    if (B) B += step_b;
    if constexpr (kLayer) mean += step;
    float s2 = 0.f, m2 = 0.f;
    uint32_t extra2[3] = {0, 0, 0};
    if (n + 1 < rows) {
      s2 = *rstd;
      if constexpr (kLayer) m2 = *mean;
      extra2[0] = load_extra(Y, k), extra2[1] = load_extra(H, k), extra2[2] = load_extra(B, k);
    }
    cp_async_wait<kStages - 1>();
    const uint8_t *row = mine + stage * 3 * kSlab;
    grad_row<kLayer, kBf16, 32, NV>(
        X, k, true, c.dH != nullptr, t, sums, s, m, inv_n, extra, nullptr,
        [&](int a, int i) {
          return *reinterpret_cast<const uint4 *>(row + a * kSlab + i * 512);
        },
        [] {});
    fill(stage);
    X += step_x;
    s = s2, m = m2;
    extra[0] = extra2[0], extra[1] = extra2[1], extra[2] = extra2[2];
    if (++stage == kStages) stage = 0;
  }
  if (part == nullptr) return;
  __syncthreads();  // the ring is free
  constexpr int kSets = kLayer ? 2 : 1;
  const int pitch = sums_at(c.cols) + 1;
  float *all = reinterpret_cast<float *>(ring), *own = all + warp * pitch;
  const int apart = warps * pitch;  // db's sums behind dw's
#pragma unroll
  for (int which = 0; which < kSets; ++which) {
    float *to = own + which * apart;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * 32 + t >= k.units) continue;
      const int j = k.head + 8 * (i * 32 + t);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        split(sums.pair(which, i, q), to[sums_at(j + 2 * q)], to[sums_at(j + 2 * q + 1)]);
    }
    if (k.extra >= 0) to[sums_at(k.extra)] = sums.last(which);
  }
  __syncthreads();
  // Eight loads in flight per thread; the adds are in warp order.
  const int stride = 32 * warps;
#pragma unroll
  for (int which = 0; which < kSets; ++which) {
    const float *sums_of = all + which * apart;
    for (int j = threadIdx.x; j < c.cols; j += 2 * stride) {
      const bool two = j + stride < c.cols;
      const int at0 = sums_at(j), at1 = sums_at(two ? j + stride : j);
      float v0 = 0.f, v1 = 0.f;
      for (int w = 0; w < warps; w += 4) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float *from = sums_of + min(w + i, warps - 1) * pitch;
          a[i] = from[at0], b[i] = from[at1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (w + i < warps) v0 += a[i], v1 += b[i];
      }
      const int64_t row = kLayer ? which * static_cast<int64_t>(gridDim.x) + blockIdx.x : blockIdx.x;
      float *out = part + row * c.cols + j;
      out[0] = v0;
      if (two) out[stride] = v1;
    }
  }
}

// Rows of any length and alignment: one block per group of rows; the partial sums of dw live
// in the block's partial row in global memory.
template <bool kLayer, bool kBf16>
__global__ void __launch_bounds__(1024, 2)
    norm_grad_long_kernel(const NormGradCall c, float *part) {
  __shared__ __align__(16) float red[2][kLayer ? 64 : 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const float inv_n = 1.f / static_cast<float>(c.cols);
  float *mine = part ? part + blockIdx.x * static_cast<int64_t>(c.cols) : nullptr;
  float *mine_b = kLayer && part ? mine + gridDim.x * static_cast<int64_t>(c.cols) : nullptr;
  int flip = 0;
  bool first = true;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const uint16_t *dY = c.dY + r * c.lddy, *H = c.H + r * c.ldh;
    const float s = c.rstd[r], m = kLayer ? c.mean[r] : 0.f;
    LongSum dots, levels;
    float dot = 0.f, level = 0.f;
    walk_long(
        c.cols,
        [&](int64_t j) {
          const float d = from16<kBf16>(dY[j]);
          const float n = (kLayer ? from16<kBf16>(H[j]) - m : from16<kBf16>(H[j])) * s;
          if constexpr (kLayer) {
            level += c.W ? d * from16<kBf16>(c.W[j]) : d;
            if (mine) mine_b[j] = first ? d : d + mine_b[j];
          }
          dot = fmaf(c.W ? d * from16<kBf16>(c.W[j]) : d, n, dot);
          if (mine) mine[j] = first ? d * n : fmaf(d, n, mine[j]);  // this thread's own element
        },
        [&] {
          dots.add(dot), dot = 0.f;
          if constexpr (kLayer) levels.add(level), level = 0.f;
        });
    dot = dots.value();
    if constexpr (kLayer) {
      level = levels.value();
      row_sums<1024>(dot, level, reinterpret_cast<float2 *>(red[flip]));
    } else {
      dot = row_sum<1024>(dot, red[flip]);
    }
    flip ^= 1;
    const float mean = dot * inv_n;
    for (int64_t j = threadIdx.x; j < c.cols; j += 1024) {
      const float d = from16<kBf16>(dY[j]);
      const float n = (kLayer ? from16<kBf16>(H[j]) - m : from16<kBf16>(H[j])) * s;
      float g = c.W ? d * from16<kBf16>(c.W[j]) : d;
      if constexpr (kLayer) g -= level * inv_n;
      const float b = c.dH ? from16<kBf16>(c.dH[r * c.lddh + j]) : 0.f;
      c.dX[r * c.lddx + j] = to16<kBf16>(fmaf(s, g - n * mean, b));
    }
    first = false;
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, int smem,
                       cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool kLayer, bool kBf16, int T>
cudaError_t launch_norm_ring(const DeviceInfo &dev, const NormCall &c, cudaStream_t stream) {
  auto kern = norm_ring_kernel<kLayer, kBf16, false, T>;
  if constexpr (!kLayer)
    if (c.scale) kern = norm_ring_kernel<kLayer, kBf16, true, T>;
  const int mats = c.R ? 2 : 1;
  const int sms = std::max(dev.sm_count / 8 * 8, 8);
  int threads = T;
  int64_t blocks;
  if (T > 32) {
    blocks = std::min(c.rows, sms * (kNormThreads / T));
  } else {
    const int most = kNormThreads / 32;
    const int per_warp = (c.rows - 1) / (sms * most) + 1, warps = (c.rows - 1) / (sms * per_warp) + 1;
    threads = 32 * warps;
    blocks = per_warp > 1 ? sms : (c.rows - 1) / warps + 1;
  }
  // Rows in flight or in work: about 64 KB per SM. (16384 x 8192 without a residual:
  // 64 KB 83 us, 192 KB 94 us; 16384 x 5280 with one: 42 KB 130 us, 84 KB 115 us,
  // 126 KB 125 us.)
  const int layer = kNormThreads / T * mats * c.cols * 2;
  const int stages = std::min(std::max((65536 + layer / 2) / layer, 2), 4);
  const int smem = threads / T * stages * mats * (kNormUnits * T * 16 + 64);
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem, dev.device);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, static_cast<unsigned>(blocks), static_cast<unsigned>(threads), smem,
                    stream, c, stages);
}

template <bool kLayer, bool kBf16>
cudaError_t launch_norm(const DeviceInfo &dev, const NormCall &c, cudaStream_t stream) {
  const int units = c.cols / 8;  // at most, whatever the alignment
  const bool alike =
      c.R == nullptr || ((reinterpret_cast<uintptr_t>(c.R) ^ reinterpret_cast<uintptr_t>(c.X)) % 16 == 0 &&
                         (c.ldr - c.ldx) % 8 == 0);
  // Blocks that walk rows, or a block per row? A block per row while about all rows
  // are in residence at once (1024 x 4096: 5.2 against 4.4 us, but 304 x 4096 2.3
  // against 2.8), and for rows of up to 512 columns (16384 x 512 8.0 against 7.7).
  // With a residual, whose reads and writes keep memory busy enough, also where the
  // row fills most of the block (16384 rows: 2048 40 against 45 us, 4096 78 against
  // 87; but 2560 58 against 54, 5280 139 against 115 and 12288, of half as many
  // rows, 185 against 131).
  const int slots = units <= 128 ? 128 : units <= 256 ? 256 : 512;
  // Layer norm, whose row takes a block longer: only where it fills 13/16 of the block and
  // all rows start on 16-byte boundaries, or the gain and bias are read value by value for
  // each row (16384 rows: 3584 79 against 83 us, but 3200 76 against 72 and 4095 107
  // against 97).
  const bool whole = reinterpret_cast<uintptr_t>(c.X) % 16 == 0 && c.ldx % 8 == 0 && c.cols % 8 == 0;
  const bool full = units > 128 && units <= 512 &&
                    (kLayer ? whole && 16 * units > 13 * slots : 4 * units > 3 * slots);
  if (alike && units > 64 && static_cast<int64_t>(c.rows) * c.cols > 10240LL * dev.sm_count &&
      !(c.R != nullptr && full)) {
    if (units <= 128) return launch_norm_ring<kLayer, kBf16, 32>(dev, c, stream);
    if (units <= 256) return launch_norm_ring<kLayer, kBf16, 64>(dev, c, stream);
    if (units <= 512) return launch_norm_ring<kLayer, kBf16, 128>(dev, c, stream);
    if (units <= 1024) return launch_norm_ring<kLayer, kBf16, 256>(dev, c, stream);
    if (units <= 2048) return launch_norm_ring<kLayer, kBf16, 512>(dev, c, stream);
  }
  const unsigned rows = static_cast<unsigned>(c.rows);
  if (units <= 16) return launch_pdl(norm_kernel<kLayer, kBf16, 16, 1>, (rows + 7) / 8, 128, 0, stream, c);
  if (units <= 32) return launch_pdl(norm_kernel<kLayer, kBf16, 16, 2>, (rows + 7) / 8, 128, 0, stream, c);
  if (units <= 64) return launch_pdl(norm_kernel<kLayer, kBf16, 32, 2>, (rows + 3) / 4, 128, 0, stream, c);
  if (units <= 128) return launch_pdl(norm_kernel<kLayer, kBf16, 128, 1>, rows, 128, 0, stream, c);
  if (units <= 256) return launch_pdl(norm_kernel<kLayer, kBf16, 128, 2>, rows, 128, 0, stream, c);
  if (units <= 512) return launch_pdl(norm_kernel<kLayer, kBf16, 256, 2>, rows, 256, 0, stream, c);
  if (units <= 1024) return launch_pdl(norm_kernel<kLayer, kBf16, 512, 2>, rows, 512, 0, stream, c);
  if (units <= 2048) return launch_pdl(norm_kernel<kLayer, kBf16, 1024, 2>, rows, 1024, 0, stream, c);
  return launch_pdl(norm_long_kernel<kLayer, kBf16>, rows, 1024, 0, stream, c);
}

// Runs launch(part) with a partial-sum matrix of `parts` rows (layer: one for db behind
// it) when dW or db is wanted, then adds its rows.
template <bool kLayer, typename F>
cudaError_t with_partials(const DeviceInfo &dev, const NormGradCall &c, int64_t parts,
                          cudaStream_t stream, F &&launch) {
  void *part = nullptr;
  cudaError_t e;
  if (c.dW != nullptr || c.db != nullptr) {
    cudaMemPool_t pool;
    e = device_pool(dev, &pool);
    if (e != cudaSuccess) return e;
    e = cudaMallocFromPoolAsync(&part, static_cast<size_t>(kLayer ? 2 : 1) * parts * c.cols * 4, pool,
                                stream);
    if (e != cudaSuccess) return e;
  }
  e = launch(static_cast<float *>(part));
  if (part != nullptr) {
    if (e == cudaSuccess)
      e = launch_col_sums(c.bf16, static_cast<const float *>(part), static_cast<int>(parts),
                          c.cols, c.cols, c.dW, stream, parts * c.cols, c.db);
    cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

// Blocks of one wave, `resident` per SM but at most 4 (each costs a partial row
// to write and add): fewer than the rows only as a multiple of 8 (a block's rows
// must be a multiple of 8 apart).
int64_t grad_blocks(const DeviceInfo &dev, int64_t rows, int resident) {
  const int64_t wave =
      static_cast<int64_t>(std::min(std::max(resident, 1), 4)) * dev.sm_count / 8 * 8;
  return std::min<int64_t>(std::max<int64_t>(wave, 8), rows);
}

template <bool kLayer, bool kBf16, int NV>
cudaError_t launch_grad_warp(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  const int64_t blocks = grad_blocks(dev, (static_cast<int64_t>(c.rows) + 3) / 4,
                                     kGradWarpBlocks<NV>);
  return with_partials<kLayer>(dev, c, blocks, stream, [&](float *part) {
    return launch_pdl(norm_grad_warp_kernel<kLayer, kBf16, NV>, static_cast<unsigned>(blocks), 128, 0,
                      stream, c, part);
  });
}

template <bool kLayer, bool kBf16, int T, int NV = 2>
cudaError_t launch_grad_ring(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  auto kern = norm_grad_kernel<kLayer, kBf16, T, NV>;
  // An SM's blocks share about 200 KB of rows in flight (220 makes three stages of
  // 12288 columns, 156 -> 121 us for 8192 rows) and hide each other's reductions.
  // At the end the ring holds the sums.
  const int units = c.cols / 8, stage = units * 16 * 3;
  const int room = (NV > 2 ? 440 : 200) * T;
  const int stages = std::max(2, std::min(kMaxGradStages, room / std::max(stage, 1)));
  const int smem = std::max(stages * stage, ((units + 27) / 32 * 32 + 4) * 8 * 4);
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem, dev.device);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, T, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = grad_blocks(dev, c.rows, per_sm);
  return with_partials<kLayer>(dev, c, blocks, stream, [&](float *part) {
    return launch_pdl(kern, static_cast<unsigned>(blocks), T, smem, stream, c, part, stages,
                      dev.err_word);
  });
}

template <bool kLayer, bool kBf16, int NV>
cudaError_t launch_grad_rows(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  auto kern = norm_grad_rows_kernel<kLayer, kBf16, NV>;
  // As few rows per warp as kGradRowWarps warps per SM allow, then as few warps as
  // that takes. A warp's rows are a multiple of 8 apart, or it has one row.
  const int sms = std::max(dev.sm_count / 8 * 8, 8);
  const int per_warp = (c.rows - 1) / (sms * kGradRowWarps<kLayer, NV>) + 1;
  int warps = (c.rows - 1) / (sms * per_warp) + 1;
  // One row each: at least 8 warps a block, for fewer partial rows and more threads
  // to add them (333 x 1001 7.0 -> 6.4 us).
  if (per_warp == 1) warps = std::max(warps, 8);
  const int64_t blocks = per_warp > 1 ? sms : (c.rows - 1) / warps + 1;
  const int smem = std::max(warps * kGradRowStages<NV> * 3 * NV * 512,
                            (kLayer ? 2 : 1) * warps * (c.cols + c.cols / 32 + 1) * 4);
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem, dev.device);
  if (e != cudaSuccess) return e;
  return with_partials<kLayer>(dev, c, blocks, stream, [&](float *part) {
    return launch_pdl(kern, static_cast<unsigned>(blocks), 32u * warps, smem, stream, c, part);
  });
}

template <bool kLayer, bool kBf16>
cudaError_t launch_grad_long(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  const int blocks = std::min(c.rows, 2 * dev.sm_count);
  return with_partials<kLayer>(dev, c, blocks, stream, [&](float *part) {
    return launch_pdl(norm_grad_long_kernel<kLayer, kBf16>, static_cast<unsigned>(blocks), 1024, 0,
                      stream, c, part);
  });
}

template <bool kLayer, bool kBf16>
cudaError_t launch_grad(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  const int units = c.cols / 8;  // at most, whatever the alignment
  auto alike = [&](const void *p, int64_t ld) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(c.dY)) % 16 == 0 &&
                            (ld - c.lddy) % 8 == 0);
  };
  const bool same = alike(c.H, c.ldh) && alike(c.dH, c.lddh) && alike(c.dX, c.lddx);
  if (!same) {
    if (units <= 32) return launch_grad_warp<kLayer, kBf16, 1>(dev, c, stream);
    if (units <= 64) return launch_grad_warp<kLayer, kBf16, 2>(dev, c, stream);
    return launch_grad_long<kLayer, kBf16>(dev, c, stream);
  }
  // A warp per row, or a block per row? The warp form keeps more rows in flight
  // (32768 x 1024 47.5 against 62.3 us, 32768 x 1536 65.3 against 85.7, 8192 x 512
  // 10.1 against 12.4 for a warp per row without the copies ahead); the block form
  // has the shorter row where there are few (256 x 1024 4.7 against 5.2 us but
  // 400 x 1024 6.2 against 5.5; 256 x 2048 5.4 against 7.4, 1300 x 2048 9.1 against
  // 10.8, 2048 x 2048 11.2 against 11.1).
  if (units <= 32) return launch_grad_rows<kLayer, kBf16, 1>(dev, c, stream);
  if (units <= 64) return launch_grad_rows<kLayer, kBf16, 2>(dev, c, stream);
  if (units <= 128 && c.rows > 2 * dev.sm_count) return launch_grad_rows<kLayer, kBf16, 4>(dev, c, stream);
  if (units <= 128) return launch_grad_ring<kLayer, kBf16, 128, 1>(dev, c, stream);
  if (units <= 256 && c.rows > 10 * dev.sm_count) return launch_grad_rows<kLayer, kBf16, 8>(dev, c, stream);
  // (Layer: 4 units per thread, 1300 x 2048 12.4 -> 11.2 us; 2 spill.)
  if (units <= 256)
    return launch_grad_ring<kLayer, kBf16, kLayer ? 64 : 128, kLayer ? 4 : 2>(dev, c, stream);
  if (units <= 512) return launch_grad_ring<kLayer, kBf16, 128, 4>(dev, c, stream);
  if (units <= 1024) return launch_grad_ring<kLayer, kBf16, 256, 4>(dev, c, stream);
  if (units <= 2048) return launch_grad_ring<kLayer, kBf16, 512, 4>(dev, c, stream);
  return launch_grad_long<kLayer, kBf16>(dev, c, stream);
}

template <bool kLayer>
cudaError_t launch_norm_form(const DeviceInfo &dev, const NormCall &c, cudaStream_t stream) {
  return c.bf16 ? launch_norm<kLayer, true>(dev, c, stream)
                : launch_norm<kLayer, false>(dev, c, stream);
}

template <bool kLayer>
cudaError_t launch_grad_form(const DeviceInfo &dev, const NormGradCall &c, cudaStream_t stream) {
  if (c.rows == 0)
    return c.dW || c.db ? launch_col_sums(c.bf16, nullptr, 0, c.cols, c.cols, c.dW, stream, 0, c.db)
                        : cudaSuccess;
  return c.bf16 ? launch_grad<kLayer, true>(dev, c, stream)
                : launch_grad<kLayer, false>(dev, c, stream);
}

}  // namespace
}  // namespace dgr

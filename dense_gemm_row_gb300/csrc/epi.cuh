// epi.cuh -- device functions of the linear-layer operators: 16-bit storage
// formats, activations and their derivatives.
//
// Everything is evaluated in fp32. The four activations and what they cost:
//   relu       max(z, 0)                                      (NaN stays NaN)
//   gelu       z * Phi(z), Phi the normal distribution function
//   gelu_tanh  z * s(2u), u = sqrt(2/pi) (z + 0.044715 z^3): the tanh form
//              0.5 z (1 + tanh u) rewritten with the logistic s, since
//              1 + tanh u = 2 s(2u): one exponential and one division
//   silu       z * s(z)
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dgr {
namespace {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;

// 16-bit storage <-> fp32; widening is exact, narrowing rounds to nearest even.
template <bool kBf16>
__device__ __forceinline__ float from16(uint32_t h) {
  if constexpr (kBf16) {
    return __uint_as_float(h << 16);
  } else {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
  }
}
template <bool kBf16>
__device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (kBf16) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  } else {
    return __half_as_ushort(__float2half_rn(v));
  }
}
// Two values per 32-bit word, the first in the low half (as stored in memory).
template <bool kBf16>
__device__ __forceinline__ void unpack16(uint32_t w, float &a, float &b) {
  if constexpr (kBf16) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
  }
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// The hardware's exponential and reciprocal, subnormals taken as zero: a few
// 2^-22 (relative), far below one 16-bit rounding (2^-9 for bf16, 2^-12 for
// fp16). One instruction each; __expf and __fdividef add the handling of
// subnormals around them, which an element-wise pass pays for.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + exp(-x)). exp(-x) overflows to +inf for x < -88, where the quotient
// is 0, its limit.
__device__ __forceinline__ float logistic(float x) { return rcp_fast(1.f + exp_fast(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The normal distribution function Phi(z), with e = exp(-z^2 / 2) returned for
// its density. Phi(-x sqrt 2) = erfc(x) / 2, and erfc(x) = exp(-x^2) t P(t)
// with t = 1 / (1 + x / 2): P is the degree-6 polynomial that minimises the
// largest relative error over 0 <= x <= 9.3 (iteratively reweighted least
// squares against a double-precision erfc; 1.5e-6 with fp32 coefficients).
// The relative error holds in the lower tail too, where 1 + erf cancels, and
// the exponential is the one the density needs: two MUFU operations in all,
// so an element-wise pass stays bound by memory.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float x = fabsf(z) * kInvSqrt2;
  const float t = rcp_fast(fmaf(0.5f, x, 1.f));
  e = exp_fast(-0.5f * z * z);
  float p = 0.08912812918424606f;
  p = fmaf(p, t, -0.35999614000320435f);
  p = fmaf(p, t, 0.39379453659057617f);
  p = fmaf(p, t, 0.03464719280600548f);
  p = fmaf(p, t, 0.28272417187690735f);
  p = fmaf(p, t, 0.2773527503013611f);
  p = fmaf(p, t, 0.2823481559753418f);
  const float q = 0.5f * e * t * p;
  return z < 0.f ? q : 1.f - q;
}

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (kAct == kActRelu) {
    return z < 0.f ? 0.f : z;
  } else if constexpr (kAct == kActGelu) {
    float e;
    return z * normal_cdf(z, e);
  } else if constexpr (kAct == kActGeluTanh) {
    return z * logistic(2.f * kGeluC * (z + kGeluA * z * z * z));
  } else if constexpr (kAct == kActSilu) {
    return z * logistic(z);
  } else {
    return z;
  }
}

template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (kAct == kActRelu) {
    return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);  // NaN stays NaN
  } else if constexpr (kAct == kActGelu) {
    float e;  // Phi(z) + z phi(z)
    const float cdf = normal_cdf(z, e);
    return fmaf(z * kInvSqrt2Pi, e, cdf);
  } else if constexpr (kAct == kActGeluTanh) {
    // s + z s (1 - s) 2u'. For |z| > 100 s (1 - s) is 0; the bound on z^2
    // keeps a finite z from making it 0 * inf.
    const float zz = fminf(z * z, 1e4f);
    const float s = logistic(2.f * kGeluC * (z + kGeluA * z * z * z));
    return fmaf(z * s * (1.f - s), 2.f * kGeluC * fmaf(3.f * kGeluA, zz, 1.f), s);
  } else if constexpr (kAct == kActSilu) {
    const float s = logistic(z);
    return fmaf(z * s, 1.f - s, s);
  } else {
    return 1.f;
  }
}

// Calls f(std::integral_constant<int, act>) for the run-time `act`. The branch
// is uniform over the grid.
template <typename F>
__device__ __forceinline__ void with_act(int act, F &&f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}

}  // namespace
}  // namespace dgr

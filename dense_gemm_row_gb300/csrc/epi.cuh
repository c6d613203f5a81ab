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

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFltMax = 3.402823466e38f;

// Two fp32 values in one register pair, and the packed operations on them: one
// instruction for two values. It keeps the element-wise gradient near the cost of
// its memory traffic, and an epilogue's gelu short: 64 columns by eight warps took
// 1.9 us of a 7.2 us call (300 x 1024 x 512) with one value per instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// Two 16-bit values of a word, widened.
template <bool kBf16>
__device__ __forceinline__ F2 unpack2(uint32_t w) {
  float a, b;
  unpack16<kBf16>(w, a, b);
  return f2(a, b);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(F2 v) {
  float a, b;
  split(v, a, b);
  return pack16<kBf16>(a, b);
}
// 2^x and 1 / x of both values: the hardware's approximations, subnormals taken
// as zero. They are a few 2^-22 (relative) off, and x's own roundings add |x| 2^-23, at
// most 2^-16 before the result underflows: far below one 16-bit rounding (2^-9 for
// bf16, 2^-12 for fp16). 1 / (1 + 2^x) needs no care at the ends: 2^x
// overflows to infinity, whose reciprocal is 0, the limit.
__device__ __forceinline__ F2 exp2_fast2(F2 x) {
  float a, b;
  split(x, a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  return f2(a, b);
}
__device__ __forceinline__ F2 rcp_fast2(F2 x) {
  float a, b;
  split(x, a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return f2(a, b);
}

// -erfc(|z| / sqrt 2) / 2, i.e. -Phi(-|z|), and e = exp(-z^2 / 2), for two z.
// With x = |z| / sqrt 2: erfc(x) = exp(-x^2) t P(t), t = 1 / (1 + x / 2), where P
// is the degree-6 polynomial that minimises the largest relative error over
// 0 <= x <= 9.3 (iteratively reweighted least squares against a double-precision
// erfc; 1.5e-6 with fp32 coefficients). Relative: it holds in the tail, where
// 1 + erf would cancel.
__device__ __forceinline__ F2 minus_tail2(F2 z, F2 mag, F2 &e) {
  e = exp2_fast2(mul2(mul2(z, z), f2(-0.5f * kLog2e)));
  const F2 t = rcp_fast2(fma2(mag, f2(0.5f * kInvSqrt2), f2(1.f)));
  F2 p = f2(-0.5f * 0.08912812918424606f);
  p = fma2(p, t, f2(-0.5f * -0.35999614000320435f));
  p = fma2(p, t, f2(-0.5f * 0.39379453659057617f));
  p = fma2(p, t, f2(-0.5f * 0.03464719280600548f));
  p = fma2(p, t, f2(-0.5f * 0.28272417187690735f));
  p = fma2(p, t, f2(-0.5f * 0.2773527503013611f));
  p = fma2(p, t, f2(-0.5f * 0.2823481559753418f));
  return mul2(mul2(e, t), p);
}
// The logistic functions of the tanh form and of silu: s(2u) and s(z).
__device__ __forceinline__ F2 tanh_gate2(F2 z, F2 zz) {
  const F2 arg =
      mul2(z, fma2(zz, f2(-2.f * kGeluC * kLog2e * kGeluA), f2(-2.f * kGeluC * kLog2e)));
  return rcp_fast2(add2(exp2_fast2(arg), f2(1.f)));
}
__device__ __forceinline__ F2 logistic2(F2 z) {
  return rcp_fast2(add2(exp2_fast2(mul2(z, f2(-kLog2e))), f2(1.f)));
}

// The activations of two values. gelu: z Phi(z) = max(z, 0) - |z| Phi(-|z|), where the
// tail is 0 at +inf: |z| has to be finite there (kFinite: z is known to be).
template <int kAct, bool kFinite = false>
__device__ __forceinline__ F2 act_value2(F2 z) {
  if constexpr (kAct == kActNone) return z;
  if constexpr (kAct == kActSilu) return mul2(z, logistic2(z));
  if constexpr (kAct == kActGeluTanh) return mul2(z, tanh_gate2(z, mul2(z, z)));
  float z0, z1;
  split(z, z0, z1);
  if constexpr (kAct == kActRelu) {  // NaN stays NaN
    return f2(z0 < 0.f ? 0.f : z0, z1 < 0.f ? 0.f : z1);
  } else {
    const F2 mag = kFinite ? f2(fabsf(z0), fabsf(z1))
                           : f2(fmaxf(fminf(z0, kFltMax), -z0), fmaxf(fminf(z1, kFltMax), -z1));
    F2 e;
    return fma2(mag, minus_tail2(z, mag, e), f2(fmaxf(z0, 0.f), fmaxf(z1, 0.f)));
  }
}
// The same for the lanes' 2 kN values, by a whole warp. gelu: a sum shows whether all
// are finite, for one addition per pair instead of two clamps (8192 x 8192 x 256: 108.0
// us without care for infinities, 109.8 checked, 114.6 clamped; four sums in turn: 110.1).
template <int kAct, int kN>
__device__ __forceinline__ void act_values(F2 (&z)[kN]) {
  if constexpr (kAct == kActGelu) {
    F2 sum = z[0];
#pragma unroll
    for (int j = 1; j < kN; ++j) sum = add2(sum, z[j]);
    float a, b;
    split(sum, a, b);
    if (__any_sync(0xffffffffu, !(fabsf(a + b) <= kFltMax))) {
#pragma unroll
      for (int j = 0; j < kN; ++j) z[j] = act_value2<kAct>(z[j]);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) z[j] = act_value2<kAct, true>(z[j]);
}
template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  float a, b;
  split(act_value2<kAct>(f2(z)), a, b);
  return a;
}

// The derivatives at two values. gelu: Phi(z) + z phi(z), with Phi as 1/2 +
// sign(z) (1/2 - erfc / 2), as the slope needs it to an absolute 2^-24 only;
// gelu_tanh: s + z s (1 - s) 2u', where for |z| > 100 s (1 - s) is 0 and a bound
// on z^2 keeps a finite z from making it 0 * inf; silu: s + z s (1 - s).
template <int kAct>
__device__ __forceinline__ F2 act_slope2(float z0, float z1) {
  const F2 z = f2(z0, z1);
  if constexpr (kAct == kActRelu) {  // NaN stays NaN
    return f2(z0 > 0.f ? 1.f : (z0 <= 0.f ? 0.f : z0), z1 > 0.f ? 1.f : (z1 <= 0.f ? 0.f : z1));
  } else if constexpr (kAct == kActGelu) {
    F2 e;
    float a, b;
    split(add2(minus_tail2(z, f2(fabsf(z0), fabsf(z1)), e), f2(0.5f)), a, b);
    const F2 cdf = add2(f2(copysignf(a, z0), copysignf(b, z1)), f2(0.5f));
    return fma2(mul2(z, f2(kInvSqrt2Pi)), e, cdf);
  } else if constexpr (kAct == kActGeluTanh) {
    const F2 zz = mul2(z, z), s = tanh_gate2(z, zz);
    float a, b;
    split(zz, a, b);
    const F2 poly = fma2(f2(fminf(a, 1e4f), fminf(b, 1e4f)), f2(6.f * kGeluC * kGeluA),
                         f2(2.f * kGeluC));
    return fma2(mul2(mul2(z, s), fma2(s, f2(-1.f), f2(1.f))), poly, s);
  } else if constexpr (kAct == kActSilu) {
    const F2 s = logistic2(z);
    return fma2(mul2(z, s), fma2(s, f2(-1.f), f2(1.f)), s);
  } else {
    return f2(1.f);
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

// e4m3.cuh -- conversion to e4m3 values with a scale.
#pragma once

#include <cstdint>

#include <cuda_fp8.h>

#include "epi.cuh"

namespace dgr {
namespace {

constexpr float kE4m3Max = 448.f;
// A row (or block) whose largest |y| is below this counts as zeros (scale 0): 448 / |y|
// must not overflow.
constexpr float kE4m3Least = 1e-30f;

// The scale of a row whose largest |y| is `most`, and its inverse; NaN and infinity
// stay visible in both the scale and the values (0 * inf and NaN).
__device__ __forceinline__ float e4m3_scale(float most) {
  return most < kE4m3Least ? 0.f : most / kE4m3Max;
}
__device__ __forceinline__ float e4m3_inverse(float most) {
  return most < kE4m3Least ? 0.f : kE4m3Max / most;
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace
}  // namespace dgr

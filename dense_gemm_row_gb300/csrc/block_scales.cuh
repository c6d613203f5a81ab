// block_scales.cuh -- what the two block-scaled kernels share: scales of four k-blocks
// at a time, and loads of 16 columns from tensor memory.
#pragma once

#include <cstdint>

namespace dgr {
namespace {

// Whether rows of scales are in whole 16-byte units.
__host__ __device__ __forceinline__ bool scales_whole(const float *p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0;
}
// The scales of k-blocks kb .. kb + 3 of one row (zeros past the last). Plain loads: the
// kernels start while the one that writes the scales may still run, and loads through the
// read-only path (ld.global.nc) are for memory that does not change while a kernel runs;
// nothing orders them behind the wait for that kernel.
__device__ __forceinline__ float4 load_scales(const float *row, int kb, int KB, bool vec) {
  if (row == nullptr) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec && kb + 4 <= KB) return *reinterpret_cast<const float4 *>(row + kb);
  float4 v;
  v.x = kb < KB ? row[kb] : 0.f;
  v.y = kb + 1 < KB ? row[kb + 1] : 0.f;
  v.z = kb + 2 < KB ? row[kb + 2] : 0.f;
  v.w = kb + 3 < KB ? row[kb + 3] : 0.f;
  return v;
}
__device__ __forceinline__ float4 scale_products(const float4 &a, const float4 &b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float pick(const float4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

}  // namespace
}  // namespace dgr

// tc_issue.cuh -- helpers of the warps that issue TMA copies and MMAs in the
// linear-layer kernels.
//
// Those warps run their loops converged, with every value derived from uniform
// ones, and let one elected lane issue. A loop under `if (lane == 0)` does the
// same work, but the compiler cannot tell that its operands are uniform, and the
// copies' and MMAs' operands live in uniform registers: such a loop took 0.29 us
// per k-block of 4 MMAs where the elected form takes under 0.2 (measured on GB300
// on the few-rows kernel at 1 x 1024 x 4096, operands in L2).
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace dgr {

// This thread's warp index, uniform over the warp to the compiler too.
__device__ __forceinline__ int uniform_warp() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(p)
               :
               : "memory");
  return p != 0;
}

// mbar_wait_bounded for the issue loops, by a whole warp: the same bound and the
// same failure, but the clock is first read after 64 polls, so a wait that is met in
// time costs its polls only. Lanes poll and read the clock for themselves, so at the
// limit some could give up a wait that others see met: the warp votes on every poll
// and on giving up, and all its lanes get the same answer. kCluster: acquires at
// cluster scope.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait_lazy(uint32_t bar, uint32_t parity, volatile int *abort,
                                               uint32_t *err_word, uint32_t code,
                                               uint64_t limit_ns = kWaitLimitNs) {
  constexpr uint32_t kWarp = 0xffffffffu;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(kWarp, kCluster ? mbar_try_wait_cluster(bar, parity)
                                   : mbar_try_wait(bar, parity)))
      return true;
    if ((it & 63u) == 0u) {
      // The kernel may have started while the previous one still runs: its time is not
      // this wait's.
      if (t0 == 0) grid_dependency_wait();
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      const uint32_t polls = limit_ns > kWaitLimitNs ? ~0u - 255u : kWaitMaxPolls;
      const bool late = now - t0 > limit_ns || it >= polls;
      if (__any_sync(kWarp, late || *abort)) {
        if (late) {
          *abort = 1;
          record_timeout(err_word, code);
        }
        return false;
      }
    }
  }
}

}  // namespace dgr

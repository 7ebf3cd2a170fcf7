// A bounded mbarrier wait for hot loops. Reading %globaltimer takes about 800 SM clocks (measured as
// the delay between an arrival and the waiter's next instruction when every poll reads it), so
// the time is looked at only once per 256 polls; each poll suspends in hardware while the phase is
// incomplete.
#pragma once

#include "pbs_device.cuh"

namespace pbs {

// Wait for the phase with the given parity; false after about `limit_ns`.
__device__ __forceinline__ bool mbar_wait_quick(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
#pragma unroll 1
  while (global_timer_ns() - t0 <= limit_ns) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (mbar_try_wait(bar, parity)) return true;
  }
  return false;
}

}  // namespace pbs

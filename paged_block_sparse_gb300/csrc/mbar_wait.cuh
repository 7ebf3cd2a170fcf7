// A bounded mbarrier wait for hot loops: the waiting thread is suspended in hardware (the time given to
// try_wait is how long at most) instead of polling. A poll loop takes issue slots from the warps that the
// wait is for, and reading %globaltimer in it delays the wake-up by some 800 SM clocks (both measured in
// the window prefill kernel).
#pragma once

#include "pbs_device.cuh"

namespace pbs {

// Wait for the phase with the given parity; false after about `limit_ns`.
__device__ __forceinline__ bool mbar_wait_quick(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  constexpr uint32_t kSuspendNs = 1000000;
  const uint32_t addr = smem_u32(bar);
  const int tries = static_cast<int>(limit_ns / kSuspendNs) + 1;
  unsigned long long t0 = 0;
#pragma unroll 1
  for (int i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok != 0) return true;
    // the hardware may return earlier than asked: past the expected number of tries the clock decides
    if (i >= tries) {
      if (t0 == 0) t0 = global_timer_ns();
      else if (global_timer_ns() - t0 > limit_ns) return false;
    }
  }
}

}  // namespace pbs

// waiter.cuh -- bounded mbarrier waits: on expiry the thread records the device
// error word and raises its CTA's abort flag; nothing traps or hangs.
#pragma once

#include "fmha_internal.h"
#include "ptx_sm100.cuh"

namespace fmha {

// Suspend-time hint of one barrier probe, in ns.
constexpr uint32_t kWaitSleepNs = 1000;

// Bounded mbarrier wait. Returns false on timeout (recorded) or CTA abort.
struct Waiter {
  volatile uint32_t* abort_flag;
  uint32_t* err;
  uint64_t budget;
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    // First a non-blocking test: try_wait may itself suspend the thread for a
    // hardware-chosen time, which would let a short limit never run out.
    if (ptx::mbar_test_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
      // The limit is checked before every sleeping probe, so a limit shorter
      // than one probe still gives up after the first unsatisfied probe.
      if (static_cast<uint64_t>(clock64() - t0) > budget) {
        *abort_flag = 1u;
        record_timeout(bar, parity);
        return false;
      }
      // Sleep in the barrier (woken when the phase completes) rather than spin:
      // a spinning warp takes issue slots from the warps sharing its scheduler.
      if (ptx::mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
      if (*abort_flag) return false;
    }
  }
  // Sets the timeout bit and, for the first timeout only, the site bits.
  __device__ __forceinline__ void record_timeout(uint32_t bar, uint32_t parity) const {
    const uint32_t site = ((bar & 0xfffu) | ((parity & 1u) << 12) | (((threadIdx.x >> 5) + 1u) << 16))
                          << kErrSiteShift;
    uint32_t old = atomicOr(err, kErrTimeout);
    for (int tries = 0; tries < 8 && (old >> kErrSiteShift) == 0u; ++tries) {
      const uint32_t seen = atomicCAS(err, old | kErrTimeout, old | kErrTimeout | site);
      if (seen == (old | kErrTimeout)) break;
      old = seen;
    }
  }
  // Teardown wait: ignores the abort flag (used to drain in-flight async work).
  // Its limit never drops below ~1 s, whatever the wait limit is set to: a copy
  // or MMA already issued always completes, and shared memory / TMEM must not
  // be released under it.
  __device__ __forceinline__ bool drain(uint32_t bar, uint32_t parity) const {
    const uint64_t limit = budget > (1ull << 31) ? budget : (1ull << 31);
    const long long t0 = clock64();
    while (!ptx::mbar_try_wait(bar, parity)) {
      if (static_cast<uint64_t>(clock64() - t0) > limit) {
        record_timeout(bar, parity);
        return false;
      }
    }
    return true;
  }
};

}  // namespace fmha

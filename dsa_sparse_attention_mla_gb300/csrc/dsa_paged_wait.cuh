// dsa_paged_wait.cuh - bounded waits of the dense paged attention's warps on one another.
#pragma once
#include <cstdint>

#include "dsa_ptx.cuh"

namespace dsa {
namespace paged {

constexpr uint64_t kWaitNs = 2000000000ull;

// The hint lets the hardware park the warp for up to a millisecond: some twenty warps wait at any time,
// and polling took a third of the issue slots.
__device__ __forceinline__ bool try_wait_parked(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}

// Waits for the phase of the given parity; false after `limit` ns, or once another warp has given up and set
// *abort (in shared memory; a wait for operations in flight, which must end before the block does, takes
// no flag).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const volatile int* abort, uint64_t limit = kWaitNs) {
  if (try_wait_parked(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    // (the time before an attempt, not after it: a block that the GPU has not run for a while tries again)
    const bool late = globaltimer_ns() - t0 > limit;
    if (try_wait_parked(bar, parity)) return true;
    if ((abort && *abort) || late) return false;
  }
}

// The same for a wait that may last a row, whose tiles can take longer than any limit for a hand-off: the limit
// starts anew whenever *progress (in shared memory) has changed.
__device__ __forceinline__ bool bar_wait_row(uint32_t bar, uint32_t parity, const volatile int* abort,
                                             const volatile int* progress, uint64_t limit = kWaitNs) {
  for (;;) {
    const int seen = *progress;
    if (bar_wait(bar, parity, abort, limit)) return true;
    if (*abort || *progress == seen) return false;
  }
}

}  // namespace paged
}  // namespace dsa

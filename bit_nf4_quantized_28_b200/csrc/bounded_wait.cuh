// bounded_wait.cuh -- the barrier wait of the kernels beside the NF4 linear.
//
// A note that holds for all of those kernels: they may start before the kernel
// ahead of them has ended, and read its results after griddepcontrol.wait with
// plain loads.  Loads through the read-only path (__ldg) promise the compiler
// data that never changes while the kernel runs, which would let it move them
// ahead of that wait.
#pragma once

#include "common.cuh"

namespace qn {

// Waits for the mbarrier phase with the given parity (completed in this CTA,
// or by another CTA of the cluster with kCluster).  Bounded like mbar_wait,
// but the timer is not read before 64 tries (each of which suspends the
// thread a while) have failed: that read would stand in a pipeline's way.
template <bool kCluster>
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             unsigned int err_bit) {
  const uint32_t addr = smem_u32(bar);
  unsigned long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (kCluster ? mbar_try_wait_cluster(addr, parity) : mbar_try_wait(addr, parity)) return true;
    if ((it & 63u) == 0u) {
      if (*abort) return false;
      const unsigned long long t = global_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > kWaitLimitNs) {
        atomicOr(&g_error_word, err_bit);
        *abort = 1;
        return false;
      }
    }
  }
}

// After a wait gave up: time for the copies in flight to land before the CTA
// leaves.
__device__ __forceinline__ void abort_grace() {
  const unsigned long long t0 = global_ns();
  while (global_ns() - t0 < 100000ull) {
  }
}

}  // namespace qn

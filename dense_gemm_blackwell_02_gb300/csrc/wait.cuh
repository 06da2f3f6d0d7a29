// Bounded mbarrier waits: every wait of a kernel ends, by the phase completing or by the
// limit in WaitCtl, which records the site in the device status word and raises a flag in
// shared memory that makes the CTA's other roles leave their loops.
#pragma once
#include <cstdint>

#include "params.h"
#include "ptx.cuh"

namespace gb300 {

struct WaitCtl {
  uint64_t limit_ns;
  uint32_t* status;
  volatile int32_t* abort_flag;
};

__device__ __forceinline__ void record_timeout(const WaitCtl& c, uint32_t site) {
  *c.abort_flag = 1;
  const uint32_t word = (kDevTimeout << 24) | (site << 16) | (blockIdx.x & 0xFFFFu);
  // the first of several stays, but what is lost weighs more than an index not followed
  const uint32_t before = atomicCAS(c.status, 0u, word);
  if ((before >> 24) == kDevBadIndex) atomicCAS(c.status, before, word);
}

// Teardown wait: ignores the abort flag (it is used while aborting) but is bounded.
static __device__ __noinline__ bool wait_parity_drain(uint32_t bar, uint32_t parity, const WaitCtl& c) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0u && (globaltimer_ns() - t0 > c.limit_ns || it > (1u << 26))) {
      record_timeout(c, kSiteDrain);
      return false;
    }
  }
}

// Warp-collective wait: all 32 lanes poll together and leave together (a phase, once
// complete, stays complete, so one lane seeing it is enough), so the warp never
// diverges around the wait.  Lane 0's clock decides the timeout for the warp.
static __device__ __noinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& c,
                                              uint32_t site) {
  if (__any_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__any_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    if ((it & 31u) == 0u) {
      const bool aborting = *c.abort_flag != 0;
      const bool expired = globaltimer_ns() - t0 > c.limit_ns || it > (1u << 26);
      if (__shfl_sync(0xFFFFFFFFu, aborting ? 1u : 0u, 0)) return false;
      if (__shfl_sync(0xFFFFFFFFu, expired ? 1u : 0u, 0)) {
        if (lane_id() == 0) record_timeout(c, site);
        __syncwarp();
        return false;
      }
    }
  }
}

// Inline fast path of the wait: a phase that is already complete costs one test here
// instead of a call (whose register saves cost about 200 cycles per wait, measured with
// clock64 in the MMA warp); the bounded loop above runs only when it is not.  Every wait
// of the kernel's roles is this warp-collective form.  An epilogue warp whose lane 0
// polled alone and broadcast the verdict with a shuffle took longer per accumulator
// hand-over: blockwise FP8 8192^3 589.8 -> 534.1 us, E4M3 4096^3 55.6 -> 51.2 us with
// every lane polling (A/B on one GPU).
__device__ __forceinline__ bool warp_wait_inl(uint32_t bar, uint32_t parity, const WaitCtl& c,
                                              uint32_t site) {
  if (__any_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, c, site);
}

// Bounded pause (used by a pair's follower while aborting, so copies it issued can land).
__device__ __forceinline__ void pause_ns(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) {
  }
}

}  // namespace gb300

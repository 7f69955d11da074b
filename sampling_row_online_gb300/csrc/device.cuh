// What the kernels of every translation unit share: device status bits,
// dependent-launch control and bounded barrier waits.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace spec {

constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;  // 1 s bound on any wait

// device status bits (per stream)
constexpr int ST_TOKEN = 1, ST_PARENT = 2, ST_TIMEOUT = 4;
constexpr int ST_LENGTH = 8;      // lengths[b] outside [0, L]
constexpr int ST_PAGE = 16;       // a page id outside [0, pages)
constexpr int ST_SLOTS = 32;      // a sequence's context and count do not fit its pages
constexpr int ST_NONFINITE = 64;  // a non-finite key or value was given to the cache

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Bounded wait on an mbarrier phase; false if it ran out.  The warp sleeps
// in hardware between polls.
// Also bounded in polls (each suspends at most ~20 us), should the clock
// not advance.
constexpr int WAIT_LIMIT_POLLS = 1 << 17;
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  const uint64_t t0 = clock_ns();
  for (int polls = 0; !mbar_try_wait_sleep(bar, parity, 20000u); ++polls)
    if (clock_ns() - t0 > WAIT_LIMIT_NS || polls > WAIT_LIMIT_POLLS) return false;
  return true;
}

}  // namespace spec

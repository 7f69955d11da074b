// A list of work items cut into equal stretches, one per worker, and the sums
// over a CTA that find a stretch's place in it.
#pragma once

#include <cstdint>

namespace spec {

// Equal stretches of `total` work items for `n` workers: the first `rem` have
// one more.  (32-bit arithmetic, one division: at a call's start and end every
// instruction is fetched for the first time, and 64-bit divisions took
// microseconds.)
struct Share {
  unsigned total, n, each, rem;
  __device__ __forceinline__ Share(unsigned total_, unsigned n_) : total(total_), n(n_), each(total_ / n_), rem(total_ - total_ / n_ * n_) {}
  __device__ __forceinline__ unsigned start(unsigned i) const { return i * each + min(i, rem); }
  __device__ __forceinline__ unsigned holder(unsigned item) const {  // each > 0
    const unsigned big = rem * (each + 1);
    return item < big ? item / (each + 1) : rem + (item - big) / each;
  }
};
// Inclusive sum over the CTA's threads; `sum` is the CTA's.
template <int WARPS>
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned *s, unsigned &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous use of s is over
  if (lane == 31) s[warp] = x;
  __syncthreads();
  sum = 0;
#pragma unroll 1
  for (int i = 0; i < WARPS; ++i) {
    if (i == warp) x += sum;
    sum += s[i];
  }
  return x;
}

}  // namespace spec

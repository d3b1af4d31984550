// The accumulators of a persistent tensor-core CTA or pair, taken in turn tile by tile, and the
// parities of their barriers' phases.  Plain C++, so that it also compiles and is tested on the
// host.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define GPTQ_HD __host__ __device__ __forceinline__
#else
#define GPTQ_HD inline
#endif

namespace gptq {

struct AccRing {
  int accs;              // accumulators
  int at = 0;            // the one whose turn it is
  uint32_t phase = 0;    // parity of its current phase: of "full" in this use, of "empty" at its end

  GPTQ_HD explicit AccRing(int n) : accs(n) {}
  GPTQ_HD void next() {
    if (++at == accs) { at = 0; phase ^= 1u; }
  }
  // Parity of the phase that the latest use of accumulator i completes.  A barrier that no use
  // has touched is in phase 0, and a wait for parity 1 passes at once there.
  GPTQ_HD uint32_t last(int i) const { return i < at ? phase : phase ^ 1u; }
};

}  // namespace gptq

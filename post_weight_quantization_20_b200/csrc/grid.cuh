// The min-max integer grid (GPTQ量化算法深度解析 §3.1, §3.3), shared by the sweep and the cache.
#pragma once
#include "common.cuh"

namespace gptq {

// Grid of a set of values with range [lo, hi] (lo <= 0 <= hi), all in IEEE fp32.
__device__ __forceinline__ void grid_params(float lo, float hi, float maxq, int sym, float& s,
                                            float& z) {
  if (sym) {
    float m = fmaxf(-lo, hi);
    if (m == 0.f) m = 1.f;
    s = __fdiv_rn(__fsub_rn(m, -m), maxq);
    z = (maxq + 1.f) * 0.5f;
  } else {
    if (lo == 0.f && hi == 0.f) { lo = -1.f; hi = 1.f; }
    s = __fdiv_rn(__fsub_rn(hi, lo), maxq);
    z = rintf(__fdiv_rn(-lo, s));
  }
}

}  // namespace gptq

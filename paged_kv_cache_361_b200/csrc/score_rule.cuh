// What pa_decode_multi and pa_prefill_window share of their score rule: capped
// scores, and the end of a row with its sink and log-sum-exp.
#pragma once

#include "common.cuh"

namespace pa {

// A capped score in base 2, cap_log2 * tanh(y), from z = 2 log2 e * y:
// tanh(y) = 1 - 2 / (2^z + 1), which is 1 and -1 where 2^z is inf and 0. Its
// absolute error, a few 2^-24, times a cap of 50 moves a score by 1e-5 at most
// (the hardware's tanh.approx, at 2^-11, would move it by 2 %).
__device__ __forceinline__ float capped_score(float z, float cap_log2) {
  return fmaf(-2.f * cap_log2, __fdividef(1.f, fast_exp2(z) + 1.f), cap_log2);
}

// The end of a row of head h: (m, l) of all its keys in base 2 with the head's
// sink, as the factor of o and the log-sum-exp. A row that sees nothing gives
// 0 and its sink, or -inf.
__device__ __forceinline__ float finish_row(const float* sinks, int h, float m, float l, float& lse) {
  const float sink = sinks ? __ldg(sinks + h) * 1.4426950408889634f : -INFINITY;
  const float M = fmaxf(m, sink);
  if (M == -INFINITY) {
    lse = -INFINITY;
    return 0.f;
  }
  const float f = exp2f(m - M);
  const float den = l * f + exp2f(sink - M);
  lse = (M + log2f(den)) * 0.6931471805599453f;
  return f / den;
}

}  // namespace pa

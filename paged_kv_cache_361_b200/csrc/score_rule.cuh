// What pa_decode_multi and pa_prefill_window share of their score rule: the range of
// the weights, capped scores, and the end of a row with its sink and log-sum-exp.
#pragma once

#include "common.cuh"

namespace pa {

// Weights that are rounded to f16 for their product with V are packed times 2^7,
// which o keeps until finish_row. They are 2^(x - m), the running maximum m moving
// when a score exceeds it by 8, so the largest one packed is between 2^7 and 2^15 of
// f16's 65504, and a weight keeps its 11 bits down to 2^-21 of the largest; below, it
// is off by 2^-32 of that at most (n keys together by n 2^-32 max|V| of the result).
// Without the factor a tail of 33000 keys behind one that outweighs each of them
// 2^25.5 times was lost whole. (A maximum taken 7 lower costs no multiplication, but
// rounds the exponents near 7 instead of near 0.)
constexpr float kWeightF16 = 128.f;

// What a raw score q.k is multiplied by, normal numbers.
struct ScoreScale {
  float scale_log2;  // scale * log2 e (times the K scale of an 8-bit cache)
  float cap_log2;    // softcap * log2 e, 0: none
  float cap_k;       // with a cap: scale / softcap (times the K scale)
  float cap_arg;     // 2 log2 e * cap_k
};

// tanh of a capped score y = scale s / cap. From z = 2 log2 e * y as 1 - 2 / (2^z +
// 1), which is 1 and -1 where 2^z is inf and 0, it has an absolute error of a few
// 2^-24: a cap of 50 makes that 5e-6 of the score, which shows where few keys are
// seen and the log-sum-exp is small. For small y, and without exponentials, it is
// y P(y^2), P(z) = 1 + z Q(z), Q of degree 1 or 3 fitted by least squares in Chebyshev
// polynomials at 400 Chebyshev nodes of z. With the fp32 coefficients y P is within
// 9e-8 of tanh(y) up to 0.2 (degree 1) and within 3e-8 up to 0.5, with a relative
// error of a few 2^-24. Four or six multiply-adds a score, where the exponentials are
// three operations of a pipe that does one for every eight multiply-adds. (The
// hardware's tanh.approx, at 2^-11, would move a score by 2 %.)
constexpr float kCapSmall = 0.2f, kCapMedium = 0.5f;
constexpr float kCapM0 = -0.333333105f, kCapM1 = 0.133305132f, kCapM2 = -0.0533910543f, kCapM3 = 0.0179992188f;

// Capped scores in base 2 from raw ones: |y| up to kCapMedium, and any.
__device__ __forceinline__ float capped_medium(const ScoreScale& a, float s) {
  const float y = s * a.cap_k, z = y * y;
  return a.cap_log2 * (y * fmaf(z, fmaf(z, fmaf(z, fmaf(z, kCapM3, kCapM2), kCapM1), kCapM0), 1.f));
}
__device__ __forceinline__ float capped_score(const ScoreScale& a, float s) {
  const float big = a.cap_log2 * fmaf(-2.f, __fdividef(1.f, fast_exp2(s * a.cap_arg) + 1.f), 1.f);
  return fabsf(s * a.cap_k) <= kCapMedium ? capped_medium(a, s) : big;
}

// P scaled by cap_log2: the capped score of y in base 2 is y times the value at
// y^2 (y = -inf gives +inf: a masked score stays -inf).
__device__ __forceinline__ float2 cap_poly(const float2 z, const float c0, const float c1, const float c2) {
  return ffma2(ffma2(make_float2(c2, c2), z, make_float2(c1, c1)), z, make_float2(c0, c0));
}
struct CapPoly {
  float one, s[2], m[4];
  __device__ __forceinline__ explicit CapPoly(float cap_log2) {
    one = cap_log2;
    s[0] = -0.333322763f * cap_log2;
    s[1] = 0.131206915f * cap_log2;
    m[0] = kCapM0 * cap_log2;
    m[1] = kCapM1 * cap_log2;
    m[2] = kCapM2 * cap_log2;
    m[3] = kCapM3 * cap_log2;
  }
  __device__ __forceinline__ float2 small(float2 y) const { return cap_poly(fmul2(y, y), one, s[0], s[1]); }
  __device__ __forceinline__ float2 medium(float2 y) const {
    const float2 z = fmul2(y, y), q = cap_poly(z, m[1], m[2], m[3]);
    return ffma2(ffma2(q, z, make_float2(m[0], m[0])), z, make_float2(one, one));
  }
};

// The weights of a softmax thread's 64 scores x (one row, raw, masked ones
// -inf), for both tcgen05 kernels: moves the running maximum m (base 2) when a
// score exceeds it by 8, scaling l by alpha and saying whether O has to be
// scaled too; adds the weights to l and packs them as f16, times kWeightF16.
//   amax: largest |score| that the row sees (capped scores)
template <bool CAPPED, int C>
__device__ __forceinline__ void row_weights(const ScoreScale& a, const float (&x)[C], float amax, const CapPoly& poly,
                                            float& m, float& l, float& alpha, bool& rescale, uint32_t (&ph)[C / 2]) {
  float pm[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) pm[u] = -INFINITY;
#pragma unroll
  for (int c = 0; c < C / 2; ++c) pm[c & 3] = fmax3(pm[c & 3], x[2 * c], x[2 * c + 1]);
  float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  if (!CAPPED)
    mx *= a.scale_log2;  // scale > 0 keeps the order
  else if (mx != -INFINITY)
    mx = capped_score(a, mx);
  alpha = 1.f;
  rescale = false;
  if (mx > m + 8.f) {
    alpha = fast_exp2(m - mx);  // 0 while m is -inf
    l *= alpha;
    rescale = m != -INFINITY;   // (O is 0 while m is -inf)
    m = mx;
  }
  const float nm = m == -INFINITY ? 0.f : -m;  // a row that has seen nothing: weights 0
  const float2 nm2 = make_float2(nm, nm);
  float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  auto weigh = [&](auto score) {
#pragma unroll
    for (int c = 0; c < C / 2; ++c) {
      const float2 y = score(make_float2(x[2 * c], x[2 * c + 1]));
      const float2 pp = make_float2(fast_exp2(y.x), fast_exp2(y.y));
      part[c & 1] = fadd2(part[c & 1], pp);
      const float2 ps = fmul2(pp, make_float2(kWeightF16, kWeightF16));
      const __half2 h = __floats2half2_rn(ps.x, ps.y);
      ph[c] = *reinterpret_cast<const uint32_t*>(&h);
    }
  };
  if constexpr (!CAPPED) {
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    weigh([&](float2 s) { return ffma2(s, sc2, nm2); });
  } else if (__all_sync(0xffffffffu, amax * a.cap_k <= kCapSmall)) {
    const float2 k2 = make_float2(a.cap_k, a.cap_k);
    weigh([&](float2 s) {
      const float2 y = fmul2(s, k2);
      return ffma2(y, poly.small(y), nm2);
    });
  } else if (__all_sync(0xffffffffu, amax * a.cap_k <= kCapMedium)) {
    const float2 k2 = make_float2(a.cap_k, a.cap_k);
    weigh([&](float2 s) {
      const float2 y = fmul2(s, k2);
      return ffma2(y, poly.medium(y), nm2);
    });
  } else {
    weigh([&](float2 s) {
      return make_float2(s.x == -INFINITY ? -INFINITY : capped_score(a, s.x) + nm,
                         s.y == -INFINITY ? -INFINITY : capped_score(a, s.y) + nm);
    });
  }
  l += (part[0].x + part[0].y) + (part[1].x + part[1].y);
}

// The reference of a row at the end of its keys. A maximum skips NaN, so a row whose
// scores are all NaN (a query of NaN) has kept -inf and would end as one that sees
// nothing; with a finite reference its NaN of l reaches the result through every merge.
__device__ __forceinline__ float final_ref(float m, float l) { return l != l ? 0.f : m; }

// Largest |x| of raw scores that the row sees, all of them or (masked_amax, which
// puts -inf in the place of the others) those of the columns lo .. hi. It chooses the
// form of the cap, whose last bits differ: bytes that no row sees must not count.
template <int C>
__device__ __forceinline__ float masked_amax(float (&x)[C], int lo, int hi) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool seen = c >= lo && c <= hi;
    if (seen) m[c & 3] = fmaxf(m[c & 3], fabsf(x[c]));
    x[c] = seen ? x[c] : -INFINITY;
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <int C>
__device__ __forceinline__ float row_amax(const float (&x)[C]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < C / 2; ++c) m[c & 3] = fmax3(m[c & 3], fabsf(x[2 * c]), fabsf(x[2 * c + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The end of a row of head h: (m, l) of all its keys in base 2 with the head's
// sink, as the factor of o (whose weights were packed times 1 / o_unit) and the
// log-sum-exp. A row that sees nothing gives 0 and its sink, or -inf. (A v_scale is
// multiplied in after the factor: the two together may be below fp32's range where
// the result is not.)
__device__ __forceinline__ float finish_row(const float* sinks, int h, float m, float l, float o_unit, float& lse) {
  const float sink = sinks ? __ldg(sinks + h) * 1.4426950408889634f : -INFINITY;
  const float M = fmaxf(m, sink);
  if (M == -INFINITY) {
    lse = -INFINITY;
    return 0.f;
  }
  const float f = exp2f(m - M);
  const float den = l * f + exp2f(sink - M);
  lse = (M + log2f(den)) * 0.6931471805599453f;
  return f / den * o_unit;
}

}  // namespace pa

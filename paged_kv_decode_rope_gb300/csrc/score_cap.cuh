// score_cap.cuh -- the tanh cap of the scored decodes, and its polynomial for the
// scored prefill.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// The cap of a score in base 2, softcap log2(e) tanh(x), of t = 2 log2(e) x
// (x = score / softcap). Beyond |x| = 0.3 it is cap - 2 cap / (2^t + 1), which
// is off by about cap 2^-23 whatever the score; a softcap far above the scores
// would lose them in that. So up to there it is x (k0 + k1 x^2 + k2 x^4 + k3
// x^6), which interpolates tanh(x) / x in x^2 at the four Chebyshev nodes of
// [0, 0.09] (relative error below 1.1e-8); both forms are computed.
struct ScoreCap {
  float cap;   // softcap * log2(e); 0: none
  float c[4];  // the polynomial's coefficients for powers 1, 3, 5, 7 of t
};
inline ScoreCap make_score_cap(float softcap) {
  constexpr double log2e = 1.4426950408889634;
  constexpr double k[4] = {0.99999999, -0.33332962, 0.13312578, -0.05022099};
  ScoreCap s;
  s.cap = static_cast<float>(softcap * log2e);
  double step = 1.0 / (2.0 * log2e);
  for (int i = 0; i < 4; ++i, step /= 4.0 * log2e * log2e) s.c[i] = static_cast<float>(softcap * log2e * k[i] * step);
  return s;
}

__device__ __forceinline__ float capped_score(const ScoreCap& s, float t) {
  constexpr float kMostT = static_cast<float>(2.0 * 1.4426950408889634 * 0.3);
  const float u = t * t;
  const float near = t * fmaf(fmaf(fmaf(s.c[3], u, s.c[2]), u, s.c[1]), u, s.c[0]);
  const float far = fmaf(-2.f * s.cap, fast_rcp(fast_exp2(t) + 1.f), s.cap);
  return fabsf(t) <= kMostT ? near : far;
}

}  // namespace pkv

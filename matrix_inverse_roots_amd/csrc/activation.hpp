// Activations of the feed-forward layers and their derivatives, in float32.
//
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution's
//   gelu_tanh  z sigma(p(z)), p(z) = 2 sqrt(2 / pi) (z + 0.044715 z^3):
//              (1 + tanh(y)) / 2 = sigma(2 y)
//   silu       z sigma(z)
// sigma(p) = 1 / (1 + 2^(-p log2 e)): one exp2 and one reciprocal instruction,
// off by some 2^-22 and, since p's roundings pass through the exponential, a few
// |p| 2^-24 relative (measured: silu 6e-7 at z = -8, gelu_tanh 4e-6 at -6).  Phi(-|z|)
// = t P(t) e^(-z^2/2) with t = 1 / (1 + 0.45 |z| / sqrt 2) and P of degree 9, fitted
// (least squares reweighted towards the largest relative error) to erfc(x) e^(x^2) /
// (2 t) over all x >= 0: 3.2e-8 relative in exact arithmetic, 3.6e-7 at most as P(t) t
// is evaluated here.  The exponential adds what rounding z^2/2 costs it, z^2/2 times
// some 2^-23: z Phi(z) is off by 4e-7 relative at most for |z| to 1, 9e-7 to 4, 2e-6 to
// 6, 2.9e-6 to 8, 7.7e-6 to 13 (measured, below zero; above it 1 - Phi(-z) is exact to
// 2^-23 from z = 2 on).  Small probabilities keep their digits, which 1 + erf would lose,
// and the exponential serves the derivative too.
//
// Values that are not finite follow the formulas: relu's derivative is [z > 0],
// so 0 at NaN; the others' are NaN at NaN and, as infinity times zero, at
// both infinities.  Finite values reach the limits 0 and 1 without overflow.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace shampoo {

struct ActNone {
  __device__ __forceinline__ float value(float z) const { return z; }
  __device__ __forceinline__ float both(float z, float& slope) const {
    slope = 1.f;
    return z;
  }
};

struct ActRelu {
  __device__ __forceinline__ float value(float z) const { return z < 0.f ? 0.f : z; }  // a NaN stays one
  __device__ __forceinline__ float both(float z, float& slope) const {
    slope = z > 0.f ? 1.f : 0.f;  // 0 at NaN
    return value(z);
  }
};

struct ActGelu {
  // Phi(z), and e^(-z^2/2)
  __device__ __forceinline__ float cdf(float z, float& bell) const {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3181980515339464f, fabsf(z), 1.f));
    bell = __builtin_amdgcn_exp2f(z * z * -0.7213475204444817f);
    float p = -0.02069614275f;
    p = __builtin_fmaf(p, t, 0.0953465046f);
    p = __builtin_fmaf(p, t, -0.1502958999f);
    p = __builtin_fmaf(p, t, 0.0712050923f);
    p = __builtin_fmaf(p, t, -0.01118165835f);
    p = __builtin_fmaf(p, t, 0.05997615575f);
    p = __builtin_fmaf(p, t, 0.0876258727f);
    p = __builtin_fmaf(p, t, 0.11413584175f);
    p = __builtin_fmaf(p, t, 0.1269415804f);
    p = __builtin_fmaf(p, t, 0.1269426604f);
    const float q = p * t * bell;
    return z < 0.f ? q : 1.f - q;
  }
  __device__ __forceinline__ float value(float z) const {
    float bell;
    return z * cdf(z, bell);
  }
  __device__ __forceinline__ float both(float z, float& slope) const {
    float bell;
    const float c = cdf(z, bell);
    slope = __builtin_fmaf(z * 0.3989422804014327f, bell, c);
    return z * c;
  }
};

// z sigma(p(z)): p(z) = z, or gelu_tanh's cubic (whose z^2 may overflow: p keeps its sign)
template <bool CUBIC> struct ActSigmoid {
  static constexpr float C1 = CUBIC ? 1.5957691216057308f : 1.f, C3 = 0.07135481627260025f;
  __device__ __forceinline__ float sigma(float z) const {
    constexpr float L2E = 1.4426950408889634f;
    const float slope = CUBIC ? __builtin_fmaf(-C3 * L2E, z * z, -C1 * L2E) : -L2E;
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(slope * z));
  }
  __device__ __forceinline__ float value(float z) const { return z * sigma(z); }
  __device__ __forceinline__ float both(float z, float& slope) const {
    const float s = sigma(z);
    if constexpr (CUBIC) {
      // behind 10^4 sigma is 0 or 1, and z p'(z) would overflow; NaN at an
      // infinity, which the bound takes away, comes back through z 0
      const float w = fminf(fmaxf(z, -1e4f), 1e4f), one = __builtin_fmaf(z, 0.f, 1.f);
      slope = __builtin_fmaf(s * (one - s), w * __builtin_fmaf(3.f * C3, w * w, C1), s);
    } else {
      slope = __builtin_fmaf(s * (1.f - s), z, s);
    }
    return z * s;
  }
};

// f(the activation of SHAMPOO_ACT_* code `act`)
template <typename F> __device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case 1: f(ActRelu{}); break;
    case 2: f(ActGelu{}); break;
    case 3: f(ActSigmoid<true>{}); break;
    case 4: f(ActSigmoid<false>{}); break;
    default: f(ActNone{}); break;
  }
}

}  // namespace shampoo

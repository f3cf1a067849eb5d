// Activations of the linear and gated feed-forward operators and their
// derivatives, in fp32.  ACT is an m3_act value.
#pragma once

#include "m3_common.hpp"

namespace m3 {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SIGMOID = 5, ACT_COUNT = 6 };

// FINE (fp32 io): the math library's exponential, erfc and division.
// Otherwise the exponential and the reciprocal are the hardware's and Phi a
// polynomial, off by about 1e-6 relative, far under the bf16 rounding of the
// result.  In both, the rounding of an exponential's argument m adds |m| units
// of 2^-24 and more in a tail: 1e-5 where Phi is 1e-38.
template <bool FINE>
__device__ __forceinline__ float exp_neg(float v) {  // exp(-v)
  if constexpr (FINE) return expf(-v);
  else return __builtin_amdgcn_exp2f(-1.4426950408889634f * v);
}
template <bool FINE>
__device__ __forceinline__ float recip(float v) {
  if constexpr (FINE) return 1.0f / v;
  else return __builtin_amdgcn_rcpf(v);
}
template <bool FINE>
__device__ __forceinline__ float sigmoid(float z) { return recip<FINE>(1.0f + exp_neg<FINE>(z)); }

// Phi(z), the normal distribution function; e receives exp(-z^2/2) (its
// density is e / sqrt(2 pi)).
template <bool FINE>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = exp_neg<FINE>(0.5f * z * z);
  if constexpr (FINE) {
    return 0.5f * erfcf(-0.7071067811865476f * z);
  } else {
    // Phi(-|z|) = exp(-z^2/2) t P(t), t = 1 / (1 + 0.46 |z| / sqrt(2)), P fitted
    // to the least relative error over t in (0, 1]: 6.8e-7.  (A fit of the least
    // absolute error with three terms less is 0.4 % off at z = -6, 2 % at -10.)
    const float t = recip<false>(1.0f + 0.325269119f * fabsf(z));
    const float a = 0.129763529f + t * (0.129778632f + t * (0.115590947f + t * 0.0934238768f));
    const float b = 0.0263053378f + t * (0.0845954819f + t * (-0.113314642f + t * 0.0338571766f));
    const float t2 = t * t;
    const float tail = e * t * (a + t2 * t2 * b);
    return z < 0.0f ? tail : 1.0f - tail;
  }
}

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <int ACT, bool FINE>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  else if constexpr (ACT == ACT_SILU) return z * sigmoid<FINE>(z);
  else if constexpr (ACT == ACT_GELU) {
    float e;
    return z * normal_cdf<FINE>(z, e);
  } else if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid<FINE>(2.0f * kGeluA * (z + kGeluB * z * z * z));
  else if constexpr (ACT == ACT_SIGMOID) return sigmoid<FINE>(z);
  else return z;
}

// act(z) and act'(z)
template <int ACT, bool FINE>
__device__ __forceinline__ void act_both(float z, float& f, float& df) {
  if constexpr (ACT == ACT_RELU) {
    f = z < 0.0f ? 0.0f : z;
    df = z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
  } else if constexpr (ACT == ACT_SILU) {
    const float p = sigmoid<FINE>(z);
    f = z * p;
    df = p * (1.0f + z * (1.0f - p));
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float p = normal_cdf<FINE>(z, e);
    f = z * p;
    df = p + z * e * 0.3989422804014327f;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // z/2 (1 + tanh u) = z sigmoid(2u); past |z| = 100 the sigmoid is 0 or 1
    // and its derivative 0, so z is held there where z^2 would overflow
    const float c = fminf(fmaxf(z, -100.0f), 100.0f);
    const float p = sigmoid<FINE>(2.0f * kGeluA * (c + kGeluB * c * c * c));
    f = z * p;
    df = p + c * p * (1.0f - p) * 2.0f * kGeluA * (1.0f + 3.0f * kGeluB * c * c);
    df = z == z ? df : z;
  } else if constexpr (ACT == ACT_SIGMOID) {
    // from exp(-|z|), so that neither tail is a difference of near-equal terms
    const float e = exp_neg<FINE>(fabsf(z)), r = recip<FINE>(1.0f + e);
    f = z < 0.0f ? e * r : r;
    df = e * r * r;
  } else {
    f = z;
    df = 1.0f;
  }
}

// Calls f(std::integral_constant<int, ACT>) for a runtime activation.
template <typename F>
inline auto with_act(int act, F&& f) {
  switch (act) {
    case ACT_RELU: return f(std::integral_constant<int, ACT_RELU>{});
    case ACT_SILU: return f(std::integral_constant<int, ACT_SILU>{});
    case ACT_GELU: return f(std::integral_constant<int, ACT_GELU>{});
    case ACT_GELU_TANH: return f(std::integral_constant<int, ACT_GELU_TANH>{});
    case ACT_SIGMOID: return f(std::integral_constant<int, ACT_SIGMOID>{});
    default: return f(std::integral_constant<int, ACT_NONE>{});
  }
}

}  // namespace m3

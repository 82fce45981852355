// linear_act.hpp -- the activations of the linear layer and their slopes, in
// fp32 (one value per call; a chain of a few v_fma, one v_exp and one v_rcp).
//
//   none       z
//   relu       max(z, 0); a NaN stays NaN
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z sigmoid(2u) = z (1 + tanh u) / 2, u = sqrt(2/pi)(z + 0.044715 z^3)
//   silu       z sigmoid(z)
//
// Phi's tail uses Q(a) = Phi(-a) = E(a) t P(t) for a >= 0 with E(a) =
// exp(-a^2 / 2) and t = 1 / (1 + 0.36 a): P is a polynomial of degree 6 fitted
// to Q / (E t) on [0, 14] by iteratively reweighted least squares of the
// relative error (largest 8.8e-7).  In fp32 the rounding of E's exponent, up to
// 3 / 2 a^2 times 2^-24, comes on top: the relative error of gelu(z) is 1.2e-6 for
// z >= -3, 3.5e-6 at -8 and 7.1e-6 at -13.  The slopes clamp their
// argument to |z| <= 20, where E is 0 in fp32 (silu: 200, where the sigmoid is 0
// or 1), so an infinity times 0 does not arise; a NaN passes the clamps (they
// compare).  z = -infinity gives NaN, as
// -infinity * 0 in the formula, with gelu, gelu_tanh and silu.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

namespace gemm_epi {

// Activation codes; the same numbers as the public header.
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2e = 1.44269504088896340736f;

// sigmoid(x) = 1 / (1 + exp(-x)); exp overflows to infinity, whose reciprocal is 0
__device__ __forceinline__ float sigmoid(float x) { return rcp_hw(1.0f + exp2_hw(-kLog2e * x)); }

// E = exp(-a^2 / 2) and Q = Phi(-a) for a >= 0
__device__ __forceinline__ void normal_tail(float a, float& E, float& Q) {
  E = exp2_hw(a * a * (-0.5f * kLog2e));
  const float t = rcp_hw(__builtin_fmaf(0.36f, a, 1.0f));
  float p = 0.04705947301089522f;
  p = __builtin_fmaf(p, t, -0.17977562615876672f);
  p = __builtin_fmaf(p, t, 0.1809689288381831f);
  p = __builtin_fmaf(p, t, 0.02653903856429528f);
  p = __builtin_fmaf(p, t, 0.13972302224815616f);
  p = __builtin_fmaf(p, t, 0.1417717685325932f);
  p = __builtin_fmaf(p, t, 0.14371309388216708f);
  Q = p * t * E;
}

constexpr float kTanhC = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kTanhK = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z < 0.0f ? 0.0f : z;
  } else if constexpr (ACT == ACT_GELU) {
    float E, Q;
    normal_tail(__builtin_fabsf(z), E, Q);
    return z * (z > 0.0f ? 1.0f - Q : Q);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float u = kTanhC * z * __builtin_fmaf(kTanhK * z, z, 1.0f);
    return z * sigmoid(2.0f * u);
  } else if constexpr (ACT == ACT_SILU) {
    return z * sigmoid(z);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_GELU) {
    const float zc = z > 20.0f ? 20.0f : (z < -20.0f ? -20.0f : z);
    const float a = __builtin_fabsf(zc);
    float E, Q;
    normal_tail(a, E, Q);
    // Phi(z) + z phi(z), phi = E / sqrt(2 pi)
    return __builtin_fmaf(zc * 0.39894228040143267794f, E, zc > 0.0f ? 1.0f - Q : Q);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float zc = z > 20.0f ? 20.0f : (z < -20.0f ? -20.0f : z);
    const float z2 = zc * zc;
    const float u2 = 2.0f * kTanhC * zc * __builtin_fmaf(kTanhK, z2, 1.0f);
    const float p = sigmoid(u2);
    // p + z p (1 - p) u2'
    return __builtin_fmaf(zc * p * (1.0f - p), 2.0f * kTanhC * __builtin_fmaf(3.0f * kTanhK, z2, 1.0f), p);
  } else if constexpr (ACT == ACT_SILU) {
    const float zc = z > 200.0f ? 200.0f : (z < -200.0f ? -200.0f : z);
    const float p = sigmoid(zc);
    return p * __builtin_fmaf(zc, 1.0f - p, 1.0f);
  } else {
    return 1.0f;
  }
}

// Calls f(act_c) with the activation code as a compile-time constant, so the
// (uniform) choice is made once per group of values.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}); break;
  }
}

}  // namespace gemm_epi

// What every linear kernel does with a finished sum: bias, activation, residual, store.
#pragma once

#include "op_common.cuh"
#include "ops.h"

namespace dit {

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + exp(-z)) from the exponential and reciprocal units: a few 1e-7 relative, also far in
// the negative tail, where a form with tanh would cancel.  z = -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * z)); }

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == DIT_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays
  // 0.5 v (1 + tanh u) = v sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
  if constexpr (ACT == DIT_ACT_GELU_TANH) {
    const float s = v * v;
    return v * sigmoid_fast(v * fmaf(s, 2.0f * 0.7978845608028654f * 0.044715f, 2.0f * 0.7978845608028654f));
  }
  // v Phi(v), Phi(-|v|) = erfc(z) / 2 at z = |v| / sqrt 2 by the rational approximation 7.1.26 of
  // Abramowitz and Stegun's handbook: erfc(z) = (a1 t + .. + a5 t^5) exp(-z^2), t = 1 / (1 + p z),
  // off by at most 1.5e-7
  if constexpr (ACT == DIT_ACT_GELU) {
    const float z = fabsf(v) * 0.7071067811865476f;
    const float t = rcp_approx(fmaf(0.3275911f, z, 1.0f));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float tail = 0.5f * p * t * ex2_approx(-1.4426950408889634f * z * z);
    return v * (v < 0.f ? tail : 1.0f - tail);
  }
  if constexpr (ACT == DIT_ACT_SILU) return v * sigmoid_fast(v);
  return v;
}

// f(std::integral_constant<int, ACT>) for the run-time act
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case DIT_ACT_RELU: f(std::integral_constant<int, DIT_ACT_RELU>()); break;
    case DIT_ACT_GELU_TANH: f(std::integral_constant<int, DIT_ACT_GELU_TANH>()); break;
    case DIT_ACT_GELU: f(std::integral_constant<int, DIT_ACT_GELU>()); break;
    case DIT_ACT_SILU: f(std::integral_constant<int, DIT_ACT_SILU>()); break;
    default: f(std::integral_constant<int, DIT_ACT_NONE>()); break;
  }
}

// residual and store of one already activated value
template <typename T, bool F32>
__device__ __forceinline__ void linear_put(const LinearArgs& a, int m, int n, float v) {
  using O = typename std::conditional<F32, float, T>::type;
  if (a.residual) v += to_f32(static_cast<const O*>(a.residual)[m * a.ldr + n]);
  static_cast<O*>(a.y)[m * a.ldy + n] = from_f32<O>(v);
}

template <typename T>
__device__ __forceinline__ void linear_store(const LinearArgs& a, int m, int n, float v) {
  if (a.bias) v += __ldg(a.bias + n);
  with_act(a.act, [&](auto act) { v = activate<decltype(act)::value>(v); });
  if (a.out_f32) linear_put<T, true>(a, m, n, v);
  else linear_put<T, false>(a, m, n, v);
}

}  // namespace dit

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

// 1 / (1 + exp(-z)) from the exponential and reciprocal units: (|z| + 8) 2^-23 relative at most, the rounding of
// the exponent, in the negative tail as well, where a form with tanh would cancel.  z = -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * z)); }

// DIT_ACT_GELU for a 16-bit output (LinearArgs::act; not an argument of the entry point)
constexpr int kActGelu16 = DIT_ACT_SILU + 1;

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == DIT_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays
  // 0.5 v (1 + tanh u) = v sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
  if constexpr (ACT == DIT_ACT_GELU_TANH) {
    const float s = v * v;
    return v * sigmoid_fast(v * fmaf(s, 2.0f * 0.7978845608028654f * 0.044715f, 2.0f * 0.7978845608028654f));
  }
  // v Phi(v), Phi(-a) = exp(-a^2 / 2) R(a) at a = |v|.  R is a polynomial in t = 1 / (1 + 0.3 a) without constant term: the
  // form of Hastings' approximations (7.1.26 of Abramowitz and Stegun's handbook is one, good to 1.5e-7 of 1 only, 1.6e-3
  // of the result at v = -5), fitted by reweighted least squares on the relative error over [0, 14].
  // float32 output: eight terms (1.5e-7, 4.3e-7 in float32), and the exponent's rounding (up to 120 2^-24 of the result)
  // is computed exactly and put back: 1e-6 as far as float32 reaches.  16 bits: six terms (8.2e-6) and no such
  // correction, 2^-15 in all, an eighth of fp16's half step (16384 x 1152 -> 4608: 148 us, a tenth more with the other).
  if constexpr (ACT == DIT_ACT_GELU || ACT == kActGelu16) {
    constexpr float c = -0.7213475108146667f, c_lo = -9.6298e-9f;  // -1 / (2 ln 2)
    const float a = fminf(fabsf(v), 15.0f);  // nothing is left of the tail there
    const float t = rcp_approx(fmaf(0.3f, a, 1.0f));
    const float s = a * a, y = s * c;
    float p, e = ex2_approx(y);
    if constexpr (ACT == DIT_ACT_GELU) {
      p = fmaf(t, 0.035674650222063065f, -0.15720251202583313f);
      p = fmaf(p, t, 0.20635241270065308f);
      p = fmaf(p, t, -0.05368255823850632f);
      p = fmaf(p, t, 0.12856101989746094f);
      p = fmaf(p, t, 0.09991368651390076f);
      p = fmaf(p, t, 0.12075392156839371f);
      p = fmaf(p, t, 0.11962930113077164f);
      const float lost = fmaf(s, c, -y) + fmaf(fmaf(a, a, -s), c, s * c_lo);
      e = fmaf(e, 0.6931472f * lost, e);
    } else {
      p = fmaf(t, -0.0770975798368454f, 0.21603742241859436f);
      p = fmaf(p, t, -0.016948366537690163f);
      p = fmaf(p, t, 0.14419648051261902f);
      p = fmaf(p, t, 0.1137419119477272f);
      p = fmaf(p, t, 0.12007423490285873f);
    }
    const float tail = p * t * e;
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
    case kActGelu16: f(std::integral_constant<int, kActGelu16>()); break;
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

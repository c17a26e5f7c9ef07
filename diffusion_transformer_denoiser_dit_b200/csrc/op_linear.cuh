// What every linear kernel does with a finished sum: bias, activation, residual, store.
#pragma once

#include "op_common.cuh"
#include "ops.h"

namespace dit {

// 1 / (1 + exp(-z)) from the exponential and reciprocal units (a few 1e-7 relative, also far
// in the negative tail, where a form with tanh would cancel)
__device__ __forceinline__ float sigmoid_fast(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case DIT_ACT_RELU:
      return v > 0.f ? v : v != v ? v : 0.f;
    case DIT_ACT_GELU_TANH:  // 0.5 v (1 + tanh u) = v sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
      return v * sigmoid_fast(2.0f * 0.7978845608028654f * fmaf(0.044715f * v, v * v, v));
    case DIT_ACT_GELU:
      return 0.5f * v * erfcf(-0.7071067811865476f * v);
    case DIT_ACT_SILU:
      return v * sigmoid_fast(v);
    default:
      return v;
  }
}

template <typename T>
__device__ __forceinline__ void linear_store(const LinearArgs& a, int m, int n, float v) {
  if (a.bias) v += __ldg(a.bias + n);
  v = activate(v, a.act);
  const long long at = m * a.ldy + n;
  if (a.out_f32) {
    if (a.residual) v += static_cast<const float*>(a.residual)[m * a.ldr + n];
    static_cast<float*>(a.y)[at] = v;
  } else {
    if (a.residual) v += to_f32(static_cast<const T*>(a.residual)[m * a.ldr + n]);
    static_cast<T*>(a.y)[at] = from_f32<T>(v);
  }
}

}  // namespace dit

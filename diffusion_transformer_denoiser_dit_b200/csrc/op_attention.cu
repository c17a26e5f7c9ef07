// Attention over packed sequences, grouped heads, causal or full.
#include <math.h>

#include "internal.h"
#include "op_common.cuh"
#include "ops.h"

namespace dit {

// One warp per (query token, head): a running maximum and sum over the keys, the dh features
// spread over the lanes.
template <typename T>
__global__ void __launch_bounds__(128) attention_rows_kernel(const PackedAttnArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + warp;
  pdl_trigger();
  pdl_wait();
  if (item >= static_cast<long long>(a.total_q) * a.H) return;
  const int tok = static_cast<int>(item / a.H), h = static_cast<int>(item % a.H);
  int lo = 0, hi = a.n_seq;  // the last sequence that starts at or before tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_q[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const int q0 = a.cu_q[lo], q1 = min(a.cu_q[lo + 1], a.total_q);
  if (tok < q0 || tok >= q1) return;
  const int k0 = min(max(a.cu_k[lo], 0), a.total_k), k1 = min(max(a.cu_k[lo + 1], k0), a.total_k);
  const int nk = k1 - k0;
  const int last = a.causal ? min(nk, tok - q0 + nk - (q1 - q0) + 1) : nk;
  const T* q = static_cast<const T*>(a.q) + tok * a.q_tok + h * a.q_head;
  const T* k = static_cast<const T*>(a.k) + k0 * a.k_tok + (h / (a.H / a.Hk)) * a.k_head;
  const T* v = static_cast<const T*>(a.v) + k0 * a.v_tok + (h / (a.H / a.Hk)) * a.v_head;
  float qf[4] = {}, o[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.dh) qf[i] = to_f32(q[lane + 32 * i]) * a.scale;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < last; ++j) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.dh) s = fmaf(qf[i], to_f32(k[j * a.k_tok + lane + 32 * i]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.dh) o[i] = fmaf(p, to_f32(v[j * a.v_tok + lane + 32 * i]), o[i] * c);
    m = mn;
  }
  const float inv = last > 0 ? 1.f / l : 0.f;
  T* out = static_cast<T*>(a.o) + tok * a.o_tok + h * a.o_head;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.dh) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
  if (lane == 0 && a.lse) a.lse[static_cast<long long>(h) * a.total_q + tok] = last > 0 ? m + logf(l) : -INFINITY;
}

cudaError_t launch_attention_packed(const PackedAttnArgs& a, int, cudaStream_t st) {
  const long long blocks = (static_cast<long long>(a.total_q) * a.H + 3) / 4;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (a.fp16) return launch_kernel(attention_rows_kernel<__half>, dim3(blocks), dim3(128), 0, st, a);
  return launch_kernel(attention_rows_kernel<__nv_bfloat16>, dim3(blocks), dim3(128), 0, st, a);
}

}  // namespace dit

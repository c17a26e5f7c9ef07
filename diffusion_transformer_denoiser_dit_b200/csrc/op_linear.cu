// y = act(x W^T + b) + r for 16-bit x, W: float32 sums and epilogue, one rounding at the end.
#include "internal.h"
#include "op_common.cuh"
#include "op_linear.cuh"
#include "ops.h"

namespace dit {

// One warp per output feature and MB rows of x; lanes stride over K, the partial sums of the
// lanes are added by shuffles.
template <typename T, int MB, bool VEC>
__global__ void __launch_bounds__(256) linear_rows_kernel(const LinearArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + warp, m0 = blockIdx.y * MB;
  pdl_trigger();
  pdl_wait();
  if (n >= a.N) return;
  const T* w = static_cast<const T*>(a.w) + n * a.ldw;
  const T* x = static_cast<const T*>(a.x) + m0 * a.ldx;
  const int nm = min(MB, a.M - m0);
  float acc[MB] = {};
  int k = 0;
  if constexpr (VEC) {
    const int kv = a.K & ~7;
    for (int kk = lane * 8; kk < kv; kk += 256) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(w + kk));
      const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (m >= nm) break;
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + m * a.ldx + kk));
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = unpack2<T>(ws[i]), q = unpack2<T>(xs[i]);
          acc[m] = fmaf(p.x, q.x, acc[m]);
          acc[m] = fmaf(p.y, q.y, acc[m]);
        }
      }
    }
    k = kv;
  }
  for (int kk = k + lane; kk < a.K; kk += 32) {
    const float p = to_f32(w[kk]);
#pragma unroll
    for (int m = 0; m < MB; ++m)
      if (m < nm) acc[m] = fmaf(p, to_f32(x[m * a.ldx + kk]), acc[m]);
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const float s = warp_sum(acc[m]);
    if (lane == 0 && m < nm) linear_store<T>(a, m0 + m, n, s);
  }
}

template <typename T, bool VEC>
static cudaError_t launch_rows(const LinearArgs& a, cudaStream_t st) {
  const unsigned gx = (a.N + 7) / 8;
  auto run = [&](auto kernel, int mb) -> cudaError_t {
    // at most 65535 row groups in one grid
    for (int m = 0; m < a.M; m += mb * 65535) {
      LinearArgs c = a;
      c.x = static_cast<const T*>(a.x) + m * a.ldx;
      const int es = a.out_f32 ? 4 : 2;
      if (a.residual) c.residual = static_cast<const char*>(a.residual) + m * a.ldr * es;
      c.y = static_cast<char*>(a.y) + m * a.ldy * es;
      c.M = a.M - m < mb * 65535 ? a.M - m : mb * 65535;
      const cudaError_t e = launch_kernel(kernel, dim3(gx, (c.M + mb - 1) / mb), dim3(256), 0, st, c);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  };
  if (a.M <= 1) return run(linear_rows_kernel<T, 1, VEC>, 1);
  if (a.M <= 4) return run(linear_rows_kernel<T, 4, VEC>, 4);
  return run(linear_rows_kernel<T, 8, VEC>, 8);
}

cudaError_t launch_linear_fused(const LinearArgs& a, int num_sms, cudaStream_t st) {
  if (a.M > 8) return launch_linear_tc(a, num_sms, st);
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0 &&
                   ((a.ldx | a.ldw) & 7) == 0;
  if (a.fp16) return vec ? launch_rows<__half, true>(a, st) : launch_rows<__half, false>(a, st);
  return vec ? launch_rows<__nv_bfloat16, true>(a, st) : launch_rows<__nv_bfloat16, false>(a, st);
}

}  // namespace dit

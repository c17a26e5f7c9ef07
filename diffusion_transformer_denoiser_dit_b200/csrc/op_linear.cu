// y = act(x W^T + b) + r for 16-bit x, W: float32 sums and epilogue, one rounding at the end.
#include "internal.h"
#include "op_common.cuh"
#include "op_linear.cuh"
#include "ops.h"

namespace dit {

// Few rows: the weights are read once, by warps that take NR output features and all MB rows of x; ks warps of
// a block share the features and split K.  Bound by HBM (8192 x 8192: 134 MB), so that the loads count: each
// lane holds NR 16-byte pieces of W at a time, and a piece of x, unpacked once, serves NR features.
template <typename T, int MB, int NR, bool VEC>
__global__ void __launch_bounds__(256) linear_rows_kernel(const LinearArgs a, const int ks) {
  constexpr int V = NR * MB;
  __shared__ float part[8][V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % ks;
  const int n0 = (blockIdx.x * (8 / ks) + warp / ks) * NR;
  pdl_trigger();
  pdl_wait();
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  const T* wr[NR];
  const T* xr[MB];
#pragma unroll
  for (int i = 0; i < NR; ++i) wr[i] = w + min(n0 + i, a.N - 1) * a.ldw;  // features past N repeat the last
#pragma unroll
  for (int m = 0; m < MB; ++m) xr[m] = x + min(m, a.M - 1) * a.ldx;
  float acc[V] = {};
  int k = 0;
  if constexpr (VEC) {
    const int kv = a.K & ~7;
#pragma unroll 2
    for (int kk = (slice * 32 + lane) * 8; kk < kv; kk += ks * 256) {
      uint4 wv[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) wv[i] = __ldg(reinterpret_cast<const uint4*>(wr[i] + kk));
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(xr[m] + kk));
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 q = unpack2<T>(xs[e]);
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const uint32_t ws[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
            const float2 p = unpack2<T>(ws[e]);
            acc[i * MB + m] = fmaf(p.x, q.x, acc[i * MB + m]);
            acc[i * MB + m] = fmaf(p.y, q.y, acc[i * MB + m]);
          }
        }
      }
    }
    k = kv;
  }
  // what is left of K; all of it where rows are not 16-byte aligned (M = 1), two bytes per load: 1151 -> 4608 9.3 us for
  // 3.8, 8191 -> 8192 81 for 22.7
  for (int kk = k + slice * 32 + lane; kk < a.K; kk += ks * 32) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float p = to_f32(wr[i][kk]);
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[i * MB + m] = fmaf(p, to_f32(xr[m][kk]), acc[i * MB + m]);
    }
  }
  // sums over the lanes: V values are halved by each exchange until a lane has one, of index lane / (32 / V)
  int o = 16;
#pragma unroll
  for (int n = V; n > 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? acc[i + n / 2] : acc[i], send = up ? acc[i] : acc[i + n / 2];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  for (; o > 0; o /= 2) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
  const int v = lane / (32 / V), n = n0 + v / MB, m = v % MB;
  if (ks > 1) {
    if (lane % (32 / V) == 0) part[warp][v] = acc[0];
    __syncthreads();
    if (slice > 0) return;
    for (int j = 1; j < ks; ++j) acc[0] += part[warp + j][v];
  }
  if (lane % (32 / V) == 0 && n < a.N && m < a.M) linear_store<T>(a, m, n, acc[0]);
}

template <typename T, int MB, int NR, bool VEC>
static cudaError_t launch_rows(const LinearArgs& a, int num_sms, cudaStream_t st) {
  const long long groups = (a.N + NR - 1) / NR;
  // 16 warps for every SM, if K has 512 values for each
  int ks = 1;
  while (ks < 8 && groups * ks < 16ll * num_sms && a.K >= 1024 * ks) ks *= 2;
  const long long blocks = (groups * ks + 7) / 8;
  return launch_kernel(linear_rows_kernel<T, MB, NR, VEC>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, ks);
}

template <typename T>
static cudaError_t launch_t(const LinearArgs& a, bool vec, int num_sms, cudaStream_t st) {
  if (a.M == 1) return vec ? launch_rows<T, 1, 1, true>(a, num_sms, st) : launch_rows<T, 1, 1, false>(a, num_sms, st);
  if (vec && a.M <= 2) return launch_rows<T, 2, 4, true>(a, num_sms, st);
  if (vec && a.M <= 4) return launch_rows<T, 4, 4, true>(a, num_sms, st);
  return launch_linear_tc(a, num_sms, st);
}

cudaError_t launch_linear_fused(const LinearArgs& args, int num_sms, cudaStream_t st) {
  LinearArgs a = args;
  if (a.act == DIT_ACT_GELU && !a.out_f32) a.act = kActGelu16;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0 &&
                   ((a.ldx | a.ldw) & 7) == 0;
  return a.fp16 ? launch_t<__half>(a, vec, num_sms, st) : launch_t<__nv_bfloat16>(a, vec, num_sms, st);
}

}  // namespace dit

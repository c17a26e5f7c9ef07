// Rotary positions: pair k of a head's first 2P features turns by the angle pos * freq_k,
//   y_a = amp (x_a cos - x_b sin),  y_b = amp (x_b cos + x_a sin),
// (a, b) = (k, k + P) in the half layout and (2k, 2k + 1) in the interleaved one.
//
// Angles: freq_k is kept as a fraction of a turn in 64-bit fixed point, so pos * freq_k modulo
// one turn is one wrapping integer multiplication, exact for every 64-bit position; the top 32
// bits go to float32 (half a turn at most, so 2^-25 of a turn) and through sincospif.  A
// float32 product pos * freq would be off by 0.004 rad at position 10^5.
//
// A block owns TT tokens: it computes their cos / sin once into shared memory and all heads of
// those tokens read them from there.  HBM-bound: x is read once and y written once.
#include "internal.h"
#include "op_common.cuh"
#include "ops.h"

namespace dit {

constexpr int kRotaryThreads = 256;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// PAIR items: V pairs of one (token, head), two vectors of V elements each; REST items: V
// elements behind the rotated part, copied.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads)
    rotary_kernel(const __grid_constant__ dit_rotary r, const RotaryArgs a, const int TT, const int rest) {
  extern __shared__ float2 cs[];  // [TT][P] (cos, sin) times the amplitude
  const int P = r.pairs, each = P / r.axes;
  const int t0 = blockIdx.x * TT, nt = min(TT, a.tokens - t0);
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < nt * P; i += kRotaryThreads) {
    const int t = i / P, k = i - t * P, axis = k / each;
    const size_t at = static_cast<size_t>(t0 + t) * r.axes + axis;
    const long long pos = a.pos64 ? static_cast<const long long*>(a.pos)[at] : static_cast<const int*>(a.pos)[at];
    const uint64_t turn = static_cast<uint64_t>(pos) * r.turns[k - axis * each];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c * r.amplitude, (a.transpose ? -s : s) * r.amplitude);
  }
  __syncthreads();
  const int pc = P / V, per = pc + rest;  // items per (token, head)
  const int items = nt * a.heads * per;
  for (int i = threadIdx.x; i < items; i += kRotaryThreads) {
    const int th = i / per, c = i - th * per, t = th / a.heads, h = th - t * a.heads;
    const T* x = static_cast<const T*>(a.x) + (t0 + t) * a.x_tok + h * a.x_head;
    T* y = static_cast<T*>(a.y) + (t0 + t) * a.y_tok + h * a.y_head;
    if (c >= pc) {
      const int e = 2 * P + (c - pc) * V;
      *reinterpret_cast<Vec<T, V>*>(y + e) = *reinterpret_cast<const Vec<T, V>*>(x + e);
      continue;
    }
    const int ea = INTERLEAVED ? 2 * V * c : V * c, eb = INTERLEAVED ? ea + V : P + V * c;
    Vec<T, V> u = *reinterpret_cast<const Vec<T, V>*>(x + ea), w = *reinterpret_cast<const Vec<T, V>*>(x + eb);
    const float2* f = cs + t * P + c * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      // pair j of this item: (u[j], w[j]), or element 2j of the two vectors back to back
      T& p = INTERLEAVED ? (2 * j < V ? u.v[(2 * j) % V] : w.v[(2 * j) % V]) : u.v[j];
      T& q = INTERLEAVED ? (2 * j + 1 < V ? u.v[(2 * j + 1) % V] : w.v[(2 * j + 1) % V]) : w.v[j];
      const float xa = to_f32(p), xb = to_f32(q);
      const float2 g = f[j];
      p = from_f32<T>(xa * g.x - xb * g.y);
      q = from_f32<T>(xb * g.x + xa * g.y);
    }
    *reinterpret_cast<Vec<T, V>*>(y + ea) = u;
    *reinterpret_cast<Vec<T, V>*>(y + eb) = w;
  }
}

template <typename T, int V>
static cudaError_t launch_v(const dit_rotary& r, const RotaryArgs& a, cudaStream_t st) {
  int TT = kRotaryThreads / r.pairs;
  TT = TT < 1 ? 1 : TT > 8 ? 8 : TT;
  const int rest = a.x == a.y ? 0 : (a.dh - 2 * r.pairs) / V;  // in place: the rest already is where it belongs
  const dim3 grid((a.tokens + TT - 1) / TT);
  const size_t smem = sizeof(float2) * TT * r.pairs;
  return a.interleaved ? launch_kernel(rotary_kernel<T, V, true>, grid, dim3(kRotaryThreads), smem, st, r, a, TT, rest)
                       : launch_kernel(rotary_kernel<T, V, false>, grid, dim3(kRotaryThreads), smem, st, r, a, TT, rest);
}

template <typename T>
static cudaError_t launch_t(const dit_rotary& r, const RotaryArgs& a, cudaStream_t st) {
  // widest vector that every address of x and y is a multiple of and that divides the parts
  auto fits = [&](int v) {
    const uint64_t bytes = sizeof(T) * v;
    const uint64_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                        sizeof(T) * static_cast<uint64_t>(a.x_tok | a.x_head | a.y_tok | a.y_head);
    return at % bytes == 0 && r.pairs % v == 0 && (a.dh - 2 * r.pairs) % v == 0;
  };
  constexpr int W = 16 / sizeof(T);
  if (fits(W)) return launch_v<T, W>(r, a, st);
  if (fits(W / 2)) return launch_v<T, W / 2>(r, a, st);
  return launch_v<T, 1>(r, a, st);
}

cudaError_t launch_rotary(const dit_rotary& r, const RotaryArgs& a, int, cudaStream_t st) {
  if (a.dtype == DIT_DTYPE_BF16) return launch_t<__nv_bfloat16>(r, a, st);
  if (a.dtype == DIT_DTYPE_FP16) return launch_t<__half>(r, a, st);
  return launch_t<float>(r, a, st);
}

}  // namespace dit

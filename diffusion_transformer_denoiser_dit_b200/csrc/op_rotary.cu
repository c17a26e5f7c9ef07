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

constexpr int kRotaryThreads = 128;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// V pairs of a row at a time, two vectors of V elements; `rest` vectors behind the turned part.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, 10)
    rotary_kernel(const __grid_constant__ dit_rotary r, const RotaryArgs a, const int TT, const int rest) {
  extern __shared__ float2 cs[];  // [TT][V][P / V] (cos, sin) times the amplitude
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
    // pair k = V c + j of a token at [j][c]: the lanes of a row read neighbouring entries
    cs[t * P + (k % V) * (P / V) + k / V] = make_float2(c * r.amplitude, (a.transpose ? -s : s) * r.amplitude);
  }
  __syncthreads();
  // A thread keeps its pairs c of a row (one head of one token) and steps through the rows of the block's
  // tokens; it also copies every pc-th vector behind the turned part.  One row at a time in small blocks:
  // ten blocks of an SM overlap their loads (32768 x 20 x 128 bf16, half turned: 54 us, 6.2 TB/s; all
  // turned: 61 us, with four rows in flight per thread and three blocks of 256: 123 us).  The bound of ten leaves 48
  // registers, which the 16-bit kernels of eight elements exceed by 8 to 16 spilled bytes; with nine blocks, and none: 59 us.
  const int pc = P / V;
  for (int c0 = 0; c0 < pc; c0 += kRotaryThreads) {
    const int wide = min(pc - c0, kRotaryThreads), together = kRotaryThreads / wide;  // rows at a time
    const int c = c0 + static_cast<int>(threadIdx.x) % wide, first = static_cast<int>(threadIdx.x) / wide;
    if (first >= together) continue;
    const int ea = INTERLEAVED ? 2 * V * c : V * c, eb = INTERLEAVED ? ea + V : P + V * c;
    const int rows = nt * a.heads;
    int t = first / a.heads, h = first - t * a.heads;
    for (int r = first; r < rows; r += together) {
      const T* x = static_cast<const T*>(a.x) + (t0 + t) * a.x_tok + h * a.x_head;
      T* y = static_cast<T*>(a.y) + (t0 + t) * a.y_tok + h * a.y_head;
      Vec<T, V> u = *reinterpret_cast<const Vec<T, V>*>(x + ea), w = *reinterpret_cast<const Vec<T, V>*>(x + eb);
      for (int e = c; e < rest; e += 2 * pc) {
        const bool two = e + pc < rest;
        Vec<T, V> m = *reinterpret_cast<const Vec<T, V>*>(x + 2 * P + e * V), l;
        if (two) l = *reinterpret_cast<const Vec<T, V>*>(x + 2 * P + (e + pc) * V);
        *reinterpret_cast<Vec<T, V>*>(y + 2 * P + e * V) = m;
        if (two) *reinterpret_cast<Vec<T, V>*>(y + 2 * P + (e + pc) * V) = l;
      }
      const float2* f = cs + t * P + c;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // pair j of this item: (u[j], w[j]), or element 2j of the two vectors back to back
        T& p = INTERLEAVED ? (2 * j < V ? u.v[(2 * j) % V] : w.v[(2 * j) % V]) : u.v[j];
        T& q = INTERLEAVED ? (2 * j + 1 < V ? u.v[(2 * j + 1) % V] : w.v[(2 * j + 1) % V]) : w.v[j];
        const float xa = to_f32(p), xb = to_f32(q);
        const float2 g = f[j * pc];
        p = from_f32<T>(xa * g.x - xb * g.y);
        q = from_f32<T>(xb * g.x + xa * g.y);
      }
      *reinterpret_cast<Vec<T, V>*>(y + ea) = u;
      *reinterpret_cast<Vec<T, V>*>(y + eb) = w;
      for (h += together; h >= a.heads; h -= a.heads) ++t;
    }
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

cudaError_t launch_rotary(const dit_rotary& r, const RotaryArgs& a, cudaStream_t st) {
  if (a.dtype == DIT_DTYPE_BF16) return launch_t<__nv_bfloat16>(r, a, st);
  if (a.dtype == DIT_DTYPE_FP16) return launch_t<__half>(r, a, st);
  return launch_t<float>(r, a, st);
}

}  // namespace dit

// Element types of the packed-layer building blocks: loads to and stores from float32.
#pragma once

#include <math.h>

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dit {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two 16-bit values in one register (lo at the lower address) to and from float32.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// v, which every lane holds, marked as one value for the warp (the compiler then keeps what depends
// on it, branches among it, in uniform registers).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ int warp_index() { return static_cast<int>(uniform(threadIdx.x >> 5)); }

// One lane of a converged warp, the same each time.  The roles that issue TMA copies and MMAs
// run their loops with the whole warp and elect a lane around the instructions alone: their
// operands then stay warp-uniform.  With the loop inside `if (lane == 0)` the four MMAs and the
// commit of one K stage took 543 cycles to issue (clock64), whatever their size.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e != 0;
}
// mbar_wait that looks at the clock only once in 1024 tries: a read of globaltimer between two
// tries costs more than most waits last.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity, int* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        record_status(status, DIT_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
}
// The same by a whole warp: false for every lane when it ran out for any.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, status));
}

// After a wait that ran out: what the warp issued (copies, products: microseconds) gets a millisecond to end
// before the block leaves its memory.
__device__ __forceinline__ void after_timeout() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 1000000u) {
  }
  __syncwarp();
}

// Maxima that keep a NaN (fmaxf drops it): a softmax whose maximum forgets a NaN score would lose the row's.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The new reference maximum of a softmax row: one of +inf (an infinite score, or one that overflowed) becomes
// NaN, as inf - inf in its exponentials is.
__device__ __forceinline__ float reference_max(float a, float b) {
  const float m = max_nan(a, b);
  return m == INFINITY ? NAN : m;
}

// Instruction descriptor, kind::f16: A and B both fp16 or both bf16, K-major, f32 accumulator.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N) {
  constexpr uint32_t f = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// A CTA's shared memory may be written by another only once it runs.  This CTA says so early, and every
// thread waits for the others just before the first remote access, so that the wait hides behind the work
// between the two.  Nothing is published: the barrier orders starts only.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_all_started() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// 16 bytes into the shared memory of a CTA of the cluster (address from mapa)
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

}  // namespace dit

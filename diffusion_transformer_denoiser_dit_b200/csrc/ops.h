// Launch interfaces of the packed-layer building blocks (op_api.cu checks the arguments and
// calls these): linear with bias, activation and residual; attention over packed sequences;
// rotary positions.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dit.h"

namespace dit {

// y[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
struct LinearArgs {
  const void *x, *w;        // 16-bit, rows ldx / ldw elements apart
  const float* bias;        // [N] or null
  const void* residual;     // the output's type, rows ldr apart, or null; may be y itself
  void* y;                  // 16-bit (x's type) or float32, rows ldy apart
  long long ldx, ldw, ldr, ldy;
  int M, N, K;
  int act;                  // DIT_ACT_*
  int fp16;                 // x, w (and a 16-bit y) are fp16, else bf16
  int out_f32;
  int* status;
};
cudaError_t launch_linear_fused(const LinearArgs& a, int num_sms, cudaStream_t st);
// The tensor-core kernels (op_linear_tc.cu).
cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t st);

// Packed attention: sequence s owns query tokens cu_q[s] .. cu_q[s+1] and keys cu_k[s] .. cu_k[s+1].
struct PackedAttnArgs {
  const void *q, *k, *v;
  void* o;
  float* lse;               // [H, total_q] or null
  const int *cu_q, *cu_k;   // [n_seq + 1]
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;  // strides in elements
  int n_seq, total_q, total_k, max_q, max_k;
  int H, Hk, dh;
  float scale;
  int causal, fp16;
  int* status;
};
cudaError_t launch_attention_packed(const PackedAttnArgs& a, cudaStream_t st);
// sequences of few rows (query tokens x at most 16 heads per key head), 16 at a time, by clusters of `split` CTAs
cudaError_t launch_attention_rows(const PackedAttnArgs& a, int split, cudaStream_t st);

struct RotaryArgs {
  const void *x, *pos;
  void* y;
  long long x_tok, x_head, y_tok, y_head;  // strides in elements
  int tokens, heads, dh;
  int dtype, pos64, interleaved, transpose;
};
cudaError_t launch_rotary(const dit_rotary& r, const RotaryArgs& a, cudaStream_t st);

// Tensor map of a strided view: dims[0] contiguous, strides_bytes[i] from dims[i] to dims[i+1],
// box[0] 128 bytes wide, 128-byte swizzle.  False where TMA cannot read it.
bool make_tmap_view(CUtensorMap* map, int dtype, const void* base, int rank, const uint64_t* dims,
                    const uint64_t* strides_bytes, const uint32_t* box);

}  // namespace dit

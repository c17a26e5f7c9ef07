// C entry points of the packed-layer building blocks: argument checks, then one launch.
#include <math.h>
#include <string.h>

#include "internal.h"
#include "ops.h"

using namespace dit;

namespace {

// SM count of the current device, or 0 when it is no sm_100 device.
int current_sms() {
  static int sms[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return 0;
  if (sms[dev] == 0) {
    int major = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major != 10 ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    sms[dev] = n;
  }
  return sms[dev];
}

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether an outer x inner array of rows of `row` elements, `so` and `si` apart, writes every
// element at one place only.
bool distinct(long long outer, long long so, long long inner, long long si, long long row) {
  if (outer <= 1) return inner <= 1 || si >= row;
  if (inner <= 1) return so >= row;
  return (si >= row && so >= si * (inner - 1) + row) || (so >= row && si >= so * (outer - 1) + row);
}

dit_status launched(cudaError_t e) {
  if (e == cudaSuccess) return DIT_OK;
  cudaGetLastError();  // reported here, not to the caller's next CUDA call
  return DIT_ERR_CUDA;
}

// sizes leave room for a tile beyond them in 32-bit arithmetic
constexpr int kMaxSize = 0x7fffffff - 4096;

}  // namespace

extern "C" {

dit_status dit_op_linear_fused(int dtype, const void* x, long long ldx, const void* w, long long ldw, const float* bias,
                               int act, const void* residual, long long ldr, void* y, long long ldy, int out_dtype,
                               int M, int N, int K, int* status, dit_stream_t stream) {
  if (dtype != DIT_DTYPE_BF16 && dtype != DIT_DTYPE_FP16) return DIT_ERR_UNSUPPORTED;
  if (out_dtype != dtype && out_dtype != DIT_DTYPE_F32) return DIT_ERR_UNSUPPORTED;
  if (M < 0 || N <= 0 || K <= 0 || act < DIT_ACT_NONE || act > DIT_ACT_SILU) return DIT_ERR_INVALID_ARG;
  if (M == 0) return DIT_OK;
  if (M > kMaxSize || N > kMaxSize || K > kMaxSize) return DIT_ERR_UNSUPPORTED;
  const uintptr_t es = out_dtype == DIT_DTYPE_F32 ? 4 : 2;
  if (x == nullptr || w == nullptr || y == nullptr || ldx < 0 || ldw < 0 || ldr < 0 || (M > 1 && ldy < N) ||
      !aligned(x, 2) || !aligned(w, 2) || !aligned(bias, 4) || !aligned(y, es) || !aligned(residual, es) ||
      (y == residual && M > 1 && ldy != ldr))
    return DIT_ERR_INVALID_ARG;
  const int sms = current_sms();
  if (sms == 0) return DIT_ERR_NO_DEVICE;
  LinearArgs a;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldr = ldr;
  a.ldy = ldy;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = act;
  a.fp16 = dtype == DIT_DTYPE_FP16;
  a.out_f32 = out_dtype == DIT_DTYPE_F32;
  a.status = status;
  return launched(launch_linear_fused(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

dit_status dit_op_attention_packed(int dtype, const void* q, const void* k, const void* v, void* o, float* lse,
                                   const int* cu_q, const int* cu_k, int n_seq, int total_q, int total_k, int max_q,
                                   int max_k, int heads, int kv_heads, int dh, const long long* strides, float scale,
                                   int causal, int* status, dit_stream_t stream) {
  if (dtype != DIT_DTYPE_BF16 && dtype != DIT_DTYPE_FP16) return DIT_ERR_UNSUPPORTED;
  if (n_seq < 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0 || heads <= 0 || kv_heads <= 0 || dh <= 0 ||
      heads % kv_heads != 0 || strides == nullptr || !(scale > 0.f) || !isfinite(scale))
    return DIT_ERR_INVALID_ARG;
  if (dh % 8 != 0 || dh > 128 || heads / kv_heads > 128) return DIT_ERR_UNSUPPORTED;
  // work items (a query tile of a key head) are counted in 31 bits
  if (total_k > kMaxSize || max_q > kMaxSize || max_k > kMaxSize ||
      (static_cast<long long>(total_q) + n_seq) * kv_heads > 0x7fff0000ll)
    return DIT_ERR_UNSUPPORTED;
  if (n_seq == 0 || total_q == 0) return DIT_OK;
  if (q == nullptr || o == nullptr || cu_q == nullptr || cu_k == nullptr ||
      (total_k > 0 && (k == nullptr || v == nullptr)))
    return DIT_ERR_INVALID_ARG;
  for (int i = 0; i < 8; ++i)
    if (strides[i] < 0 || strides[i] % 8 != 0 || strides[i] >= (1ll << 38)) return DIT_ERR_INVALID_ARG;
  // the copies into shared memory step through q, k and v by these
  if ((total_q > 1 && strides[0] == 0) || (heads > 1 && strides[1] == 0) ||
      (total_k > 1 && (strides[2] == 0 || strides[4] == 0)) || (kv_heads > 1 && (strides[3] == 0 || strides[5] == 0)))
    return DIT_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4) || !distinct(total_q, strides[6], heads, strides[7], dh))
    return DIT_ERR_INVALID_ARG;
  if (current_sms() == 0) return DIT_ERR_NO_DEVICE;
  PackedAttnArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.q_tok = strides[0];
  a.q_head = strides[1];
  a.k_tok = strides[2];
  a.k_head = strides[3];
  a.v_tok = strides[4];
  a.v_head = strides[5];
  a.o_tok = strides[6];
  a.o_head = strides[7];
  a.n_seq = n_seq;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_q = max_q;
  a.max_k = max_k;
  a.H = heads;
  a.Hk = kv_heads;
  a.dh = dh;
  a.scale = scale;
  a.causal = causal != 0;
  a.fp16 = dtype == DIT_DTYPE_FP16;
  a.status = status;
  return launched(launch_attention_packed(a, reinterpret_cast<cudaStream_t>(stream)));
}

dit_status dit_rotary_frequencies(int scaling, int pairs, double base, double factor, int original_length, double* freq,
                                  float* amplitude) {
  if (pairs <= 0 || freq == nullptr || amplitude == nullptr || !(base > 0.0) || !isfinite(base) || !(factor > 0.0) ||
      !isfinite(factor))
    return DIT_ERR_INVALID_ARG;
  if (scaling < DIT_ROTARY_NONE || scaling > DIT_ROTARY_YARN) return DIT_ERR_INVALID_ARG;
  if (scaling == DIT_ROTARY_YARN && original_length <= 0) return DIT_ERR_INVALID_ARG;
  if (scaling == DIT_ROTARY_NTK && pairs < 2) return DIT_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  if (scaling == DIT_ROTARY_NTK) base *= pow(factor, static_cast<double>(pairs) / (pairs - 1));
  for (int i = 0; i < pairs; ++i) {
    double f = pow(base, -static_cast<double>(i) / pairs);
    if (scaling == DIT_ROTARY_LINEAR) {
      f /= factor;
    } else if (scaling == DIT_ROTARY_YARN) {
      double keep = (original_length * f / two_pi - 1.0) / 31.0;
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = keep * f + (1.0 - keep) * f / factor;
    }
    freq[i] = f;
  }
  *amplitude = scaling == DIT_ROTARY_YARN && factor > 1.0 ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  return DIT_OK;
}

dit_status dit_rotary_init(dit_rotary* r, const double* freq, int pairs_per_axis, int axes, float amplitude) {
  if (r == nullptr || freq == nullptr || pairs_per_axis <= 0 || axes <= 0 || !isfinite(amplitude))
    return DIT_ERR_INVALID_ARG;
  if (axes > DIT_ROTARY_MAX_PAIRS || pairs_per_axis > DIT_ROTARY_MAX_PAIRS / axes) return DIT_ERR_UNSUPPORTED;
  for (int i = 0; i < pairs_per_axis; ++i)
    if (!isfinite(freq[i])) return DIT_ERR_INVALID_ARG;
  memset(r, 0, sizeof(*r));
  r->pairs = pairs_per_axis * axes;
  r->axes = axes;
  r->amplitude = amplitude;
  // fraction of a turn per position, times 2^64
  const long double inv_two_pi = 0.159154943091895335768883763372514362L;
  for (int i = 0; i < pairs_per_axis; ++i) {
    long double t = static_cast<long double>(freq[i]) * inv_two_pi;
    t -= floorl(t);
    // t in [0, 1): the product with 2^64 fits but for a t that rounds up to 1, a whole turn
    r->turns[i] = t >= 1.0L ? 0u : static_cast<uint64_t>(ldexpl(t, 64));
  }
  return DIT_OK;
}

dit_status dit_op_rotary(const dit_rotary* r, int dtype, const void* x, long long x_tok, long long x_head,
                         const void* positions, int positions_64bit, void* y, long long y_tok, long long y_head,
                         int tokens, int heads, int dh, int interleaved, int transpose, dit_stream_t stream) {
  if (r == nullptr || r->pairs <= 0 || r->pairs > DIT_ROTARY_MAX_PAIRS || r->axes <= 0 || r->pairs % r->axes != 0)
    return DIT_ERR_INVALID_ARG;
  if (dtype != DIT_DTYPE_F32 && dtype != DIT_DTYPE_BF16 && dtype != DIT_DTYPE_FP16) return DIT_ERR_UNSUPPORTED;
  if (tokens < 0 || heads <= 0 || dh <= 0 || 2 * r->pairs > dh) return DIT_ERR_INVALID_ARG;
  if (tokens == 0) return DIT_OK;
  const uintptr_t es = dtype == DIT_DTYPE_F32 ? 4 : 2;
  if (x == nullptr || y == nullptr || positions == nullptr || x_tok < 0 || x_head < 0 || y_tok < 0 || y_head < 0 ||
      !aligned(x, es) || !aligned(y, es) || !aligned(positions, positions_64bit ? 8 : 4) ||
      !distinct(tokens, y_tok, heads, y_head, dh) || (x == y && (x_tok != y_tok || x_head != y_head)))
    return DIT_ERR_INVALID_ARG;
  if (static_cast<long long>(heads) * dh > (1 << 24) || tokens > kMaxSize) return DIT_ERR_UNSUPPORTED;
  if (current_sms() == 0) return DIT_ERR_NO_DEVICE;
  RotaryArgs a;
  a.x = x;
  a.pos = positions;
  a.y = y;
  a.x_tok = x_tok;
  a.x_head = x_head;
  a.y_tok = y_tok;
  a.y_head = y_head;
  a.tokens = tokens;
  a.heads = heads;
  a.dh = dh;
  a.dtype = dtype;
  a.pos64 = positions_64bit != 0;
  a.interleaved = interleaved != 0;
  a.transpose = transpose != 0;
  return launched(launch_rotary(*r, a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

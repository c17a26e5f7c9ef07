// Attention over packed sequences for single tokens: o_i = sum_j softmax_j(scale q_i . k_j) v_j where a
// sequence has so few query tokens that all rows of one key head (tokens x heads per key head) are at most
// 16.  Every byte of K and V is used once, so what bounds it is memory.
//
// A cluster of CTAs takes one key head of a sequence, its CTAs consecutive parts of the keys, the four
// warps of a CTA 16 keys of every 64.  A warp keeps its 16 rows' running maximum, sum and output
// (float32) in registers and reads K and V straight into the operands of m16n8k16 products, 16 bytes per
// lane: the order of the features in Q K^T is free, so a lane's eight are two steps' operands as they lie,
// and V's keys are paired by byte permutations.  The loads of the next 16 keys are on their way while
// these are worked on; eight warps per SM (twelve up to 64 features) keep 64 KB in flight.
//
// Products of 16 rows, not of 128 in tensor memory: the tiles of the other kernel (csrc/op_attention.cu) hand
// keys through shared memory, tensor memory and four roles, 7 us for a sequence of 300 keys however few its
// rows.  Here a CTA lasts 3.4 us and 1.1 us per step, beside others on its SM: 200 x 300 keys, 16 heads of 64,
// 160 -> 70 us; 256 x 1024 keys, 8 key heads of 128, 195 -> 185 us (5.8 TB/s).  The step is a chain (loads,
// Q K^T, maximum, exponentials, P V), so few long sequences stay with the other kernel.  Tried: K and V staged
// in shared memory three steps ahead, slower (211 us; 20 x 300 keys 11.8 against 9.0: fewer CTAs per SM).
// P is rounded to the type of V, as the products' operands need it; its sum is not.  That is a rounding per key beside that of
// the output: against 64 bits, 256 x 1024 keys of 128, 2.3e-3 of the norm in bfloat16 for 1.7e-3 with P in float32.
// Partial rows are joined in a fixed order: warps in shared memory, CTAs over distributed shared memory.
#include <math.h>

#include "internal.h"
#include "op_common.cuh"
#include "ops.h"

namespace dit {

namespace {

constexpr int kRowWarps = 4;

template <typename T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes that are read once, or zeros
__device__ __forceinline__ uint4 load_once(const void* p, bool in) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (in)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

struct RowArgs {
  PackedAttnArgs a;
  int G, TQ;    // heads per key head, query tokens per item
  int split;    // CTAs per cluster
  float sc;     // scale * log2(e)
};

// NA 64-feature blocks of a head
template <int NA, typename T>
__global__ void __launch_bounds__(32 * kRowWarps, NA == 1 ? 3 : 2) attention_rows_kernel(const __grid_constant__ RowArgs f) {
  constexpr int W = NA * 64, S = W + 4;  // a partial row, its stride (other banks for other rows)
  __shared__ __align__(16) float part[kRowWarps][16][S];
  __shared__ __align__(16) float joined[16][S];
  __shared__ float2 stat[kRowWarps][16], joined_stat[16];  // (maximum, sum)
  __shared__ __align__(16) int lengths[32];
  __shared__ int4 found;  // q0, lq, k0, lk
  const PackedAttnArgs& a = f.a;
  const int warp = warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  pdl_trigger();
  pdl_wait();
  // This cluster's sequence and key head.  Longest first within 32 sequences: what starts last should end
  // soon.  Offsets beyond the totals are cut: nothing outside the tensors is used.
  const unsigned item = blockIdx.x / f.split;
  const int place = static_cast<int>(item / static_cast<unsigned>(a.Hk)), hk = static_cast<int>(item - static_cast<unsigned>(place) * a.Hk);
  if (warp == 0) {
    const int block = place & ~31, sq = block + lane;
    int4 e = make_int4(0, 0, 0, -1);
    if (sq < a.n_seq) {
      e.x = min(max(a.cu_q[sq], 0), a.total_q);
      e.y = min(max(a.cu_q[sq + 1], e.x), a.total_q) - e.x;
      e.z = min(max(a.cu_k[sq], 0), a.total_k);
      e.w = min(max(a.cu_k[sq + 1], e.z), a.total_k) - e.z;
    }
    lengths[lane] = e.w;
    __syncwarp();
    int before = 0;
#pragma unroll 4
    for (int o = 0; o < 32; o += 4) {
      const int4 l4 = *reinterpret_cast<const int4*>(lengths + o);
      const int l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) before += l[x] > e.w || (l[x] == e.w && o + x < lane);
    }
    if (before == place - block) found = e;
  }
  __syncthreads();
  const int q0 = found.x, lq = found.y, k0 = found.z, lk = found.w;
  const T* kp = static_cast<const T*>(a.k) + k0 * a.k_tok + hk * a.k_head;
  const T* vp = static_cast<const T*>(a.v) + k0 * a.v_tok + hk * a.v_head;

  for (int tok0 = 0; tok0 < lq; tok0 += f.TQ) {
    const int ntok = min(f.TQ, lq - tok0), rows = ntok * f.G, off = tok0 + lk - lq;
    // keys that row r of the item sees
    auto seen = [&](int r) { return r >= rows ? 0 : a.causal ? max(min(lk, off + r / f.G + 1), 0) : lk; };
    const int keys = seen(rows - 1);
    const int steps = (keys + 63) >> 6;
    const int begin = static_cast<int>(static_cast<long long>(steps) * rank / f.split);
    const int end = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / f.split);
    const int lim[2] = {seen(g), seen(g + 8)}, stop = min(keys, end * 64);

    // Q: rows g and g + 8, features 32 i + 8 t ..
    uint4 qf[2 * NA][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h, tok = r / f.G, head = hk * f.G + r - tok * f.G;
      const T* qp = static_cast<const T*>(a.q) + (r < rows ? (q0 + tok0 + tok) * a.q_tok + head * a.q_head : 0);
#pragma unroll
      for (int i = 0; i < 2 * NA; ++i) qf[i][h] = load_once(qp + 32 * i + 8 * t, r < rows && 32 * i + 8 * t < a.dh);
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[NA][8][4];
#pragma unroll
    for (int j = 0; j < NA; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][e][c] = 0.f;

    uint4 kf[2 * NA][2], vf[NA][4];
    auto load_k = [&](int key0) {  // keys g and g + 8, features 32 i + 8 t ..
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = key0 + g + 8 * h;
        const T* p = kp + key * a.k_tok + 8 * t;
#pragma unroll
        for (int i = 0; i < 2 * NA; ++i) kf[i][h] = load_once(p + 32 * i, key < stop && 32 * i + 8 * t < a.dh);
      }
    };
    auto load_v = [&](uint4 (&v)[NA][4], int key0) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, features 64 j + 8 g ..
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = key0 + 2 * t + (c & 1) + 8 * (c >> 1);
        const T* p = vp + key * a.v_tok + 8 * g;
#pragma unroll
        for (int j = 0; j < NA; ++j) v[j][c] = load_once(p + 64 * j, key < stop && 64 * j + 8 * g < a.dh);
      }
    };
    if (begin < end) {
      load_k((begin * kRowWarps + warp) * 16);
      load_v(vf, (begin * kRowWarps + warp) * 16);
    }
#pragma unroll 1
    for (int step = begin; step < end; ++step) {
      const int key0 = (step * kRowWarps + warp) * 16;
      float sc[2][4] = {};  // keys 8 x + 2 t, + 1 of row g, then of row g + 8
#pragma unroll
      for (int i = 0; i < 2 * NA; ++i) {
        const uint32_t q4[2][4] = {{qf[i][0].x, qf[i][1].x, qf[i][0].y, qf[i][1].y}, {qf[i][0].z, qf[i][1].z, qf[i][0].w, qf[i][1].w}};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mma_16x8x16<T>(sc[x], q4[0], kf[i][x].x, kf[i][x].y);
          mma_16x8x16<T>(sc[x], q4[1], kf[i][x].z, kf[i][x].w);
        }
      }
      uint4 vn[NA][4];
      load_k(key0 + 16 * kRowWarps);      // beyond this CTA's keys: zeros, without an access
      load_v(vn, key0 + 16 * kRowWarps);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (key0 + 8 * x + 2 * t + (c & 1) >= lim[c >> 1]) sc[x][c] = -INFINITY;
          mx[c >> 1] = max_nan(mx[c >> 1], sc[x][c]);
        }
      bool grew = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * f.sc;
        grew = grew || !(mx[h] <= m[h] + 8.0f);
      }
      // the reference moves only when a maximum grew by more than 2^8 (or is the first); a NaN maximum stays
      if (__any_sync(0xffffffffu, grew)) {
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = reference_max(m[h], mx[h]);
          alpha[h] = mn == m[h] ? 1.0f : ex2_approx(m[h] - mn);
          m[h] = mn;
          l[h] *= alpha[h];
        }
#pragma unroll
        for (int j = 0; j < NA; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][e][c] *= alpha[c >> 1];
      }
      uint32_t p4[4];  // row g keys 2 t, + 1; row g + 8; the same of keys 8 further
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mu = m[h] == -INFINITY ? 0.f : m[h];
          const float pa = ex2_approx(fmaf(sc[x][2 * h], f.sc, -mu)), pb = ex2_approx(fmaf(sc[x][2 * h + 1], f.sc, -mu));
          l[h] += pa + pb;
          p4[2 * x + h] = pack2<T>(pa, pb);
        }
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        const uint32_t v4[4][4] = {{vf[j][0].x, vf[j][0].y, vf[j][0].z, vf[j][0].w},
                                   {vf[j][1].x, vf[j][1].y, vf[j][1].z, vf[j][1].w},
                                   {vf[j][2].x, vf[j][2].y, vf[j][2].z, vf[j][2].w},
                                   {vf[j][3].x, vf[j][3].y, vf[j][3].z, vf[j][3].w}};
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // feature 64 j + 8 g + e is column g of this product
          const uint32_t pick = e & 1 ? 0x7632u : 0x5410u;
          mma_16x8x16<T>(o[j][e], p4, __byte_perm(v4[0][e >> 1], v4[1][e >> 1], pick), __byte_perm(v4[2][e >> 1], v4[3][e >> 1], pick));
        }
      }
#pragma unroll
      for (int j = 0; j < NA; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) vf[j][c] = vn[j][c];
    }
    // ---------------- this warp's rows: features 64 j + 16 t .. + 15 of rows g and g + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const int r = g + 8 * h;
      if (r < rows) {
#pragma unroll
        for (int j = 0; j < NA; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x)  // columns 2 t and 2 t + 1: two runs of eight features
            *reinterpret_cast<float4*>(&part[warp][r][64 * j + 16 * t + 4 * x]) =
                make_float4(o[j][4 * (x & 1)][2 * h + (x >> 1)], o[j][4 * (x & 1) + 1][2 * h + (x >> 1)],
                            o[j][4 * (x & 1) + 2][2 * h + (x >> 1)], o[j][4 * (x & 1) + 3][2 * h + (x >> 1)]);
        if (t == 0) stat[warp][r] = make_float2(m[h], l[h]);
      }
    }
    __syncthreads();
    // ---------------- the CTA's warps, in their order; four features per thread and turn
    for (int i = threadIdx.x; i < rows * (W / 4); i += 32 * kRowWarps) {
      const int r = i / (W / 4), c = i % (W / 4) * 4;
      float mx = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) mx = max_nan(mx, stat[w][r].x);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float2 st = stat[w][r];
        const float4 v = *reinterpret_cast<const float4*>(&part[w][r][c]);
        if (st.x == -INFINITY) continue;  // saw no key
        const float k = ex2_approx(st.x - mx);
        sum += k * st.y;
        acc.x += k * v.x, acc.y += k * v.y, acc.z += k * v.z, acc.w += k * v.w;
      }
      *reinterpret_cast<float4*>(&joined[r][c]) = acc;
      if (c == 0) joined_stat[r] = make_float2(mx, sum);
    }
    if (f.split > 1) cluster_sync_all();
    else __syncthreads();
    // ---------------- the cluster's CTAs, in their order; eight features per thread, CTA after CTA
    const int units = a.dh / 8;
    for (int i = rank * 32 * kRowWarps + threadIdx.x; i < rows * units; i += f.split * 32 * kRowWarps) {
      const int r = i / units, c = (i - r * units) * 8;
      const uint32_t at = smem_u32(&joined[r][c]), st_at = smem_u32(&joined_stat[r]);
      float mx = -INFINITY, sum = 0.f, acc[8] = {};
      for (int p = 0; p < f.split; ++p) mx = max_nan(mx, ld_cluster_f2(mapa_shared(st_at, p)).x);
#pragma unroll 2
      for (int p = 0; p < f.split; ++p) {
        const float2 st = ld_cluster_f2(mapa_shared(st_at, p));
        const uint32_t peer = mapa_shared(at, p);
        const float4 x = ld_cluster_f4(peer), y = ld_cluster_f4(peer + 16);
        if (st.x == -INFINITY) continue;
        const float k = ex2_approx(st.x - mx);
        sum += k * st.y;
        acc[0] += k * x.x, acc[1] += k * x.y, acc[2] += k * x.z, acc[3] += k * x.w;
        acc[4] += k * y.x, acc[5] += k * y.y, acc[6] += k * y.z, acc[7] += k * y.w;
      }
      const bool any = mx != -INFINITY;
      const float inv = any ? 1.0f / sum : 0.f;
      const int tok = r / f.G, head = hk * f.G + r - tok * f.G, row = q0 + tok0 + tok;
      *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + row * a.o_tok + head * a.o_head + c) =
          make_uint4(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv),
                     pack2<T>(acc[4] * inv, acc[5] * inv), pack2<T>(acc[6] * inv, acc[7] * inv));
      if (c == 0 && a.lse)
        a.lse[static_cast<long long>(head) * a.total_q + row] = any ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    // no CTA leaves, or writes its rows again, while another reads them
    if (f.split > 1) cluster_sync_all();
    else __syncthreads();
  }
}

template <int NA, typename T>
cudaError_t launch_rows_t(const PackedAttnArgs& a, int split, cudaStream_t st) {
  RowArgs f;
  f.a = a;
  f.G = a.H / a.Hk;
  f.TQ = 16 / f.G;
  f.sc = a.scale * 1.4426950408889634f;
  const long long items = static_cast<long long>(a.n_seq) * a.Hk;
  f.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * f.split));
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(f.split), 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = g_pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attention_rows_kernel<NA, T>, f);
}

}  // namespace

cudaError_t launch_attention_rows(const PackedAttnArgs& a, int split, cudaStream_t st) {
  if (a.fp16) return a.dh <= 64 ? launch_rows_t<1, __half>(a, split, st) : launch_rows_t<2, __half>(a, split, st);
  return a.dh <= 64 ? launch_rows_t<1, __nv_bfloat16>(a, split, st) : launch_rows_t<2, __nv_bfloat16>(a, split, st);
}

}  // namespace dit

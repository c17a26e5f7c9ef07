// Attention over packed sequences on the tensor cores: o_i = sum_j softmax_j(scale q_i . k_j) v_j.
//
// A query tile is 128 rows: TQ = 128 / G tokens of one sequence times the G heads that share a
// key head, so K and V are read once per key head and one new token with G heads is one tile.
// Two softmax groups of eight warps each own a query tile:
//   S = Q K^T (128 x 128 keys) into TMEM, half a row in each of two threads' registers, running
//   maximum and sum in base 2 (float32), probabilities as 16-bit back into TMEM, O += P V with P
//   read from there.  Two threads per row: with one, the two warps of a scheduler left it idle half
//   the time (period of a tile pair at dh = 64: 3100 cycles for 1536 of exponentials).
// O is rescaled only when the maximum grew by more than 2^8 (then in place, by its own threads),
// so P <= 2^8 before the final division.  P is rounded to the type of V, since the MMA takes both operands in one
// 16-bit type: one rounding per key, averaged over the keys, beside that of the output (against 64 bits, 8192 tokens bfloat16,
// 2.0e-3 of the norm for 1.5e-3 with P in float32).  Its sum l, by which O is divided, is not rounded.  V is used as it lies (keys x features: the MN-major B
// operand of the MMA).
//
// Pair form: an item is two neighbouring query tiles of one key head; both read the same K / V
//   tiles from one ring.
// Split form (single tokens, or too few tiles to fill the GPU): an item is one query tile; the
//   CTAs of a cluster take consecutive parts of its keys, the two groups of a CTA every other
//   key tile, from a ring each.  Partial (max, sum, O) rows are sent to the CTA that finishes the
//   row over distributed shared memory and joined there in a fixed order.
//
// Roles: warp 0 TMA loads; warp 1 issues the MMAs; warp 3 finds the items
// (sequence, tile, head) from the offsets in device memory, 32 sequences at a time, and hands
// them to the others; warps 4-11, 12-19 softmax.  Rows outside the item's sequence are read by
// TMA as they come: query rows are independent and not stored, scores of such keys are masked,
// and their V rows are set to zero in shared memory, since 0 * NaN is NaN.
// Every wait is bounded; no TMA multicast.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "op_common.cuh"
#include "ops.h"

namespace dit {

// One pair of probabilities in every kPolyEvery is exponentiated by a polynomial on the FMA pipe: the MUFU
// unit gives 16 exponentials a cycle and SM, as long for a 128 x 128 tile as its two products at dh = 128.
constexpr int kPolyEvery = 5;

// 2^x of a pair of numbers (a NaN's row has it in its maximum and sum), 0 below -126 (a masked probability has to be 0 itself: 2^-126 of a bfloat16 value near the
// type's largest is 4): x = n + f with n the nearest integer (adding and subtracting
// 1.5 * 2^23), 2^f by a quartic fitted on [-1/2, 1/2] by reweighted least squares on the relative error (at
// most 2.7e-6 in float32, 4e-8 on average: the sum of the probabilities is returned in float32 as well), and n
// added to the exponent field from the low mantissa bits of x + 1.5 * 2^23.
__device__ __forceinline__ uint64_t ex2_quartic_f2(uint64_t x2) {
  constexpr float c0 = 0.9999992847442627f, c1 = 0.6931217908859253f, c2 = 0.240247443318367f, c3 = 0.05591785907745361f,
                  c4 = 0.009570100344717503f;
  const uint64_t t2 = f2_add(x2, f2_pack(12582912.0f, 12582912.0f));
  const uint64_t n2 = f2_add(t2, f2_pack(-12582912.0f, -12582912.0f));
  const uint64_t fr = f2_fma(n2, f2_pack(-1.0f, -1.0f), x2);
  uint64_t p = f2_fma(f2_pack(c4, c4), fr, f2_pack(c3, c3));
  p = f2_fma(p, fr, f2_pack(c2, c2));
  p = f2_fma(p, fr, f2_pack(c1, c1));
  p = f2_fma(p, fr, f2_pack(c0, c0));
  float a, b, lo, hi, tl, th;
  f2_unpack(x2, a, b);
  f2_unpack(p, lo, hi);
  f2_unpack(t2, tl, th);
  return f2_pack(a >= -126.0f ? __uint_as_float(__float_as_uint(lo) + (__float_as_uint(tl) << 23)) : 0.f,
                 b >= -126.0f ? __uint_as_float(__float_as_uint(hi) + (__float_as_uint(th) << 23)) : 0.f);
}

template <int NA, bool SPLIT>
struct FaCfg {
  static constexpr int ATOM = 128 * 128;             // 128 rows x 64 features
  static constexpr int TILE = NA * ATOM;
  static constexpr int QT = SPLIT ? 1 : 2;           // query tiles per item
  static constexpr int QB = NA == 1 ? 2 : 1;         // Q buffers
  static constexpr int Q_BYTES = QB * QT * TILE;
  static constexpr int SLOTS = (224 * 1024 - Q_BYTES) / TILE;  // K / V tiles in flight, all rings
  static constexpr int RINGS = SPLIT ? 2 : 1;
  static constexpr int RS = SPLIT ? (SLOTS - 2) / 2 : SLOTS;   // slots per ring; the split form keeps two for
  static constexpr int OFF_X = Q_BYTES + RINGS * RS * TILE;    // the exchange of few rows
  static constexpr int OFF_KV = Q_BYTES;
  static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE;
  static constexpr int OFF_SORT = OFF_BAR + 448;     // 32 lane numbers
  static constexpr int OFF_ROW = OFF_SORT + 128;      // one float per query row: the halves' exchange
  static constexpr int SMEM = 1024 + OFF_ROW + 1024;
  static constexpr int THREADS = 640, REG_CTRL = 64, REG_SOFTMAX = 104;
  static constexpr int REG_POOL = 128 * REG_CTRL + 512 * REG_SOFTMAX;
  static_assert(SMEM <= 232448 && RS >= 2, "shared memory");
  // split form with at most this many rows per tile: the partial rows of one item, two groups of up to
  // eight CTAs with the rows rounded up to a multiple of the CTAs, fit one slot
  static constexpr int LIGHT_ROWS = 24;
  static_assert(LIGHT_ROWS % 8 == 0 && 2 * LIGHT_ROWS * (NA * 256 + 8) <= TILE, "exchange slot");
  // with all 128 rows: all slots
  static_assert(2 * 128 * (NA * 256 + 8) <= SLOTS * TILE, "exchange of a full tile");
};

struct FaItem {
  int tok0, ntok;   // first query token, query tokens (<= QT * TQ); ntok < 0: no more items
  int k0, nk;       // first key token, keys of the sequence
  int off;          // query token i of the item sees keys j <= off + i (causal)
  int hk;           // key head
  int t0, t1;       // pair: key tiles of group 0, 1; split: this CTA's key tiles t0 .. t1 - 1
};

template <int NA, bool SPLIT>
struct FaBars {
  using C = FaCfg<NA, SPLIT>;
  enum { IF = 0, IE = 2, QF = 4, QE = 6, SF = 8, PF = 10, OD = 12, OF = 14, XF = 16, KF = 18, KE = KF + C::SLOTS, N = KE + C::SLOTS };
  static_assert(8 * N + 16 + 2 * sizeof(FaItem) <= 448, "barrier area");
};

// V tile in shared memory, rows of keys, 64 features (128 bytes) per atom: MN-major, 128-byte
// swizzle; 8-key groups 1024 bytes apart (stride), the next 64 features one atom on (leading)
// (the low word; the high word is kSdescHiSw128)
__device__ __forceinline__ uint32_t sdesc_mn_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (((128u * 128u) >> 4) << 16);
}

// S = Q K^T over STEPS x 16 features (operands in 64-feature atoms)
template <int STEPS>
__device__ __forceinline__ void mma_qk(uint32_t tS, uint32_t qd, uint32_t kd, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const uint32_t o = ((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4;
    mma_bf16_ss(tS, sdesc_make(qd + o, kSdescHiSw128), sdesc_make(kd + o, kSdescHiSw128), idesc, k > 0 ? 1u : 0u);
  }
}
// O (+)= P V over STEPS x 16 keys; P of keys 64-127 starts 64 columns behind P of keys 0-63, each in
// the place of its own scores
template <int STEPS>
__device__ __forceinline__ void mma_pv(uint32_t tO, uint32_t tP, uint32_t vd, uint32_t idesc, uint32_t more) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    mma_bf16_ts(tO, tP + (k >> 2) * 64 + 8 * (k & 3), sdesc_make(vd + k * (2048 >> 4), kSdescHiSw128), idesc, k > 0 ? 1u : more);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// whether v holds for any thread of the two warps that meet at barrier `id`
__device__ __forceinline__ bool any_of_pair(uint32_t id, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned p, %2, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ float2 ld_shared_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f1(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// wait for arrivals from other CTAs of the cluster and see what they wrote before them
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, int* status) {
  const bool ok = mbar_wait_warp(bar, parity, status);
  fence_cluster();
  return ok;
}

struct FaArgs {
  PackedAttnArgs a;
  int G, TQ;        // heads per key head, query tokens per tile
  int split;        // CTAs per cluster (split form)
  int light;        // split form with few rows per tile
  float sc;         // scale * log2(e)
};

template <int NA, typename T, bool SPLIT>
__global__ void __launch_bounds__(640, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FaArgs f) {
  using C = FaCfg<NA, SPLIT>;
  using B = FaBars<NA, SPLIT>;
  const PackedAttnArgs& a = f.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  volatile FaItem* items = reinterpret_cast<volatile FaItem*>(smem + C::OFF_BAR + 8 * B::N);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * B::N + 2 * sizeof(FaItem));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B::IF + i), 1);
      mbar_init(bar(B::IE + i), 19);              // one arrival per warp that reads items
      mbar_init(bar(B::QF + i), 1);
      mbar_init(bar(B::QE + i), 1);
      mbar_init(bar(B::SF + i), 1);
      mbar_init(bar(B::PF + i), 8);               // the group's warps have written P
      mbar_init(bar(B::OD + i), 1);
      mbar_init(bar(B::OF + i), 8);
      mbar_init(bar(B::XF + i), 4 * f.split);     // the partial rows of four warps of each CTA
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(bar(B::KF + i), 1);
      mbar_init(bar(B::KE + i), 1);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  if constexpr (SPLIT) {  // the barriers are there before another CTA of the cluster arrives on them
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem_base = uniform(*holder);
  pdl_trigger();
  pdl_wait();

  // the item of use n, read by a whole warp, its ring entry released at once
  auto next_item = [&](int n, FaItem& it) -> bool {
    const bool ok = mbar_wait_warp(bar(B::IF + (n & 1)), (n >> 1) & 1, a.status);
    const volatile FaItem& s = items[n & 1];
    it.tok0 = uniform(s.tok0), it.ntok = uniform(s.ntok), it.k0 = uniform(s.k0), it.nk = uniform(s.nk);
    it.off = uniform(s.off), it.hk = uniform(s.hk), it.t0 = uniform(s.t0), it.t1 = uniform(s.t1);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B::IE + (n & 1)));
    return ok && it.ntok >= 0;
  };
  // Split form, many rows: they are exchanged through the K / V slots once every CTA is done with them.  A role
  // whose wait ran out does no more work, but keeps step here.
  auto exchange_others = [&]() {
    if (SPLIT && !f.light) {
      __syncwarp();
      cluster_sync_all();
      cluster_sync_all();
      named_barrier_sync(9, C::THREADS);
    }
  };

  if (warp < 4) {
    regs_dec<C::REG_CTRL>();
    FaItem it;
    if (warp == 0) {  // ---------------- loads
      int slot[C::RINGS] = {};
      uint32_t ph[C::RINGS] = {};
      const uint32_t q_bytes = static_cast<uint32_t>(f.G * f.TQ) * 128;
      bool ok = true;
      for (int n = 0; next_item(n, it); ++n) {
        const int j0 = SPLIT ? it.t0 : 0, j1 = SPLIT ? it.t1 : max(it.t0, it.t1);
        auto load_tile = [&](int r, int j, const CUtensorMap* map) {
          const int at = r * C::RS + slot[r];
          ok = ok && mbar_wait_warp(bar(B::KE + at), ph[r] ^ 1u, a.status);
          if (ok && elect_one()) {
            mbar_arrive_expect_tx(bar(B::KF + at), C::TILE);
#pragma unroll
            for (int c = 0; c < NA; ++c)
              tma_load_3d(sbase + C::OFF_KV + at * C::TILE + c * C::ATOM, map, bar(B::KF + at), c * 64, it.hk, it.k0 + j * 128);
          }
          __syncwarp();
          if (++slot[r] == C::RS) {
            slot[r] = 0;
            ph[r] ^= 1u;
          }
        };
        // K of the first tile before Q: its slot is free earlier than Q's place
        if (j0 < j1) load_tile(0, j0, &tmK);
        const int qb = n % C::QB, ng = !SPLIT && it.ntok > f.TQ ? 2 : 1;
        ok = ok && mbar_wait_warp(bar(B::QE + qb), ((n / C::QB) & 1) ^ 1, a.status);
        if (ok && elect_one()) {
          mbar_arrive_expect_tx(bar(B::QF + qb), ng * NA * q_bytes);
          for (int g = 0; g < ng; ++g)
#pragma unroll
            for (int c = 0; c < NA; ++c)
              tma_load_3d(sbase + (qb * C::QT + g) * C::TILE + c * C::ATOM, &tmQ, bar(B::QF + qb), c * 64, it.hk * f.G,
                          it.tok0 + g * f.TQ);
        }
        __syncwarp();
        if (j0 < j1) load_tile(0, j0, &tmV);
        for (int j = j0 + 1; j < j1; j += C::RINGS) {
#pragma unroll
          for (int r = 0; r < C::RINGS; ++r) {  // split form: the second ring is due first
            const int at = C::RINGS == 2 ? 1 - r : 0;
            if (j + r < j1) {
              load_tile(at, j + r, &tmK);
              load_tile(at, j + r, &tmV);
            }
          }
        }
        exchange_others();
      }
      if (!ok) after_timeout();
    } else if (warp == 3) {  // ---------------- items
      const int per = C::QT * f.TQ;                       // query tokens per item
      // Items are dealt out in rounds, every other one in reverse, so that who got a long one gets a short
      // one next (sequences are taken longest first).
      const unsigned step = SPLIT ? gridDim.x / f.split : gridDim.x, place = SPLIT ? blockIdx.x / f.split : blockIdx.x;
      int sb = -32;                                        // sequences sb + lane are in registers
      unsigned cum = 0;                                    // items (per head) before them
      int q0 = 0, lq = 0, k0 = 0, lk = 0, tiles = 0, incl = 0;
      unsigned total = 0;
      for (int n = 0;; ++n) {
        const unsigned id = n & 1 ? (n + 1) * step - 1 - place : n * step + place, t = id / static_cast<unsigned>(a.Hk);
        while (sb < a.n_seq && t >= cum + total) {
          cum += total;
          sb += 32;
          if (sb >= a.n_seq) break;
          const int s = sb + lane;
          q0 = lq = k0 = lk = tiles = 0;
          if (s < a.n_seq) {  // offsets beyond the totals are cut: nothing outside the tensors is used
            q0 = min(max(a.cu_q[s], 0), a.total_q);
            lq = min(max(a.cu_q[s + 1], q0), a.total_q) - q0;
            k0 = min(max(a.cu_k[s], 0), a.total_k);
            lk = min(max(a.cu_k[s + 1], k0), a.total_k) - k0;
            tiles = (lq + per - 1) / per;
          }
          // longest first within the 32: lane i takes the sequence of rank i
          if (a.n_seq > 1) {
            // (lengths read from shared memory, four at once: by 31 shuffles the first item came 1.5 us later)
            volatile int* sorted = reinterpret_cast<volatile int*>(smem + C::OFF_SORT);
            sorted[lane] = lk;
            __syncwarp();
            int rank_of = 0;
#pragma unroll 4
            for (int o = 0; o < 32; o += 4) {
              const uint4 v = ld_shared_v4(sbase + C::OFF_SORT + 4 * o);
              const int l4[4] = {static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w)};
#pragma unroll
              for (int e = 0; e < 4; ++e) rank_of += l4[e] > lk || (l4[e] == lk && o + e < lane);
            }
            __syncwarp();
            sorted[rank_of] = lane;
            __syncwarp();
            const int from = sorted[lane];
            __syncwarp();
            q0 = __shfl_sync(0xffffffffu, q0, from), lq = __shfl_sync(0xffffffffu, lq, from);
            k0 = __shfl_sync(0xffffffffu, k0, from), lk = __shfl_sync(0xffffffffu, lk, from);
            tiles = __shfl_sync(0xffffffffu, tiles, from);
          }
          incl = tiles;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
          }
          total = __shfl_sync(0xffffffffu, incl, 31);
        }
        FaItem e{};
        e.ntok = -1;
        if (sb < a.n_seq) {
          const int left = static_cast<int>(t - cum);
          const int src = __ffs(__ballot_sync(0xffffffffu, incl > left)) - 1;
          int tile = left - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, tiles, src));
          if (a.causal) tile = __shfl_sync(0xffffffffu, tiles, src) - 1 - tile;  // the longest first
          const int Lq = __shfl_sync(0xffffffffu, lq, src), Lk = __shfl_sync(0xffffffffu, lk, src);
          e.tok0 = __shfl_sync(0xffffffffu, q0, src) + tile * per;
          e.ntok = min(per, Lq - tile * per);
          e.k0 = __shfl_sync(0xffffffffu, k0, src);
          e.nk = Lk;
          e.off = tile * per + Lk - Lq;
          e.hk = static_cast<int>(id - t * static_cast<unsigned>(a.Hk));
          // key tiles that query tokens up to the item's last-th see
          auto seen = [&](int last) {
            const int keys = a.causal ? min(Lk, e.off + last + 1) : Lk;
            return keys > 0 ? (keys + 127) / 128 : 0;
          };
          if constexpr (SPLIT) {
            const int nt = seen(e.ntok - 1);  // at most 2^24
            e.t0 = nt * rank / f.split;
            e.t1 = nt * (rank + 1) / f.split;
          } else {
            e.t0 = seen(min(e.ntok, f.TQ) - 1);
            e.t1 = e.ntok > f.TQ ? seen(e.ntok - 1) : 0;
          }
        }
        const bool room = mbar_wait_warp(bar(B::IE + (n & 1)), ((n >> 1) & 1) ^ 1, a.status);
        if (room && elect_one()) {
          volatile FaItem& s = items[n & 1];
          s.tok0 = e.tok0, s.ntok = e.ntok, s.k0 = e.k0, s.nk = e.nk, s.off = e.off, s.hk = e.hk, s.t0 = e.t0, s.t1 = e.t1;
          mbar_arrive(bar(B::IF + (n & 1)));
        }
        __syncwarp();
        if (n > 0) exchange_others();  // of the item before: this one was looked up meanwhile
        if (!room || e.ntok < 0) break;
      }
    } else if (warp == 1) {  // ---------------- MMA issue
      // One warp issues for both groups in turn, O_g += P_g V_j and S_g = Q_g K_j+1 of one before those of
      // the other, so that the groups work half a period apart: one's exponentials run beside the other's
      // products.  (Issued by a warp per group, both groups' products finished together and the two took
      // turns with the tensor cores as one: period 5000 cycles at dh = 128 for 2048 of products.)
      constexpr uint32_t idesc_s = idesc_16<T>(128, 128);
      const int n16 = (a.dh + 15) / 16;
      const uint32_t idesc_o = idesc_16<T>(128, 16 * n16) | (1u << 16);  // B (V) is MN-major
      int np[2] = {}, ni[2] = {};  // per group: PV issued; items with tiles
      bool ok = true;
      // K and V alternate in a ring: K of tile j + 1 lies two slots behind K of tile j, V of tile j between
      int kslot[C::RINGS] = {}, vslot[C::RINGS];
      uint32_t kph[C::RINGS] = {}, vph[C::RINGS] = {};
#pragma unroll
      for (int i = 0; i < C::RINGS; ++i) vslot[i] = 1;
      auto step2 = [&](int& s, uint32_t& p) {
        s += 2;
        if (s >= C::RS) {
          s -= C::RS;
          p ^= 1u;
        }
      };
      auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && mbar_wait_warp(b, parity, a.status); };
      bool more = next_item(0, it);
      for (int n = 0; more; ++n) {
        const int qb = n % C::QB;
        int mine[2];  // key tiles of each group
        if constexpr (SPLIT) {
          mine[0] = (it.t1 - it.t0 + 1) >> 1;
          mine[1] = (it.t1 - it.t0) >> 1;
        } else {
          mine[0] = it.t0;
          mine[1] = it.t1;
        }
        const int all = max(mine[0], mine[1]);
        wait(bar(B::QF + qb), (n / C::QB) & 1);
        // S_g = Q_g K_j from the slot `at`
        auto issue_qk = [&](int g, int at) {
          // S is free: the product that reads P in its place was issued before this one
          tc_fence_after();
          const uint32_t qd = sdesc_lo(sbase + (qb * C::QT + (SPLIT ? 0 : g)) * C::TILE);
          const uint32_t kd = sdesc_lo(sbase + C::OFF_KV + at * C::TILE), tS = tmem_base + g * 128;
          // 16 features a step; features past dh are zeros in shared memory, so the step count is one of few
          // and the products are issued without a branch between them (about 40 cycles each; with a
          // condition at each, 85, more than most of them run)
          if (ok && elect_one()) {
            if (NA == 1) mma_qk<4>(tS, qd, kd, idesc_s);
            else if (n16 == 5) mma_qk<5>(tS, qd, kd, idesc_s);
            else if (n16 == 6) mma_qk<6>(tS, qd, kd, idesc_s);
            else mma_qk<8>(tS, qd, kd, idesc_s);
            mma_commit(bar(B::SF + g));
          }
          __syncwarp();
        };
        // O_g (+)= P_g V_j from the slot `at`, whose keys start at key0
        auto issue_pv = [&](int g, int at, int j, int key0) {
          // O of the previous item has been read
          if (j == 0 && ni[g] > 0) wait(bar(B::OF + g), (ni[g] - 1) & 1);
          const int steps = min(8, (it.nk - key0 + 15) >> 4);
          const uint32_t vd = sdesc_mn_lo(sbase + C::OFF_KV + at * C::TILE);
          const uint32_t tO = tmem_base + 256 + g * (NA == 1 ? 64 : 128);
          const uint32_t tP = tmem_base + g * 128;
          wait(bar(B::PF + g), np[g] & 1);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t more = j > 0 ? 1u : 0u;
            if (steps == 8) {
              mma_pv<8>(tO, tP, vd, idesc_o, more);
            } else {
              mma_pv<1>(tO, tP, vd, idesc_o, more);
              for (int k = 1; k < steps; ++k)
                mma_pv<1>(tO, tP + (k >> 2) * 64 + 8 * (k & 3), vd + k * (2048 >> 4), idesc_o, 1u);
            }
            mma_commit(bar(B::OD + g));
          }
          __syncwarp();
          ++np[g];
        };
        // keys behind the sequence inside the last 16 of a V tile: their rows become zero
        auto clear_tail = [&](int at, int key0) {
          const int valid = it.nk - key0;
          if (valid >= 128 || (valid & 15) == 0) return;
          const int rows = 16 - (valid & 15);
          for (int i = lane; i < rows * 8 * NA; i += 32) {
            const int c = i / (rows * 8), r = valid + (i >> 3) % rows;
            *reinterpret_cast<uint4*>(smem + C::OFF_KV + at * C::TILE + c * C::ATOM + r * 128 + (i & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        };
        auto release = [&](uint32_t b) {  // once the products issued so far are complete
          if (elect_one()) mma_commit(b);
          __syncwarp();
        };
        if constexpr (SPLIT) {
          auto k_of = [&](int g) {
            const int at = g * C::RS + kslot[g % C::RINGS];
            wait(bar(B::KF + at), kph[g % C::RINGS]);
            issue_qk(g, at);
            release(bar(B::KE + at));
            step2(kslot[g % C::RINGS], kph[g % C::RINGS]);
          };
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (mine[g] > 0) k_of(g);
          for (int j = 0; j < all; ++j) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (j >= mine[g]) continue;
              const int at = g * C::RS + vslot[g % C::RINGS], key0 = (it.t0 + 2 * j + g) * 128;
              wait(bar(B::KF + at), vph[g % C::RINGS]);
              clear_tail(at, key0);
              issue_pv(g, at, j, key0);
              release(bar(B::KE + at));
              step2(vslot[g % C::RINGS], vph[g % C::RINGS]);
              if (j + 1 < mine[g]) k_of(g);
            }
            if (j + 2 == all) release(bar(B::QE + qb));  // that was Q's last product
          }
        } else {
          if (all > 0) {
            wait(bar(B::KF + kslot[0]), kph[0]);
#pragma unroll
            for (int g = 0; g < 2; ++g)
              if (mine[g] > 0) issue_qk(g, kslot[0]);
            release(bar(B::KE + kslot[0]));
            step2(kslot[0], kph[0]);
          }
          for (int j = 0; j < all; ++j) {
            const int kat = kslot[0], vat = vslot[0];
            if (j + 1 < all) wait(bar(B::KF + kat), kph[0]);
            wait(bar(B::KF + vat), vph[0]);
            clear_tail(vat, j * 128);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (j < mine[g]) issue_pv(g, vat, j, j * 128);
              if (j + 1 < mine[g]) issue_qk(g, kat);
            }
            release(bar(B::KE + vat));
            step2(vslot[0], vph[0]);
            if (j + 1 < all) {
              release(bar(B::KE + kat));
              step2(kslot[0], kph[0]);
            }
            if (j + 2 == all) release(bar(B::QE + qb));  // that was Q's last product
          }
        }
        if (all <= 1) release(bar(B::QE + qb));
#pragma unroll
        for (int g = 0; g < 2; ++g) ni[g] += mine[g] > 0;
        more = next_item(n + 1, it);
        exchange_others();
      }
      if (!ok) after_timeout();
    } else {  // ---------------- warp 2 only keeps step
      for (int n = 0; next_item(n, it); ++n) exchange_others();
    }
  } else {  // ---------------- softmax: group g, two threads per query row, 64 keys of a tile each
    regs_inc<C::REG_SOFTMAX>();
    const int g = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, q = warp & 3, r = q * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + g * 128 + hf * 64, tO = tmem_base + lane_off + 256 + g * (NA == 1 ? 64 : 128);
    const int rt = r / f.G, rh = r - rt * f.G;  // token and head of this row within the tile
    const uint32_t pair = 1 + g * 4 + q;        // named barrier of the two warps that share 32 rows
    volatile float* row = reinterpret_cast<volatile float*>(smem + C::OFF_ROW) + g * 128 + r;
    // f(half 0's value, half 1's value) to both halves of a row
    auto join = [&](float v, auto&& fn) {
      if (hf == 1) *row = v;
      named_barrier_sync(pair, 64);
      if (hf == 0) *row = v = fn(v, *row);
      named_barrier_sync(pair, 64);
      return hf == 1 ? static_cast<float>(*row) : v;
    };
    int cnt = 0;  // key tiles of this group so far
    bool ok = true;
    FaItem it;
    for (int n = 0; next_item(n, it); ++n) {
      const int tok = (SPLIT ? 0 : g * f.TQ) + rt;          // of the item
      const bool row_ok = r < f.TQ * f.G && tok < it.ntok;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok); // else this warp only keeps step
      const int lim = !row_ok ? 0 : a.causal ? min(it.nk, it.off + tok + 1) : it.nk;  // keys this row sees
      const int mine = SPLIT ? (it.t1 - it.t0 + 1 - g) >> 1 : g == 0 ? it.t0 : it.t1;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < mine && ok; ++j, ++cnt) {
        const int key0 = (SPLIT ? it.t0 + 2 * j + g : j) * 128 + hf * 64;
        if (!mbar_wait_warp(bar(B::SF + g), cnt & 1, a.status)) ok = false;
        if (!warp_ok) {
          __syncwarp();
          if (elect_one()) mbar_arrive(bar(B::PF + g));
          __syncwarp();
          continue;
        }
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32(tS, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld_wait<64>(s);
        const int nvalid = lim - key0;
        if (__any_sync(0xffffffffu, nvalid < 64)) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= nvalid) s[i] = __float_as_uint(-INFINITY);
        }
        float mp[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mp[e] = max_nan(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
        for (int i = 8; i < 64; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mp[e] = max_nan(mp[e], __uint_as_float(s[i + 2 * e]), __uint_as_float(s[i + 2 * e + 1]));
        const float mx = max_nan(max_nan(mp[0], mp[1], mp[2]), mp[3]) * f.sc;
        // The reference moves only when a row's maximum grew by more than 2^8 (or is the first): the two
        // warps of the row agree on that by a barrier that also ors, and only then exchange their maxima.  A NaN
        // maximum stays, and makes every later sum of its row NaN.
        if (any_of_pair(pair, !(mx <= m_ref + 8.0f))) {
          const float m_new = reference_max(m_ref, join(mx, [](float x, float y) { return max_nan(x, y); }));
          const float alpha = m_ref == m_new ? 1.0f : ex2_approx(m_ref - m_new);
          m_ref = m_new;
          l *= alpha;
          if (j > 0) {
            // O moves to the new maximum, each half every other 16 columns.  Its last product is complete: it
            // came before this S in the same pipe.
#pragma unroll 1
            for (int c = 16 * hf; c < a.dh; c += 32) {
              uint32_t o[16];
              tmem_ld16(tO + c, o);
              tmem_ld_wait<16>(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + c, o);
            }
            tmem_st_wait();
            tc_fence_before();
            named_barrier_sync(pair, 64);  // all of O before either half's P lets the next product start
          }
        }
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;  // a row that has seen no key yet
        const uint64_t sc2 = f2_pack(f.sc, f.sc), nm2 = f2_pack(-mu, -mu);
        uint64_t rs2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 16 * h; i < 16 * h + 16; ++i) {
            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, nm2);
            uint64_t p2;
            if (i % kPolyEvery == kPolyEvery - 1) {
              p2 = ex2_quartic_f2(x2);
            } else {
              float x0, x1;
              f2_unpack(x2, x0, x1);
              p2 = f2_pack(ex2_approx(x0), ex2_approx(x1));
            }
            rs2[i & 1] = f2_add(rs2[i & 1], p2);
            float p0, p1;
            f2_unpack(p2, p0, p1);
            pk[i - 16 * h] = pack2<T>(p0, p1);
          }
          tmem_st16(tS + 16 * h, pk);  // P, in the place of S
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(bar(B::PF + g));
        __syncwarp();
        float r0, r1, r2, r3;
        f2_unpack(rs2[0], r0, r1);
        f2_unpack(rs2[1], r2, r3);
        l += (r0 + r1) + (r2 + r3);
      }
      ok = ok && (mine == 0 || mbar_wait_warp(bar(B::OD + g), (cnt - 1) & 1, a.status));
      if (!SPLIT && !ok) break;
      tc_fence_after();
      if (warp_ok) l = join(l, [](float x, float y) { return x + y; });
      const int head = it.hk * f.G + rh;
      if constexpr (!SPLIT) {
        if (warp_ok) {
          const bool any = !(l == 0.f);  // some key has a weight (or NaN)
          const float inv = any ? 1.0f / l : 0.f;
          // 32 columns at a time (each half every other 32): a lane's row is four 16-byte units; four lanes
          // exchange them so that lane i of the four holds unit i of their four rows, and a store covers
          // 64 bytes of each of eight rows instead of 16 of 32
          const long long row_at = row_ok ? (it.tok0 + tok) * a.o_tok + head * a.o_head : -1;
          const int sub = lane & 3;
#pragma unroll 1
          for (int c = 32 * hf; c < a.dh; c += 64) {
            uint32_t u[4][4];
            if (mine > 0) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_ld_wait<32>(o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                u[i >> 2][i & 3] = any ? pack2<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) u[i >> 2][i & 3] = 0u;
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1)  // swap unit i ^ x of this lane with unit i of lane ^ x
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!(i & x))
#pragma unroll
                  for (int w = 0; w < 4; ++w) {
                    const bool up = sub & x;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? u[i][w] : u[i ^ x][w], x);
                    if (up) u[i][w] = got;
                    else u[i ^ x][w] = got;
                  }
            // u[i] is now unit `sub` of the row of lane (lane & ~3) + i
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const long long at = __shfl_sync(0xffffffffu, row_at, (lane & ~3) + i);
              if (at >= 0 && c + 8 * sub < a.dh)
                *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + at + c + 8 * sub) = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
            }
          }
          if (row_ok && hf == 0 && a.lse)
            a.lse[static_cast<long long>(head) * a.total_q + it.tok0 + tok] =
                any ? (m_ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        tc_fence_before();
        __syncwarp();
        if (mine > 0 && elect_one()) mbar_arrive(bar(B::OF + g));
        __syncwarp();
      } else {
        // Rows go to the CTA that finishes them: CTA r / share keeps rows share * CTA ..; the partial
        // of CTA c, group g is slot 2 c + g: O rows [slot][row][16 n16] float32, then (max, sum) [slot][row].
        // Few rows: a place of their own that alternates by item, and a barrier that the warps with rows
        // arrive at; those of group 1, which end last, wait there and finish the rows, while group 0 and
        // the loads go on with the next item.  A place is written again two items later: before that its
        // writer has passed the barrier of the item between, where the finishing warps arrived after they
        // were done with this item's rows.
        // Many rows: the K / V slots, between two barriers of the whole cluster.
        const int rows = min(f.TQ, it.ntok) * f.G, share = (rows + f.split - 1) / f.split;
        const uint32_t wide = (a.dh + 15) / 16 * 64;  // bytes of a row
        const uint32_t part = sbase + (f.light ? C::OFF_X + (n & 1) * C::TILE : C::OFF_KV), stats = part + 2 * f.split * share * wide;
        if (!f.light) cluster_sync_all();
        else if (g == 0 && q == 0 && n > 0)
          ok = mbar_wait_cluster(bar(B::XF + ((n - 1) & 1)), ((n - 1) >> 1) & 1, a.status) && ok;
        if (q * 32 < rows) {
          const int owner = min(r / share, f.split - 1), pr = (2 * rank + g) * share + r - owner * share;
          // a row's 16-byte units are rotated by its number: neighbouring rows meet other banks
          const uint32_t peer = mapa_shared(part, owner) + pr * wide, turn = (pr * 16) % wide;
#pragma unroll 1
          for (int c = 16 * hf; c < a.dh && mine > 0; c += 32) {
            uint32_t o[16];
            tmem_ld16(tO + c, o);
            tmem_ld_wait<16>(o);
            if (r < rows)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t at = c * 4 + i * 16 + turn;
                if (at >= wide) at -= wide;
                st_cluster_v4(peer + at, o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              }
          }
          if (r < rows && hf == 0) st_cluster_v2(mapa_shared(stats, owner) + pr * 8, m_ref, l);
        }
        tc_fence_before();
        __syncwarp();
        if (mine > 0 && elect_one()) mbar_arrive(bar(B::OF + g));
        __syncwarp();
        if (f.light) {
          if (q == 0) {
            fence_cluster();
            __syncwarp();
            if (lane < f.split) mbar_arrive_cluster(mapa_shared(bar(B::XF + (n & 1)), lane));
            __syncwarp();
            if (g == 1) ok = mbar_wait_cluster(bar(B::XF + (n & 1)), (n >> 1) & 1, a.status) && ok;
            __syncwarp();
          }
        } else {
          cluster_sync_all();
        }
        const int mrows = min(share, rows - rank * share);
        const uint32_t slots = 2 * f.split, skip = (share * 16) % wide;
        if (!f.light) {
          // Many rows: a thread per row and slot turns (max, sum) into a weight in its place (-1: nothing seen,
          // its O row was not written), slot 0's sum into the factor; then eight columns per thread.
          // (With both done by a half-warp per row, four rows deep, they took 6600 cycles for a tile on
          // one CTA; with a thread per row, 4200 for the 16 slots of eight.)
          const int i = threadIdx.x - 128, lr0 = i / static_cast<int>(slots);
          if (i - lane < mrows * static_cast<int>(slots)) {
            const uint32_t at = stats + ((i & (slots - 1)) * share + min(lr0, mrows - 1)) * 8;
            const float2 st = ld_shared_f2(at);
            float mx = st.x;
            for (uint32_t x = 1; x < slots; x <<= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float w = st.x == -INFINITY ? -1.f : ex2_approx(st.x - mx);
            float sum = w < 0.f ? 0.f : w * st.y;
            for (uint32_t x = 1; x < slots; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            if (lr0 < mrows) {
              st_shared_f1(at, w);
              if ((i & (slots - 1)) == 0) {
                const bool any = mx != -INFINITY;
                st_shared_f1(at + 4, any ? 1.0f / sum : 0.f);
                if (a.lse) {
                  const int row = rank * share + lr0, t = row / f.G, hd = it.hk * f.G + row - t * f.G;
                  a.lse[static_cast<long long>(hd) * a.total_q + it.tok0 + t] = any ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                }
              }
            }
          }
          named_barrier_sync(10, 512);
          constexpr int LPR = NA == 1 ? 8 : 16;  // threads per row
          const int u = i % LPR;
          if (8 * u < a.dh) {
#pragma unroll 1
            for (int lr = i / LPR; lr < mrows; lr += 512 / LPR) {
              float o[8] = {};
              uint32_t pr = lr, turn = (lr * 16) % wide;
#pragma unroll 4
              for (uint32_t p = 0; p < slots; ++p, pr += share) {
                const float w = ld_shared_f2(stats + pr * 8).x;
                uint32_t a0 = u * 32 + turn, a1 = a0 + 16;
                if (a0 >= wide) a0 -= wide;
                if (a1 >= wide) a1 -= wide;
                turn += skip;
                if (turn >= wide) turn -= wide;
                const uint4 x = ld_shared_v4(part + pr * wide + a0), y = ld_shared_v4(part + pr * wide + a1);
                const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += w < 0.f ? 0.f : w * __uint_as_float(v[e]);
              }
              const float inv = ld_shared_f2(stats + lr * 8).y;
              const int row = rank * share + lr, t = row / f.G, hd = it.hk * f.G + row - t * f.G;
              T* out = static_cast<T*>(a.o) + (it.tok0 + t) * a.o_tok + hd * a.o_head + 8 * u;
              *reinterpret_cast<uint4*>(out) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                          pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
            }
          }
        }
        // few rows: a half-warp per row, eight columns per lane
        const int u = lane & 15, top = lane & 16;
#pragma unroll 1
        for (int l0 = 2 * hf; f.light && q == 0 && g == 1 && l0 < mrows; l0 += 4) {
          const int lr = l0 + (lane >> 4);
          // lane p holds (max, sum) of slot p
          float2 st = make_float2(-INFINITY, 0.f);
          if (u < slots && lr < mrows) st = ld_shared_f2(stats + (u * share + lr) * 8);
          float mx = st.x;
#pragma unroll
          for (int x = 8; x > 0; x >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          const float w = st.x == -INFINITY ? 0.f : ex2_approx(st.x - mx);
          float sum = w * st.y;
#pragma unroll
          for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          float o[8] = {};
          uint32_t pr = lr, turn = (lr * 16) % wide;
#pragma unroll 2
          for (uint32_t p = 0; p < slots; ++p) {
            const float wp = __shfl_sync(0xffffffffu, w, top + p), mp = __shfl_sync(0xffffffffu, st.x, top + p);
            if (mp != -INFINITY && lr < mrows && 8 * u < a.dh) {  // else nothing seen: its O row was not written
              uint32_t a0 = u * 32 + turn, a1 = a0 + 16;
              if (a0 >= wide) a0 -= wide;
              if (a1 >= wide) a1 -= wide;
              const uint4 x = ld_shared_v4(part + pr * wide + a0), y = ld_shared_v4(part + pr * wide + a1);
              o[0] += wp * __uint_as_float(x.x), o[1] += wp * __uint_as_float(x.y);
              o[2] += wp * __uint_as_float(x.z), o[3] += wp * __uint_as_float(x.w);
              o[4] += wp * __uint_as_float(y.x), o[5] += wp * __uint_as_float(y.y);
              o[6] += wp * __uint_as_float(y.z), o[7] += wp * __uint_as_float(y.w);
            }
            pr += share;
            turn += skip;
            if (turn >= wide) turn -= wide;
          }
          if (lr < mrows) {
            const bool any = mx != -INFINITY;
            const float inv = any ? 1.0f / sum : 0.f;
            const int row = rank * share + lr, t = row / f.G, hd = it.hk * f.G + row - t * f.G;
            if (8 * u < a.dh) {
              T* out = static_cast<T*>(a.o) + (it.tok0 + t) * a.o_tok + hd * a.o_head + 8 * u;
              *reinterpret_cast<uint4*>(out) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                          pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
            }
            if (u == 0 && a.lse)
              a.lse[static_cast<long long>(hd) * a.total_q + it.tok0 + t] = any ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
          }
        }
        if (!f.light) {
          fence_proxy_async_smem();  // the slots are TMA's again
          __syncwarp();
          named_barrier_sync(9, C::THREADS);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (SPLIT) cluster_sync_all();  // no CTA leaves while another may write to it
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// One-time set-up on the current device, and how many clusters of 1, 2, 4 and 8 CTAs run at one time (those
// of 4 and 8 do not reach every SM; a persistent cluster that has to wait for another would double the time).
template <int NA, typename T, bool SPLIT>
static cudaError_t set_up_fa(int (&places)[4]) {
  using C = FaCfg<NA, SPLIT>;
  auto kernel = attention_tc_kernel<NA, T, SPLIT>;
  static std::atomic<int> of[kMaxDevices][4];  // published together, the first last: threads may come at once
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (of[dev][0].load(std::memory_order_acquire) == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    // the register split (setmaxnreg) must fit in the launch allocation, or it would wait forever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * C::THREADS < C::REG_POOL) return cudaErrorInvalidConfiguration;
    for (int i = 3; i >= 0; --i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1184);
      cfg.blockDim = dim3(C::THREADS);
      cfg.dynamicSmemBytes = C::SMEM;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim = {1u << i, 1, 1};
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n <= 0) return cudaErrorInvalidConfiguration;
      places[i] = n;
    }
    for (int i = 3; i >= 0; --i) of[dev][i].store(places[i], std::memory_order_release);
    return cudaSuccess;
  }
  for (int i = 0; i < 4; ++i) places[i] = of[dev][i].load(std::memory_order_relaxed);
  return cudaSuccess;
}

template <int NA, typename T, bool SPLIT>
static cudaError_t launch_fa(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FaArgs& f, int ctas,
                             cudaStream_t st) {
  using C = FaCfg<NA, SPLIT>;
  auto kernel = attention_tc_kernel<NA, T, SPLIT>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (SPLIT) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n++].val.clusterDim = {static_cast<unsigned>(f.split), 1, 1};
  }
  if (g_pdl) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, f);
}

template <int NA, typename T>
static cudaError_t launch_form(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, FaArgs& f,
                               cudaStream_t st) {
  const PackedAttnArgs& a = f.a;
  // Form and slices, by what was measured in cycles: a key tile step 2600 (either form: two query tiles, or
  // two key tiles of one), a pair item 5000 besides, a split item 8000 or, with many rows, 13000; the longest item, or all items over
  // the places where they run, whichever lasts longer.  Lengths beyond the longest are averages:
  // the totals are known here, the offsets are not.
  auto tiles = [](long long n, long long per) { return (n + per - 1) / per; };
  const long long avg_q = a.total_q / a.n_seq, avg_k = a.total_k / a.n_seq;
  auto items = [&](long long per) { return a.n_seq * tiles(avg_q > 0 ? avg_q : 1, per) * a.Hk; };
  // Up to two rounds are whole ones (52 x 3 items on 148 CTAs: 37.6 us, as pairs in one round 33.3); of more, the
  // long items of one run beside short ones of the next (8192 tokens causal, 3.5 rounds of pairs: 216 us, in the
  // form that whole rounds would choose 274).  Single tokens wait for memory, which fewer share in the last round.
  auto rounds = [&](long long n, long long cost, long long at) { return !f.light && n <= 2 * at ? tiles(n, at) * cost : n * cost / at; };
  const long long nt_max = tiles(a.max_k, 128), nt_avg = tiles(avg_k, 128);
  int places[4];
  cudaError_t e = set_up_fa<NA, T, true>(places);
  if (e != cudaSuccess) return e;
  const long long pair_all = rounds(items(2 * f.TQ), nt_avg * 2600 + 5000, places[0]);
  long long best = f.light ? -1 : nt_max * 2600 + 5000 > pair_all ? nt_max * 2600 + 5000 : pair_all;
  int split = 0;  // the pair form
  const long long extra = f.light ? 8000 : 13000;
  for (int i = 0, c = 1; i < 4; ++i, c *= 2) {
    long long cost = tiles(nt_max, 2 * c) * 2600 + extra;
    const long long all = rounds(items(f.TQ), tiles(nt_avg, 2 * c) * 2600 + extra, places[i]);
    if (all > cost) cost = all;
    if (best < 0 || cost < best) {
      best = cost;
      split = c;
    }
  }
  if (f.G <= 16 && a.max_q <= 16 / f.G) {
    // Few enough rows for the kernel without tiles (csrc/op_attention_rows.cu): a CTA takes 5200 and a step of
    // 64 keys 1300 (dh to 64) or 1850, three or two CTAs per SM.  It wins where sequences are short (200 x
    // 300 keys, 16 heads of 64: 160 -> 70 us; 512 keys, 8 of 128: 9.4 -> 7.2) or memory limits both (256 x 1024
    // keys, 8 of 128: 195 -> 185), the tiles where few sequences are long (60000 keys: 134 against 72).
    const long long per_step = NA == 1 ? 1300 : 1850, at = (NA == 1 ? 3 : 2) * places[0], n = static_cast<long long>(a.n_seq) * a.Hk;
    const long long memory = 4ll * a.total_k * a.Hk * a.dh / 3800;
    long long least = best > memory ? best : memory;
    int rows_split = 0;
    for (int c = 1; c <= 8; c *= 2) {
      long long cost = tiles(a.max_k, 64 * c) * per_step + 5200;
      const long long one = tiles(avg_k, 64 * c) * per_step + 5200;
      const long long all = n * c <= 2 * at ? tiles(n * c, at) * one : n * c * one / at;
      if (all > cost) cost = all;
      if (memory > cost) cost = memory;
      if (cost < least || (rows_split == 0 && cost == least)) {
        least = cost;
        rows_split = c;
      }
    }
    if (rows_split > 0) return launch_attention_rows(a, rows_split, st);
  }
  // items there can be at most: every sequence ends inside a tile
  auto most = [&](long long per) { return (a.total_q / per + a.n_seq) * a.Hk; };
  if (split == 0) {
    e = set_up_fa<NA, T, false>(places);
    if (e != cudaSuccess) return e;
    const long long n = most(2 * f.TQ);
    return launch_fa<NA, T, false>(tq, tk, tv, f, static_cast<int>(n < places[0] ? n : places[0]), st);
  }
  f.split = split;
  const int fit = places[split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3];
  const long long n = most(f.TQ);
  return launch_fa<NA, T, true>(tq, tk, tv, f, static_cast<int>(n < fit ? n : fit) * split, st);
}

template <typename T>
static cudaError_t launch_t(const PackedAttnArgs& a, cudaStream_t st) {
  FaArgs f;
  f.a = a;
  f.G = a.H / a.Hk;
  // few rows per sequence (single tokens): small tiles, whose partial rows are exchanged lightly
  f.light = f.G <= FaCfg<1, true>::LIGHT_ROWS && a.max_q <= FaCfg<1, true>::LIGHT_ROWS / f.G;
  f.TQ = (f.light ? FaCfg<1, true>::LIGHT_ROWS : 128) / f.G;
  f.split = 1;
  f.sc = a.scale * 1.4426950408889634f;
  const int dt = a.fp16 ? DIT_DTYPE_FP16 : DIT_DTYPE_BF16;
  CUtensorMap tq, tk, tv;
  auto map = [&](CUtensorMap* m, const void* p, long long heads, long long tokens, long long head, long long tok, int box_h,
                 int box_t) {
    // an axis of length 1 is never stepped along: any valid stride does
    const uint64_t sh = heads > 1 ? 2 * head : 2 * a.dh, stk = tokens > 1 ? 2 * tok : 2 * a.dh;
    const uint64_t dims[3] = {static_cast<uint64_t>(a.dh), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {sh, stk};
    const uint32_t box[3] = {64, static_cast<uint32_t>(box_h), static_cast<uint32_t>(box_t)};
    return make_tmap_view(m, dt, p, 3, dims, strides, box);
  };
  if (!map(&tq, a.q, a.H, a.total_q, a.q_head, a.q_tok, f.G, f.TQ)) return cudaErrorInvalidValue;
  if (a.total_k == 0) {
    tk = tv = tq;  // no key tile is ever loaded
  } else if (!map(&tk, a.k, a.Hk, a.total_k, a.k_head, a.k_tok, 1, 128) ||
             !map(&tv, a.v, a.Hk, a.total_k, a.v_head, a.v_tok, 1, 128)) {
    return cudaErrorInvalidValue;
  }
  return a.dh <= 64 ? launch_form<1, T>(tq, tk, tv, f, st) : launch_form<2, T>(tq, tk, tv, f, st);
}

cudaError_t launch_attention_packed(const PackedAttnArgs& a, cudaStream_t st) {
  return a.fp16 ? launch_t<__half>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace dit

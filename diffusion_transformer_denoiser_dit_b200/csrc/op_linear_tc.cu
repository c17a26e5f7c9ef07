// y = act(x W^T + b) + r on the tensor cores: two kernels.
//
// linear_pair_kernel: 256 x BN output tiles on SM pairs (tcgen05 cta_group::2), persistent.
//   A pair moves 256 + BN operand rows per 256 x BN x 64 multiply-adds, half of what two single
//   SMs would.  Warp 0 of each CTA loads its 128 rows of x and BN/2 rows of W per 64-wide K
//   stage by TMA; one thread of the leader issues the MMAs of both SMs; warps 4-11 of each CTA
//   finish 32 rows x BN/2 columns each.  Two accumulators in TMEM: the epilogue of one tile
//   runs beside the main loop of the next.  The residual is loaded by TMA into the staging
//   tile while the main loop still runs, added there, and stored from there by TMA.
//
// linear_split_kernel: 128 x BN tiles, one CTA per tile and K slice; the CTAs of a cluster hold
//   the slices of one tile, send each row of their float32 partial tiles to the CTA that finishes
//   that row (distributed shared memory), and each adds up its rows in the order of the slices,
//   so that results repeat bit for bit.  For products with too few 256-row
//   tiles to fill the GPU.  Operands whose rows do not start on 16-byte boundaries are copied
//   into shared memory by the epilogue warps instead of TMA (GATHER).
//
// float32 outputs: tcgen05 drops bits below the accumulator's last place at every 16-wide step,
// a one-sided error that grows with K (5e-6 of the result's norm at K = 4608, where float32
// summation has 7e-7).  So the sum is taken over every 512 products, in round-to-nearest: in registers
// (pairs), or by another accumulator in tensor memory (split K).  16-bit outputs (rounded by up to 2^-9 or
// 2^-12) run 8192 products in one go, whose truncation is at most 2^-22 per 16 of them of the sum so far: 6e-5 of a sum
// that grows evenly (measured 3.5e-5 with bfloat16 products, 5.3e-5 with fp16 ones), an eighth of fp16's half step.
//
// Every wait is bounded; no TMA multicast.
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "op_common.cuh"
#include "op_linear.cuh"
#include "ops.h"

namespace dit {

// 64-wide K blocks per accumulator when the output is float32, and when it has 16 bits
constexpr int kF32ChunkBlocks = 8, k16ChunkBlocks = 128;

// v[i] += bias[n + i] for i < W; columns at or past N get nothing
template <int W>
__device__ __forceinline__ void add_bias(const LinearArgs& a, int n, float* v) {
  if (a.bias == nullptr) return;
  if (n + W <= a.N && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(a.bias + n + i));
      v[i] += b.x;
      v[i + 1] += b.y;
      v[i + 2] += b.z;
      v[i + 3] += b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (n + i < a.N) v[i] += __ldg(a.bias + n + i);
  }
}

// ------------------------------------------------------------------------- SM pairs
template <int BN, bool F32>
struct PairCfg {
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int COLS = BN / 2;             // columns per epilogue warp
  static constexpr int CW = F32 ? 32 : 64;        // columns per 128-byte staging row
  static constexpr int CHUNKS = F32 ? COLS / CW : 2;  // at most, per epilogue warp
  static constexpr int BUF = 32 * 128;            // one staging tile: 32 rows of 128 bytes
  static constexpr int STAGING = 8 * 2 * BUF;
  static constexpr int FIT = (232448 - 1024 - 512 - STAGING) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = 1024 + STAGES * STAGE + STAGING + 512;
  static constexpr int THREADS = 384;             // warpgroup 0: loads, MMA; 1, 2: epilogue
  static constexpr int REG_CTRL = 80, REG_EPI = 208;
  static constexpr int REG_POOL = 128 * REG_CTRL + 256 * REG_EPI;  // must fit the launch allocation
  static_assert(STAGES >= 4 && B_BYTES % 1024 == 0 && COLS % 32 == 0, "tile shape");
};

// Tiles in groups of 8 tile rows, columns outermost inside a group: the tiles that run at one
// time are a block of the output, whose rows of x and W stay in L2 between their uses.
__device__ __forceinline__ void tile_at(int tile, int m_tiles, int n_tiles, int& mt, int& nt) {
  const int per = 8 * n_tiles, g = tile / per, left = tile - g * per, h = min(8, m_tiles - 8 * g);
  nt = left / h;
  mt = 8 * g + left - nt * h;
}

template <int BN, typename T, bool F32>
__global__ void __launch_bounds__(384, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmY,
                       const LinearArgs a, const int tma_out) {
  using C = PairCfg<BN, F32>;
  using O = typename std::conditional<F32, float, T>::type;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t staging = sbase + C::STAGES * C::STAGE;
  const uint32_t bar0 = staging + C::STAGING;
  // barriers: stage full, stage empty, accumulator full, accumulator empty, residual landed
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto TFULL = [&](int i) { return bar0 + 8u * (2 * C::STAGES + i); };
  auto TEMPTY = [&](int i) { return bar0 + 8u * (2 * C::STAGES + 2 + i); };
  auto RES = [&](int w, int b) { return bar0 + 8u * (2 * C::STAGES + 4 + 2 * w + b); };
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::STAGES * C::STAGE + C::STAGING + 8 * (2 * C::STAGES + 20));

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int m_tiles = (a.M + 255) / 256, n_tiles = (a.N + BN - 1) / BN, num_tiles = m_tiles * n_tiles;
  const int kblocks = (a.K + 63) / 64;
  const int chunk = F32 ? kF32ChunkBlocks : k16ChunkBlocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(TFULL(i), 1);
      mbar_init(TEMPTY(i), 512);  // 256 epilogue threads in each CTA of the pair
    }
    for (int i = 0; i < 16; ++i) mbar_init(RES(i >> 1, i & 1), 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(holder), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = uniform(*holder);
  pdl_trigger();
  pdl_wait();

  if (warp < 4) {
    regs_dec<C::REG_CTRL>();
    if (warp == 0) {  // ---------------- loads (both CTAs)
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cid; tile < num_tiles && ok; tile += nclusters) {
        int mt, nt;
        tile_at(tile, m_tiles, n_tiles, mt, nt);
        const int m0 = mt * 256 + 128 * rank, n0 = nt * BN + BN / 2 * rank;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait_warp(EMPTY(s), ph ^ 1u, a.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + s * C::STAGE, full = mapa_shared(FULL(s), 0);
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(FULL(s), 2 * C::STAGE);
            tma_load_2d_pair(sa, &tmX, full, kb * 64, m0);
            tma_load_2d_pair(sa + C::A_BYTES, &tmW, full, kb * 64, n0);
          }
          __syncwarp();
          if (++s == C::STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every stage this CTA filled has been released: no commit is on its way to its barriers
      for (int i = 0; i < C::STAGES && ok; ++i) {
        if (!mbar_wait_warp(EMPTY(s), ph ^ 1u, a.status)) break;
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) after_timeout();
    } else if (warp == 1 && leader) {  // ---------------- MMA issuer
      constexpr uint32_t idesc = idesc_16<T>(256, BN);
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cid; tile < num_tiles && ok; tile += nclusters) {
        for (int kb0 = 0; kb0 < kblocks && ok; kb0 += chunk, ++it) {
          if (!mbar_wait_warp(TEMPTY(it & 1), ((it >> 1) & 1) ^ 1u, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dt = tmem_base + (it & 1) * 256;
          const int kb1 = min(kb0 + chunk, kblocks);
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(FULL(s), ph, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = sbase + s * C::STAGE, sb = sa + C::A_BYTES;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_pair(dt, sdesc_k_sw128(sa + k * 32), sdesc_k_sw128(sb + k * 32), idesc, kb > kb0 || k > 0 ? 1u : 0u);
              mma_commit_pair(EMPTY(s));
              mma_commit_pair(mapa_shared(EMPTY(s), 1));
            }
            __syncwarp();
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (ok && elect_one()) {
            mma_commit_pair(TFULL(it & 1));
            mma_commit_pair(mapa_shared(TFULL(it & 1), 1));
          }
          __syncwarp();
        }
      }
      // every epilogue release, the partner's remote arrivals among them, has landed
      for (int i = it >= 2 ? it - 2 : 0; i < it && ok; ++i)
        if (!mbar_wait_warp(TEMPTY(i & 1), (i >> 1) & 1, a.status)) break;
      if (!ok) after_timeout();
    }
  } else {  // ------------------------ epilogue warps 4..11 (both CTAs)
    regs_inc<C::REG_EPI>();
    const int q = warp & 3, w = warp - 4, half = w >> 2;
    const uint32_t buf0 = staging + w * 2 * C::BUF;
    const uint32_t row = static_cast<uint32_t>(lane) * 128, r7 = lane & 7;
    const bool res_tma = tma_out && a.residual != nullptr;
    int it = 0, use = 0, turn = 0;  // accumulators read; staging tiles used; tiles
    bool ok = true;
    for (int tile = cid; tile < num_tiles && ok; tile += nclusters) {
      int mt, nt;
      tile_at(tile, m_tiles, n_tiles, mt, nt);
      const int m0 = mt * 256 + 128 * rank + 32 * q, n0 = nt * BN;
      // chunk c of this warp starts at tile column col(c): a half of contiguous float32 chunks, or
      // every other 64-wide chunk (of three, two or one, the two halves taking turns by tile)
      const int hh = half ^ (BN % 128 != 0 ? turn & 1 : 0);
      ++turn;
      auto col = [&](int c) { return F32 ? half * C::COLS + c * C::CW : 64 * (hh + 2 * c); };
      int nchunks = 0;
      if (m0 < a.M)
        for (int c = 0; c < C::CHUNKS; ++c) nchunks += col(c) < BN && n0 + col(c) < a.N;
      // residual of chunk c into the staging tile of that chunk's use
      auto load_residual = [&](int c, int ahead) {
        if (lane == 0) {
          bulk_wait_read_all();  // what was staged there has been stored
          const int b = (use + ahead) & 1;
          mbar_arrive_expect_tx(RES(w, b), C::BUF);
          tma_load_2d(buf0 + b * C::BUF, &tmR, RES(w, b), n0 + col(c), m0);
        }
      };
      if (res_tma)
        for (int c = 0; c < 2 && c < nchunks; ++c) load_residual(c, c);
      // 16-bit outputs read the accumulator piece by piece below; float32 sums are taken over here
      float acc[F32 ? C::COLS : 1];
#pragma unroll
      for (int i = 0; i < (F32 ? C::COLS : 1); ++i) acc[i] = 0.f;
      const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (F32) {
        for (int kb0 = 0; kb0 < kblocks; kb0 += chunk, ++it) {
          ok = mbar_wait_spin(TFULL(it & 1), (it >> 1) & 1, a.status);
          __syncwarp();
          if (__any_sync(0xffffffffu, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::COLS; c += 16) {
            uint32_t r[16];
            tmem_ld16(tq + (it & 1) * 256 + half * C::COLS + c, r);
            tmem_ld_wait<16>(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += __uint_as_float(r[i]);
          }
          tc_fence_before();
          mbar_arrive_cluster(mapa_shared(TEMPTY(it & 1), 0));
        }
      } else {
        for (int kb0 = 0;; kb0 += chunk, ++it) {
          ok = mbar_wait_spin(TFULL(it & 1), (it >> 1) & 1, a.status);
          __syncwarp();
          ok = !__any_sync(0xffffffffu, !ok);
          tc_fence_after();
          if (!ok) break;
          if (kb0 > 0) {  // a long sum: what came before onto this accumulator, in the columns that this warp finishes
            const uint32_t now = tq + (it & 1) * 256, before = tq + (~it & 1) * 256;
#pragma unroll 1
            for (int c = 0; c < 4 * nchunks; ++c) {
              const int at = col(c >> 2) + 16 * (c & 3);
              uint32_t v[16], u[16];
              tmem_ld16(now + at, v);
              tmem_ld16(before + at, u);
              tmem_ld_wait<16>(v);
              tmem_ld_wait<16>(u);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(v[i]));
              tmem_st16(now + at, v);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_cluster(mapa_shared(TEMPTY(~it & 1), 0));
          }
          if (kb0 + chunk >= kblocks) break;
        }
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) {
        if (c >= nchunks) break;
        const int n = n0 + col(c), b = use & 1;
        const uint32_t buf = buf0 + b * C::BUF;
        float own[F32 ? 1 : C::CW];
        float* v = F32 ? acc + c * C::CW : own;  // registers: every index below is a constant
        if constexpr (!F32) {
          uint32_t* r = reinterpret_cast<uint32_t*>(v);
          tmem_ld32(tq + (it & 1) * 256 + col(c), r);
          tmem_ld32(tq + (it & 1) * 256 + col(c) + 32, r + 32);
          tmem_ld_wait<C::CW>(*reinterpret_cast<uint32_t(*)[C::CW]>(r));
          if (c + 1 >= nchunks) {  // the last read of this accumulator
            tc_fence_before();
            mbar_arrive_cluster(mapa_shared(TEMPTY(it & 1), 0));
          }
        }
        add_bias<C::CW>(a, n, v);
        with_act(a.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < C::CW; ++i) v[i] = activate<decltype(act)::value>(v[i]);
        });
        if (tma_out) {
          if (res_tma) {
            ok = mbar_wait_spin(RES(w, b), (use >> 1) & 1, a.status);
            __syncwarp();
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
          } else if (use >= 2) {  // the store two uses ago has read this tile
            if (lane == 0) bulk_wait_read_but1();
            __syncwarp();
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint32_t at = buf + row + ((u ^ r7) << 4);
            uint32_t p[4];
            if (res_tma) {
              const uint4 rr = ld_shared_v4(at);
              p[0] = rr.x, p[1] = rr.y, p[2] = rr.z, p[3] = rr.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (F32) {
                float z = v[4 * u + i];
                if (res_tma) z += __uint_as_float(p[i]);
                p[i] = __float_as_uint(z);
              } else {
                float z0 = v[8 * u + 2 * i], z1 = v[8 * u + 2 * i + 1];
                if (res_tma) {
                  const float2 rr = unpack2<T>(p[i]);
                  z0 += rr.x;
                  z1 += rr.y;
                }
                p[i] = pack2<T>(z0, z1);
              }
            }
            st_shared_v4(at, p[0], p[1], p[2], p[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmY, buf, n, m0);  // rows past M and columns past N are clipped
            bulk_commit_group();
          }
          if (res_tma && c + 2 < nchunks) load_residual(c + 2, 2);  // the same staging tile, once stored
        } else {
          // 32 float32 columns at a time through the staging tile, then a row per step: lane = column
#pragma unroll
          for (int h = 0; h < C::CW; h += 32) {
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u)
              st_shared_v4(buf + row + ((u ^ r7) << 4), __float_as_uint(v[h + 4 * u]), __float_as_uint(v[h + 4 * u + 1]),
                           __float_as_uint(v[h + 4 * u + 2]), __float_as_uint(v[h + 4 * u + 3]));
            __syncwarp();
            const int nn = n + h + lane, rows = min(32, a.M - m0);
            const uint8_t* src = smem + (buf - sbase);
            if (nn < a.N) {
#pragma unroll 2
              for (int r = 0; r < rows; ++r)
                linear_put<T, F32>(a, m0 + r, nn,
                                   *reinterpret_cast<const float*>(src + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4));
            }
          }
        }
        ++use;
      }
      if (!F32) {
        if (nchunks == 0) {
          tc_fence_before();
          mbar_arrive_cluster(mapa_shared(TEMPTY(it & 1), 0));
        }
        ++it;
      }
    }
    if (lane == 0) bulk_wait_all();  // this warp's stores are complete
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its partner may still signal it or use its TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

static bool map_rows(CUtensorMap* m, int dtype, const void* p, long long rows, long long cols, long long ld, int box_rows,
                     int box_cols) {
  const uint64_t es = dtype == DIT_DTYPE_F32 ? 4 : 2;
  // one row has no stride; any aligned one will do
  const uint64_t stride = rows > 1 ? ld * es : (cols * es + 15) / 16 * 16;
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, strides[1] = {stride};
  const uint32_t box[2] = {static_cast<uint32_t>(box_cols), static_cast<uint32_t>(box_rows)};
  if (rows > 1 && ld < cols) return false;
  return make_tmap_view(m, dtype, p, 2, dims, strides, box);
}

template <int BN, typename T, bool F32>
static cudaError_t launch_pair(const LinearArgs& a, const CUtensorMap& tx, const CUtensorMap& tw, int num_sms,
                               cudaStream_t st) {
  using C = PairCfg<BN, F32>;
  auto kernel = linear_pair_kernel<BN, T, F32>;
  static int clusters_of[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {2, 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  if (clusters_of[dev] == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    // the register split (setmaxnreg) must fit in the launch allocation, or it would wait forever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * C::THREADS < C::REG_POOL) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(2 * (num_sms / 2));
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    clusters_of[dev] = n < num_sms / 2 ? n : num_sms / 2;
  }
  const int od = F32 ? DIT_DTYPE_F32 : a.fp16 ? DIT_DTYPE_FP16 : DIT_DTYPE_BF16;
  CUtensorMap ty = tx, tr = tx;
  int tma_out = map_rows(&ty, od, a.y, a.M, a.N, a.ldy, 32, C::CW);
  if (tma_out && a.residual) tma_out = map_rows(&tr, od, a.residual, a.M, a.N, a.ldr, 32, C::CW);
  const long long tiles = static_cast<long long>((a.M + 255) / 256) * ((a.N + BN - 1) / BN);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < clusters_of[dev] ? tiles : clusters_of[dev]));
  cfg.numAttrs = g_pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tx, tw, tr, ty, a, tma_out);
}

// ------------------------------------------------------------------------- split K in a cluster
template <int BN>
struct SplitCfg {
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int PART = 128 * BN * 4;          // partial rows of all slices for this CTA's share
  // One CTA per SM with all of its memory in flight: a round trip of a stage (load, product,
  // release) took 1.6 us measured, so 96 KB of stages fed an SM 31 bytes a cycle and no more.
  static constexpr int STAGES = (232448 - 1024 - 256 - PART) / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + PART + 256;
  static constexpr int TMEM = 4 * BN;                // four accumulators: the first chunk's, which takes over the
                                                     // later ones of a long sum, and three in turn
  // 16-byte unit u of partial row r: rows 8 apart in one bank group, neighbours in others
  static __device__ __forceinline__ uint32_t part_at(int r, int u) {
    return static_cast<uint32_t>(r) * (BN * 4) + static_cast<uint32_t>((u & ~7) | ((u ^ r) & 7)) * 16;
  }
};

// `rows` rows (a multiple of 8) of 128 bytes into a 128-byte-swizzled tile by 128 threads, GRAIN bytes (4 or
// 8) per cp.async: this thread's column of them, `bytes` of it inside the matrix, rows row0, row0 + GRAIN, ..;
// rows from `real` on are zeros.  Addresses advance by additions (with the row times the stride formed
// anew for each, an iteration took 166 cycles).
template <int GRAIN>
__device__ __forceinline__ void gather_async(uint32_t dst, const uint8_t* src, long long ld_bytes, int row0, int rows,
                                             int real, int col_bytes, int bytes) {
#pragma unroll
  for (int sub = 0; sub < 8 / GRAIN; ++sub) {  // the row modulo 8, and so the swizzle, stays in this loop
    const int r = row0 + sub * GRAIN;
    uint32_t to = dst + r * 128 + ((col_bytes & 112) ^ ((r & 7) << 4)) + (col_bytes & 15);
    const uint8_t* from = src + r * ld_bytes;
    const long long step = 8 * ld_bytes;
    int left = (real - r + 7) >> 3;           // rows of this thread inside the matrix
    if (left <= 0) from = src;
#pragma unroll 4
    for (int i = r; i < rows; i += 8) {
      const int n = left > 0 ? bytes : 0;
      if constexpr (GRAIN == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
      to += 1024;
      if (--left > 0) from += step;           // never past the last row
    }
  }
}

// 128 bytes (64 values) of `rows` rows from p (row r0, column k0) into a 128-byte-swizzled tile, by 128
// threads; values outside [R, K] are zero.  Rows aligned to 4 or 8 bytes are copied asynchronously (the
// caller waits for its group), others through registers.
template <typename T>
__device__ __forceinline__ void gather_tile(uint32_t dst, const T* p, long long ld, int r0, int R, int k0, int K, int rows,
                                            int grain, int tid) {
  if (grain >= 4) {
    const int c = grain == 8 ? tid & 15 : tid & 31, row0 = grain == 8 ? tid >> 4 : tid >> 5, k = k0 + c * (grain >> 1);
    const int bytes = min(max(K - k, 0) * 2, grain);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(p + r0 * ld + (k < K ? k : 0));
    if (grain == 8) gather_async<8>(dst, src, ld * 2, row0, rows, R - r0, c * 8, bytes);
    else gather_async<4>(dst, src, ld * 2, row0, rows, R - r0, c * 4, bytes);
    return;
  }
  // Odd element offsets: a thread takes 16 bytes of every 16th row from the aligned words around them (a word
  // that holds a value of the matrix can be read whole) and shifts; four rows in flight.
  const int u = tid & 7, row0 = tid >> 3, k = k0 + u * 8, n = min(max(K - k, 0), 8);
  const uintptr_t base = reinterpret_cast<uintptr_t>(p + r0 * ld + k);
  const long long step = 16 * ld * 2;
  uintptr_t at = base + row0 * ld * 2;
  const uint32_t to = dst + row0 * 128 + ((u ^ (row0 & 7)) << 4);
  for (int i = 0; row0 + i * 16 < rows; i += 4) {
    uint32_t w[4][5];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = r0 + row0 + (i + j) * 16 < R && row0 + (i + j) * 16 < rows;
      const uintptr_t src = at + j * step;
      const int words = in && n > 0 ? static_cast<int>(((src & 2) + 2 * n + 3) >> 2) : 0;
#pragma unroll
      for (int e = 0; e < 5; ++e) w[j][e] = e < words ? reinterpret_cast<const uint32_t*>(src & ~uintptr_t(3))[e] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t shift = static_cast<uint32_t>((at + j * step) & 2) * 8;
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __funnelshift_r(w[j][e], w[j][e + 1], shift);
        if (n < 2 * e + 2) v[e] = n == 2 * e + 1 ? v[e] & 0xffffu : 0u;  // values past K
      }
      if (row0 + (i + j) * 16 < rows) st_shared_v4(to + (i + j) * 16 * 128, v[0], v[1], v[2], v[3]);
    }
    at += 4 * step;
  }
}

struct SplitArgs {
  int split;            // CTAs per cluster: K slices of a tile
  int grain_x, grain_w; // 0: by TMA; else bytes that its rows are aligned to (2, 4 or 8)
  int vec;              // y and residual rows allow four values at a time
};

// Accumulator b, once it is complete, onto the first, by one of four warps (its 32 rows).  Not inlined into the gathering
// loop: 1111 x 588 -> 1153, which never comes here, 21.3 us for 21.6.
template <int BN>
__device__ __noinline__ bool split_take_over(uint32_t t, int b, uint32_t complete, uint32_t taken, uint32_t parity, int* status) {
  if (!mbar_wait_warp(complete, parity, status)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < BN; c += 16) {
    uint32_t v[16], w[16];
    tmem_ld16(t + c, v);
    tmem_ld16(t + b * BN + c, w);
    tmem_ld_wait<16>(v);
    tmem_ld_wait<16>(w);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
    tmem_st16(t + c, v);
  }
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(taken);
  return true;
}

template <int BN, typename T, bool GATHER>
__global__ void __launch_bounds__(192)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                        const LinearArgs a, const SplitArgs sp, const int box_rows) {
  using C = SplitCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), part = sbase + C::STAGES * C::STAGE, bar0 = part + C::PART;
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  const uint32_t done = bar0 + 8u * (2 * C::STAGES);  // the last product of this CTA is complete
  // sums of more than four chunks: a chunk is complete; it has been added to the first, its place is free
  auto CHUNK = [&](int b) { return done + 8u * b; };        // b = 1, 2, 3
  auto TAKEN = [&](int b) { return done + 8u * (3 + b); };
  static_assert(8 * (2 * C::STAGES + 7) + 4 <= 256, "barrier area");
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::STAGES * C::STAGE + C::PART + 8 * (2 * C::STAGES + 7));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int m_tiles = (a.M + 127) / 128;
  const int tile = blockIdx.x / sp.split;
  const int m0 = (tile % m_tiles) * 128, n0 = (tile / m_tiles) * BN;
  const int kblocks_all = (a.K + 63) / 64;
  const int kb_begin = static_cast<int>(static_cast<long long>(kblocks_all) * rank / sp.split);
  const int kb_end = static_cast<int>(static_cast<long long>(kblocks_all) * (rank + 1) / sp.split);
  // blocks per accumulator: 8192 products, or 512.  Chunk 0 is in accumulator 0, chunk i in 1 + (i - 1) % 3.
  const int nkb = kb_end - kb_begin;
  const int chunk = a.out_f32 ? kF32ChunkBlocks : k16ChunkBlocks, nchunks = (nkb + chunk - 1) / chunk;
  // rows of the tile that one CTA of the cluster finishes
  const int share = (min(128, a.M - m0) + sp.split - 1) / sp.split;
  const int gathered = GATHER ? (sp.grain_x != 0) + (sp.grain_w != 0) : 0;
  const int gather_rows = min(128, (a.M - m0 + 7) & ~7);  // the rest of the tile only reaches rows past M

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(FULL(s), (gathered < 2 ? 1 : 0) + (gathered > 0 ? 128 : 0));
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(done, 1);
    for (int b = 1; b < 4; ++b) {
      mbar_init(CHUNK(b), 1);
      mbar_init(TAKEN(b), 4);  // one arrival per warp with rows
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(holder), C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_started();  // the others are waited for before the first partial row is sent
  const uint32_t tmem_base = uniform(*holder);
  pdl_trigger();
  pdl_wait();
  // the residual of this CTA's rows on its way to L2 beside the main loop (4096 x 2052 -> 4096 with residual:
  // 328 -> 304 us; nothing where it is there already)
  if (a.residual != nullptr && threadIdx.x >= 64 && static_cast<int>(threadIdx.x) - 64 < min(share, a.M - m0 - rank * share)) {
    const long long row = m0 + rank * share + static_cast<int>(threadIdx.x) - 64, size = a.out_f32 ? 4 : 2;
    const uint8_t* p = static_cast<const uint8_t*>(a.residual) + (row * a.ldr + n0) * size;
    const int bytes = min(BN, a.N - n0) * static_cast<int>(size);
    for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + bytes - 1));
  }

  if (warp == 0) {
    if (gathered < 2) {  // ---------------- TMA loads
      int s = 0;
      uint32_t ph = 0, armed = 0;
      bool ok = true;
      const bool bx = !GATHER || sp.grain_x == 0, bw = !GATHER || sp.grain_w == 0;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_wait_warp(EMPTY(s), ph ^ 1u, a.status)) {
          ok = false;
          break;
        }
        const uint32_t sa = sbase + s * C::STAGE;
        if (elect_one()) {
          mbar_arrive_expect_tx(FULL(s), (bx ? box_rows * 128 : 0) + (bw ? C::B_BYTES : 0));
          // rows of the tile past box_rows keep what they held: they only reach rows past M
          if (bx) tma_load_2d(sa, &tmX, FULL(s), kb * 64, m0);
          if (bw) tma_load_2d(sa + C::A_BYTES, &tmW, FULL(s), kb * 64, n0);
        }
        __syncwarp();
        armed |= 1u << s;
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok)  // a wait ran out: let the copies that were issued land before leaving
        for (int j = 0; j < C::STAGES; ++j)
          if (armed & (1u << j)) mbar_wait_warp(FULL(j), j < s ? ph : ph ^ 1u, a.status);
    }
    cluster_all_started();
  } else if (warp == 1) {
    // ---------------- MMA issuer
    constexpr uint32_t idesc = idesc_16<T>(128, BN);
    int s = 0, left = chunk, i = 0, b = 0;  // chunk i in accumulator b
    uint32_t ph = 0, acc = tmem_base, fresh = 0;
    for (int kb = 0; kb < nkb; ++kb) {
      if (i >= 4 && fresh == 0 && !mbar_wait_warp(TAKEN(b), ((i - 1) / 3 - 1) & 1, a.status)) break;
      if (!mbar_wait_warp(FULL(s), ph, a.status)) break;
      tc_fence_after();
      const uint32_t sa = sbase + s * C::STAGE, sb = sa + C::A_BYTES;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ss(acc, sdesc_k_sw128(sa + k * 32), sdesc_k_sw128(sb + k * 32), idesc, k > 0 ? 1u : fresh);
        mma_commit(EMPTY(s));
      }
      __syncwarp();
      fresh = 1;
      if (--left == 0) {
        if (i > 0 && i + 4 <= nchunks) {
          if (elect_one()) mma_commit(CHUNK(b));
          __syncwarp();
        }
        left = chunk;
        b = b == 3 ? 1 : b + 1;
        ++i;
        acc = tmem_base + b * BN;
        fresh = 0;
      }
      if (++s == C::STAGES) {
        s = 0;
        ph ^= 1u;
      }
    }
    // also after a wait that ran out: what was issued finishes before TMEM is freed
    if (elect_one()) mma_commit(done);
    __syncwarp();
    mbar_wait_warp(done, 0, a.status);
    cluster_all_started();
  } else {  // ------------------------ warps 2..5: gather, then one row of sums per thread
    const int tid = threadIdx.x - 64, q = warp & 3, r = q * 32 + lane;
    // chunk i (0 < i <= nchunks - 4) onto the first accumulator, in the order of the chunks
    auto take_over = [&](int i) -> bool {
      const int b = 1 + (i - 1) % 3;
      return split_take_over<BN>(tmem_base + (static_cast<uint32_t>(q * 32) << 16), b, CHUNK(b), TAKEN(b), ((i - 1) / 3) & 1, a.status);
    };
    if (!(GATHER && gathered > 0))
      for (int i = 1; i + 4 <= nchunks; ++i)
        if (!take_over(i)) break;
    if (GATHER && gathered > 0) {
      // copies of up to AHEAD stages are in flight; a stage is handed over when this thread's share landed
      constexpr int AHEAD = 3;
      static_assert(C::STAGES > AHEAD, "stages");
      int s = 0, full = 0;
      uint32_t ph = 0;
      bool ok = true;
      // up to where chunk `next` is taken over, a whole chunk behind its end: all of its stages have been handed over
      // then, and its products do not wait for this warp
      for (int begin = kb_begin, next = 1;; ++next) {
        const bool last = next + 4 > nchunks;
        const int stop = last ? kb_end + AHEAD : kb_begin + (next + 2) * chunk;
        for (int kb = begin; kb < stop; ++kb) {
          if (kb < kb_end) {
            ok = ok && mbar_wait_spin(EMPTY(s), ph ^ 1u, a.status);
            if (ok) {
              const uint32_t sa = sbase + s * C::STAGE;
              if (sp.grain_x)
                gather_tile(sa, static_cast<const T*>(a.x), a.ldx, m0, a.M, kb * 64, a.K, gather_rows, sp.grain_x, tid);
              if (sp.grain_w)
                gather_tile(sa + C::A_BYTES, static_cast<const T*>(a.w), a.ldw, n0, a.N, kb * 64, a.K, BN, sp.grain_w, tid);
            }
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (kb - AHEAD >= kb_begin) {
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
            fence_proxy_async_smem();
            if (ok) mbar_arrive(FULL(full));
            if (++full == C::STAGES) full = 0;
          }
        }
        if (last) break;
        ok = __all_sync(0xffffffffu, ok) && take_over(next);
        begin = stop;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    cluster_all_started();
    // Row r goes to the CTA that finishes it: CTA r / share keeps rows share * CTA .. of the tile,
    // slice after slice.  A short loop: code that runs once per launch costs its fetch.
    if (m0 + q * 32 < a.M && mbar_wait_warp(done, 0, a.status)) {
      tc_fence_after();
      const int owner = r / share, pr = rank * share + (r - owner * share);
      const uint32_t base = mapa_shared(part, min(owner, sp.split - 1)), t = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const bool mine = m0 + r < a.M;
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        uint32_t v[16];
        tmem_ld16(t + c, v);
        tmem_ld_wait<16>(v);
#pragma unroll 1
        for (int j = max(1, nchunks - 3); j < nchunks; ++j) {
          uint32_t w[16];
          tmem_ld16(t + (1 + (j - 1) % 3) * BN + c, w);
          tmem_ld_wait<16>(w);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
        }
        if (mine)
#pragma unroll
          for (int i = 0; i < 4; ++i) st_cluster_v4(base + C::part_at(pr, c / 4 + i), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // the partial rows of all slices are where they are finished
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM);
  }
  // this CTA's rows: a thread keeps its four columns and steps through the rows, slices added in their order;
  // four rows at a time, whose residuals are on their way together
  constexpr int UNITS = BN / 4, STEP = 192 / UNITS, BATCH = 4;
  static_assert(192 % UNITS == 0, "whole rows per step");
  const int u = threadIdx.x % UNITS, n = n0 + 4 * u, r0 = m0 + rank * share, rows = min(share, a.M - r0);
  if (n >= a.N) return;
  const bool vec = sp.vec && n + 4 <= a.N;
  const int cols = min(4, a.N - n);
  float bias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) bias[e] = a.bias && e < cols ? __ldg(a.bias + n + e) : 0.f;
  with_act(a.act, [&](auto act) {
#pragma unroll 1
    for (int r = threadIdx.x / UNITS; r < rows; r += BATCH * STEP) {
      float v[BATCH][4], res[BATCH][4];
      if (a.residual) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const long long at = (r0 + min(r + k * STEP, rows - 1)) * a.ldr + n;
          if (a.out_f32) {
            const float* p = static_cast<const float*>(a.residual) + at;
            if (vec) *reinterpret_cast<float4*>(res[k]) = *reinterpret_cast<const float4*>(p);
            else
#pragma unroll
              for (int e = 0; e < 4; ++e) res[k][e] = e < cols ? p[e] : 0.f;
          } else {
            const T* p = static_cast<const T*>(a.residual) + at;
            if (vec) {
              const uint2 w = *reinterpret_cast<const uint2*>(p);
              const float2 y0 = unpack2<T>(w.x), y1 = unpack2<T>(w.y);
              res[k][0] = y0.x, res[k][1] = y0.y, res[k][2] = y1.x, res[k][3] = y1.y;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) res[k][e] = e < cols ? to_f32(p[e]) : 0.f;
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) res[k][e] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = bias[e];
      for (int j = 0; j < sp.split; ++j)
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const uint4 p = ld_shared_v4(part + C::part_at(j * share + min(r + k * STEP, rows - 1), u));
          v[k][0] += __uint_as_float(p.x), v[k][1] += __uint_as_float(p.y);
          v[k][2] += __uint_as_float(p.z), v[k][3] += __uint_as_float(p.w);
        }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (r + k * STEP >= rows) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = activate<decltype(act)::value>(v[k][e]) + res[k][e];
        const long long at = (r0 + r + k * STEP) * a.ldy + n;
        if (a.out_f32) {
          float* p = static_cast<float*>(a.y) + at;
          if (vec) *reinterpret_cast<float4*>(p) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
          else
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < cols) p[e] = v[k][e];
        } else {
          T* p = static_cast<T*>(a.y) + at;
          if (vec) *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[k][0], v[k][1]), pack2<T>(v[k][2], v[k][3]));
          else
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < cols) p[e] = from_f32<T>(v[k][e]);
        }
      }
    }
  });
}

template <int BN, typename T, bool GATHER>
static cudaError_t launch_split(const LinearArgs& a, const CUtensorMap& tx, const CUtensorMap& tw, SplitArgs sp,
                                int box_rows, cudaStream_t st) {
  using C = SplitCfg<BN>;
  auto kernel = linear_split_kernel<BN, T, GATHER>;
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const long long ctas = static_cast<long long>((a.M + 127) / 128) * ((a.N + BN - 1) / BN) * sp.split;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(sp.split), 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = g_pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a, sp, box_rows);
}

// clusters of 1, 2, 4 and 8 CTAs of the split kernel that the device runs at one time; first calls may come
// from several threads at once, so the counts are published together, the last with release
template <typename T>
static bool split_clusters(int* fit) {
  static std::atomic<int> of[kMaxDevices][4];
  const int dev = current_device();
  if (dev < 0) return false;
  if (of[dev][3].load(std::memory_order_acquire) == 0) {
    auto kernel = linear_split_kernel<64, T, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SplitCfg<64>::SMEM) != cudaSuccess) return false;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(8 * 148);
      cfg.blockDim = dim3(192);
      cfg.dynamicSmemBytes = SplitCfg<64>::SMEM;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim = {1u << i, 1, 1};
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&fit[i], kernel, &cfg) != cudaSuccess || fit[i] <= 0) return false;
    }
    for (int i = 0; i < 4; ++i) of[dev][i].store(fit[i], std::memory_order_release);
    return true;
  }
  for (int i = 0; i < 4; ++i) fit[i] = of[dev][i].load(std::memory_order_relaxed);
  return true;
}

template <typename T>
static cudaError_t launch_tc(const LinearArgs& a, int num_sms, cudaStream_t st) {
  const int dt = a.fp16 ? DIT_DTYPE_FP16 : DIT_DTYPE_BF16;
  const int kblocks = (a.K + 63) / 64;
  CUtensorMap tx, tw;
  // Tile width: a 64-wide K stage costs a pair 512 cycles at 256 columns (tensor cores) and
  // about 400 at 192, so the narrower tile pays where it leaves fewer or fuller rounds
  // (N = 1152 at 8192 rows: 3 rounds of either).
  const long long mt2 = (a.M + 255) / 256, pairs = num_sms / 2;
  auto rounds = [&](int bn) { return (mt2 * ((a.N + bn - 1) / bn) + pairs - 1) / pairs; };
  const int bn2 = rounds(192) * 400 < rounds(256) * 512 ? 192 : 256;
  // fewer tiles than half the pairs: the split kernel (1024 x 1152 -> 4608, 72 of 74 pairs busy: 12.9
  // against 24.6 us; 512 x 768 -> 2304, 24 busy: 8.5 against 8.0).  Tiles of 256 rows are counted, full or not: up to
  // 128 rows by 7200 features and more the split kernel would mostly last less (in a graph, 5 x 4608 -> 7200 12.6 against
  // 30.8 us, 128 x 1152 -> 16384 10.0 against 11.9; 64 x 1152 -> 32768 17.6 against 16.7), above 128 not
  // (192 x 1152 -> 16384 18.9 against 12.0).
  if (mt2 * ((a.N + 191) / 192) >= pairs / 2 && map_rows(&tx, dt, a.x, a.M, a.K, a.ldx, 128, 64) &&
      map_rows(&tw, dt, a.w, a.N, a.K, a.ldw, bn2 / 2, 64)) {
    if (a.out_f32) return bn2 == 192 ? launch_pair<192, T, true>(a, tx, tw, num_sms, st) : launch_pair<256, T, true>(a, tx, tw, num_sms, st);
    return bn2 == 192 ? launch_pair<192, T, false>(a, tx, tw, num_sms, st) : launch_pair<256, T, false>(a, tx, tw, num_sms, st);
  }
  // the split kernel
  auto grain = [](const void* p, long long ld) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 2);
    return v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
  };
  // Tile width and slices, from what was measured in cycles: a K block is 370 whatever the tile (the
  // issue of its four MMAs), a round of CTAs 5300 besides and 3600 / 7600 more to finish 128 rows of
  // 64 / 128 columns.  A round is what fits at one time: clusters of 4 and 8 do not reach every SM.
  SplitArgs sp;
  const long long mt = (a.M + 127) / 128;
  const int rows = a.M >= 128 ? 128 : a.M;
  int fit[4];
  if (!split_clusters<T>(fit)) return cudaErrorInvalidConfiguration;
  const bool gather = !(map_rows(&tx, dt, a.x, a.M, a.K, a.ldx, 8, 64) && map_rows(&tw, dt, a.w, a.N, a.K, a.ldw, 64, 64));
  bool narrow = false;
  long long best = -1;
  for (int bn = 128; bn >= 64; bn -= 64)
    for (int i = 0, split = 1; i < 4 && 2 * split <= kblocks + 1; ++i, split *= 2) {
      const long long rounds = (mt * ((a.N + bn - 1) / bn) + fit[i] - 1) / fit[i];
      const long long cost = rounds * (5300 + (kblocks + split - 1) / split * (gather ? 900 : 370) + (bn == 64 ? 3600 : 7600) * rows / 128);
      if (best < 0 || cost < best) {
        best = cost;
        sp.split = split;
        narrow = bn == 64;
      }
    }
  const int bn = narrow ? 64 : 128;
  const int box_rows = a.M >= 128 ? 128 : (a.M + 7) / 8 * 8;
  sp.grain_x = map_rows(&tx, dt, a.x, a.M, a.K, a.ldx, box_rows, 64) ? 0 : grain(a.x, a.ldx);
  sp.grain_w = map_rows(&tw, dt, a.w, a.N, a.K, a.ldw, bn, 64) ? 0 : grain(a.w, a.ldw);
  const int es = a.out_f32 ? 4 : 2;
  auto four = [&](const void* p, long long ld) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es)) & (4 * es - 1)) == 0;
  };
  sp.vec = four(a.y, a.ldy) && (a.residual == nullptr || four(a.residual, a.ldr));
  if (sp.grain_x && sp.grain_w) tx = tw = CUtensorMap{};
  else if (sp.grain_x) tx = tw;
  else if (sp.grain_w) tw = tx;
  if (narrow)
    return gather ? launch_split<64, T, true>(a, tx, tw, sp, box_rows, st)
                  : launch_split<64, T, false>(a, tx, tw, sp, box_rows, st);
  return gather ? launch_split<128, T, true>(a, tx, tw, sp, box_rows, st)
                : launch_split<128, T, false>(a, tx, tw, sp, box_rows, st);
}

cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t st) {
  return a.fp16 ? launch_tc<__half>(a, num_sms, st) : launch_tc<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace dit

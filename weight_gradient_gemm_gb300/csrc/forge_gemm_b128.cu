// The 8-bit products of a linear layer, with one scale per 128 columns of a
// token's row and per 128 x 128 block of the weight:
//   forward          Y[t][p]  = sum_b sx[t][b] sw[p/128][b] sum_{q in b} X[t][q] W[p][q]
//   input gradient   dX[t][q] = sum_b sd[t][b] sw[b][q/128] sum_{p in b} dY[t][p] W[p][q]
// The same stored weight serves both: the forward pass reads it K-major, the
// input gradient MN-major.
//
// The inner sums over one block of 128 are plain e4m3 products, which the
// tensor core forms (tcgen05.mma kind::f8f6f4, four instructions 32 deep) into
// a fresh TMEM accumulator.  The scales change from block to block, so the
// outer sum cannot stay in TMEM: the epilogue warps read each block's
// accumulator and add it, times the row's and the block's scale, to fp32
// registers that hold the output tile.  Several TMEM buffers let the tensor
// core run ahead of that.
//
// Warp roles (320 threads): warp 0 loads operand stages of 128 columns with
// TMA, warp 1 issues the MMAs, warps 2-9 add up (two per TMEM lane quadrant,
// each half of the tile's columns) and store.  Every wait is bounded, as in
// forge_gemm.cuh.
#include <cuda_bf16.h>

#include "forge_internal.h"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

constexpr int kThreads8 = 320;
constexpr int kEpiWarps = 8;
constexpr int kSmemMax = 232448;   // dynamic shared memory of one CTA (227 KB)

// CG CTAs compute a (128 CG) x BN tile; a CTA loads its 128 rows of A and
// BN / CG columns of B per stage.
template <int CG, int BN>
struct Traits8 {
  static constexpr int TM = kBM * CG;
  static constexpr int BNL = BN / CG;
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int STAGE_BYTES = A_BYTES + BNL * 128;
  static constexpr int OUT_BYTES = kEpiWarps * 4096;   // one 32-row slab of 128-byte rows a warp
  static constexpr int STAGES = 6;
  static constexpr int NBUF = 512 / BN;                // TMEM accumulators
  static constexpr int NC = BN / 2;                    // columns per epilogue thread
  static constexpr int OFF_OUT = STAGES * STAGE_BYTES;
  static constexpr int OFF_BARS = OFF_OUT + OUT_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NBUF + 1;
  static constexpr int OFF_TMEM = OFF_BARS + 8 * NUM_BARS;
  static constexpr int SMEM_USED = OFF_TMEM + 8;
  static constexpr int SMEM_ALLOC = SMEM_USED + 1024 < kSmemMax ? SMEM_USED + 1024 : kSmemMax;
  static_assert(SMEM_USED <= kSmemMax, "shared memory budget exceeded");
};

// Tile order: groups of group_m tile rows, column by column inside a group,
// so that the tiles in flight share operands in L2.
__device__ __forceinline__ void tile_of(int t, const B128Args& a, int& tm, int& tn) {
  const int per = a.group_m * a.tiles_n;
  const int g = t / per, r = t - g * per;
  const int m0 = g * a.group_m;
  const int gm = min(a.group_m, a.tiles_m - m0);
  tn = r / gm;
  tm = m0 + r - tn * gm;
}

template <int CG, int BN, bool DGRAD>
__global__ void __launch_bounds__(kThreads8, 1) gemm_b128_kernel(const __grid_constant__ B128Args a) {
  using T = Traits8<CG, BN>;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  if (base - raw + T::SMEM_USED > T::SMEM_ALLOC) {   // uniform: nothing has started
    if (threadIdx.x == 0) atomicCAS(a.err, 0, kErrDeviceConfig);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit0 = kPair ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = kPair ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

  const uint32_t bars = base + T::OFF_BARS;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (T::STAGES + s); };
  auto bar_tfull = [&](int b) { return bars + 8u * (2 * T::STAGES + b); };
  auto bar_tempty = [&](int b) { return bars + 8u * (2 * T::STAGES + T::NBUF + b); };
  const uint32_t bar_drain = bars + 8u * (2 * T::STAGES + 2 * T::NBUF);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM + 4);
  const WaitCtx wc{abort_flag, a.err, a.err_site, a.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < T::NBUF; ++b) {
      mbar_init(bar_tfull(b), 1);
      mbar_init(bar_tempty(b), CG * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.a);
    tma_prefetch_desc(&a.b);
    tma_prefetch_desc(&a.out);
  }
  if constexpr (kPair) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(base + T::OFF_TMEM, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(base + T::OFF_TMEM, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      uint32_t cnt = 0;
      int32_t last_armed[T::STAGES];
#pragma unroll
      for (int s = 0; s < T::STAGES; ++s) last_armed[s] = -1;
      bool ok = true;
      for (int t = unit0; ok && t < a.num_tiles; t += units) {
        int tm, tn;
        tile_of(t, a, tm, tn);
        const int ya = tm * T::TM + static_cast<int>(rank) * kBM;
        const int nb = tn * BN + static_cast<int>(rank) * T::BNL;
        for (int k = 0; k < a.num_kb; ++k, ++cnt) {
          const int s = cnt % T::STAGES;
          if (!wait_stage<!kPair>(bar_empty(s), ((cnt / T::STAGES) & 1u) ^ 1u, wc,
                                  kSiteProducerEmpty)) { ok = false; break; }
          const uint32_t dst = base + s * T::STAGE_BYTES;
          // the weight's box: [BNL rows][128 of K], or for the input gradient
          // [128 of K][128 columns] per 128 columns
          if constexpr (kPair) {
            const uint32_t fb = mapa_shared(bar_full(s), 0);
            if (leader) mbar_arrive_expect_tx(bar_full(s), 2 * T::STAGE_BYTES);
            tma_load_2d_pair(dst, &a.a, k * 128, ya, fb, pol);
            if constexpr (DGRAD) {
#pragma unroll
              for (int c = 0; c < T::BNL / 128; ++c)
                tma_load_2d_pair(dst + T::A_BYTES + c * 16384, &a.b, nb + c * 128, k * 128, fb, pol);
            } else {
              tma_load_2d_pair(dst + T::A_BYTES, &a.b, k * 128, nb, fb, pol);
            }
          } else {
            mbar_arrive_expect_tx(bar_full(s), T::STAGE_BYTES);
            tma_load_2d(dst, &a.a, k * 128, ya, bar_full(s), pol);
            if constexpr (DGRAD) {
#pragma unroll
              for (int c = 0; c < T::BNL / 128; ++c)
                tma_load_2d(dst + T::A_BYTES + c * 16384, &a.b, nb + c * 128, k * 128, bar_full(s),
                            pol);
            } else {
              tma_load_2d(dst + T::A_BYTES, &a.b, k * 128, nb, bar_full(s), pol);
            }
          }
          if (leader) last_armed[s] = static_cast<int32_t>(cnt);
        }
      }
      // let every armed load land before the CTA can exit
      for (int s = 0; s < T::STAGES; ++s)
        if (last_armed[s] >= 0)
          wait_bounded(bar_full(s), (static_cast<uint32_t>(last_armed[s]) / T::STAGES) & 1u, wc,
                       kSiteDrainOperands, false);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = make_idesc_e4m3(T::TM, BN, false, DGRAD);
      uint32_t cnt = 0;
      bool ok = true;
      for (int t = unit0; ok && t < a.num_tiles; t += units) {
        for (int k = 0; k < a.num_kb; ++k, ++cnt) {
          const int buf = cnt % T::NBUF;
          if (!wait_bounded(bar_tempty(buf), ((cnt / T::NBUF) & 1u) ^ 1u, wc, kSiteMmaTmemEmpty)) {
            ok = false;
            break;
          }
          const int s = cnt % T::STAGES;
          if (!wait_stage<!kPair>(bar_full(s), (cnt / T::STAGES) & 1u, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d = tmem_base + buf * BN;
          const uint32_t a0 = base + s * T::STAGE_BYTES;
          const uint32_t b0 = a0 + T::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {   // 32 of K: 32 bytes K-major, 32 rows MN-major
            const uint64_t ad = make_sdesc_k_sw128(a0 + kk * 32, 1024);
            const uint64_t bd = DGRAD ? make_sdesc_mn_sw128(b0 + kk * 4096, 16384, 1024)
                                      : make_sdesc_k_sw128(b0 + kk * 32, 1024);
            if constexpr (kPair) umma_e4m3_pair(d, ad, bd, idesc, kk != 0);
            else umma_e4m3(d, ad, bd, idesc, kk != 0);
          }
          if constexpr (kPair) {
            umma_commit_pair_mc(bar_empty(s), 0x3);
            umma_commit_pair_mc(bar_tfull(buf), 0x3);
          } else {
            umma_commit(bar_empty(s));
            umma_commit(bar_tfull(buf));
          }
        }
      }
      // every MMA issued must complete before the tensor memory is freed
      if constexpr (kPair) umma_commit_pair_mc(bar_drain, 0x1); else umma_commit(bar_drain);
      wait_bounded(bar_drain, 0u, wc, kSiteDrainMma, false);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                       // TMEM lane quadrant this warp may read
    const int h = (warp - 2) >> 2;                // half of the tile's columns
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t slab = base + T::OFF_OUT + (warp - 2) * 4096;
    uint8_t* gslab = gbase + T::OFF_OUT + (warp - 2) * 4096;
    uint32_t cnt = 0;
    bool ok = true;
    for (int t = unit0; ok && t < a.num_tiles; t += units) {
      int tm, tn;
      tile_of(t, a, tm, tn);
      const int row0 = tm * T::TM + static_cast<int>(rank) * kBM + q * 32;
      const int row = row0 + lane;
      const int col0 = tn * BN + h * T::NC;
      // this row's scales, and the weight's for this half's block of columns
      // (a half lies within one block); rows and blocks outside count zero
      const bool row_ok = row < a.m;
      const float* sa = a.sa + static_cast<int64_t>(row_ok ? row : 0) * a.num_kb;
      const bool col_ok = col0 < a.n;
      const float* sw = a.sw + static_cast<int64_t>(col_ok ? col0 / 128 : 0) * a.sw_n;
      const bool live = row_ok && col_ok;
      float2 acc[T::NC / 2];
#pragma unroll
      for (int i = 0; i < T::NC / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      float ra = live ? __ldg(sa) : 0.0f, rw = live ? __ldg(sw) : 0.0f;
      for (int k = 0; k < a.num_kb; ++k, ++cnt) {
        const float2 s2 = dup2(ra * rw);
        if (live && k + 1 < a.num_kb) {   // the next block's scales, ahead of the wait
          ra = __ldg(sa + k + 1);
          rw = __ldg(sw + static_cast<int64_t>(k + 1) * a.sw_k);
        }
        const int buf = cnt % T::NBUF;
        const bool good = wait_bounded(bar_tfull(buf), (cnt / T::NBUF) & 1u, wc, kSiteEpiTmemFull);
        if (!__all_sync(0xffffffffu, good)) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t taddr = tmem_base + lane_addr + buf * BN + h * T::NC;
#pragma unroll
        for (int c = 0; c < T::NC / 32; ++c) {
          uint32_t r[32];
          tmem_ld_x32(taddr + 32 * c, r);
          tmem_ld_wait();
          if (c == T::NC / 32 - 1) {   // this warp has read its part of the buffer
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              if constexpr (kPair) mbar_arrive_cluster(mapa_shared(bar_tempty(buf), 0));
              else mbar_arrive(bar_tempty(buf));
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] = fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                   s2, acc[c * 16 + i]);
        }
      }
      if (!ok) break;
      // store through this warp's slab: boxes of 32 rows x 128 bytes
      if (row0 < a.m && col_ok) {
        if (a.out_fp32) {
#pragma unroll
          for (int c = 0; c < T::NC / 32; ++c) {
            if (col0 + 32 * c >= a.n) break;
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x = acc[c * 16 + 2 * i], y = acc[c * 16 + 2 * i + 1];
              *reinterpret_cast<float4*>(gslab + sw128_off(lane, i)) = make_float4(x.x, x.y, y.x, y.y);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&a.out, col0 + 32 * c, row0, slab);
              bulk_commit_group();
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < T::NC / 64; ++c) {
            if (col0 + 64 * c >= a.n) break;
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2* x = acc + c * 32 + 4 * i;
              *reinterpret_cast<uint4*>(gslab + sw128_off(lane, i)) =
                  make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                             pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&a.out, col0 + 64 * c, row0, slab);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  if constexpr (kPair) {
    if (*abort_flag) {   // let copies in flight into this CTA land (see forge_gemm.cuh)
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

template <int CG, int BN, bool DGRAD>
cudaError_t launch_t(const B128Args& a, int num_sms, cudaStream_t stream) {
  using T = Traits8<CG, BN>;
  auto kern = gemm_b128_kernel<CG, BN, DGRAD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       T::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(kThreads8, 1, 1);
  lc.dynamicSmemBytes = T::SMEM_ALLOC;
  lc.stream = stream;
  const int units = num_sms / CG;
  lc.gridDim = dim3(CG * (a.num_tiles < units ? a.num_tiles : units), 1, 1);
  return cudaLaunchKernelEx(&lc, kern, a);
}

}  // namespace

cudaError_t launch_gemm_b128(const B128Config& c, bool dgrad, const B128Args& a, int num_sms,
                             cudaStream_t stream) {
  if (c.cg == 1 && c.bn == 128)
    return dgrad ? launch_t<1, 128, true>(a, num_sms, stream)
                 : launch_t<1, 128, false>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace forge

// The forward product of a linear layer in 16 bits with its epilogue:
//   Z = X W^T + bias,   Y = residual + drop(act(Z) * mul).
// X [m, k] and W [n, k] are both K-major; a tile's whole reduction stays in tensor
// memory (fp32), and the epilogue works on it while the next tile's products run in
// the other accumulator.
//
// Warp roles (384 threads): warp 0 loads operand stages 64 deep with TMA, warp 1
// issues the MMAs, warps 4-11 are the epilogue (two per TMEM lane quadrant, each half
// of the tile's columns).  An epilogue warp works on boxes of 32 rows x 64 columns:
// residual and mul come into its two slabs of shared memory by TMA, ahead of the
// accumulator, and Y and Z leave from the same slabs, whose every 16 bytes one thread
// reads before it writes them.  Every wait is bounded, as in forge_gemm.cuh.
#include <cuda_bf16.h>

#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_layer.cuh"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

constexpr int kThreadsL = 384;
constexpr int kEpiWarpsL = 8;
constexpr int kSmemMaxL = 232448;   // dynamic shared memory of one CTA (227 KB)

// CG CTAs compute a (128 CG) x BN tile; a CTA loads its 128 rows of X and BN / CG
// rows of W per stage.
template <int CG, int BN>
struct TraitsL {
  static constexpr int TM = kBM * CG;
  static constexpr int BNL = BN / CG;
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int STAGE_BYTES = A_BYTES + BNL * 128;
  static constexpr int SLAB = 4096;                      // 32 rows x 128 bytes
  static constexpr int OUT_BYTES = kEpiWarpsL * 2 * SLAB;
  static constexpr int STAGES = 5;
  static constexpr int GROUPS = BN / 128;                // boxes of 64 columns per epilogue warp
  static constexpr int TMEM_COLS = 2 * BN;               // two accumulators
  static constexpr int OFF_OUT = STAGES * STAGE_BYTES;
  static constexpr int OFF_BARS = OFF_OUT + OUT_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 4 + 1 + kEpiWarpsL;
  static constexpr int OFF_TMEM = OFF_BARS + 8 * NUM_BARS;
  static constexpr int SMEM_USED = OFF_TMEM + 8;
  static constexpr int SMEM_ALLOC = SMEM_USED + 1024 < kSmemMaxL ? SMEM_USED + 1024 : kSmemMaxL;
  static_assert(SMEM_USED <= kSmemMaxL, "shared memory budget exceeded");
};

// Tile order: groups of group_m tile rows, column by column inside a group, so that
// the tiles in flight share operands in L2.
__device__ __forceinline__ void tile_of(int t, const LinearArgs& a, int& tm, int& tn) {
  const int per = a.group_m * a.tiles_n;
  const int g = t / per, r = t - g * per;
  const int m0 = g * a.group_m;
  const int gm = min(a.group_m, a.tiles_m - m0);
  tn = r / gm;
  tm = m0 + r - tn * gm;
}

template <int CG, int BN>
__global__ void __launch_bounds__(kThreadsL, 1)
    gemm_linear_kernel(const __grid_constant__ LinearArgs a) {
  using T = TraitsL<CG, BN>;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  if (base - raw + T::SMEM_USED > T::SMEM_ALLOC) {   // uniform: nothing has started
    grid_dependency_wait();   // the launch after this one may rely on those before it
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
  auto bar_tempty = [&](int b) { return bars + 8u * (2 * T::STAGES + 2 + b); };
  const uint32_t bar_drain = bars + 8u * (2 * T::STAGES + 4);
  auto bar_in = [&](int w) { return bars + 8u * (2 * T::STAGES + 5 + w); };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM + 4);
  const WaitCtx wc{abort_flag, a.err, a.err_site, a.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull(b), 1);
      mbar_init(bar_tempty(b), CG * kEpiWarpsL);
    }
    mbar_init(bar_drain, 1);
    for (int w = 0; w < kEpiWarpsL; ++w) mbar_init(bar_in(w), 1);
    *abort_flag = 0u;
    fence_mbarrier_init();
    drop_first_arrival(a.drop_first_arrival, bar_full(0));
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.a);
    tma_prefetch_desc(&a.b);
    tma_prefetch_desc(&a.y);
  }
  if constexpr (kPair) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(base + T::OFF_TMEM, T::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(base + T::OFF_TMEM, T::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM);

  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        const uint64_t pol = l2_policy_evict_normal();
        uint32_t s = 0, ph = 0;   // next stage, and its phase
        uint32_t armed = 0;       // stages filled so far, at most STAGES
        bool ok = true;
        for (int t = unit0; ok && t < a.num_tiles; t += units) {
          int tm, tn;
          tile_of(t, a, tm, tn);
          const int ya = tm * T::TM + static_cast<int>(rank) * kBM;
          const int yb = tn * BN + static_cast<int>(rank) * T::BNL;
          for (int k = 0; k < a.num_kb; ++k) {
            if (!wait_bounded(bar_empty(s), ph ^ 1u, wc, kSiteProducerEmpty)) { ok = false; break; }
            const uint32_t dst = base + s * T::STAGE_BYTES;
            if constexpr (kPair) {
              const uint32_t fb = mapa_shared(bar_full(s), 0);
              if (leader) mbar_arrive_expect_tx(bar_full(s), 2 * T::STAGE_BYTES);
              tma_load_2d_pair(dst, &a.a, k * 64, ya, fb, pol);
              tma_load_2d_pair(dst + T::A_BYTES, &a.b, k * 64, yb, fb, pol);
            } else {
              mbar_arrive_expect_tx(bar_full(s), T::STAGE_BYTES);
              tma_load_2d(dst, &a.a, k * 64, ya, bar_full(s), pol);
              tma_load_2d(dst + T::A_BYTES, &a.b, k * 64, yb, bar_full(s), pol);
            }
            if (armed < T::STAGES) ++armed;
            if (++s == T::STAGES) { s = 0; ph ^= 1u; }
          }
        }
        // Before the CTA can exit, every stage's last release has to arrive (on a pair
        // the leader's MMAs signal it from afar); after a timeout, every load that is
        // under way has to land (a pair's complete on the leader's barriers).
        for (uint32_t i = 0; i < armed; ++i) {
          if (s == 0) { s = T::STAGES; ph ^= 1u; }
          --s;
          const bool freed = ok && wait_bounded(bar_empty(s), ph, wc, kSiteDrainOperands);
          if (!freed && leader) wait_bounded(bar_full(s), ph, wc, kSiteDrainOperands, false);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp walks the stages, so that addresses and descriptors stay in
      // uniform registers, and one elected lane issues.
      if (leader) {
        constexpr uint32_t idesc = make_idesc_bf16(T::TM, BN, false, false);
        const uint64_t ad0 = make_sdesc_k_sw128(base, 1024);
        const uint64_t bd0 = make_sdesc_k_sw128(base + T::A_BYTES, 1024);
        const bool issue = elect_one();
        uint32_t s = 0, ph = 0, buf = 0, bph = 1;
        bool ok = true;
        for (int t = unit0; ok && t < a.num_tiles; t += units) {
          ok = __all_sync(0xffffffffu,
                          wait_bounded(bar_tempty(buf), bph, wc, kSiteMmaTmemEmpty));
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t d = tmem_base + buf * BN;
#pragma unroll 1
          for (int k = 0; k < a.num_kb; ++k) {
            ok = __all_sync(0xffffffffu, wait_bounded(bar_full(s), ph, wc, kSiteMmaFull));
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t ad = ad0 + s * (T::STAGE_BYTES >> 4);
            const uint64_t bd = bd0 + s * (T::STAGE_BYTES >> 4);
            if (issue) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {   // 16 of K: 32 bytes
                if constexpr (kPair)
                  umma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
                else
                  umma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
              }
              if constexpr (kPair) umma_commit_pair_mc(bar_empty(s), 0x3);
              else umma_commit(bar_empty(s));
            }
            if (++s == T::STAGES) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          if (issue) {
            if constexpr (kPair) umma_commit_pair_mc(bar_tfull(buf), 0x3);
            else umma_commit(bar_tfull(buf));
          }
          if (++buf == 2) { buf = 0; bph ^= 1u; }
        }
        // every MMA issued must complete before the tensor memory is freed
        if (issue) {
          if constexpr (kPair) umma_commit_pair_mc(bar_drain, 0x1); else umma_commit(bar_drain);
        }
        wait_bounded(bar_drain, 0u, wc, kSiteDrainMma, false);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                       // TMEM lane quadrant this warp may read
    const int h = (warp - 4) >> 2;                // half of the tile's columns
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t slab_y = base + T::OFF_OUT + (warp - 4) * 2 * T::SLAB;
    const uint32_t slab_z = slab_y + T::SLAB;
    uint8_t* gy = gbase + T::OFF_OUT + (warp - 4) * 2 * T::SLAB;
    uint8_t* gz = gy + T::SLAB;
    const uint32_t bin = bar_in(warp - 4);
    const uint64_t pol = l2_policy_evict_first();
    const bool loads = a.e.mul || a.e.residual;
    const uint32_t in_bytes = (a.e.mul ? T::SLAB : 0) + (a.e.residual ? T::SLAB : 0);
    const uint64_t offset = drop_offset(a.e.drop);
    const int64_t nv = a.n / 8;

    // The boxes of this warp in order: group g of tile t.  (Those outside the matrix
    // are passed over by loads, arithmetic and stores alike.)
    auto place = [&](int t, int g, int& row0, int& col) {
      int tm, tn;
      tile_of(t, a, tm, tn);
      row0 = tm * T::TM + static_cast<int>(rank) * kBM + q * 32;
      col = tn * BN + h * (BN / 2) + g * 64;
      return row0 < a.m && col < a.n;
    };
    auto next = [&](int& t, int& g) {
      if (++g == T::GROUPS) { g = 0; t += units; }
    };
    // loads the inputs of the next box there is from (t, g) on
    auto ask = [&](int t, int g) {
      int row0, col;
      while (t < a.num_tiles && !place(t, g, row0, col)) next(t, g);
      if (t >= a.num_tiles) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bin, in_bytes);
        if (a.e.residual) tma_load_2d(slab_y, &a.residual, col, row0, bin, pol);
        if (a.e.mul) tma_load_2d(slab_z, &a.mul, col, row0, bin, pol);
      }
      return true;
    };
    uint32_t buf = 0, bph = 0, iph = 0;
    bool ok = true, asked = loads && ask(unit0, 0);
    for (int t = unit0; ok && t < a.num_tiles; t += units) {
      ok = __all_sync(0xffffffffu,
                      wait_bounded_inline(bar_tfull(buf), bph, wc, kSiteEpiTmemFull));
      if (!ok) break;
      tc_fence_after_sync();
      auto release = [&]() {   // this warp has read its part of the accumulator
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_cluster_relaxed(mapa_shared(bar_tempty(buf), 0));
          else mbar_arrive(bar_tempty(buf));
        }
      };
#pragma unroll 1
      for (int g = 0; g < T::GROUPS; ++g) {
        const bool last = g == T::GROUPS - 1;
        int row0, col;
        if (!place(t, g, row0, col)) {
          if (last) release();
          continue;
        }
        if (loads) {
          ok = __all_sync(0xffffffffu, wait_bounded_inline(bin, iph, wc, kSiteEpiSlotFull));
          if (!ok) break;
          asked = false;
          iph ^= 1u;
        } else {   // the slabs are free once the stores before have read them
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        }
        const uint32_t taddr = tmem_base + lane_addr + buf * BN + h * (BN / 2) + g * 64;
        const uint64_t block0 = static_cast<uint64_t>(row0 + lane) * nv + col / 8;
        // an fp32 box holds half the columns, in the place of all the residual's
        uint4 later[4];
        if (a.e.y_fp32 && a.e.residual) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            later[c] = *reinterpret_cast<const uint4*>(gy + sw128_off(lane, 4 + c));
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          tmem_ld_x32(taddr + 32 * half, r);
          tmem_ld_wait();
          if (last && half == 1) release();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int cc = 4 * half + c;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[8 * c + k]);
            const uint32_t at = sw128_off(lane, cc);
            uint4 mul = make_uint4(0, 0, 0, 0), res = mul;
            if (a.e.mul) mul = *reinterpret_cast<const uint4*>(gz + at);
            if (a.e.residual)
              res = a.e.y_fp32 && half == 1 ? later[c] : *reinterpret_cast<const uint4*>(gy + at);
            // columns past the last: the bias is not read there
            const int64_t bc = col + 8 * cc < a.n ? col + 8 * cc : 0;
            const uint4 z = epilogue8(v, a.e, bc, mul, res, offset, block0 + cc);
            if (a.e.z) *reinterpret_cast<uint4*>(gz + at) = z;
            if (!a.e.y_fp32) {
              *reinterpret_cast<uint4*>(gy + at) = pack8(v);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) r[8 * c + k] = __float_as_uint(v[k]);
            }
          }
          if (a.e.y_fp32 && col + 32 * half < a.n) {   // a box of 32 columns
            if (half == 1) {
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(gy + sw128_off(lane, i)) =
                  make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&a.y, col + 32 * half, row0, slab_y);
              bulk_commit_group();
            }
          }
        }
        if (!a.e.y_fp32 || a.e.z) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!a.e.y_fp32) tma_store_2d(&a.y, col, row0, slab_y);
            if (a.e.z) tma_store_2d(&a.z, col, row0, slab_z);
            bulk_commit_group();
          }
        }
        if (loads) {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          int nt = t, ng = g;
          next(nt, ng);
          asked = ask(nt, ng);
        }
      }
      if (!ok) break;
      if (++buf == 2) { buf = 0; bph ^= 1u; }
    }
    if (asked) wait_bounded(bin, iph, wc, kSiteDrainState, false);   // after a timeout
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  grid_dependency_trigger();
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
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, T::TMEM_COLS);
    else tmem_dealloc(tmem_base, T::TMEM_COLS);
  }
}

template <int CG, int BN>
cudaError_t launch_t(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  using T = TraitsL<CG, BN>;
  auto kern = gemm_linear_kernel<CG, BN>;
  // the units that can be resident: CTAs, or (known to the occupancy) pairs
  static PerDevice resident;
  int units = 0;
  const cudaError_t e = resident.get(&units, [&](int* n) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         T::SMEM_ALLOC);
    *n = num_sms;
    if (CG == 1 || r != cudaSuccess) return r;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(2 * (num_sms / 2), 1, 1);
    lc.blockDim = dim3(kThreadsL, 1, 1);
    lc.dynamicSmemBytes = T::SMEM_ALLOC;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    r = cudaOccupancyMaxActiveClusters(n, kern, &lc);
    if (r == cudaSuccess && *n <= 0) r = cudaErrorInvalidConfiguration;
    *n = *n < num_sms / 2 ? *n : num_sms / 2;
    return r;
  });
  if (e != cudaSuccess) return e;
  return launch_chained(kern, CG * (a.num_tiles < units ? a.num_tiles : units), kThreadsL,
                        T::SMEM_ALLOC, CG == 2 ? 2 : 0, stream, a);
}

}  // namespace

cudaError_t launch_gemm_linear(const LinearConfig& c, const LinearArgs& a, int num_sms,
                               cudaStream_t stream) {
  if (c.cg == 1 && c.bn == 128) return launch_t<1, 128>(a, num_sms, stream);
  if (c.cg == 2 && c.bn == 256) return launch_t<2, 256>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace forge

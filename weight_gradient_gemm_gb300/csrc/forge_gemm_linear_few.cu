// The forward product of a linear layer in 16 bits (see forge_gemm_linear.cu) for few
// tokens, where reading the weight is all the time there is.
//
// As in the 8-bit form (forge_gemm_b128_few.cu) the operands change places: 128
// outputs lie along the MMA's M and the tokens along its N, 16 to 128 of them (more
// tokens: several tiles of 128), and the reduction is split over the CTAs of a cluster (up
// to 8), which send slices of their fp32 sums to the CTAs that own them through distributed
// shared memory; the owners add them in a fixed order, apply the epilogue and store.  One
// launch, no workspace, the same result on every run.
//
// Warp roles: 0 loads (TMA), 1 issues the MMAs, from 4 on a warp takes the 32 outputs
// of a TMEM lane quadrant and up to 32 tokens; all threads join in the end.  Every
// wait is bounded.
//
// Bound by the weight's bytes: 4096 -> 14336 (117 MB, 17.3 us at 6.79 TB/s) 18.8 us for
// one token (19.1 gated), 19.2 for 16, 21.3 for 64, 23.1 for 128; 4096 -> 4096 (4.9) 8.6, 9.1,
// 10.3 and 11.8, of which about 3.5 are a launch from its first load to its last store.  More
// tokens: by the operands at 64 bytes a cycle an SM (512 cycles a step of 128 x 128) and
// the exchange of shares: 300 tokens, 4096 -> 1024, 9.7 us; 200, 14336 -> 4096, 31.1.  The
// shares go out as [token][output], 128 bytes a warp and store; as [output][token] in
// stores of 16 bytes a lane the exchange cost more (333 tokens, 1032 -> 520, with everything,
// 9.3 us, 7.9 so).
#include <cuda_bf16.h>

#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_layer.cuh"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

template <int NT>
struct FewL {
  static constexpr int EPI = NT <= 32 ? 4 : NT / 8;     // epilogue warps
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int NC = NT <= 32 ? NT : 32;         // tokens per epilogue thread
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int STAGE_BYTES = A_BYTES + NT * 128;
  // Operand stages: as many as let two CTAs share an SM, or, where the grid has no
  // more than one CTA for each, as many as fit.
  static constexpr int STAGES = NT <= 16 ? 6 : (NT == 32 ? 5 : 4);
  static constexpr int DEEP = NT <= 16 ? 12 : (NT == 32 ? 11 : (NT == 64 ? 9 : 7));
  static constexpr int ACC_COLS = NT < 32 ? 32 : NT;
  // Shared memory from a 1024-aligned base: barriers (the most there can be), abort
  // flag, stages.  The shares, one tile of fp32 sums, take the stages' place once the
  // products of all the cluster's CTAs have run.
  static constexpr int NUM_BARS = 2 * DEEP + 5;
  static constexpr int OFF_TMEM = 8 * NUM_BARS;
  static constexpr int OFF_STAGES = 1024;
  static constexpr int smem(int stages) { return OFF_STAGES + stages * STAGE_BYTES + 1024; }
  static_assert(OFF_TMEM + 8 <= OFF_STAGES, "barriers");
  static_assert(NT * kBM * 4 <= STAGES * STAGE_BYTES, "shares");
  static_assert(NT > 64 || 2 * smem(STAGES) <= 228 * 1024 - 2 * 1024, "two CTAs an SM");
  static_assert(smem(DEEP) <= 232448, "shared memory budget");
};

// F32: Y in fp32, whose sums are added up in registers a few steps at a time (see
// kLinearChunk), from two accumulators in turn.  (128 tokens, 4096 -> 14336, 24.4 us; Y in
// bf16, one sum, 23.1.  A kernel of its own: as a loop of one turn it cost Y in bf16 3 to 6 %.)
template <int NT, bool F32>
__global__ void __launch_bounds__(FewL<NT>::THREADS, NT <= 64 ? 2 : 1)
    gemm_linear_few_kernel(const __grid_constant__ LinearArgs a) {
  using T = FewL<NT>;
  constexpr int TMEM_COLS = (F32 ? 2 : 1) * T::ACC_COLS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  // the same offset in every CTA of the cluster: remote stores use it
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = a.splits;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / splits;
  const int tile = unit / a.tiles_m, t0 = (unit - tile * a.tiles_m) * NT;   // outputs, first token
  const int m = min(a.m - t0, NT);
  // this CTA's steps of the reduction
  const int kb = b128_first_block(rank, splits, a.num_kb);
  const int ke = b128_first_block(rank + 1, splits, a.num_kb);

  const uint32_t stages = a.stages;
  const uint32_t bars = base, stage0 = base + T::OFF_STAGES;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (T::DEEP + s); };
  const uint32_t bar_done = bars + 8u * (2 * T::DEEP);   // all products have run
  auto bar_acc = [&](int b) { return bars + 8u * (2 * T::DEEP + 1 + b); };    // an accumulator's
  auto bar_free = [&](int b) { return bars + 8u * (2 * T::DEEP + 3 + b); };   // has been read
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM + 4);
  const WaitCtx wc{abort_flag, a.err, a.err_site, a.timeout_ns};
  // A weight that is read once passes through L2 as the first to leave it (one token,
  // 4096 -> 14336, when only that was changed: 22.7 -> 19.9 us).
  const uint64_t wpol = a.tiles_m > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
  const uint64_t xpol = l2_policy_evict_last();

  // Warp 0 sets up the barriers while warp 1 takes the tensor memory; one block
  // barrier covers both.
  if (warp == 0) {
    for (int i = lane; i < T::NUM_BARS; i += 32)
      mbar_init(bars + 8u * i, i >= 2 * T::DEEP + 3 ? T::EPI : 1);
    if (lane == 0) *abort_flag = 0u;
    fence_mbarrier_init();
    __syncwarp();
    if (lane == 0) drop_first_arrival(a.drop_first_arrival, bar_full(0));
  } else if (warp == 1) {
    tmem_alloc(base + T::OFF_TMEM, TMEM_COLS);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  // While the kernel before still runs, the weight's first steps are asked for as far
  // as L2, where all writes meet (see forge_gemm_b128_few.cu): calls back to back on one
  // token, 4096 -> 14336, gated, 19.1 us with 16 steps ahead, 20.7 with eight, 21.6 with none.
  if (warp == 0 && lane == 0) {
    for (int k = kb; k < min(ke, kb + 16); ++k) tma_prefetch_l2_2d(&a.b, k * 64, tile * 128);
  }
  grid_dependency_wait();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM);

  // The outputs that this CTA owns, eight neighbouring ones at a time: token e >> shift.
  // The first ones' inputs are asked for now, under the reduction.
  const int slice = kBM / splits;   // splits divides 128
  const int shift = 31 - __clz(slice >> 3), total = m << shift;
  const int64_t nv = a.n / 8;
  auto place = [&](int e, int& t, int& j, int64_t& at) {
    t = e >> shift;
    j = (e - (t << shift)) * 8;
    const int o = tile * 128 + rank * slice + j;
    at = static_cast<int64_t>(t0 + t) * nv + o / 8;
    return e < total && o < a.n;
  };
  uint4 mul0 = make_uint4(0, 0, 0, 0), res0 = mul0;
  uint64_t offset = 0;
  if (warp != 0 && warp != 1) {
    int t, j;
    int64_t at;
    if (place(threadIdx.x, t, j, at)) {
      if (a.e.mul) mul0 = reinterpret_cast<const uint4*>(a.e.mul)[at];
      if (a.e.residual) res0 = reinterpret_cast<const uint4*>(a.e.residual)[at];
    }
  }

  float acc[T::NC];   // epilogue threads: one output, NC tokens
  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, armed = 0;   // next stage, its phase, stages in use
      for (int k = kb; k < ke; ++k) {
        if (!wait_bounded(bar_empty(s), ph ^ 1u, wc, kSiteProducerEmpty)) break;
        const uint32_t dst = stage0 + s * T::STAGE_BYTES;
        mbar_arrive_expect_tx(bar_full(s), T::STAGE_BYTES);
        tma_load_2d(dst, &a.b, k * 64, tile * 128, bar_full(s), wpol);
        tma_load_2d(dst + T::A_BYTES, &a.a, k * 64, t0, bar_full(s), xpol);
        if (armed < stages) ++armed;
        if (++s == stages) { s = 0; ph ^= 1u; }
      }
      for (uint32_t i = 0; i < armed; ++i) {   // the last load of every stage lands
        if (s == 0) { s = stages; ph ^= 1u; }
        --s;
        wait_bounded(bar_full(s), ph, wc, kSiteDrainOperands, false);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = make_idesc_bf16(128, NT, false, false);
    const uint64_t ad0 = make_sdesc_k_sw128(stage0, 1024);
    const uint64_t bd0 = make_sdesc_k_sw128(stage0 + T::A_BYTES, 1024);
    const bool issue = elect_one();
    uint32_t s = 0, ph = 0, buf = 0, bph = 1;
    for (int k0 = kb, k1; k0 < ke; k0 = k1) {
      k1 = F32 ? min(ke, k0 + a.chunk) : ke;
      if (F32 && !__all_sync(0xffffffffu, wait_bounded(bar_free(buf), bph, wc, kSiteMmaTmemEmpty)))
        break;
      if (F32) tc_fence_after_sync();
      bool ok = true;
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        ok = __all_sync(0xffffffffu, wait_bounded(bar_full(s), ph, wc, kSiteMmaFull));
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t ad = ad0 + s * (T::STAGE_BYTES >> 4), bd = bd0 + s * (T::STAGE_BYTES >> 4);
        if (issue) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem_base + buf * T::ACC_COLS, ad + 2 * kk, bd + 2 * kk, idesc, (k - k0) | kk);
          umma_commit(bar_empty(s));
        }
        if (++s == stages) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (F32) {
        if (issue) umma_commit(bar_acc(buf));
        if (++buf == 2) { buf = 0; bph ^= 1u; }
      }
    }
    if (issue) umma_commit(bar_done);
    wait_bounded(bar_done, 0u, wc, kSiteDrainMma, false);
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t tcol = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + h * T::NC;
    auto sums = [&](uint32_t from, auto&& take) {   // take(i, the i-th token's)
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < T::NC / 16; ++c) {
        uint32_t r[16];
        tmem_ld_x16(from + 16 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) take(16 * c + i, __uint_as_float(r[i]));
      }
    };
#pragma unroll
    for (int i = 0; i < T::NC; ++i) acc[i] = 0.0f;   // (a CTA without steps adds nothing)
    if constexpr (F32) {
      uint32_t buf = 0, bph = 0;
#pragma unroll 1
      for (int k0 = kb; k0 < ke; k0 += a.chunk) {
        if (!__all_sync(0xffffffffu, wait_bounded(bar_acc(buf), bph, wc, kSiteEpiTmemFull))) break;
        sums(tcol + buf * T::ACC_COLS, [&](int i, float v) { acc[i] += v; });
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free(buf));
        if (++buf == 2) { buf = 0; bph ^= 1u; }
      }
    } else if (__all_sync(0xffffffffu, wait_bounded(bar_done, 0u, wc, kSiteEpiTmemFull)) &&
               ke > kb) {
      sums(tcol, [&](int i, float v) { acc[i] = v; });
    }
  }
  tc_fence_before_sync();

  // ------------------------------------------------------------ join and store
  grid_dependency_trigger();
  constexpr uint32_t off_part = T::OFF_STAGES;
  // every CTA's products have run and its loads have landed (warps 0 and 1 waited)
  if (splits > 1) cluster_sync_all(); else __syncthreads();
  if (warp >= 4) {
    const int h = (warp - 4) >> 2, o = (warp & 3) * 32 + lane;
    // [rank of the sender][token][output of the slice]
    const uint32_t to = base + off_part + 4u * ((rank * NT + h * T::NC) * slice + o % slice);
    const uint32_t dst = splits > 1 ? mapa_shared(to, o / slice) : 0u;
    float* here = reinterpret_cast<float*>(gbase + (to - base));
#pragma unroll
    for (int i = 0; i < T::NC; ++i)
      if (h * T::NC + i < m) {
        if (splits > 1) st_cluster_f32(dst + 4u * i * slice, acc[i]);
        else here[i * slice] = acc[i];
      }
  }
  if (splits > 1) cluster_sync_all(); else __syncthreads();
  if (a.e.drop.threshold) offset = drop_offset(a.e.drop);
  if (!*abort_flag) {
    const float* part = reinterpret_cast<const float*>(gbase + off_part);
    for (int e = threadIdx.x; e < total; e += T::THREADS) {
      int t, j;
      int64_t at;
      if (!place(e, t, j, at)) continue;
      if (e != static_cast<int>(threadIdx.x) || warp < 2) {
        if (a.e.mul) mul0 = reinterpret_cast<const uint4*>(a.e.mul)[at];
        if (a.e.residual) res0 = reinterpret_cast<const uint4*>(a.e.residual)[at];
      }
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      for (int z = 0; z < splits; ++z) {
        const float4* p = reinterpret_cast<const float4*>(part + (z * NT + t) * slice + j);
        const float4 x = p[0], y = p[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      if (a.e.bias) {
        float b[8];
        load_bias8(a.e.bias, a.e.bias_bf16, tile * 128 + rank * slice + j, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
      }
      uint4 z;
      with_act(a.e.act, [&](auto act) {
        z = epilogue8<decltype(act)::value>(v, a.e, mul0, res0, offset, static_cast<uint64_t>(at));
      });
      if (a.e.z) reinterpret_cast<uint4*>(a.e.z)[at] = z;
      if constexpr (F32) {
        float4* y = reinterpret_cast<float4*>(a.e.y) + 2 * at;
        y[0] = make_float4(v[0], v[1], v[2], v[3]);
        y[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        reinterpret_cast<uint4*>(a.e.y)[at] = pack8(v);
      }
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// The clusters of `splits` CTAs that can be resident at once with as many stages as fit.
template <int NT, bool F32>
cudaError_t resident(int splits, int num_sms, int* n) {
  using T = FewL<NT>;
  static PerDevice kept[4];
  auto kern = gemm_linear_few_kernel<NT, F32>;
  return kept[splits == 1 ? 0 : (splits == 2 ? 1 : (splits == 4 ? 2 : 3))].get(n, [&](int* v) {
    cudaError_t r =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    *v = num_sms;
    if (splits == 1 || r != cudaSuccess) return r;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(num_sms / splits * splits, 1, 1);
    lc.blockDim = dim3(T::THREADS, 1, 1);
    lc.dynamicSmemBytes = T::smem(T::DEEP);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    r = cudaOccupancyMaxActiveClusters(v, kern, &lc);
    if (r == cudaSuccess && *v <= 0) r = cudaErrorInvalidConfiguration;
    return r;
  });
}

template <int NT, bool F32>
cudaError_t launch_t(LinearArgs a, int num_sms, cudaStream_t stream) {
  using T = FewL<NT>;
  int clusters = 0;
  const cudaError_t e = resident<NT, F32>(a.splits, num_sms, &clusters);
  if (e != cudaSuccess) return e;
  const int steps = (a.num_kb + a.splits - 1) / a.splits;
  a.stages = a.num_tiles <= clusters ? T::DEEP : T::STAGES;
  if (steps < a.stages) a.stages = steps < 2 ? 2 : steps;
  // (the shares take the stages' place)
  while (a.stages * T::STAGE_BYTES < NT * kBM * 4) ++a.stages;
  return launch_chained(gemm_linear_few_kernel<NT, F32>, a.num_tiles * a.splits, T::THREADS,
                        T::smem(a.stages), a.splits > 1 ? a.splits : 0, stream, a);
}

template <int NT>
cudaError_t launch_nt(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.e.y_fp32 ? launch_t<NT, true>(a, num_sms, stream) : launch_t<NT, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t linear_few_clusters(int nt, int splits, int num_sms, int* n) {
  switch (nt) {
    case 16: return resident<16, false>(splits, num_sms, n);
    case 32: return resident<32, false>(splits, num_sms, n);
    case 64: return resident<64, false>(splits, num_sms, n);
    case 128: return resident<128, false>(splits, num_sms, n);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_gemm_linear_few(int nt, const LinearArgs& a, int num_sms, cudaStream_t stream) {
  switch (nt) {
    case 16: return launch_nt<16>(a, num_sms, stream);
    case 32: return launch_nt<32>(a, num_sms, stream);
    case 64: return launch_nt<64>(a, num_sms, stream);
    case 128: return launch_nt<128>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace forge

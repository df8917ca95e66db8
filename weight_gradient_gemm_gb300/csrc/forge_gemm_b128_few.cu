// The 8-bit products of a linear layer (see forge_gemm_b128.cu) for few tokens,
// where reading the weight is all the time there is:
//   out[t][o] = sum_b (sx[t][b] sw(o, b)) P_b[t][o].
//
// The operands change places: 128 outputs (rows of the weight, or its columns
// for the input gradient) lie along the MMA's M and the tokens along its N, 16
// to 128 of them, so a block's accumulator is as small as the tokens are few
// and the weight's scale is one number per block.  To keep every SM loading,
// the reduction is split over the CTAs of a cluster (up to 8): each walks its
// share of the blocks, then sends slices of its partial sums to the CTAs that
// own them, through distributed shared memory, and the owners add the shares
// in a fixed order and store.  One launch, no workspace, the same result on
// every run.
//
// Bound by the weight's bytes and, below about 10 MB, by the 3.5 us that a launch
// takes from its first load to its last store.  4096 -> 14336 (58.7 MB, 8.7 us at
// 6.79 TB/s): 12.8 us a call for one token, 13.4 for 16, 14.8 for 64, 17.3 for 128,
// where every CTA reads all the tokens again (117 MB through L2; without any adding
// up 2 us less); 4096 -> 4096 (2.5 us): 6.3, 6.9, 8.0 and 9.4; the input gradient
// 14336 -> 4096: 13.4, 13.6, 14.4 and 17.9.  4096 -> 128256, with more tiles than SMs
// and two CTAs on each (525 MB, 77.4 us): 86.6 for one token, 90.9 for 32.
//
// Warp roles: 0 loads (TMA), 1 issues the MMAs, 2 multiplies the scales, from
// 4 on the epilogue (the 32 outputs of a TMEM lane quadrant and up to 32
// tokens a warp).  Every wait is bounded.
#include <cuda_bf16.h>

#include "forge_b128.cuh"
#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

template <int NT>
struct Few {
  static constexpr int EPI = NT <= 32 ? 4 : NT / 8;     // epilogue warps
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int NC = NT <= 32 ? NT : 32;         // tokens per epilogue thread
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int STAGE_BYTES = A_BYTES + NT * 128;
  // Operand stages: as many as let two CTAs share an SM, or, where the grid
  // has no more than one CTA for each, as many as fit.
  static constexpr int STAGES = NT <= 16 ? 5 : 4;
  static constexpr int DEEP = NT <= 16 ? 11 : (NT == 32 ? 9 : (NT == 64 ? 8 : 6));
  static constexpr int NBUF = NT <= 32 ? 8 : 4;         // TMEM accumulators
  static constexpr int TMEM_COLS = NT * NBUF;           // two CTAs fit an SM up to 64 tokens
  static constexpr int SC_BATCH = 8;
  static constexpr int SC_BYTES = 2 * SC_BATCH * NT * 4;
  static constexpr int PART_BYTES = NT * kBM * 4;       // one tile of fp32 sums
  // Shared memory from a 1024-aligned base: barriers (the most there can be),
  // abort flag, scales (and per batch of them a word, and each token's factor and
  // exponent: forge_b128.cuh), stages, and where the reduction is split the shares.
  // (In the stages' place the shares would have to wait for every CTA's last
  // load and product: a cluster barrier more.)
  static constexpr int NUM_BARS = 2 * DEEP + 2 * NBUF + 5;
  static constexpr int OFF_TMEM = 8 * NUM_BARS;
  static constexpr int OFF_WORD = OFF_TMEM + 8;
  static constexpr int OFF_SC = (OFF_WORD + 8 + 15) & ~15;
  static constexpr int OFF_FACTOR = OFF_SC + SC_BYTES;
  static constexpr int OFF_EXPONENT = OFF_FACTOR + 2 * NT * 4;
  static constexpr int OFF_STAGES = (OFF_EXPONENT + 2 * NT * 4 + 1023) & ~1023;
  static constexpr int smem(int stages, bool split) {
    return OFF_STAGES + stages * STAGE_BYTES + (split ? PART_BYTES : 0) + 1024;
  }
  static constexpr int SPLIT_DEEP = NT <= 32 ? DEEP : (NT == 64 ? 6 : 4);   // beside the shares
  static_assert(NT > 64 || 2 * smem(STAGES, false) <= 228 * 1024 - 2 * 1024, "two CTAs an SM");
  static_assert(smem(DEEP, false) <= 232448 && smem(SPLIT_DEEP, true) <= 232448,
                "shared memory budget");
};

__device__ __forceinline__ void store_out(const B128Args& a, int64_t idx, float v) {
  if (a.out_fp32) reinterpret_cast<float*>(a.out_ptr)[idx] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out_ptr)[idx] = __float2bfloat16_rn(v);
}

template <int NT, bool DGRAD>
__global__ void __launch_bounds__(Few<NT>::THREADS, NT <= 64 ? 2 : 1)
    gemm_b128_few_kernel(const __grid_constant__ B128Args a) {
  using T = Few<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  // the same offset in every CTA of the cluster: remote stores use it
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = a.splits;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  // this CTA's blocks (none where more CTAs than blocks are asked for)
  const int kb = b128_first_block(rank, splits, a.num_kb);
  const int ke = b128_first_block(rank + 1, splits, a.num_kb);

  const uint32_t stages = a.stages;
  const uint32_t bars = base, stage0 = base + T::OFF_STAGES;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (T::DEEP + s); };
  auto bar_tfull = [&](int b) { return bars + 8u * (2 * T::DEEP + b); };
  auto bar_tempty = [&](int b) { return bars + 8u * (2 * T::DEEP + T::NBUF + b); };
  auto bar_sfull = [&](int b) { return bars + 8u * (2 * T::DEEP + 2 * T::NBUF + b); };
  auto bar_sempty = [&](int b) { return bars + 8u * (2 * T::DEEP + 2 * T::NBUF + 2 + b); };
  const uint32_t bar_drain = bars + 8u * (2 * T::DEEP + 2 * T::NBUF + 4);
  float* scales = reinterpret_cast<float*>(gbase + T::OFF_SC);   // [2][SC_BATCH][NT]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM + 4);
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_WORD);
  float* factors = reinterpret_cast<float*>(gbase + T::OFF_FACTOR);     // [2][NT]
  int* exponents = reinterpret_cast<int*>(gbase + T::OFF_EXPONENT);     // [2][NT]
  const WaitCtx wc{abort_flag, a.err, a.err_site, a.timeout_ns};

  const uint64_t wpol = l2_policy_evict_normal(), xpol = l2_policy_evict_last();
  auto load = [&](uint32_t s, int k) {
    const uint32_t dst = stage0 + s * T::STAGE_BYTES;
    mbar_arrive_expect_tx(bar_full(s), T::STAGE_BYTES);
    tma_load_2d(dst, &a.b, DGRAD ? tile * 128 : k * 128, DGRAD ? k * 128 : tile * 128, bar_full(s),
                wpol);
    tma_load_2d(dst + T::A_BYTES, &a.a, k * 128, 0, bar_full(s), xpol);
  };
  // Warp 0 sets up the barriers, a lane each, while warp 1 takes the tensor
  // memory; one block barrier covers both.
  if (warp == 0) {
    for (int i = lane; i < T::NUM_BARS; i += 32) {
      const bool tempty = i >= 2 * T::DEEP + T::NBUF && i < 2 * T::DEEP + 2 * T::NBUF;
      const bool sfull = i == 2 * T::DEEP + 2 * T::NBUF || i == 2 * T::DEEP + 2 * T::NBUF + 1;
      const bool sempty = i == 2 * T::DEEP + 2 * T::NBUF + 2 || i == 2 * T::DEEP + 2 * T::NBUF + 3;
      mbar_init(bars + 8u * i, sfull ? 32 : (tempty || sempty ? T::EPI : 1));
    }
    if (lane == 0) *abort_flag = 0u;
    fence_mbarrier_init();
    if (lane == 0) drop_first_arrival(a.drop_first_arrival, bar_full(0));
  } else if (warp == 1) {
    tmem_alloc(base + T::OFF_TMEM, T::TMEM_COLS);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  if (splits > 1) cluster_arrive();   // waited for before the first remote store
  tc_fence_after_sync();
  // While the kernel before still runs, the weight's first blocks are asked for
  // as far as L2.  (L2 is where all writes meet: were that kernel writing them,
  // the loads after the wait would still find what it wrote.)  One token, norm,
  // 4096 -> 14336, quantiser, 14336 -> 4096: 28.1 us, 28.8 without; of up to 128
  // tokens four blocks gain more than half the share (64 tokens: 32.0 and 32.6).
  if (warp == 0 && lane == 0) {
    const int ahead = NT <= 16 ? max(4, (ke - kb) / 2) : 4;
    for (int k = kb; k < min(ke, kb + ahead); ++k)
      tma_prefetch_l2_2d(&a.b, DGRAD ? tile * 128 : k * 128, DGRAD ? k * 128 : tile * 128);
  }
  grid_dependency_wait();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM);

  float2 acc[T::NC / 2];   // epilogue threads: one output, NC tokens
  if (warp == 0) {
    if (lane == 0) {
      uint32_t ps = 0, pph = 0, armed = 0;   // next stage, its phase, stages in use
      for (int k = kb; k < ke; ++k) {
        if (!wait_bounded(bar_empty(ps), pph ^ 1u, wc, kSiteProducerEmpty)) break;
        load(ps, k);
        if (armed < stages) ++armed;
        if (++ps == stages) { ps = 0; pph ^= 1u; }
      }
      for (uint32_t i = 0; i < armed; ++i) {   // the last load of every stage lands
        if (ps == 0) { ps = stages; pph ^= 1u; }
        --ps;
        wait_bounded(bar_full(ps), pph, wc, kSiteDrainOperands, false);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = make_idesc_e4m3(128, NT, DGRAD, false);
    const uint64_t ad0 = DGRAD ? make_sdesc_mn_sw128(stage0, 16384, 1024)
                               : make_sdesc_k_sw128(stage0, 1024);
    const uint64_t bd0 = make_sdesc_k_sw128(stage0 + T::A_BYTES, 1024);
    constexpr uint32_t kStepA = (DGRAD ? 4096 : 32) >> 4, kStepB = 32 >> 4;
    const bool issue = elect_one();
    uint32_t s = 0, ph = 0, buf = 0, bph = 1;
#pragma unroll 1
    for (int k = kb; k < ke; ++k) {
      const bool ok = wait_bounded(bar_tempty(buf), bph, wc, kSiteMmaTmemEmpty) &&
                      wait_bounded(bar_full(s), ph, wc, kSiteMmaFull);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      const uint64_t ad = ad0 + s * (T::STAGE_BYTES >> 4), bd = bd0 + s * (T::STAGE_BYTES >> 4);
      if (issue) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_e4m3(tmem_base + buf * NT, ad + kk * kStepA, bd + kk * kStepB, idesc, kk != 0);
        umma_commit(bar_empty(s));
        umma_commit(bar_tfull(buf));
      }
      if (++s == stages) { s = 0; ph ^= 1u; }
      if (++buf == T::NBUF) { buf = 0; bph ^= 1u; }
    }
    if (issue) umma_commit(bar_drain);
    wait_bounded(bar_drain, 0u, wc, kSiteDrainMma, false);
    __syncwarp();
  } else if (warp == 2) {
    // sx[t][k] sw[tile][k]; tokens past the last count zero.  A batch's loads
    // all start before any is used.
    constexpr int PT = (NT + 31) / 32;   // tokens per lane
    uint32_t b = 0, ph = 1;
    TokenExponents te;
    for (int k0 = kb; k0 < ke; k0 += T::SC_BATCH) {
      float rx[PT][T::SC_BATCH];
#pragma unroll
      for (int i = 0; i < T::SC_BATCH; ++i) {
        const int k = min(k0 + i, ke - 1);   // past the end: loaded again, not used
#pragma unroll
        for (int j = 0; j < PT; ++j) {
          const int t = lane + 32 * j;
          rx[j][i] = a.sa[static_cast<int64_t>(min(t, a.m - 1)) * a.num_kb + k];
        }
      }
      // a lane for each of the batch's weight blocks
      const float rl = a.sw[static_cast<int64_t>(tile) * a.sw_n +
                            static_cast<int64_t>(min(k0 + (lane & 7), ke - 1)) * a.sw_k];
      const bool any_w = __any_sync(0xffffffffu, rl != 0.0f);
      float rw[T::SC_BATCH];
#pragma unroll
      for (int i = 0; i < T::SC_BATCH; ++i) rw[i] = __shfl_sync(0xffffffffu, rl, i);
      // (what lies past the last token or block repeats it)
      bool apart = false;
#pragma unroll
      for (int j = 0; j < PT; ++j) {
        float most = 0.0f;
        uint32_t any = 0u;   // whether the token has a scale other than zero
#pragma unroll
        for (int i = 0; i < T::SC_BATCH; ++i) {
          any |= __float_as_uint(rx[j][i]);
          rx[j][i] *= rw[i];
          most = fmaxf(most, fabsf(rx[j][i]));
        }
        apart |= te.add(j, most, any_w && any != 0u);
      }
      const bool good = wait_bounded(bar_sempty(b), ph, wc, kSiteLoaderEmpty);
      if (!__all_sync(0xffffffffu, good)) break;
      uint32_t word = 0u;
      if (__any_sync(0xffffffffu, apart)) {
        word = scales_apart<1, NT, T::SC_BATCH>(a, te, scales + b * T::SC_BATCH * NT,
                                                factors + b * NT, exponents + b * NT, lane, lane,
                                                tile, k0, ke);
      } else {
#pragma unroll
        for (int i = 0; i < T::SC_BATCH; ++i)
#pragma unroll
          for (int j = 0; j < PT; ++j) {
            const int t = lane + 32 * j;
            if (t < NT) scales[(b * T::SC_BATCH + i) * NT + t] = t < a.m ? rx[j][i] : 0.0f;
          }
      }
      if (lane == 0) words[b] = word;
      mbar_arrive(bar_sfull(b));
      if (++b == 2) { b = 0; ph ^= 1u; }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t tcol = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + h * T::NC;
#pragma unroll
    for (int i = 0; i < T::NC / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
    uint32_t buf = 0, bph = 0, sb = 0, sph = 0;
    bool ok = true;
    for (int k0 = kb; ok && k0 < ke; k0 += T::SC_BATCH) {
      const int kn = min(T::SC_BATCH, ke - k0);
      const float* sc_row = scales + sb * T::SC_BATCH * NT + h * T::NC;
      ok = __all_sync(0xffffffffu, wait_bounded_inline(bar_sfull(sb), sph, wc, kSiteEpiSlotFull));
      if (!ok) break;
      if (words[sb] & kBatchFactors) {
#pragma unroll
        for (int i = 0; i < T::NC / 2; ++i) {
          const float* f = factors + sb * NT + h * T::NC + 2 * i;
          acc[i] = mul2(acc[i], make_float2(f[0], f[1]));
        }
      }
#pragma unroll 1
      for (int k = 0; k < kn; ++k) {
        ok = __all_sync(0xffffffffu,
                        wait_bounded_inline(bar_tfull(buf), bph, wc, kSiteEpiTmemFull));
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < T::NC / 16; ++c) {
          uint32_t r[16];
          tmem_ld_x16(tcol + buf * NT + 16 * c, r);
          float4 f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = *reinterpret_cast<const float4*>(sc_row + k * NT + 16 * c + 4 * i);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            fma2_loaded(acc[c * 8 + 2 * i], r[4 * i], r[4 * i + 1], make_float2(f[i].x, f[i].y));
            fma2_loaded(acc[c * 8 + 2 * i + 1], r[4 * i + 2], r[4 * i + 3],
                        make_float2(f[i].z, f[i].w));
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_tempty(buf));
        if (++buf == T::NBUF) { buf = 0; bph ^= 1u; }
      }
      if (!ok) break;
      if (k0 + T::SC_BATCH >= ke && (words[sb] & kBatchExponents)) {
#pragma unroll
        for (int i = 0; i < T::NC / 2; ++i) {
          const int* e = exponents + sb * NT + h * T::NC + 2 * i;
          acc[i] = make_float2(times_pow2_64(acc[i].x, e[0]), times_pow2_64(acc[i].y, e[1]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sempty(sb));
      if (++sb == 2) { sb = 0; sph ^= 1u; }
    }
  }

  // ------------------------------------------------------------ join and store
  grid_dependency_trigger();
  tc_fence_before_sync();
  if (splits == 1) {
    __syncthreads();
    if (warp >= 4 && !*abort_flag) {
      const int h = (warp - 4) >> 2, o = tile * 128 + (warp & 3) * 32 + lane;
      if (o < a.n) {
#pragma unroll
        for (int i = 0; i < T::NC; ++i) {
          const int t = h * T::NC + i;
          if (t < a.m)
            store_out(a, static_cast<int64_t>(t) * a.n + o, i & 1 ? acc[i / 2].y : acc[i / 2].x);
        }
      }
    }
  } else {
    __syncthreads();
    cluster_wait();   // every CTA has started
    const uint32_t off_part = T::OFF_STAGES + a.stages * T::STAGE_BYTES;
    const int slice = kBM / splits;   // outputs each CTA of the cluster owns (splits divides 128)
    if (warp >= 4) {
      const int h = (warp - 4) >> 2, o = (warp & 3) * 32 + lane;
      // [rank of the sender][token][output of the slice]
      const uint32_t dst = mapa_shared(base + off_part, o / slice) +
                           4u * ((rank * NT + h * T::NC) * slice + o % slice);
#pragma unroll
      for (int i = 0; i < T::NC; ++i)
        if (h * T::NC + i < a.m)
          st_cluster_f32(dst + 4u * i * slice, i & 1 ? acc[i / 2].y : acc[i / 2].x);
    }
    cluster_sync_all();
    if (!*abort_flag) {
      const float* part = reinterpret_cast<const float*>(gbase + off_part);
      // four outputs at a time: a slice is a power of two of at least 16, and an
      // output row a multiple of 16
      const int shift = 31 - __clz(slice >> 2), total = a.m << shift;
      for (int e = threadIdx.x; e < total; e += T::THREADS) {
        const int t = e >> shift, j = (e - (t << shift)) * 4, o = tile * 128 + rank * slice + j;
        if (o >= a.n) continue;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int z = 0; z < splits; ++z) {
          const float4 p = *reinterpret_cast<const float4*>(part + (z * NT + t) * slice + j);
          v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
        }
        const int64_t idx = static_cast<int64_t>(t) * a.n + o;
        if (a.out_fp32) {
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out_ptr) + idx) = v;
        } else {
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out_ptr) + idx) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
      }
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, T::TMEM_COLS);
  }
}

template <int NT, bool DGRAD>
cudaError_t launch_t(B128Args a, int num_sms, cudaStream_t stream) {
  using T = Few<NT>;
  auto kern = gemm_b128_few_kernel<NT, DGRAD>;
  static PerDevice once;
  const cudaError_t e = allow_smem(once, kern, 232448);
  if (e != cudaSuccess) return e;
  const bool split = a.splits > 1;
  a.stages = split ? T::SPLIT_DEEP : (a.num_tiles <= num_sms ? T::DEEP : T::STAGES);
  return launch_chained(kern, a.num_tiles * a.splits, T::THREADS, T::smem(a.stages, split),
                        a.splits > 1 ? a.splits : 0, stream, a);
}

template <int NT>
cudaError_t launch_dir(bool dgrad, const B128Args& a, int num_sms, cudaStream_t stream) {
  return dgrad ? launch_t<NT, true>(a, num_sms, stream) : launch_t<NT, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_gemm_b128_few(int nt, bool dgrad, const B128Args& a, int num_sms,
                                 cudaStream_t stream) {
  switch (nt) {
    case 16: return launch_dir<16>(dgrad, a, num_sms, stream);
    case 32: return launch_dir<32>(dgrad, a, num_sms, stream);
    case 64: return launch_dir<64>(dgrad, a, num_sms, stream);
    case 128: return launch_dir<128>(dgrad, a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace forge

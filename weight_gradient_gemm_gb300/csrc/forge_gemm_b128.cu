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
// Warp roles (384 threads): warp 0 loads operand stages of 128 columns with
// TMA, warps 1 and 3 issue the MMAs, warp 2 multiplies the scales and leaves the
// products in shared memory eight blocks ahead, warps 4-11 add up (two per
// TMEM lane quadrant, each half of the tile's columns) and store.  The first
// four warps give most of their registers to the other eight, whose threads
// hold up to 128 output values.  Every wait is bounded, as in forge_gemm.cuh.
//
// What bounds it: a pair takes 720 to 770 cycles for a block of 128 whose
// products take 512.  8192 tokens, 4096 -> 14336: 335 us (2.9 PFLOP/s; 386 in
// long runs, under the power limit) where twice the bf16 rate would take 253.
// 294 of them stay without any work in the epilogue: with two TMEM buffers a
// piece the tensor core waits for the hand-off to the epilogue and back.  The
// rest is the adding up, half of the SM's issue slots.  2000 tokens, 14336 ->
// 4096: 90 us, 128 tiles on 76 pairs, the second wave 68 % full; 512 tokens,
// 4096 -> 4096: 13.7 us, one wave of single CTAs at 490 cycles a block.  Tried and
// slower: 16 epilogue warps (405 us where 8 took 362), the two issuers in a fixed turn
// (354 for 333), waits that poll.
#include <cuda_bf16.h>

#include "forge_b128.cuh"
#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

constexpr int kThreads8 = 384;
// Registers a thread after the split: 128 x 104 + 256 x 200 = 384 x 168, what
// the block is launched with.  (With 88 and 208 the scales' warp has too few: 2000
// tokens, 14336 -> 4096, 91.2 us for 89.8; with 96 and 200 90.2, 112 and 192 94.0.)
constexpr int kRegsRole = 104, kRegsEpi = 200;
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
  static constexpr int NC = BN / 2;                    // columns per epilogue thread
  static constexpr int GROUPS = NC / 64;               // runs of 64 neighbouring columns among them
  // One slab of 32 rows x 128 bytes a warp for its output.  (Two, with four
  // operand stages, measured the same on pairs and 19 % slower on one CTA.)
  static constexpr int SLAB = 4096;
  static constexpr int OUT_BYTES = kEpiWarps * SLAB;
  static constexpr int STAGES = 5;
  // The tile's accumulator is cut into pieces of 128 columns with TMEM buffers
  // of their own, so that a piece's next product waits for the warps that read
  // that piece only.
  static constexpr int PIECES = BN / 128;
  static constexpr int NBUF = 4 / PIECES;              // buffers per piece (512 columns in all)
  static constexpr int PIECE_WARPS = kEpiWarps / PIECES;
  static constexpr int NWB = BN / 128;                 // weight blocks across the tile
  static constexpr int SC_BATCH = 8;                   // 128-blocks whose scales move together
  static constexpr int SC_BYTES = 2 * SC_BATCH * NWB * kBM * 4;
  // columns per tensor-memory load: 32 where two of them fit beside the sums
  // (with 128 sums they spill, and the kernel ran 19 % slower)
  static constexpr int LD = NC == 64 ? 32 : 16;
  static constexpr int OFF_OUT = STAGES * STAGE_BYTES;
  static constexpr int OFF_SC = OFF_OUT + OUT_BYTES;
  static constexpr int OFF_BARS = OFF_SC + SC_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 8 + 5;
  static constexpr int OFF_TMEM = OFF_BARS + 8 * NUM_BARS;
  // per scale batch: a word, and each token's factor and exponent (forge_b128.cuh)
  static constexpr int OFF_WORD = OFF_TMEM + 8;
  static constexpr int OFF_FACTOR = OFF_WORD + 8;
  static constexpr int OFF_EXPONENT = OFF_FACTOR + 2 * kBM * 4;
  static constexpr int SMEM_USED = OFF_EXPONENT + 2 * kBM * 4;
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
__global__ void __launch_bounds__(kThreads8, 1)
    gemm_b128_kernel(const __grid_constant__ B128Args a) {
  using T = Traits8<CG, BN>;
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
  // b: one of the four TMEM buffers, piece * NBUF + buffer
  auto bar_tfull = [&](int b) { return bars + 8u * (2 * T::STAGES + b); };
  auto bar_tempty = [&](int b) { return bars + 8u * (2 * T::STAGES + 4 + b); };
  auto bar_sfull = [&](int b) { return bars + 8u * (2 * T::STAGES + 8 + b); };
  auto bar_sempty = [&](int b) { return bars + 8u * (2 * T::STAGES + 10 + b); };
  const uint32_t bar_drain = bars + 8u * (2 * T::STAGES + 12);
  float* scales = reinterpret_cast<float*>(gbase + T::OFF_SC);   // [2][SC_BATCH][NWB][128]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM + 4);
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_WORD);
  float* factors = reinterpret_cast<float*>(gbase + T::OFF_FACTOR);        // [2][128]
  int* exponents = reinterpret_cast<int*>(gbase + T::OFF_EXPONENT);        // [2][128]
  const WaitCtx wc{abort_flag, a.err, a.err_site, a.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 2);   // both issuers
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(bar_tfull(b), 1);
      mbar_init(bar_tempty(b), CG * T::PIECE_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_sfull(b), 32);
      mbar_init(bar_sempty(b), kEpiWarps);
    }
    mbar_init(bar_drain, 2);
    *abort_flag = 0u;
    fence_mbarrier_init();
    drop_first_arrival(a.drop_first_arrival, bar_full(0));
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
  grid_dependency_wait();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gbase + T::OFF_TMEM);

  if (warp < 4) {
    regs_dec<kRegsRole>();
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
          const int nb = tn * BN + static_cast<int>(rank) * T::BNL;
          for (int k = 0; k < a.num_kb; ++k) {
            if (!wait_bounded(bar_empty(s), ph ^ 1u, wc, kSiteProducerEmpty)) { ok = false; break; }
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
                  tma_load_2d_pair(dst + T::A_BYTES + c * 16384, &a.b, nb + c * 128, k * 128, fb,
                                   pol);
              } else {
                tma_load_2d_pair(dst + T::A_BYTES, &a.b, k * 128, nb, fb, pol);
              }
            } else {
              mbar_arrive_expect_tx(bar_full(s), T::STAGE_BYTES);
              tma_load_2d(dst, &a.a, k * 128, ya, bar_full(s), pol);
              if constexpr (DGRAD) {
#pragma unroll
                for (int c = 0; c < T::BNL / 128; ++c)
                  tma_load_2d(dst + T::A_BYTES + c * 16384, &a.b, nb + c * 128, k * 128,
                              bar_full(s), pol);
              } else {
                tma_load_2d(dst + T::A_BYTES, &a.b, k * 128, nb, bar_full(s), pol);
              }
            }
            if (armed < T::STAGES) ++armed;
            if (++s == T::STAGES) { s = 0; ph ^= 1u; }
          }
        }
        // Before the CTA can exit, every stage's last release has to arrive (on a
        // pair the leader's MMAs signal it from afar); after a timeout, every
        // load that is under way has to land (a pair's complete on the leader's
        // barriers).
        for (uint32_t i = 0; i < armed; ++i) {
          if (s == 0) { s = T::STAGES; ph ^= 1u; }
          --s;
          const bool freed = ok && wait_bounded(bar_empty(s), ph, wc, kSiteDrainOperands);
          if (!freed && leader) wait_bounded(bar_full(s), ph, wc, kSiteDrainOperands, false);
        }
      }
      __syncwarp();
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------ MMA issuers
      // A product costs its issuing thread about 39 cycles, a commit 41 and a
      // wait that is ready 60, so one thread's 8 products, 3 commits and 3 waits
      // per block of a pair (634 cycles measured) would be slower than the tensor
      // core (512).  Two warps share them: each a piece of a pair's tile, or
      // every other block of a single CTA's.  They walk the blocks with the
      // whole warp, so that addresses and descriptors stay in uniform registers,
      // and one elected lane issues.
      if (leader) {
        constexpr uint32_t idesc = make_idesc_e4m3(T::TM, 128, false, DGRAD);
        const uint64_t ad0 = make_sdesc_k_sw128(base, 1024);
        const uint64_t bd0 = DGRAD ? make_sdesc_mn_sw128(base + T::A_BYTES, 16384, 1024)
                                   : make_sdesc_k_sw128(base + T::A_BYTES, 1024);
        // 32 of K further: 32 bytes K-major, 32 rows MN-major
        constexpr uint32_t kStepA = 32 >> 4, kStepB = (DGRAD ? 4096 : 32) >> 4;
        // 64 of each CTA's columns further (pairs): 64 rows K-major, 64 bytes MN-major
        constexpr uint32_t kPieceB = (DGRAD ? 64 : 8192) >> 4;
        const bool issue = elect_one();
        const uint32_t me = warp >> 1;   // issuer 0 or 1
        const uint32_t pc = T::PIECES == 1 ? 0 : me;
        uint32_t s = 0, ph = 0, buf = 0, bph = 1, turn = 0;
        bool ok = true;
        for (int t = unit0; ok && t < a.num_tiles; t += units) {
#pragma unroll 1
          for (int k = 0; k < a.num_kb; ++k) {
            // Both issuers wait for every block's stage and release it, also where
            // the block is the other's: a stage goes from one to the other, and a
            // parity wait that skipped or lagged a phase would take another for
            // its own.  (TMEM buffers stay with one issuer: their number is even.)
            const bool mine = T::PIECES > 1 || turn == me;
            const uint32_t b = pc * T::NBUF + buf;
            ok = wait_bounded(bar_full(s), ph, wc, kSiteMmaFull) &&
                 (!mine || wait_bounded(bar_tempty(b), bph, wc, kSiteMmaTmemEmpty));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (mine) {
              tc_fence_after_sync();
              const uint64_t ad = ad0 + s * (T::STAGE_BYTES >> 4);
              const uint64_t bd = bd0 + s * (T::STAGE_BYTES >> 4) + pc * kPieceB;
              const uint32_t d = tmem_base + b * 128;
              if (issue) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  if constexpr (kPair)
                    umma_e4m3_pair(d, ad + kk * kStepA, bd + kk * kStepB, idesc, kk != 0);
                  else
                    umma_e4m3(d, ad + kk * kStepA, bd + kk * kStepB, idesc, kk != 0);
                }
                // the stage is free, and the piece complete, once these have run
                if constexpr (kPair) {
                  umma_commit_pair_mc(bar_empty(s), 0x3);
                  umma_commit_pair_mc(bar_tfull(b), 0x3);
                } else {
                  umma_commit(bar_empty(s));
                  umma_commit(bar_tfull(b));
                }
              }
            } else if (issue) {
              mbar_arrive(bar_empty(s));
            }
            turn ^= 1u;
            if (++s == T::STAGES) { s = 0; ph ^= 1u; }
            if (++buf == T::NBUF) { buf = 0; bph ^= 1u; }
          }
        }
        // every MMA issued must complete before the tensor memory is freed
        if (issue) {
          if constexpr (kPair) umma_commit_pair_mc(bar_drain, 0x1); else umma_commit(bar_drain);
        }
        wait_bounded(bar_drain, 0u, wc, kSiteDrainMma, false);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ scales
      // sa[row][k] sw[column block][k] for the tile's 128 rows, a batch of
      // blocks at a time.  (Read by the epilogue threads themselves, one block
      // ahead, their latency bounded the whole kernel: 462 ns per block of a
      // 128 x 128 tile.)  Rows and column blocks outside count zero.  The weight's
      // scales are loaded before the wait too, a lane each (one by one after it, 16
      // latencies follow one another: 2000 tokens, 14336 -> 4096, 89.2 us for 87.5).
      uint32_t cnt = 0;
      bool ok = true;
      for (int t = unit0; ok && t < a.num_tiles; t += units) {
        int tm, tn;
        tile_of(t, a, tm, tn);
        const int row0 = tm * T::TM + static_cast<int>(rank) * kBM + lane;
        const int wb0 = tn * T::NWB;
        TokenExponents te;
        for (int k0 = 0; k0 < a.num_kb; k0 += T::SC_BATCH, ++cnt) {
          float ra[4][T::SC_BATCH];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = row0 + 32 * j;
            const float* p = a.sa + static_cast<int64_t>(row < a.m ? row : 0) * a.num_kb + k0;
#pragma unroll
            for (int i = 0; i < T::SC_BATCH; ++i)
              ra[j][i] = row < a.m && k0 + i < a.num_kb ? p[i] : 0.0f;
          }
          float most[4];
          uint32_t any[4];   // whether a token has a scale other than zero
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            most[j] = 0.0f;
            any[j] = 0u;
#pragma unroll
            for (int i = 0; i < T::SC_BATCH; ++i) any[j] |= __float_as_uint(ra[j][i]);
          }
          // a lane for each of the batch's weight blocks
          const int lk = k0 + lane / T::NWB, lw = wb0 + lane % T::NWB;
          const float rl = lane < T::SC_BATCH * T::NWB && lk < a.num_kb && lw * 128 < a.n
                               ? a.sw[static_cast<int64_t>(lw) * a.sw_n +
                                      static_cast<int64_t>(lk) * a.sw_k]
                               : 0.0f;
          const bool any_w = __any_sync(0xffffffffu, rl != 0.0f);
          const int b = cnt & 1;
          const bool good =
              wait_bounded(bar_sempty(b), ((cnt >> 1) & 1u) ^ 1u, wc, kSiteLoaderEmpty);
          if (!__all_sync(0xffffffffu, good)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < T::SC_BATCH; ++i)
#pragma unroll
            for (int w = 0; w < T::NWB; ++w) {
              const float rw = __shfl_sync(0xffffffffu, rl, i * T::NWB + w);
              float* dst = scales + ((b * T::SC_BATCH + i) * T::NWB + w) * kBM + lane;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float p = ra[j][i] * rw;
                dst[32 * j] = p;
                most[j] = fmaxf(most[j], fabsf(p));
              }
            }
          bool apart = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) apart |= te.add(j, most[j], any_w && any[j] != 0u);
          uint32_t word = 0u;
          if (__any_sync(0xffffffffu, apart))
            word = scales_apart<T::NWB, kBM, T::SC_BATCH>(
                a, te, scales + b * T::SC_BATCH * T::NWB * kBM, factors + b * kBM,
                exponents + b * kBM, row0, lane, wb0, k0, a.num_kb);
          if (lane == 0) words[b] = word;
          mbar_arrive(bar_sfull(b));
        }
      }
      __syncwarp();
    }
  } else {
    regs_inc<kRegsEpi>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                       // TMEM lane quadrant this warp may read
    const int h = (warp - 4) >> 2;                // piece (pairs), or half of the one piece
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t slab = base + T::OFF_OUT + (warp - 4) * T::SLAB;
    uint8_t* gslab = gbase + T::OFF_OUT + (warp - 4) * T::SLAB;
    const uint32_t bpiece = T::PIECES == 1 ? 0 : h * T::NBUF;   // first buffer of this warp's piece
    uint32_t buf = 0, bph = 0, sb = 0, sph = 0;
    bool ok = true;
    for (int t = unit0; ok && t < a.num_tiles; t += units) {
      int tm, tn;
      tile_of(t, a, tm, tn);
      const int row0 = tm * T::TM + static_cast<int>(rank) * kBM + q * 32;
      // A pair's piece holds 64 columns of each CTA's 128, so of both weight
      // blocks: columns p * 64 and 128 + p * 64 of the tile.
      const int col0 = tn * BN + h * 64;
      float2 acc[T::NC / 2];
#pragma unroll
      for (int i = 0; i < T::NC / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      bool ready = false;   // the next accumulator has been seen complete
      for (int k0 = 0; ok && k0 < a.num_kb; k0 += T::SC_BATCH) {
        const int kn = min(T::SC_BATCH, a.num_kb - k0);
        const float* sc_row = scales + sb * T::SC_BATCH * T::NWB * kBM + q * 32 + lane;
        ok = __all_sync(0xffffffffu, wait_bounded_inline(bar_sfull(sb), sph, wc, kSiteEpiSlotFull));
        if (!ok) break;
        if (words[sb] & kBatchFactors) {
          const float2 f = dup2(factors[sb * kBM + q * 32 + lane]);
#pragma unroll
          for (int i = 0; i < T::NC / 2; ++i) acc[i] = mul2(acc[i], f);
        }
#pragma unroll 1
        for (int k = 0; k < kn; ++k) {
          float sc[T::GROUPS];
#pragma unroll
          for (int g = 0; g < T::GROUPS; ++g) sc[g] = sc_row[(k * T::NWB + g) * kBM];
          const uint32_t b = bpiece + buf;
          if (!__all_sync(0xffffffffu, ready)) {
            ok = __all_sync(0xffffffffu,
                            wait_bounded_inline(bar_tfull(b), bph, wc, kSiteEpiTmemFull));
            if (!ok) break;
          }
          tc_fence_after_sync();
          const uint32_t taddr = tmem_base + lane_addr + b * 128 + (T::PIECES == 1 ? h * 64 : 0);
          if (++buf == T::NBUF) { buf = 0; bph ^= 1u; }
          // some columns at a time, the next ones in flight while these are added
          uint32_t r[2][T::LD];
          tmem_ld(taddr, r[0]);
#pragma unroll
          for (int c = 0; c < T::NC / T::LD; ++c) {
            tmem_ld_wait();
            if (c + 1 < T::NC / T::LD) {
              tmem_ld(taddr + T::LD * (c + 1), r[(c + 1) & 1]);
            } else {   // this warp has read its part of the buffer
              tc_fence_before_sync();
              __syncwarp();
              if (lane == 0) {
                if constexpr (kPair) mbar_arrive_cluster_relaxed(mapa_shared(bar_tempty(b), 0));
                else mbar_arrive(bar_tempty(b));
              }
            }
            // asked early, so that the answer is there when the loop comes round
            if (c == T::NC / T::LD - 2) ready = mbar_test_wait(bar_tfull(bpiece + buf), bph);
#pragma unroll
            for (int i = 0; i < T::LD / 2; ++i)
              fma2_loaded(acc[c * (T::LD / 2) + i], r[c & 1][2 * i], r[c & 1][2 * i + 1],
                          sc[c * T::LD / 64]);
          }
        }
        if (!ok) break;
        if (k0 + T::SC_BATCH >= a.num_kb && (words[sb] & kBatchExponents)) {
          const int e = exponents[sb * kBM + q * 32 + lane];
#pragma unroll
          for (int i = 0; i < T::NC / 2; ++i)
            acc[i] = make_float2(times_pow2_64(acc[i].x, e), times_pow2_64(acc[i].y, e));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sempty(sb));   // the batch's scales are read
        if (++sb == 2) { sb = 0; sph ^= 1u; }
      }
      if (!ok) break;
      // store through this warp's slab: boxes of 32 rows x 128 bytes
      // the slab is free once the store before has read it
      auto claim = [&]() {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
      };
      auto send = [&](int col) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&a.out, col, row0, slab);
          bulk_commit_group();
        }
      };
      if (row0 >= a.m) continue;
#pragma unroll
      for (int g = 0; g < T::GROUPS; ++g) {
        const int col = col0 + g * 128;
        if (col >= a.n) continue;
        const float2* v = acc + g * 32;
        if (a.out_fp32) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (col + 32 * c >= a.n) break;
            claim();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x = v[c * 16 + 2 * i], y = v[c * 16 + 2 * i + 1];
              *reinterpret_cast<float4*>(gslab + sw128_off(lane, i)) =
                  make_float4(x.x, x.y, y.x, y.y);
            }
            send(col + 32 * c);
          }
        } else {
          claim();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2* x = v + 4 * i;
            *reinterpret_cast<uint4*>(gslab + sw128_off(lane, i)) =
                make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                           pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
          }
          send(col);
        }
      }
    }
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
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

template <int CG, int BN, bool DGRAD>
cudaError_t launch_t(const B128Args& a, int num_sms, cudaStream_t stream) {
  using T = Traits8<CG, BN>;
  auto kern = gemm_b128_kernel<CG, BN, DGRAD>;
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
    lc.blockDim = dim3(kThreads8, 1, 1);
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
  return launch_chained(kern, CG * (a.num_tiles < units ? a.num_tiles : units), kThreads8,
                        T::SMEM_ALLOC, CG == 2 ? 2 : 0, stream, a);
}

template <int CG, int BN>
cudaError_t launch_dir(bool dgrad, const B128Args& a, int num_sms, cudaStream_t stream) {
  return dgrad ? launch_t<CG, BN, true>(a, num_sms, stream)
               : launch_t<CG, BN, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_gemm_b128(const B128Config& c, bool dgrad, const B128Args& a, int num_sms,
                             cudaStream_t stream) {
  if (c.cg == 1 && c.bn == 128) return launch_dir<1, 128>(dgrad, a, num_sms, stream);
  if (c.cg == 2 && c.bn == 256) return launch_dir<2, 256>(dgrad, a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace forge

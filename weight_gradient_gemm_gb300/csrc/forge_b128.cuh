// What the two kernels of the 8-bit products share: products of scales that leave
// fp32's range.
//
// A block's sum P meets the scale of its tokens and that of its weight block as
// their product p, with one multiply-add a value.  In a format whose scales go
// from 2^-126 to 2^119, p may leave fp32's normal range although the result does
// not (gradients of 2^-115 and weights of 2^-20; or a token of 2^100 that meets a
// weight of 2^40 in a few small entries).  So every token has an exponent e,
// normally 0: its sums are kept times 2^-e, its products are formed times 2^-e, and
// the result is multiplied by 2^e.  The warp that multiplies the scales chooses e
// by the largest product of a batch of blocks and of those before: 0 where that
// lies from 2^-120 to 2^100, else a multiple of 64 that brings it to 2^-32 .. 2^32.
// Once a product has been seen e only rises, so a product's rounding is at most
// 2^-30 of the token's largest (2^-150 against 2^-120).  The epilogue's loop over
// blocks stays as it is; only a batch that raises some e multiplies the sums once.
// Measured, without and with exponents: 8192 tokens, 4096 -> 14336, 332 and 335 us;
// 2000 tokens, 14336 -> 4096, 89.0 and 90.0; one token, 4096 -> 4096, 6.15 and 6.28;
// 128 tokens, 4096 -> 14336, 17.4 and 17.3.  (A second loop with the products in fp64
// took that loop's registers: 385 and 149 us for the first two.)  Where e is not 0 the
// scales' warp forms its products in fp64 from global memory: 2000 tokens, 4096 ->
// 14336, with every product below 2^-120, take 1016 us for 87.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "forge_internal.h"

namespace forge {

constexpr float kScalesLow = 0x1p-120f, kScalesHigh = 0x1p100f;
// Bits of a batch's word in shared memory: the sums take factors; some e is not 0.
constexpr uint32_t kBatchFactors = 1u, kBatchExponents = 2u;

// A lane's tokens (up to four, 32 apart): e / 64 of each in a byte, and whether a
// product other than zero has been seen (bits 0 to 3 of `seen`).
struct TokenExponents {
  uint32_t e = 0u, seen = 0u;

  // Takes in token j's products of a batch, of which `most` is the largest; `any`:
  // it and the weight have a scale other than zero (the products may all be lost).
  // True where the batch has to go through scales_apart.
  __device__ __forceinline__ bool add(int j, float most, bool any) {
    const uint32_t bit = 1u << j;
    if (most > kScalesHigh || (most < kScalesLow && any && !(seen & bit))) return true;
    if (most > 0.0f) seen |= bit;
    return e != 0u;
  }
};

// 2^(64 n) for n from -8 to 8.
__device__ __forceinline__ double pow2_64(int n) {
  return __hiloint2double((1023 + 64 * n) << 20, 0);
}

// A batch with some product outside the range, or some e other than 0: moves the
// lane's exponents on, writes the batch's products again ([blocks][NWB][LD] floats
// in `slot`) and what the epilogue reads ([LD] factors, [LD] e / 64), and returns
// the batch's word.  row: the lane's first token, `local` its place among LD.
template <int NWB, int LD, int BLOCKS>
__device__ __noinline__ uint32_t scales_apart(const B128Args& a, TokenExponents& t, float* slot,
                                              float* factor, int* exponent, int row, int local,
                                              int wb0, int k0, int ke) {
  uint32_t word = 0u;
#pragma unroll 1
  for (int j = 0; j < 4 && local + 32 * j < LD; ++j) {
    const int r = row + 32 * j, at = local + 32 * j;
    const int old = static_cast<int8_t>(t.e >> (8 * j));
    double most = 0.0;
#pragma unroll 4
    for (int i = 0; i < BLOCKS * NWB; ++i) {
      const int k = k0 + i / NWB, wb = wb0 + i % NWB;
      if (r < a.m && k < ke && wb * 128 < a.n) {
        const double p = static_cast<double>(a.sa[static_cast<int64_t>(r) * a.num_kb + k]) *
                         static_cast<double>(a.sw[static_cast<int64_t>(wb) * a.sw_n +
                                                  static_cast<int64_t>(k) * a.sw_k]);
        if (fabs(p) > most && fabs(p) < 0x1p300) most = fabs(p);   // finite scales
      }
    }
    int e = old;
    if (most > 0.0) {
      int want = 0;
      if (most < kScalesLow || most > kScalesHigh) {
        const int x = (__double2hiint(most) >> 20) - 1023;   // most is 2^x to 2^(x + 1)
        want = (x + 32) >> 6;
      }
      e = (t.seen >> j) & 1u ? max(old, want) : want;
      t.seen |= 1u << j;
    }
    t.e = (t.e & ~(0xFFu << (8 * j))) | ((static_cast<uint32_t>(e) & 0xFFu) << (8 * j));
#pragma unroll 4
    for (int i = 0; i < BLOCKS * NWB; ++i) {
      const int k = k0 + i / NWB, wb = wb0 + i % NWB;
      float p = 0.0f;
      if (r < a.m && k < ke && wb * 128 < a.n)
        p = static_cast<float>(static_cast<double>(a.sa[static_cast<int64_t>(r) * a.num_kb + k]) *
                               static_cast<double>(a.sw[static_cast<int64_t>(wb) * a.sw_n +
                                                        static_cast<int64_t>(k) * a.sw_k]) *
                               pow2_64(-e));
      slot[i * LD + at] = p;
    }
    // the sums so far go from 2^-old to 2^-e (they are zero where e falls)
    factor[at] = e > old ? static_cast<float>(pow2_64(old - e)) : 1.0f;
    exponent[at] = e;
    word |= (e > old ? kBatchFactors : 0u) | (e != 0 ? kBatchExponents : 0u);
  }
  return __reduce_or_sync(0xffffffffu, word);
}

// v times 2^(64 e), in steps that stay in range.
__device__ __forceinline__ float times_pow2_64(float v, int e) {
  const float s = __uint_as_float((127 + 16 * e) << 23);
  return v * s * s * s * s;
}

}  // namespace forge

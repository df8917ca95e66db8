// The 128-block e4m3 format of the norm, the quantiser and the 8-bit products:
// a block with largest magnitude a is stored as codes e4m3(x / s) and one fp32
// scale s = a / 448, so its largest entry takes the largest code.
#pragma once

#include "forge_math.cuh"

namespace forge {

constexpr int kBlock = 128;   // columns (and, for weights, rows) per scale

struct BlockScale {
  float scale;   // value = e4m3(code) * scale
  float inv;     // code = e4m3(value * inv)
};
// A scale is never subnormal: below 2^-126 it would lose its own digits and
// its reciprocal would overflow; entries that small keep the scale 2^-126 and
// use fewer of the codes.  An all-zero block has scale 0 and codes 0.  A
// block that holds a NaN or an infinity has a NaN or infinite scale and
// decodes to NaN throughout.  inv is 448 / a rounded once rather than
// 1 / scale, which would round twice.
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale s{amax, amax};
  if (amax > 0.0f) {
    s.scale = fmaxf(__fdiv_rn(amax, kE4m3Max), 0x1p-126f);
    s.inv = fminf(__fdiv_rn(kE4m3Max, amax), 0x1p126f);
  }
  return s;
}

// max that returns NaN if either input is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The largest of a value over each aligned group of 16 lanes (128 columns, 8
// a lane).
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The same over aligned groups of 8 lanes.
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Eight floats times inv as eight codes (the first in the low byte).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 q = mul2(make_float2(x[2 * k], x[2 * k + 1]), dup2(inv));
    c[k] = float2_to_e4m3x2(q.x, q.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The same for bf16 values of a block whose amax is bf16 too, with the codes of
// the true quotients 448 x / amax, ties to even.  Such a quotient is a tie
// between two codes or at least 2^-13 of itself away from one (8-bit
// significands, ties of 5 bits), but x * inv is up to 2 ulp off and falls on
// either side of a tie.  With 448 / amax as inv + lo the product is right to
// 2^-40 before its rounding, and a tie comes out as the tie.  lo >= 0, so that a
// zero keeps its sign.  Measured, without and with lo: 8192 x 14336 51.7 and
// 51.8 us, 8192 x 4104 19.8 and 20.2, 4096 x 4096 in 128 x 128 blocks 10.1 and 10.4.
struct QuotientScale {
  float scale, inv, lo;
};
__device__ __forceinline__ QuotientScale quotient_scale(float amax) {
  QuotientScale s{amax, amax, 0.0f};
  if (amax > 0.0f) {
    s.scale = fmaxf(__fdiv_rn(amax, kE4m3Max), 0x1p-126f);
    float inv = fminf(__fdiv_rn(kE4m3Max, amax), 0x1p126f);
    // rounded down: the remainder 448 - inv amax, exact, is not negative
    if (fmaf(-inv, amax, kE4m3Max) < 0.0f) inv = __uint_as_float(__float_as_uint(inv) - 1u);
    const float lo = fmaf(-inv, amax, kE4m3Max) * (inv * (1.0f / kE4m3Max));
    s.inv = inv;
    s.lo = inv < 0x1p126f ? lo : 0.0f;
  }
  return s;
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const QuotientScale& s) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = make_float2(x[2 * k], x[2 * k + 1]);
    const float2 q = fma2(v, dup2(s.inv), mul2(v, dup2(s.lo)));
    c[k] = float2_to_e4m3x2(q.x, q.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = bf16_lo(u[k]);
    f[2 * k + 1] = bf16_hi(u[k]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

}  // namespace forge

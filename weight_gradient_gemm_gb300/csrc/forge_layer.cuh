// What the operators between a layer's 16-bit products share: activations and their
// derivatives, the dropout generator, and the product's epilogue on eight
// neighbouring outputs.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "forge_e4m3.cuh"
#include "forge_internal.h"

namespace forge {

// ---------------------------------------------------------------- activations
// The forward value and the derivative with respect to z, in fp32.  1 / (1 + e^-x)
// uses the hardware's exponential (2 + 1.2 |x| ulp) and quotient (2 ulp): in all the
// places where it is not negligible far below bf16's half step of 2^-9.
__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}
constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The normal distribution function, (1 + erf(z / sqrt 2)) / 2 = erfc(-z / sqrt 2) / 2.
// erfc by the Chebyshev fit of Press et al., "Numerical Recipes" (erfcc): t e^(P(t) - x^2)
// with t = 1 / (1 + x / 2), its relative error below 1.2 10^-7 for all x >= 0, so that the
// tail below zero keeps its digits.  Without branches: in the product's epilogue erfcf
// cost 8192 tokens, 4096 -> 14336, 35 us.
__device__ __forceinline__ float normal_cdf(float z) {
  const float x = fabsf(z) * kInvSqrt2;
  const float t = __fdividef(1.0f, fmaf(0.5f, x, 1.0f));
  float p = fmaf(t, 0.17087277f, -0.82215223f);
  p = fmaf(t, p, 1.48851587f);
  p = fmaf(t, p, -1.13520398f);
  p = fmaf(t, p, 0.27886807f);
  p = fmaf(t, p, -0.18628806f);
  p = fmaf(t, p, 0.09678418f);
  p = fmaf(t, p, 0.37409196f);
  p = fmaf(t, p, 1.00002368f);
  p = fmaf(t, p, -1.26551223f);
  const float tail = 0.5f * t * __expf(fmaf(-x, x, p));
  return z > 0.0f ? 1.0f - tail : tail;
}
// tanh(u) as 2 sigmoid(2u) - 1, so that z (1 + tanh u) / 2 = z sigmoid(2u).
__device__ __forceinline__ float gelu_arg(float z) {
  return 2.0f * kGeluC * fmaf(kGeluB * z * z, z, z);
}
// Beyond +-128 the smooth activations are 0 or z and their derivatives 0 or 1, in fp32;
// held there, infinities give that too, and no product leaves fp32's range.  (NaN stays
// NaN.)
__device__ __forceinline__ float hold_low(float z) { return z < -128.0f ? -128.0f : z; }
__device__ __forceinline__ float hold(float z) { return z > 128.0f ? 128.0f : hold_low(z); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;   // NaN stays NaN
  if constexpr (ACT == kActNone) return z;
  z = hold_low(z);
  if constexpr (ACT == kActGelu) return z * normal_cdf(z);
  if constexpr (ACT == kActGeluTanh) return z * sigmoid(gelu_arg(z));
  return z * sigmoid(z);   // kActSilu
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == kActGelu) {
    const float h = hold(z);
    return fmaf(h * kInvSqrt2Pi, __expf(-0.5f * h * h), normal_cdf(h));
  }
  if constexpr (ACT == kActGeluTanh) {
    const float h = hold(z), s = sigmoid(gelu_arg(h));
    const float du = 2.0f * kGeluC * fmaf(3.0f * kGeluB * h, h, 1.0f);
    return fmaf(h * du * s, 1.0f - s, s);
  }
  if constexpr (ACT == kActSilu) {
    const float h = hold(z), s = sigmoid(h);
    return fmaf(h * s, 1.0f - s, s);
  }
  return 1.0f;
}
// f(integral_constant) with the activation of a call, which is the same in all threads.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    default: f(ActTag<kActNone>{});
  }
}

// ---------------------------------------------------------------- dropout
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): block `b` of eight neighbouring
// elements draws 128 bits, 16 for each.  16 bits resolve the probability to 2^-16 and
// halve the generator's work per element against 32; its 32-bit products cost half
// of those of the 64-bit form that the stochastic rounding uses.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c.x;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
    c = make_uint4(static_cast<uint32_t>(p1 >> 32) ^ c.y ^ k0, static_cast<uint32_t>(p1),
                   static_cast<uint32_t>(p0 >> 32) ^ c.w ^ k1, static_cast<uint32_t>(p0));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}
// The call's offset (its device word read after the wait for earlier launches).
__device__ __forceinline__ uint64_t drop_offset(const DropArgs& d) {
  return d.offset + (d.counter ? __ldcg(reinterpret_cast<const unsigned long long*>(d.counter)) : 0);
}
// Which elements of block b are kept, a bit each.
__device__ __forceinline__ uint32_t kept8(const DropArgs& d, uint64_t offset, uint64_t b) {
  const uint4 w = philox4x32_10(
      make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32),
                 static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)),
      static_cast<uint32_t>(d.seed), static_cast<uint32_t>(d.seed >> 32));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t kept = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((u[j] & 0xFFFFu) >= d.threshold) kept |= 1u << (2 * j);
    if ((u[j] >> 16) >= d.threshold) kept |= 2u << (2 * j);
  }
  return kept;
}
// v = 0 where dropped (whatever it was), v * scale elsewhere.
__device__ __forceinline__ void drop8(float (&v)[8], const DropArgs& d, uint32_t kept) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = kept >> k & 1u ? v[k] * d.scale : 0.0f;
}

// ---------------------------------------------------------------- the epilogue
// Eight values at column c of `bias` (fp32 or bf16).
__device__ __forceinline__ void load_bias8(const void* bias, int bf16, int64_t c, float (&b)[8]) {
  if (bf16) {
    unpack8(reinterpret_cast<const uint4*>(bias)[c / 8], b);
  } else {
    const float4 x = reinterpret_cast<const float4*>(bias)[c / 4];
    const float4 y = reinterpret_cast<const float4*>(bias)[c / 4 + 1];
    b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
    b[4] = y.x; b[5] = y.y; b[6] = y.z; b[7] = y.w;
  }
}
// With z (the bias is in it): returns it packed, for the stored pre-activation, and
// makes it residual + drop(act(z) mul).  mul, residual: eight bf16 values, read where the
// call has them; block: the elements' dropout block.
template <int ACT>
__device__ __forceinline__ uint4 epilogue8(float (&v)[8], const EpiArgs& e, uint4 mul,
                                           uint4 residual, uint64_t offset, uint64_t block) {
  uint4 z = make_uint4(0, 0, 0, 0);
  if (e.z) z = pack8(v);
  if constexpr (ACT != kActNone) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value<ACT>(v[k]);
  }
  if (e.mul) {
    float m[8];
    unpack8(mul, m);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= m[k];
  }
  if (e.drop.threshold) drop8(v, e.drop, kept8(e.drop, offset, block));
  if (e.residual) {
    float r[8];
    unpack8(residual, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += r[k];
  }
  return z;
}

}  // namespace forge

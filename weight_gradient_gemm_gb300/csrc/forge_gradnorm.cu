// The global norm of a model's gradients and the clipping coefficient,
//   norm = sqrt(sum over all tensors of g^2),  coef = min(1, max_norm / (norm + 1e-6)),
// left in device memory for the optimizer step that reads the gradients next.
//
// One pass over the gradients.  The tensors are cut into units of kNormUnit
// elements so that blocks share the work evenly whatever the tensors' sizes;
// each block leaves one partial sum, and a second launch adds the partials in
// a fixed order, so the norm is the same on every run.
//
// Bound by memory: the 218 M fp32 gradients of a 4096-wide layer (872 MB) take
// 127 us, 6.9 TB/s, a plain copy's rate; in bf16 71 us, 6.1 TB/s, of which about
// 6 us are the two launches and their tails.  Few values cost the launches alone
// (5.4 us for six small tensors; one launch of a single cluster, whose blocks
// join through shared memory, took 8.2 where two took 6.8).
#include "forge_internal.h"
#include "forge_launch.cuh"

namespace forge {
namespace {

constexpr int kThreads = 256;

// Sum of squares of N values as a double: in fp32 where no square can overflow
// or lose digits to underflow, else element by element in fp64.  A sum of at
// least 2^-100 bounds what underflowed squares could add to it (N x 2^-126)
// below its rounding; all-zero runs, common in embedding gradients, leave
// before the slow path.  fp64 runs at 1/64 of the fp32 rate, so a conversion
// and an addition for every 32 values keep it out of the way.
template <int N>
__device__ __forceinline__ double squares(const float (&g)[N]) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < N; ++k) s[k & 3] = fmaf(g[k], g[k], s[k & 3]);
  const float t = (s[0] + s[1]) + (s[2] + s[3]);
  if (t >= 0x1p-100f && t <= 0x1p126f) return static_cast<double>(t);
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) any |= __float_as_uint(g[k]) & 0x7FFFFFFFu;
  double d = 0.0;
  if (any) {
#pragma unroll
    for (int k = 0; k < N; ++k) d += static_cast<double>(g[k]) * static_cast<double>(g[k]);
  }
  return d;
}

// The sum over the block, in every thread and in a fixed order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += red[w];
  return v;
}

// Values 8 i8 .. 8 i8 + 7 of a tensor.
__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t i8, float* g) {
  if (bf16) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i8);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) { g[2 * k] = bf16_lo(u[k]); g[2 * k + 1] = bf16_hi(u[k]); }
  } else {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i8);
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i8 + 1);
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  }
}

// One block's share of the units, as a sum of squares (in every thread).
__device__ __forceinline__ double units_sum(const GradNormArgs& a) {
  double sum = 0.0;
  const int units = a.unit0[a.n];
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int lo = 0, hi = a.n - 1;   // the tensor with unit0[t] <= u < unit0[t + 1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.unit0[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const bool bf16 = (a.bf16[lo >> 6] >> (lo & 63)) & 1;
    const int64_t begin = static_cast<int64_t>(u - a.unit0[lo]) * kNormUnit;
    const int64_t left = a.numel[lo] - begin;
    const int count = static_cast<int>(left < kNormUnit ? left : kNormUnit);
    const void* p = a.ptr[lo];
    // 32 values a thread at a time, in four vectors kThreads apart
    int e = threadIdx.x * 8;
    for (; e + 3 * kThreads * 8 + 8 <= count; e += 4 * kThreads * 8) {
      float g[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) load8(p, bf16, (begin + e + j * kThreads * 8) >> 3, g + 8 * j);
      sum += squares(g);
    }
    for (; e < count; e += kThreads * 8) {
      float g[8];
      if (e + 8 <= count) {
        load8(p, bf16, (begin + e) >> 3, g);
      } else {   // the tensor's last, partial vector
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          g[k] = 0.0f;
          if (e + k < count)
            g[k] = bf16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p)[begin + e + k])
                        : reinterpret_cast<const float*>(p)[begin + e + k];
        }
      }
      sum += squares(g);
    }
  }
  return block_sum(sum);
}

// norm = sqrt(s) and the coefficient, from the sum of squares.
__device__ __forceinline__ void write_norm(double s, float max_norm, float* out) {
  const double norm = sqrt(s);
  const double c = static_cast<double>(max_norm) / (norm + 1e-6);
  out[0] = static_cast<float>(norm);
  out[1] = c >= 1.0 ? 1.0f : static_cast<float>(c);   // NaN stays NaN
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ GradNormArgs a) {
  grid_dependency_wait();
  const double sum = units_sum(a);
  grid_dependency_trigger();
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) grad_norm_final_kernel(const double* __restrict__ part,
                                                                   int n, float max_norm,
                                                                   float* __restrict__ out) {
  grid_dependency_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += __ldcg(part + i);
  s = block_sum(s);
  if (threadIdx.x == 0) write_norm(s, max_norm, out);
}

}  // namespace

int grad_norm_blocks(int64_t units, int num_sms) {
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(units < most ? units : most);
}

cudaError_t launch_grad_norm(const GradNormArgs& a, int blocks, cudaStream_t stream) {
  return launch_chained(grad_norm_kernel, blocks, kThreads, 0, 0, stream, a);
}

cudaError_t launch_grad_norm_final(const double* part, int n, float max_norm, float* out,
                                   cudaStream_t stream) {
  return launch_chained(grad_norm_final_kernel, 1, kThreads, 0, 0, stream, part, n, max_norm, out);
}

}  // namespace forge

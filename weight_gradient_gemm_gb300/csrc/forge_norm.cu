// The RMS norm in front of a linear layer, its backward pass, and the
// quantiser of the 128-block e4m3 format.  All three stream their tensors
// once; a row (or a block) stays in registers between the reduction it needs
// and the values that depend on it.
#include <cuda_bf16.h>

#include "forge_e4m3.cuh"
#include "forge_internal.h"

namespace forge {
namespace {

// Sum of v over the block, the same in every thread and on every run.  `red`
// holds one float per warp; a caller that reduces again passes another array
// (or synchronises in between).
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void load_gain8(const void* gain, int bf16, int v, float (&g)[8]) {
  if (bf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(gain) + v), g);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(gain) + 2 * v);
    const float4 b = __ldg(reinterpret_cast<const float4*>(gain) + 2 * v + 1);
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  }
}

//   h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gain
// in fp32 from the bf16 inputs (the sum is rounded only where it is stored).
// One block per row (grid-stride); thread t owns the vectors of 8 columns t,
// t + threads, ..., so 16 neighbouring lanes hold the 128 columns of a scale.
template <int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  const int nvec = a.cols / 8;
  const int nblk = (a.cols + kBlock - 1) / kBlock;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const int64_t base = row * nvec;
    float h[VPT][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = 0.0f;
      if (v < nvec) {
        unpack8(__ldcs(reinterpret_cast<const uint4*>(a.x) + base + v), h[i]);
        if (a.residual) {
          float r[8];
          unpack8(__ldcs(reinterpret_cast<const uint4*>(a.residual) + base + v), r);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][k] += r[k];
        }
        if (a.sum) __stcs(reinterpret_cast<uint4*>(a.sum) + base + v, pack8(h[i]));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(h[i][k], h[i][k], ss);
    }
    ss = block_sum(ss, red[parity]);
    const float rstd = rsqrtf(__fdiv_rn(ss, static_cast<float>(a.cols)) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      float amax = 0.0f;
      if (v < nvec) {
        float g[8];
        load_gain8(a.gain, a.gain_bf16, v, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[i][k] = h[i][k] * rstd * g[k];
          amax = max_nan(amax, fabsf(h[i][k]));
        }
        if (a.y) __stcs(reinterpret_cast<uint4*>(a.y) + base + v, pack8(h[i]));
      }
      if (a.codes) {
        const BlockScale s = block_scale(max16(amax));
        if (v < nvec) {
          __stcs(reinterpret_cast<uint2*>(a.codes) + base + v, encode8(h[i], s.inv));
          if (v % 16 == 0) a.scales[row * nblk + v / 16] = s.scale;
        }
      }
    }
  }
}

// With xh = h rstd and u = dy gain, the gradient of y = xh gain with respect
// to h is rstd (u - xh mean(u xh)); dsum, the gradient that reaches h along
// the residual stream, is added.  dgain = sum over rows of dy xh: a block
// adds its rows in registers and leaves one partial row, which
// rmsnorm_dgain_kernel adds in a fixed order.
template <int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[2][32];
  const int nvec = a.cols / 8;
  int parity = 0;
  float dg[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i][k] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const int64_t base = row * nvec;
    const float rstd = __ldg(a.rstd + row);
    uint4 hv[VPT], dv[VPT];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      hv[i] = dv[i] = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        hv[i] = __ldcs(reinterpret_cast<const uint4*>(a.h) + base + v);
        dv[i] = __ldcs(reinterpret_cast<const uint4*>(a.dy) + base + v);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        float h[8], d[8], g[8];
        unpack8(hv[i], h);
        unpack8(dv[i], d);
        load_gain8(a.gain, a.gain_bf16, v, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float t = d[k] * (h[k] * rstd);
          dg[i][k] += t;
          dot = fmaf(t, g[k], dot);
        }
      }
    }
    const float c = __fdiv_rn(block_sum(dot, red[parity]), static_cast<float>(a.cols));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        float h[8], d[8], g[8], o[8];
        unpack8(hv[i], h);
        unpack8(dv[i], d);
        load_gain8(a.gain, a.gain_bf16, v, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = rstd * fmaf(-c, h[k] * rstd, d[k] * g[k]);
        if (a.dsum) {
          float r[8];
          unpack8(__ldcs(reinterpret_cast<const uint4*>(a.dsum) + base + v), r);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] += r[k];
        }
        __stcs(reinterpret_cast<uint4*>(a.dx) + base + v, pack8(o));
      }
    }
  }
  if (a.dgain) {
    float4* part = reinterpret_cast<float4*>(a.part) + static_cast<int64_t>(blockIdx.x) * nvec * 2;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        part[2 * v] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
        part[2 * v + 1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
      }
    }
  }
}

// dgain[c] = sum over the blocks' partial rows: 32 columns a block, 8 runs of
// rows side by side, added in a fixed order.
__global__ void __launch_bounds__(256) rmsnorm_dgain_kernel(const float* __restrict__ part,
                                                            int blocks, int cols,
                                                            float* __restrict__ dgain) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int b = run; b < blocks; b += 8) s += part[static_cast<int64_t>(b) * cols + c];
  sum[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sum[k][lane];
    dgain[c] = s;
  }
}

// Largest magnitude of eight bf16 values; NaN if one of them is.
__device__ __forceinline__ float amax8(uint4 v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[0]));
#pragma unroll
  for (int k = 1; k < 4; ++k)
    m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[k])));
  return max_nan(__low2float(m), __high2float(m));
}

// Blocks of 1 x 128: 8 lanes per block, two vectors of 8 columns a lane, so
// that one reduction and one pair of divisions serve 16 of a lane's values.
constexpr int kQuantUnroll = 4;   // blocks per lane group whose loads are in flight at once

// Rows of whole blocks: the blocks of all rows follow one another, and a
// warp's groups take 4 x kQuantUnroll neighbouring ones.
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const uint4* __restrict__ x,
                                                              uint2* __restrict__ codes,
                                                              float* __restrict__ scales,
                                                              int64_t blocks) {
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t b0 =
      (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (4 * kQuantUnroll) + (lane >> 3);
  uint4 v[kQuantUnroll][2];
#pragma unroll
  for (int j = 0; j < kQuantUnroll; ++j) {
    const int64_t b = b0 + 4 * j;
    v[j][0] = v[j][1] = make_uint4(0, 0, 0, 0);
    if (b < blocks) {
      v[j][0] = __ldcs(x + b * 16 + sub);
      v[j][1] = __ldcs(x + b * 16 + 8 + sub);
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantUnroll; ++j) {
    const int64_t b = b0 + 4 * j;
    const BlockScale s = block_scale(max8(max_nan(amax8(v[j][0]), amax8(v[j][1]))));
    if (b < blocks) {
      float f[8];
      unpack8(v[j][0], f);
      __stcs(codes + b * 16 + sub, encode8(f, s.inv));
      unpack8(v[j][1], f);
      __stcs(codes + b * 16 + 8 + sub, encode8(f, s.inv));
      if (sub == 0) scales[b] = s.scale;
    }
  }
}

// Any row length: the last block of a row may be partial.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint4* __restrict__ x,
                                                            uint2* __restrict__ codes,
                                                            float* __restrict__ scales,
                                                            int64_t rows, int nvec) {
  const int nblk = (nvec + 15) / 16, sub = threadIdx.x & 7;
  const int64_t total = rows * nblk, groups = static_cast<int64_t>(gridDim.x) * 32;
  // every lane of a warp takes the same number of trips (the shuffles)
  for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * 32 + ((threadIdx.x >> 5) << 2); b0 < total;
       b0 += groups) {
    const int64_t b = b0 + ((threadIdx.x >> 3) & 3);
    const int64_t row = total <= INT32_MAX ? static_cast<int>(b) / nblk : b / nblk;
    const int vec = static_cast<int>(b - row * nblk) * 16 + sub;
    const bool in0 = b < total && vec < nvec, in1 = b < total && vec + 8 < nvec;
    const int64_t at = row * nvec + vec;
    const uint4 v0 = in0 ? __ldcs(x + at) : make_uint4(0, 0, 0, 0);
    const uint4 v1 = in1 ? __ldcs(x + at + 8) : make_uint4(0, 0, 0, 0);
    const BlockScale s = block_scale(max8(max_nan(amax8(v0), amax8(v1))));
    float f[8];
    if (in0) {
      unpack8(v0, f);
      __stcs(codes + at, encode8(f, s.inv));
    }
    if (in1) {
      unpack8(v1, f);
      __stcs(codes + at + 8, encode8(f, s.inv));
    }
    if (in0 && sub == 0) scales[b] = s.scale;
  }
}

// Blocks of 128 x 128: one CTA per block, the block in registers.
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const uint16_t* __restrict__ x,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales,
                                                             int64_t rows, int64_t cols) {
  __shared__ float red[8];
  const int64_t nblk = (cols + kBlock - 1) / kBlock;
  const int64_t br = blockIdx.x / nblk, bc = blockIdx.x % nblk;
  const int64_t col = bc * kBlock + (threadIdx.x & 15) * 8;
  const int64_t row0 = br * kBlock + (threadIdx.x >> 4);
  uint4 v[8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (col < cols && row0 + 16 * i < rows)
      v[i] = __ldcs(reinterpret_cast<const uint4*>(x + (row0 + 16 * i) * cols + col));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_nan(amax, amax8(v[i]));
  amax = max16(amax);
  amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = max_nan(amax, red[w]);
  const BlockScale s = block_scale(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col < cols && row0 + 16 * i < rows) {
      float f[8];
      unpack8(v[i], f);
      __stcs(reinterpret_cast<uint2*>(codes + (row0 + 16 * i) * cols + col), encode8(f, s.inv));
    }
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

// Threads a row needs with VPT vectors each, a multiple of 32.
int row_threads(int cols, int vpt) {
  const int t = (cols / 8 + vpt - 1) / vpt;
  return (t + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int vpt = a.cols <= 8192 ? 1 : (a.cols <= 16384 ? 2 : 4);
  const int threads = row_threads(a.cols, vpt);
  const int64_t most = static_cast<int64_t>(num_sms) * (2048 / threads);
  const int grid = static_cast<int>(a.rows < most ? a.rows : most);
  switch (vpt) {
    case 1: rmsnorm_kernel<1><<<grid, threads, 0, stream>>>(a); break;
    case 2: rmsnorm_kernel<2><<<grid, threads, 0, stream>>>(a); break;
    default: rmsnorm_kernel<4><<<grid, threads, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

int rmsnorm_bwd_blocks(int64_t rows, int cols, int num_sms) {
  const int64_t most = static_cast<int64_t>(num_sms) * 2;
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int num_sms, cudaStream_t stream) {
  const int vpt = a.cols <= 8192 ? 1 : (a.cols <= 16384 ? 2 : 4);
  const int threads = row_threads(a.cols, vpt);
  const int grid = rmsnorm_bwd_blocks(a.rows, a.cols, num_sms);
  switch (vpt) {
    case 1: rmsnorm_bwd_kernel<1><<<grid, threads, 0, stream>>>(a); break;
    case 2: rmsnorm_bwd_kernel<2><<<grid, threads, 0, stream>>>(a); break;
    default: rmsnorm_bwd_kernel<4><<<grid, threads, 0, stream>>>(a); break;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dgain) return e;
  rmsnorm_dgain_kernel<<<(a.cols + 31) / 32, 256, 0, stream>>>(a.part, grid, a.cols, a.dgain);
  return cudaGetLastError();
}

cudaError_t launch_quantize_b128(const uint16_t* x, uint8_t* codes, float* scales, int64_t rows,
                                 int64_t cols, int block_rows, int num_sms, cudaStream_t stream) {
  const int64_t nblk = (cols + kBlock - 1) / kBlock;
  if (block_rows == 1) {
    const uint4* xv = reinterpret_cast<const uint4*>(x);
    uint2* cv = reinterpret_cast<uint2*>(codes);
    const int64_t blocks = rows * nblk;
    const int64_t grid = (blocks + 32 * kQuantUnroll - 1) / (32 * kQuantUnroll);
    if (cols % kBlock == 0 && grid <= INT32_MAX) {
      quantize_blocks_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(xv, cv, scales, blocks);
    } else {
      const int64_t want = (blocks + 31) / 32, most = static_cast<int64_t>(num_sms) * 8;
      quantize_rows_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, stream>>>(
          xv, cv, scales, rows, static_cast<int>(cols / 8));
    }
  } else {
    const int64_t grid = (rows + kBlock - 1) / kBlock * nblk;
    quantize_tiles_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(x, codes, scales, rows,
                                                                          cols);
  }
  return cudaGetLastError();
}

}  // namespace forge

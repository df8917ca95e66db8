// The gradient of the 16-bit product's epilogue, and dropout by itself.
#include <cuda_bf16.h>

#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_layer.cuh"
#include "forge_ptx.cuh"

namespace forge {
namespace {

// ---------------------------------------------------------------- dropout
// y = residual + drop(x), eight elements (one generator block) a thread and vector.
// U vectors' loads are in flight at once.  Bound by memory (the generator is 9
// instructions an element): 8191 x 4096 with the residual 30.4 us, 29.6 at the copy rate;
// 64 x 520 1.4 on the device, 3.2 through Python.
template <int U>
__global__ void __launch_bounds__(256) dropout_kernel(const uint4* x, const uint4* residual,
                                                      uint4* y, int64_t nvec, const DropArgs d) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * U) + threadIdx.x;
  grid_dependency_wait();
  grid_dependency_trigger();
  uint4 xv[U], rv[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + 256 * i;
    if (v < nvec) {
      xv[i] = __ldcs(x + v);
      if (residual) rv[i] = __ldcs(residual + v);
    }
  }
  const uint64_t offset = drop_offset(d);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + 256 * i;
    if (v < nvec) {
      float f[8];
      unpack8(xv[i], f);
      if (d.threshold) drop8(f, d, kept8(d, offset, static_cast<uint64_t>(v)));
      if (residual) {
        float r[8];
        unpack8(rv[i], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] += r[k];
      }
      __stcs(y + v, pack8(f));
    }
  }
}

// ---------------------------------------------------------------- backward
//   dA = drop(dY),  dmul = dA act(Z),  dZ = dA mul act'(Z),  dbias = sum over rows of dZ
// in fp32 (dZ rounded only where it is stored).  Where an element was dropped all its
// gradients are zero, also where Z or mul is NaN or infinite there.
template <int ACT, bool MUL>
__device__ __forceinline__ void bwd8(const EpiBwdArgs& a, uint4 dyv, uint4 zv, uint4 mv,
                                     uint64_t offset, int64_t at, float (&dz)[8]) {
  unpack8(dyv, dz);
  uint32_t kept = 0xFFu;
  if (a.drop.threshold) {
    kept = kept8(a.drop, offset, static_cast<uint64_t>(at));
    drop8(dz, a.drop, kept);
  }
  float z[8];
  if (ACT != kActNone || MUL) unpack8(zv, z);
  if constexpr (MUL) {
    float m[8];
    unpack8(mv, m);
    if (a.dmul) {
      float dm[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) dm[k] = kept >> k & 1u ? dz[k] * act_value<ACT>(z[k]) : 0.0f;
      __stcs(reinterpret_cast<uint4*>(a.dmul) + at, pack8(dm));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) dz[k] *= m[k];
  }
  if constexpr (ACT != kActNone) {
#pragma unroll
    for (int k = 0; k < 8; ++k) dz[k] *= act_slope<ACT>(z[k]);
  }
  if (kept != 0xFFu) {
#pragma unroll
    for (int k = 0; k < 8; ++k) dz[k] = kept >> k & 1u ? dz[k] : 0.0f;
  }
  if (a.dz) __stcs(reinterpret_cast<uint4*>(a.dz) + at, pack8(dz));
}

// Without dbias: vectors in memory order.  8192 x 14336 with SILU and mul, 1.17 GB, 171.5 us
// (6.8 TB/s, the copy rate; three fifths of it reads).
template <int ACT, bool MUL>
__global__ void __launch_bounds__(256) epilogue_bwd_kernel(const EpiBwdArgs a) {
  constexpr int U = 2;
  const int64_t nvec = a.rows * (a.cols / 8);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * U) + threadIdx.x;
  grid_dependency_wait();
  grid_dependency_trigger();
  uint4 dy[U], z[U], m[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + 256 * i;
    dy[i] = z[i] = m[i] = make_uint4(0, 0, 0, 0);
    if (v < nvec) {
      dy[i] = __ldcs(reinterpret_cast<const uint4*>(a.dy) + v);
      if (ACT != kActNone || (MUL && a.dmul)) z[i] = __ldcs(reinterpret_cast<const uint4*>(a.z) + v);
      if (MUL) m[i] = __ldcs(reinterpret_cast<const uint4*>(a.mul) + v);
    }
  }
  const uint64_t offset = drop_offset(a.drop);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + 256 * i;
    float dz[8];
    if (v < nvec) bwd8<ACT, MUL>(a, dy[i], z[i], m[i], offset, v, dz);
  }
}

// With dbias: a block takes a strip of 8 L columns and a run of rows, L lanes to a row; a
// thread adds its eight columns over its rows, and the block's sums are joined in shared
// memory.  Up to eight runs of rows are the blocks of a cluster, whose first adds up the
// others' sums through distributed shared memory: one launch.  More leave a partial row
// each for a second one.  333 x 520 with GELU and dropout 4.4 us; 2000 x 4096 with dropout
// 18.8, 8192 x 4096 46.3 (its bytes 19.8), dbias alone 24.1 (9.9); 8192 x 14336 with SILU and
// mul 314 (173), with GELU 225 (104): twice what the bytes take, for reasons not looked into
// (121 registers a thread leave two blocks an SM).
constexpr int kBiasCluster = 8;
template <int ACT, bool MUL>
__global__ void __launch_bounds__(256) epilogue_bwd_bias_kernel(const EpiBwdArgs a, int lanes,
                                                                int parts, int cluster) {
  constexpr int U = MUL ? 2 : 4;   // rows whose loads are in flight at once
  __shared__ float4 sums[512];     // [row of the block][column / 4]
  __shared__ float some[256], joined[128];
  const int64_t nv = a.cols / 8;
  const int strip = static_cast<int>(blockIdx.x) / parts, part = blockIdx.x - strip * parts;
  const int lane = threadIdx.x & (lanes - 1), cols = 8 * lanes, rows = 256 / lanes;
  const int64_t v = static_cast<int64_t>(strip) * lanes + lane;
  const int64_t each = (a.rows + parts - 1) / parts;
  const int64_t r0 = each * part, r1 = min(a.rows, r0 + each);
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  grid_dependency_wait();
  const uint64_t offset = drop_offset(a.drop);
  if (v < nv) {
    for (int64_t row = r0 + threadIdx.x / lanes; row < r1; row += rows * U) {
      uint4 dy[U], z[U], m[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t at = (row + rows * i) * nv + v;
        dy[i] = z[i] = m[i] = make_uint4(0, 0, 0, 0);
        if (row + rows * i < r1) {
          dy[i] = __ldcs(reinterpret_cast<const uint4*>(a.dy) + at);
          if (ACT != kActNone || (MUL && a.dmul))
            z[i] = __ldcs(reinterpret_cast<const uint4*>(a.z) + at);
          if (MUL) m[i] = __ldcs(reinterpret_cast<const uint4*>(a.mul) + at);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (row + rows * i < r1) {
          float dz[8];
          bwd8<ACT, MUL>(a, dy[i], z[i], m[i], offset, (row + rows * i) * nv + v, dz);
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[k] += dz[k];
        }
    }
  }
  grid_dependency_trigger();
  sums[2 * threadIdx.x] = make_float4(sum[0], sum[1], sum[2], sum[3]);
  sums[2 * threadIdx.x + 1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
  __syncthreads();
  // a column's sums: `runs` threads each add some, the first adds theirs
  const int col = threadIdx.x & (cols - 1), runs = 256 / cols;
  float s = 0.0f;
  for (int r = threadIdx.x / cols; r < rows; r += runs)
    s += reinterpret_cast<const float*>(sums)[r * cols + col];
  some[threadIdx.x] = s;
  __syncthreads();
  const bool mine = static_cast<int>(threadIdx.x) < cols;
  if (mine)
    for (int r = 1; r < runs; ++r) s += some[r * cols + col];
  if (cluster) {   // its rank is `part`
    if (mine) joined[col] = s;
    cluster_sync_all();
    if (part == 0 && mine) {
      const uint32_t at = smem_u32(joined + col);
      for (int r = 1; r < parts; ++r) s += ld_cluster_f32(mapa_shared(at, r));
    }
    cluster_sync_all();   // no block leaves before its sums are read
  }
  const int64_t c = static_cast<int64_t>(strip) * cols + col;
  if (mine && c < a.cols) {
    if (!cluster && parts > 1) a.part[part * a.cols + c] = s;
    else if (part == 0) a.dbias[c] = s;
  }
}

// Strips of 128 columns and about six blocks an SM in all, with 32 rows at least; where
// that makes few more runs of rows than a cluster holds, as many as it holds.  Where it
// leaves SMs without a block, narrower strips (333 x 520: 4.3 us with strips of 128 and 40
// blocks).
struct BiasPlan {
  int lanes, parts;
};
BiasPlan bias_plan(int64_t rows, int64_t cols, int num_sms) {
  BiasPlan p{16, 1};
  auto strips = [&] { return (cols + 8 * p.lanes - 1) / (8 * p.lanes); };
  auto parts = [&] {
    const int64_t most = (rows * p.lanes + 511) / 512, blocks = 6LL * num_sms;
    const int64_t want = (blocks + strips() - 1) / strips(), n = want < most ? want : most;
    if (n > kBiasCluster && n <= 2 * kBiasCluster) return kBiasCluster;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  p.parts = parts();
  while (p.lanes > 4 && p.parts <= kBiasCluster && strips() * p.parts < num_sms) {
    p.lanes /= 2;
    p.parts = parts();
  }
  return p;
}

template <int ACT, bool MUL>
cudaError_t launch_t(const EpiBwdArgs& a, int num_sms, cudaStream_t stream) {
  if (!a.dbias) {
    const int64_t blocks = (a.rows * (a.cols / 8) + 511) / 512;
    return launch_chained(epilogue_bwd_kernel<ACT, MUL>, static_cast<unsigned>(blocks), 256, 0, 0,
                          stream, a);
  }
  const BiasPlan p = bias_plan(a.rows, a.cols, num_sms);
  const int64_t strips = (a.cols + 8 * p.lanes - 1) / (8 * p.lanes);
  const bool cluster = p.parts > 1 && p.parts <= kBiasCluster;
  const cudaError_t e = launch_chained(
      epilogue_bwd_bias_kernel<ACT, MUL>, static_cast<unsigned>(strips * p.parts), 256, 0,
      cluster ? p.parts : 0, stream, a, p.lanes, p.parts, static_cast<int>(cluster));
  if (e != cudaSuccess || p.parts == 1 || cluster) return e;
  return launch_join_rows(a.part, p.parts, static_cast<int>(a.cols), a.dbias, stream);
}

template <bool MUL>
cudaError_t launch_act(const EpiBwdArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.act) {
    case kActRelu: return launch_t<kActRelu, MUL>(a, num_sms, stream);
    case kActGelu: return launch_t<kActGelu, MUL>(a, num_sms, stream);
    case kActGeluTanh: return launch_t<kActGeluTanh, MUL>(a, num_sms, stream);
    case kActSilu: return launch_t<kActSilu, MUL>(a, num_sms, stream);
    default: return launch_t<kActNone, MUL>(a, num_sms, stream);
  }
}

}  // namespace

int epilogue_bwd_rows(int64_t rows, int64_t cols, int num_sms) {
  const int parts = bias_plan(rows, cols, num_sms).parts;
  return parts > kBiasCluster ? parts : 0;
}

cudaError_t launch_epilogue_bwd(const EpiBwdArgs& a, int num_sms, cudaStream_t stream) {
  return a.mul ? launch_act<true>(a, num_sms, stream) : launch_act<false>(a, num_sms, stream);
}

cudaError_t launch_dropout(const uint16_t* x, const uint16_t* residual, uint16_t* y, int64_t rows,
                           int64_t cols, const DropArgs& drop, cudaStream_t stream) {
  const int64_t nvec = rows * (cols / 8);
  const uint4 *xv = reinterpret_cast<const uint4*>(x), *rv = reinterpret_cast<const uint4*>(residual);
  uint4* yv = reinterpret_cast<uint4*>(y);
  const int64_t blocks = (nvec + 511) / 512;
  return launch_chained(dropout_kernel<2>, static_cast<unsigned>(blocks), 256, 0, 0, stream, xv, rv,
                        yv, nvec, drop);
}

}  // namespace forge

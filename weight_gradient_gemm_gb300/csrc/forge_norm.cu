// The RMS norm in front of a linear layer, its backward pass, and the
// quantiser of the 128-block e4m3 format.  All three stream their tensors
// once; a row (or a block) stays in registers between the reduction it needs
// and the values that depend on it.
#include <cuda_bf16.h>

#include "forge_e4m3.cuh"
#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_ptx.cuh"
#include "forge_wait.cuh"

namespace forge {
namespace {

// Sum of v over a row's threads, the same in every one of them and on every
// run: a warp, or the whole block with one float per warp in `red` (a caller
// that reduces again passes another array, or synchronises in between).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < nw ? red[lane] : 0.0f);
}

// Fewer blocks than SMs: the next kernel can set up beside them at once (and the
// products for few tokens begin to read their weight).  Not for more: its blocks
// would take places unevenly (a backward pass of 1000 x 2048 6.8 -> 11.8 us).
__device__ __forceinline__ void early_trigger() {
  if (gridDim.x <= 128) grid_dependency_trigger();
}

__device__ __forceinline__ void load_gain8(const void* gain, int bf16, int v, float (&g)[8]) {
  if (bf16) {
    unpack8(reinterpret_cast<const uint4*>(gain)[v], g);
  } else {
    const float4 a = reinterpret_cast<const float4*>(gain)[2 * v];
    const float4 b = reinterpret_cast<const float4*>(gain)[2 * v + 1];
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  }
}

// A row's columns are cut into vectors of 8; thread t of a row's `width`
// threads owns the vectors t, t + width, ..., so 16 neighbouring lanes hold the
// 128 columns of a scale.  Three ways to walk the rows share the arithmetic:
//   a warp per row (up to 512 columns): no barrier at all;
//   a block per row: few rows, where every row is in flight at once;
//   persistent blocks whose rows are copied ahead into shared memory (many
//   rows): the copies keep HBM busy through the reductions.
// Memory bounds all three: a row is read once and written once.  Measured, with
// the time of the bytes a call must move at the copy rate, 6.79 TB/s, in
// brackets (calls back to back on inputs that together are larger than L2):
//   8191 x 4096, x + residual -> sum, y       43.6 us (39.5)
//   the same with codes and scales            50.2 us (44.6)
//   8192 x 8192                               88.8 us (79.1)
//   8192 x 1024                               12.8 us (9.9)
//   8192 x 512 (a warp per row)                7.7 us (4.9): a warp has one row in
//                                              flight, none between its reduction
//                                              and its stores
//   512 x 4096 (a block per row)               5.0 us (2.5), launch and tail; 3.4
//                                              with its inputs in L2
//   1 x 4096                                   1.9 us: the latency of a launch,
//                                              the loads and one reduction
// With a block per row throughout, 8191 x 4096 took 55 us: between its reads and
// its stores a block waits at a barrier with nothing in flight.

// ---------------------------------------------------------------- forward
//   h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gain
// in fp32 from the bf16 inputs (the sum is rounded only where it is stored).
// h of one vector, and its share of the sum of squares.
__device__ __forceinline__ float norm_h(const NormArgs& a, uint4 x, uint4 r, int64_t at,
                                        float (&h)[8]) {
  unpack8(x, h);
  if (a.residual) {
    float f[8];
    unpack8(r, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] += f[k];
  }
  if (a.sum) __stcs(reinterpret_cast<uint4*>(a.sum) + at, pack8(h));
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) ss = fmaf(h[k], h[k], ss);
  return ss;
}
__device__ __forceinline__ float norm_rstd(const NormArgs& a, float ss) {
  return rsqrtf(__fdiv_rn(ss, static_cast<float>(a.cols)) + a.eps);
}
// One vector's outputs.  Every lane of the warp takes part (the shuffles);
// `in` is false past the row's end.
__device__ __forceinline__ void norm_out(const NormArgs& a, const float (&h)[8],
                                         const float (&g)[8], float rstd, int64_t row, int v,
                                         bool in) {
  const int64_t at = row * (a.cols / 8) + v;
  if (a.y && in) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = h[k] * rstd * g[k];
    __stcs(reinterpret_cast<uint4*>(a.y) + at, pack8(y));
  }
  if (a.codes) {
    // rstd is common to the row, so the codes are those of h gain, with one
    // rounding less than y's; only the scale carries it.  Outside a range that
    // no model's activations leave, y itself is encoded.
    float t[8], amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      t[k] = in ? h[k] * g[k] : 0.0f;
      amax = max_nan(amax, fabsf(t[k]));
    }
    amax = max16(amax);
    const float top = amax * rstd;
    BlockScale s{0.0f, 0.0f};
    const bool usual = amax >= 0x1p-100f && amax <= 0x1p100f && top >= 0x1p-100f && top <= 0x1p100f;
    if (__all_sync(0xffffffffu, usual)) {
      s.scale = __fdiv_rn(top, kE4m3Max);
      s.inv = __fdiv_rn(kE4m3Max, amax);
    } else {
      amax = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        t[k] = in ? h[k] * rstd * g[k] : 0.0f;
        amax = max_nan(amax, fabsf(t[k]));
      }
      s = block_scale(max16(amax));
    }
    if (in) {
      __stcs(reinterpret_cast<uint2*>(a.codes) + at, encode8(t, s.inv));
      if (v % 16 == 0) a.scales[row * ((a.cols + kBlock - 1) / kBlock) + v / 16] = s.scale;
    }
  }
}

// WARP: a warp per row; else a block per row (both grid-stride).
template <int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  const int nvec = a.cols / 8;
  const int width = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first =
      WARP ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * 8 : gridDim.x;
  int parity = 0;
  grid_dependency_wait();
  early_trigger();
  for (int64_t row = first; row < a.rows; row += step, parity ^= 1) {
    const int64_t base = row * nvec;
    uint4 x[VPT], r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * width;
      x[i] = r[i] = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        x[i] = __ldcs(reinterpret_cast<const uint4*>(a.x) + base + v);
        if (a.residual) r[i] = __ldcs(reinterpret_cast<const uint4*>(a.residual) + base + v);
      }
    }
    float h[VPT][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (me + i * width < nvec) ss += norm_h(a, x[i], r[i], base + me + i * width, h[i]);
    ss = WARP ? warp_sum(ss) : block_sum(ss, red[parity]);
    const float rstd = norm_rstd(a, ss);
    if (a.rstd && me == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * width;
      float g[8];
      if (v < nvec) load_gain8(a.gain, a.gain_bf16, v, g);
      norm_out(a, h[i], g, rstd, row, v, v < nvec);
    }
  }
}

// The rows of one persistent block (blockIdx.x, + gridDim.x, ...), copied ahead
// into a ring of two slots of S rows (one of each input) by bulk copies.  Two
// keep HBM busy; more reads in flight only meet the stores (8191 x 4096 with a
// residual: 44.0 us, with three slots 46.7, with six 48.7).  The inputs pass
// through L2 as the first to leave it, which the backward pass needs most
// (8192 x 8192 with three slots: 91.6 us, 103.3 without; with two 94).  A slot
// is read into registers before the row's reduction, so it is free, and
// thread 0 refills it, as soon as the reduction's barrier is passed.  A wait
// that runs out records its error and lets the block run on (its barriers stay
// matched; what it writes is unspecified).
constexpr int kRing = 2;
template <int S>
struct RowRing {
  uint32_t smem, bars, row_bytes;
  const uint8_t* src[S];
  int64_t rows;
  WaitCtx wc;
  int drop;   // testing aid
  int slot = 0;
  uint32_t ph = 0;
  bool ok = true;

  __device__ uint32_t at(int s, int i) const { return smem + (s * S + i) * row_bytes; }
  __device__ void fill(int s, int64_t row) const {
    const uint64_t policy = l2_policy_evict_first();
    mbar_arrive_expect_tx(bars + 8u * s, S * row_bytes);
#pragma unroll
    for (int i = 0; i < S; ++i)
      bulk_load(at(s, i), src[i] + row * row_bytes, row_bytes, bars + 8u * s, policy);
  }
  // thread 0, before anything is read
  __device__ void start() const {
    for (int s = 0; s < kRing; ++s) mbar_init(bars + 8u * s, 1);
    fence_mbarrier_init();
    drop_first_arrival(drop, bars);
    int64_t row = blockIdx.x;
    for (int s = 0; s < kRing && row < rows; ++s, row += gridDim.x) fill(s, row);
  }
  __device__ void wait() {
    ok = ok && wait_bounded(bars + 8u * slot, ph, wc, kSiteDrainState);
  }
  // after the barrier that follows the slot's last read
  __device__ void next(int64_t row) {
    if (threadIdx.x == 0 && ok) {
      const int64_t ahead = row + static_cast<int64_t>(kRing) * gridDim.x;
      if (ahead < rows) fill(slot, ahead);
    }
    if (++slot == kRing) { slot = 0; ph ^= 1u; }
  }
  // After a timeout: time for copies still under way to land before the block
  // leaves its shared memory.
  __device__ void finish() const {
    if (ok) return;
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
};
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// Shared memory: the ring, 16-byte aligned, then its barriers and an abort flag.
template <int S>
__device__ __forceinline__ RowRing<S> make_ring(uint8_t* smem, uint32_t row_bytes, int64_t rows,
                                                const NormWait& w) {
  RowRing<S> r;
  r.smem = smem_u32(smem);
  r.row_bytes = row_bytes;
  r.rows = rows;
  r.bars = r.smem + kRing * S * row_bytes;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + kRing * S * row_bytes + 8 * kRing);
  r.wc = WaitCtx{abort_flag, w.err, w.err_site, w.timeout_ns};
  r.drop = w.drop_first_arrival;
  return r;
}

template <int VPT, bool RES>
__global__ void __launch_bounds__(1024, 1) rmsnorm_stream_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float red[2][32];
  const int nvec = a.cols / 8;
  RowRing<RES ? 2 : 1> ring =
      make_ring<RES ? 2 : 1>(smem_raw, static_cast<uint32_t>(a.cols) * 2, a.rows, a.wait);
  ring.src[0] = reinterpret_cast<const uint8_t*>(a.x);
  if constexpr (RES) ring.src[1] = reinterpret_cast<const uint8_t*>(a.residual);
  grid_dependency_wait();
  if (threadIdx.x == 0) {
    *ring.wc.abort_flag = 0u;
    ring.start();
  }
  float g[8];   // the gain of the first vector; wider rows read theirs again (L1)
  if (static_cast<int>(threadIdx.x) < nvec) load_gain8(a.gain, a.gain_bf16, threadIdx.x, g);
  __syncthreads();
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    ring.wait();
    float h[VPT][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        const uint4 x = lds16(ring.at(ring.slot, 0) + 16 * v);
        uint4 r = make_uint4(0, 0, 0, 0);
        if constexpr (RES) r = lds16(ring.at(ring.slot, 1) + 16 * v);
        ss += norm_h(a, x, r, row * nvec + v, h[i]);
      }
    }
    ss = block_sum(ss, red[parity]);
    ring.next(row);
    const float rstd = norm_rstd(a, ss);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (VPT > 1 && v < nvec) load_gain8(a.gain, a.gain_bf16, v, g);
      norm_out(a, h[i], g, rstd, row, v, v < nvec);
    }
  }
  grid_dependency_trigger();
  ring.finish();
}

// ---------------------------------------------------------------- backward
// With xh = h rstd and u = dy gain, the gradient of y = xh gain with respect
// to h is rstd (u - xh mean(u xh)); dsum, the gradient that reaches h along
// the residual stream, is added.  dgain = sum over rows of dy xh, in one of two
// ways, each in a fixed order:
//   few rows: blocks of their own beside those of the rows read dy and h again
//   (from L2) and add down 16 or 32 columns; one launch;
//   many rows: a block adds its rows in registers and leaves one partial row,
//   and rmsnorm_dgain_kernel adds those.
// Bound by memory: 8192 x 4096 with dsum, 268 MB, 47.2 us with the second
// launch (39.5 at the copy rate; a block per row 71); without dsum 512 x 4096
// 5.4 us (1.9), 2048 x 4096 14.2 (7.4), 8192 x 1024 14.8 (7.4), 333 x 1032 2.9 a
// call, the launch.
// One vector's share of the row's dot product; dgain's terms are added to dg.
__device__ __forceinline__ float bwd_dot(uint4 hv, uint4 dv, const float (&g)[8], float rstd,
                                         float (&dg)[8]) {
  float h[8], d[8], dot = 0.0f;
  unpack8(hv, h);
  unpack8(dv, d);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = d[k] * (h[k] * rstd);
    dg[k] += t;
    dot = fmaf(t, g[k], dot);
  }
  return dot;
}
__device__ __forceinline__ void bwd_out(const NormBwdArgs& a, uint4 hv, uint4 dv, uint4 sv,
                                        const float (&g)[8], float rstd, float c, int64_t at) {
  float h[8], d[8], o[8];
  unpack8(hv, h);
  unpack8(dv, d);
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = rstd * fmaf(-c, h[k] * rstd, d[k] * g[k]);
  if (a.dsum) {
    float r[8];
    unpack8(sv, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] += r[k];
  }
  __stcs(reinterpret_cast<uint4*>(a.dx) + at, pack8(o));
}
template <int VPT>
__device__ __forceinline__ void write_part(const NormBwdArgs& a, const float (&dg)[VPT][8], int me,
                                           int width) {
  const int nvec = a.cols / 8;
  float4* part = reinterpret_cast<float4*>(a.part) + static_cast<int64_t>(blockIdx.x) * nvec * 2;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = me + i * width;
    if (v < nvec) {
      part[2 * v] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
      part[2 * v + 1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
  }
}

// dgain of 8 L columns from dy, h and rstd: L lanes hold a row's columns, every
// run of L lanes its own rows.
template <int L>
__device__ __forceinline__ void dgain_columns(const NormBwdArgs& a, int cb, float (&red)[32][32]) {
  constexpr int kBatch = 4;   // rows whose loads are in flight at once
  const int lane = threadIdx.x & 31, sub = lane & (L - 1), runs = blockDim.x / L;
  const int nvec = a.cols / 8, v = cb * L + sub;
  float dg[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (v < nvec) {
    for (int64_t row = threadIdx.x / L; row < a.rows; row += kBatch * runs) {
      uint4 hv[kBatch], dv[kBatch];
      float rs[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t r = row + j * runs;
        hv[j] = dv[j] = make_uint4(0, 0, 0, 0);
        rs[j] = 0.0f;
        if (r < a.rows) {
          hv[j] = reinterpret_cast<const uint4*>(a.h)[r * nvec + v];
          dv[j] = reinterpret_cast<const uint4*>(a.dy)[r * nvec + v];
          rs[j] = a.rstd[r];
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        float h[8], d[8];
        unpack8(hv[j], h);
        unpack8(dv[j], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[k] += d[k] * (h[k] * rs[j]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) dg[k] += __shfl_xor_sync(0xffffffffu, dg[k], o);
    if (lane < L) red[threadIdx.x >> 5][sub * 8 + k] = dg[k];
  }
  __syncthreads();
  if (threadIdx.x < 8 * L && cb * 8 * L + static_cast<int>(threadIdx.x) < a.cols) {
    float sum = 0.0f;
    for (int w = 0; w < (blockDim.x >> 5); ++w) sum += red[w][threadIdx.x];
    a.dgain[cb * 8 * L + threadIdx.x] = sum;
  }
}

// DIRECT: the first col_blocks blocks add up dgain, the others take the rows.
template <int VPT, bool WARP, bool DIRECT>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
    rmsnorm_bwd_kernel(const NormBwdArgs a, int col_blocks, int lanes) {
  __shared__ float red[2][32];
  __shared__ float4 parts[DIRECT ? 256 : (WARP ? 8 * 64 * VPT : 1)];   // [warp][vector][2]
  const int nvec = a.cols / 8;
  const int width = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
  int block = blockIdx.x, blocks = gridDim.x;
  if constexpr (DIRECT) {
    if (block < col_blocks) {
      grid_dependency_wait();
      if (lanes == 4) dgain_columns<4>(a, block, reinterpret_cast<float(&)[32][32]>(parts));
      else dgain_columns<2>(a, block, reinterpret_cast<float(&)[32][32]>(parts));
      return;
    }
    block -= col_blocks;
    blocks -= col_blocks;
  }
  const int64_t first = WARP ? static_cast<int64_t>(block) * 8 + (threadIdx.x >> 5) : block;
  const int64_t step = WARP ? static_cast<int64_t>(blocks) * 8 : blocks;
  int parity = 0;
  float dg[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i][k] = 0.0f;
  grid_dependency_wait();
  for (int64_t row = first; row < a.rows; row += step, parity ^= 1) {
    const int64_t base = row * nvec;
    const float rstd = a.rstd[row];
    uint4 hv[VPT], dv[VPT], sv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * width;
      if (v < nvec) {
        hv[i] = __ldcs(reinterpret_cast<const uint4*>(a.h) + base + v);
        dv[i] = __ldcs(reinterpret_cast<const uint4*>(a.dy) + base + v);
        if (a.dsum) sv[i] = __ldcs(reinterpret_cast<const uint4*>(a.dsum) + base + v);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * width;
      if (v < nvec) {
        float g[8];
        load_gain8(a.gain, a.gain_bf16, v, g);
        dot += bwd_dot(hv[i], dv[i], g, rstd, dg[DIRECT ? 0 : i]);   // DIRECT: not used
      }
    }
    dot = WARP ? warp_sum(dot) : block_sum(dot, red[parity]);
    const float c = __fdiv_rn(dot, static_cast<float>(a.cols));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * width;
      if (v < nvec) {
        float g[8];
        load_gain8(a.gain, a.gain_bf16, v, g);
        bwd_out(a, hv[i], dv[i], sv[i], g, rstd, c, base + v);
      }
    }
  }
  grid_dependency_trigger();
  if (DIRECT || !a.dgain) return;
  if constexpr (WARP && !DIRECT) {   // the block's warps join in a fixed order
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me + i * 32;
      parts[(warp * 32 * VPT + v) * 2] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
      parts[(warp * 32 * VPT + v) * 2 + 1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * nvec; e += 256) {
      float4 s = parts[e];
      for (int w = 1; w < 8; ++w) {
        const float4 p = parts[w * 64 * VPT + e];
        s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
      }
      reinterpret_cast<float4*>(a.part)[static_cast<int64_t>(blockIdx.x) * nvec * 2 + e] = s;
    }
  } else if constexpr (!DIRECT) {
    write_part<VPT>(a, dg, me, width);
  }
}

template <int VPT, bool DSUM>
__global__ void __launch_bounds__(1024, 1)
    rmsnorm_bwd_stream_kernel(const NormBwdArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float red[2][32];
  constexpr int S = DSUM ? 3 : 2;
  const int nvec = a.cols / 8;
  RowRing<S> ring = make_ring<S>(smem_raw, static_cast<uint32_t>(a.cols) * 2, a.rows, a.wait);
  ring.src[0] = reinterpret_cast<const uint8_t*>(a.h);
  ring.src[1] = reinterpret_cast<const uint8_t*>(a.dy);
  if constexpr (DSUM) ring.src[2] = reinterpret_cast<const uint8_t*>(a.dsum);
  grid_dependency_wait();
  if (threadIdx.x == 0) {
    *ring.wc.abort_flag = 0u;
    ring.start();
  }
  float g[8], dg[VPT][8];
  if (static_cast<int>(threadIdx.x) < nvec) load_gain8(a.gain, a.gain_bf16, threadIdx.x, g);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i][k] = 0.0f;
  __syncthreads();
  int parity = 0;
  float rstd = a.rstd[blockIdx.x];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const float rstd_next = row + gridDim.x < a.rows ? a.rstd[row + gridDim.x] : 0.0f;
    ring.wait();
    uint4 hv[VPT], dv[VPT], sv[VPT];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        hv[i] = lds16(ring.at(ring.slot, 0) + 16 * v);
        dv[i] = lds16(ring.at(ring.slot, 1) + 16 * v);
        if constexpr (DSUM) sv[i] = lds16(ring.at(ring.slot, S - 1) + 16 * v);
        if (VPT > 1) load_gain8(a.gain, a.gain_bf16, v, g);
        dot += bwd_dot(hv[i], dv[i], g, rstd, dg[i]);
      }
    }
    dot = block_sum(dot, red[parity]);
    ring.next(row);
    const float c = __fdiv_rn(dot, static_cast<float>(a.cols));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        if (VPT > 1) load_gain8(a.gain, a.gain_bf16, v, g);
        bwd_out(a, hv[i], dv[i], sv[i], g, rstd, c, row * nvec + v);
      }
    }
    rstd = rstd_next;
  }
  grid_dependency_trigger();
  if (a.dgain) write_part<VPT>(a, dg, threadIdx.x, blockDim.x);
  ring.finish();
}

// dgain[c] = sum over the blocks' partial rows: W columns a block, 1024 / W runs of
// rows side by side, added in a fixed order.  16 columns up to 1024, where 32
// leave most SMs without a block (the whole backward pass of 8192 x 1024 17.3 us
// with 32, 16.0 with 16; of 8192 x 256 8.7 and 7.8).
template <int W>
__global__ void __launch_bounds__(1024) rmsnorm_dgain_kernel(const float* __restrict__ part,
                                                             int blocks, int cols,
                                                             float* __restrict__ dgain) {
  constexpr int RUNS = 1024 / W;
  __shared__ float sum[RUNS][W + 1];
  const int col = threadIdx.x % W, run = threadIdx.x / W;
  const int c = blockIdx.x * W + col;
  grid_dependency_wait();
  early_trigger();
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int b = run; b < blocks; b += RUNS)
      s += __ldcg(part + static_cast<int64_t>(b) * cols + c);
  }
  sum[run][col] = s;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp a column
  if (warp >= W || blockIdx.x * W + warp >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int r = 0; r < RUNS; r += 32) s += sum[r + lane][warp];
  s = warp_sum(s);
  if (lane == 0) dgain[blockIdx.x * W + warp] = s;
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

// The quantisers: per block s = amax / 448, codes = 448 x / amax rounded to e4m3.
// One pass; a block stays in registers between its maximum and its codes.
//
// Blocks of 1 x 128: 8 lanes per block, two vectors of 8 columns a lane, so
// that one reduction and one pair of divisions serve 16 of a lane's values.
// 8192 x 14336: 51.8 us, the copy rate (100 us with 16 lanes a block, one block
// at a time: bound by its instructions and by loads that waited for the block
// before).  No persistent walk, no barrier: the blocks' many independent loads
// keep HBM busy by themselves.
constexpr int kQuantUnroll = 4;   // blocks per lane group whose loads are in flight at once

// Rows of whole blocks: the blocks of all rows follow one another, and a
// warp's groups take 4 x kQuantUnroll neighbouring ones.
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const uint4* __restrict__ x,
                                                              uint2* __restrict__ codes,
                                                              float* __restrict__ scales,
                                                              int64_t blocks) {
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t b0 =
      (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (4 * kQuantUnroll) +
      (lane >> 3);
  uint4 v[kQuantUnroll][2];
  grid_dependency_wait();
  early_trigger();
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
    const QuotientScale s = quotient_scale(max8(max_nan(amax8(v[j][0]), amax8(v[j][1]))));
    if (b < blocks) {
      float f[8];
      unpack8(v[j][0], f);
      __stcs(codes + b * 16 + sub, encode8(f, s));
      unpack8(v[j][1], f);
      __stcs(codes + b * 16 + 8 + sub, encode8(f, s));
      if (sub == 0) scales[b] = s.scale;
    }
  }
}

// Any row length: the last block of a row may be partial.  One block a lane group in
// flight: 8192 x 4104 21.3 us (15.0 at the copy rate), 8192 x 2880 15.1 (10.5).
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint4* __restrict__ x,
                                                            uint2* __restrict__ codes,
                                                            float* __restrict__ scales,
                                                            int64_t rows, int nvec) {
  const int nblk = (nvec + 15) / 16, sub = threadIdx.x & 7;
  const int64_t total = rows * nblk, groups = static_cast<int64_t>(gridDim.x) * 32;
  grid_dependency_wait();
  early_trigger();
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
    const QuotientScale s = quotient_scale(max8(max_nan(amax8(v0), amax8(v1))));
    float f[8];
    if (in0) {
      unpack8(v0, f);
      __stcs(codes + at, encode8(f, s));
    }
    if (in1) {
      unpack8(v1, f);
      __stcs(codes + at + 8, encode8(f, s));
    }
    if (in0 && sub == 0) scales[b] = s.scale;
  }
}

// Blocks of 128 x 128: persistent CTAs, four an SM, each with one block's 32 KB
// copied ahead by TMA (which fills zeros outside the matrix).  A block is read
// into registers before its maximum is formed, so the next copy starts at that
// reduction's barrier and runs under the codes and stores.  14336 x 4096: 30.0 us,
// 5.9 TB/s (33.2 us with loads into registers, where a CTA's loads, barrier and
// stores follow one another; more copies in flight only meet the stores: two
// slots, three CTAs an SM, 29.9 us where one took 28.9); 4096 x 4096 10.4 us;
// 1000 x 4112 4.5, or 3.5 with its values in L2.
// A wait that runs out records its error and lets the CTA run on, as in RowRing.
constexpr int kTileBytes = kBlock * kBlock * 2;
__global__ void __launch_bounds__(256)
    quantize_tiles_kernel(const __grid_constant__ CUtensorMap x, uint8_t* __restrict__ codes,
                          float* __restrict__ scales, int64_t rows, int64_t cols, int64_t blocks,
                          NormWait w) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float red[2][8];
  __shared__ uint64_t bar_word;
  __shared__ uint32_t abort_word;
  const uint32_t tile = smem_u32(smem_raw), bar = smem_u32(&bar_word);
  const WaitCtx wc{&abort_word, w.err, w.err_site, w.timeout_ns};
  const int64_t nblk = (cols + kBlock - 1) / kBlock;
  auto load = [&](int64_t b) {
    mbar_arrive_expect_tx(bar, kTileBytes);
    tma_load_2d(tile, &x, static_cast<int>(b % nblk) * kBlock, static_cast<int>(b / nblk) * kBlock,
                bar, l2_policy_evict_first());
  };
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    abort_word = 0u;
    fence_mbarrier_init();
    drop_first_arrival(w.drop_first_arrival, bar);
  }
  grid_dependency_wait();
  if (threadIdx.x == 0) load(blockIdx.x);
  __syncthreads();
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, ph ^= 1u) {
    ok = ok && wait_bounded(bar, ph, wc, kSiteDrainState);
    uint4 v[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lds16(tile + threadIdx.x * 16 + i * 4096);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, amax8(v[i]));
    amax = max16(amax);
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
    if ((threadIdx.x & 31) == 0) red[ph][threadIdx.x >> 5] = amax;
    __syncthreads();
    if (threadIdx.x == 0 && ok && b + gridDim.x < blocks) load(b + gridDim.x);
#pragma unroll
    for (int q = 0; q < 8; ++q) amax = max_nan(amax, red[ph][q]);
    const QuotientScale s = quotient_scale(amax);
    const int64_t col = b % nblk * kBlock + (threadIdx.x & 15) * 8;
    const int64_t row0 = b / nblk * kBlock + (threadIdx.x >> 4);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col < cols && row0 + 16 * i < rows) {
        float f[8];
        unpack8(v[i], f);
        __stcs(reinterpret_cast<uint2*>(codes + (row0 + 16 * i) * cols + col), encode8(f, s));
      }
    if (threadIdx.x == 0) scales[b] = s.scale;
  }
  grid_dependency_trigger();
  if (!ok) {   // time for a copy still under way to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
}

// Threads a row needs with VPT vectors each, a multiple of 32.
int row_threads(int cols, int vpt) {
  const int t = (cols / 8 + vpt - 1) / vpt;
  return (t + 31) / 32 * 32;
}

// How a call walks its rows.
enum Walk { kWalkWarp, kWalkBlock, kWalkStream };
struct RowPlan {
  Walk walk;
  int vpt, threads, grid, smem;   // smem: the stream's ring
  bool direct;                    // backward: dgain in the same launch
  int lanes;                      // and the lanes that hold a row's columns there
};

// A warp per row up to 512 columns (8192 x 768 with codes: 14.9 us so, 11.3
// through the stream).  Above, the stream for rows enough to fill its persistent
// blocks twice, while a ring of two rows fits (else a block per row).  Blocks of
// about 1024 threads in all share an SM.
//
// (Whether dgain is asked for changes nothing here, so dX has the same bits.)
// The backward pass adds up dgain in the same launch while a run of lanes has at
// most 16 rows, and in place of the stream up to 2^23 values (two rounds through
// L2 cost less than the second launch).  With the second launch, then without:
// 333 x 1032 5.7 and 2.6 us, 512 x 4096 9.5 and 6.5, 1024 x 4096 12.4 and 9.8,
// 2048 x 4096 17.0 and 15.7; 2000 x 8192 28.8 and 31.2.  Up to 2048 columns
// two lanes a row, for more column blocks (1000 x 2048: 7.0 us, 9.2 with four;
// 2048 x 4096 16.6 and 15.7).  More rows take the stream (2000 x 1024: 10.2 us,
// 12.6 with a few blocks that read as they go).
constexpr int64_t kDirectValues = 1 << 23;
RowPlan row_plan(int64_t rows, int cols, int streams, bool backward, int num_sms) {
  RowPlan p{kWalkBlock, 1, 0, 0, 0, false, cols <= 2048 ? 2 : 4};
  if (cols <= 512) {
    p.walk = kWalkWarp;
    p.vpt = cols <= 256 ? 1 : 2;
    p.threads = 256;
    p.direct = backward && rows <= 16 * p.threads / p.lanes;
    const int64_t want = (rows + 7) / 8, most = static_cast<int64_t>(num_sms) * 4;
    p.grid = static_cast<int>(want < most ? want : most);
    return p;
  }
  p.vpt = cols <= 8192 ? 1 : (cols <= 16384 ? 2 : 4);
  p.threads = row_threads(cols, p.vpt);
  int per_sm = 1024 / p.threads;
  per_sm = per_sm > 8 ? 8 : per_sm;
  const int64_t direct_rows = 16 * p.threads / p.lanes;
  p.direct = backward && rows <= direct_rows && rows * cols <= kDirectValues;
  p.smem = kRing * (streams * cols * 2 + 8) + 8;
  const bool many = rows >= 2 * per_sm * num_sms || (backward && rows > direct_rows);
  if (!p.direct && many && p.vpt <= 2 && p.smem * per_sm <= 222 * 1024) {
    p.walk = kWalkStream;
    p.grid = static_cast<int>(rows < per_sm * num_sms ? rows : per_sm * num_sms);
    return p;
  }
  // Every row in flight at once: where a vector a thread leaves rows for a second
  // wave, two vectors and half the threads (512 x 4096, inputs in L2: 3.4 us;
  // when it was chosen 4.6, and 5.8 with one vector; 304 rows the same, 152 rows
  // 3.0 and 2.8).  Where the backward pass leaves partial rows, few blocks.
  p.direct = backward && rows <= direct_rows;
  if ((!backward || p.direct) && p.vpt == 1 && rows > per_sm * num_sms) {
    p.vpt = 2;
    p.threads = row_threads(cols, 2);
  }
  const int64_t most = backward && !p.direct ? static_cast<int64_t>(num_sms) * 2 : INT32_MAX;
  p.grid = static_cast<int>(rows < most ? rows : most);
  return p;
}

// Launches a stream kernel with its ring.
template <typename Kern, typename Args>
cudaError_t launch_stream(Kern kern, PerDevice& once, const RowPlan& p, const Args& a,
                          cudaStream_t stream) {
  const cudaError_t e = allow_smem(once, kern, 224 * 1024);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, p.grid, p.threads, p.smem, 0, stream, a);
}
template <int VPT, bool RES>
cudaError_t launch_fwd_stream(const RowPlan& p, const NormArgs& a, cudaStream_t stream) {
  static PerDevice once;
  return launch_stream(rmsnorm_stream_kernel<VPT, RES>, once, p, a, stream);
}
template <int VPT, bool DSUM>
cudaError_t launch_bwd_stream(const RowPlan& p, const NormBwdArgs& a, cudaStream_t stream) {
  static PerDevice once;
  return launch_stream(rmsnorm_bwd_stream_kernel<VPT, DSUM>, once, p, a, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const RowPlan p = row_plan(a.rows, a.cols, a.residual ? 2 : 1, false, num_sms);
  if (p.walk == kWalkStream) {
    if (p.vpt == 1)
      return a.residual ? launch_fwd_stream<1, true>(p, a, stream)
                        : launch_fwd_stream<1, false>(p, a, stream);
    return a.residual ? launch_fwd_stream<2, true>(p, a, stream)
                      : launch_fwd_stream<2, false>(p, a, stream);
  }
  auto go = [&](auto kern) { return launch_chained(kern, p.grid, p.threads, 0, 0, stream, a); };
  if (p.walk == kWalkWarp)
    return p.vpt == 1 ? go(rmsnorm_kernel<1, true>) : go(rmsnorm_kernel<2, true>);
  return p.vpt == 1 ? go(rmsnorm_kernel<1, false>)
                    : (p.vpt == 2 ? go(rmsnorm_kernel<2, false>) : go(rmsnorm_kernel<4, false>));
}

int rmsnorm_bwd_blocks(int64_t rows, int cols, int num_sms) {
  // with and without dsum: one workspace serves both
  const RowPlan a = row_plan(rows, cols, 2, true, num_sms);
  const RowPlan b = row_plan(rows, cols, 3, true, num_sms);
  const int na = a.direct ? 1 : a.grid, nb = b.direct ? 1 : b.grid;   // direct: none read
  return na > nb ? na : nb;
}

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int num_sms, cudaStream_t stream) {
  const RowPlan p = row_plan(a.rows, a.cols, a.dsum ? 3 : 2, true, num_sms);
  cudaError_t e = cudaSuccess;
  if (p.walk == kWalkStream) {
    if (p.vpt == 1)
      e = a.dsum ? launch_bwd_stream<1, true>(p, a, stream)
                 : launch_bwd_stream<1, false>(p, a, stream);
    else
      e = a.dsum ? launch_bwd_stream<2, true>(p, a, stream)
                 : launch_bwd_stream<2, false>(p, a, stream);
  } else if (p.direct) {
    const int cb = a.dgain ? (a.cols + 8 * p.lanes - 1) / (8 * p.lanes) : 0;
    auto go = [&](auto kern) {
      return launch_chained(kern, cb + p.grid, p.threads, 0, 0, stream, a, cb, p.lanes);
    };
    if (p.walk == kWalkWarp)
      return p.vpt == 1 ? go(rmsnorm_bwd_kernel<1, true, true>)
                        : go(rmsnorm_bwd_kernel<2, true, true>);
    return p.vpt == 1 ? go(rmsnorm_bwd_kernel<1, false, true>)
                      : (p.vpt == 2 ? go(rmsnorm_bwd_kernel<2, false, true>)
                                    : go(rmsnorm_bwd_kernel<4, false, true>));
  } else {
    auto go = [&](auto kern) {
      return launch_chained(kern, p.grid, p.threads, 0, 0, stream, a, 0, 0);
    };
    if (p.walk == kWalkWarp)
      e = p.vpt == 1 ? go(rmsnorm_bwd_kernel<1, true, false>)
                     : go(rmsnorm_bwd_kernel<2, true, false>);
    else
      e = go(rmsnorm_bwd_kernel<4, false, false>);   // up to 16384 columns: direct or the stream
  }
  if (e != cudaSuccess || !a.dgain) return e;
  return launch_join_rows(a.part, p.grid, a.cols, a.dgain, stream);
}

cudaError_t launch_join_rows(const float* part, int blocks, int cols, float* out,
                             cudaStream_t stream) {
  auto join = [&](auto kern, int w) {
    return launch_chained(kern, (cols + w - 1) / w, 1024, 0, 0, stream, part, blocks, cols, out);
  };
  return cols <= 1024 ? join(rmsnorm_dgain_kernel<16>, 16) : join(rmsnorm_dgain_kernel<32>, 32);
}

cudaError_t launch_quantize_b128(const uint16_t* x, uint8_t* codes, float* scales, int64_t rows,
                                 int64_t cols, int block_rows, int num_sms, const NormWait& wait,
                                 cudaStream_t stream) {
  const int64_t nblk = (cols + kBlock - 1) / kBlock;
  if (block_rows == 1) {
    const uint4* xv = reinterpret_cast<const uint4*>(x);
    uint2* cv = reinterpret_cast<uint2*>(codes);
    const int64_t blocks = rows * nblk;
    const int64_t grid = (blocks + 32 * kQuantUnroll - 1) / (32 * kQuantUnroll);
    if (cols % kBlock == 0 && grid <= INT32_MAX)
      return launch_chained(quantize_blocks_kernel, static_cast<unsigned>(grid), 256, 0, 0, stream,
                            xv, cv, scales, blocks);
    const int64_t want = (blocks + 31) / 32, most = static_cast<int64_t>(num_sms) * 8;
    return launch_chained(quantize_rows_kernel, static_cast<unsigned>(want < most ? want : most),
                          256, 0, 0, stream, xv, cv, scales, rows, static_cast<int>(cols / 8));
  }
  CUtensorMap map;
  if (!host_map(&map, x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cols, rows, cols * 2, kBlock, kBlock,
                CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int64_t blocks = (rows + kBlock - 1) / kBlock * nblk;
  const int64_t most = static_cast<int64_t>(num_sms) * 4;
  return launch_chained(quantize_tiles_kernel, static_cast<unsigned>(blocks < most ? blocks : most),
                        256, kTileBytes, 0, stream, map, codes, scales, rows, cols, blocks, wait);
}

}  // namespace forge

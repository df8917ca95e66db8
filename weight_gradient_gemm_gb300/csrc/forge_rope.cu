// Rotary positions, and the norm of queries and keys with the rotation, forward and
// backward.
//
// The rotation.  Pair i of a head at position p turns by the angle 2 pi p f_i.  f_i, in
// turns per position, is a 64-bit fraction F_i / 2^64, so p F_i modulo 2^64 is the
// angle in fractions of a turn, exact for every position (one 64-bit integer product in
// place of a 64-bit floating one and a reduction by pi): its upper 32 bits, as a signed
// number, are the argument of sincospi.  Its rounding to fp32 is 2^-24 of half a turn.
//
// The layout of the work.  A head's row is cut into vectors of VEC elements.  A lane
// holds two of them: where pairs lie half the rotated part apart, the two vectors that
// turn into each other; where they lie side by side, two neighbouring ones.  P lanes (a
// power of two) hold a head, 32 / P heads a warp at a time.  A lane's pairs are the same
// in all heads, so a warp forms the sines and cosines once for its token and walks the
// heads of queries and keys with them; the next heads' loads are in flight meanwhile.
#include <cuda_bf16.h>

#include "forge_e4m3.cuh"
#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_layer.cuh"

namespace forge {
namespace {

enum RopeMode { kRope = 0, kQkNorm = 1, kQkNormBwd = 2 };

// VEC bf16 values.
template <int VEC>
struct Raw;
template <>
struct Raw<8> {
  using V = uint4;
  static __device__ __forceinline__ V zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void unpack(V v, float (&f)[8]) { unpack8(v, f); }
  static __device__ __forceinline__ V pack(const float (&f)[8]) { return pack8(f); }
};
template <>
struct Raw<4> {
  using V = uint2;
  static __device__ __forceinline__ V zero() { return make_uint2(0, 0); }
  static __device__ __forceinline__ void unpack(V v, float (&f)[4]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  }
  static __device__ __forceinline__ V pack(const float (&f)[4]) {
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
};

// What a lane's two vectors are: their first elements in the head, whether they exist
// and whether they turn.
struct LanePart {
  int a, b;
  bool has_a, has_b, rot_a, rot_b;
};
template <int VEC, bool INTER>
__device__ __forceinline__ LanePart lane_part(int u, int dim, int rot) {
  LanePart p;
  if constexpr (INTER) {
    p.a = 2 * VEC * u;
    p.b = p.a + VEC;
    p.rot_a = p.a < rot;
    p.rot_b = p.b < rot;
  } else {
    const int turning = rot / (2 * VEC);
    p.rot_a = p.rot_b = u < turning;
    p.a = u < turning ? u * VEC : rot + 2 * VEC * (u - turning);
    p.b = u < turning ? rot / 2 + u * VEC : p.a + VEC;
  }
  p.has_a = p.a < dim;
  p.has_b = p.b < dim;
  return p;
}

// Sines and cosines of the lane's VEC pairs at a position, times the magnitude.
template <int VEC, bool INTER>
__device__ __forceinline__ void turn_of(const RopeArgs& r, const LanePart& p, int64_t pos,
                                        float (&c)[VEC], float (&s)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    // HALF: pairs a, a + 1, ...; INTER: half of them in each vector
    const bool in = INTER ? (i < VEC / 2 ? p.rot_a : p.rot_b) : p.rot_a;
    const int pair = INTER ? (i < VEC / 2 ? p.a / 2 + i : p.b / 2 + i - VEC / 2) : p.a + i;
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (in) {
      const uint64_t at = static_cast<uint64_t>(pos) * r.freqs[pair];
      const float half_turns = static_cast<float>(static_cast<int32_t>(at >> 32)) * 0x1p-31f;
      sincospif(half_turns, &s[i], &c[i]);
      c[i] *= r.magnitude;
      s[i] *= r.magnitude;
    }
  }
}

// (a, b) turned: by the angle, or with `back` by its opposite.
template <int VEC, bool INTER>
__device__ __forceinline__ void turn(const LanePart& p, const float (&c)[VEC],
                                     const float (&s)[VEC], bool back, float (&a)[VEC],
                                     float (&b)[VEC]) {
  const float sign = back ? -1.0f : 1.0f;
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float sa = sign * s[i], x = a[2 * i], y = a[2 * i + 1];
      if (p.rot_a) {
        a[2 * i] = fmaf(x, c[i], -y * sa);
        a[2 * i + 1] = fmaf(y, c[i], x * sa);
      }
      const float cb = c[i + VEC / 2], sb = sign * s[i + VEC / 2], z = b[2 * i], w = b[2 * i + 1];
      if (p.rot_b) {
        b[2 * i] = fmaf(z, cb, -w * sb);
        b[2 * i + 1] = fmaf(w, cb, z * sb);
      }
    }
  } else if (p.rot_a) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float si = sign * s[i], x = a[i], y = b[i];
      a[i] = fmaf(x, c[i], -y * si);
      b[i] = fmaf(y, c[i], x * si);
    }
  }
}

template <int VEC>
__device__ __forceinline__ void load_gain(const void* gain, int bf16, int at, bool has,
                                          float (&g)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    g[i] = !has ? 0.0f
                : (bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(gain)[at + i])
                        : static_cast<const float*>(gain)[at + i]);
}

// Sum over the P lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp's units are the pairs (token, chunk): chunk c takes the c-th of `chunks` even
// shares of the head groups (those of queries, then those of keys).
template <int VEC, bool INTER, int MODE>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs r, int lanes, int chunks) {
  using R = Raw<VEC>;
  using V = typename R::V;
  constexpr bool kBwd = MODE == kQkNormBwd;
  const int lane = threadIdx.x & 31;
  const int u = lane & (lanes - 1), g = lane / lanes, groups = 32 / lanes;
  const LanePart p = lane_part<VEC, INTER>(u, r.dim, r.rot);
  const int its0 = (r.set[0].heads + groups - 1) / groups;
  const int its = its0 + (r.sets > 1 ? (r.set[1].heads + groups - 1) / groups : 0);
  float dga[2][kBwd ? VEC : 1], dgb[2][kBwd ? VEC : 1];
  if constexpr (kBwd) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) dga[k][i] = dgb[k][i] = 0.0f;
  }
  grid_dependency_wait();
  const int64_t units = r.tokens * chunks;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); unit < units;
       unit += warps) {
    const int64_t t = chunks == 1 ? unit : unit / chunks;
    const int chunk = static_cast<int>(unit - t * chunks);
    const int first = static_cast<int>(static_cast<int64_t>(its) * chunk / chunks);
    const int last = static_cast<int>(static_cast<int64_t>(its) * (chunk + 1) / chunks);
    const int64_t pos = r.positions ? r.positions[t] : t;
    float c[VEC], s[VEC];
    turn_of<VEC, INTER>(r, p, pos, c, s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const HeadSet& set = r.set[k];
      const int from = k == 0 ? first : max(first - its0, 0);
      const int to = k == 0 ? min(last, its0) : last - its0;
      if (from >= to) continue;
      float ga[VEC], gb[VEC];
      if constexpr (MODE != kRope) {
        load_gain<VEC>(set.gain, r.gain_bf16, p.a, p.has_a, ga);
        load_gain<VEC>(set.gain, r.gain_bf16, p.b, p.has_b, gb);
      }
      const uint16_t* x = set.x + t * set.x_token;
      const uint16_t* dy = kBwd ? set.dy + t * set.dy_token : nullptr;
      V xa, xb, da, db;
      auto load = [&](int it) {
        const int head = it * groups + g;
        const bool in = it < to && head < set.heads;
        xa = xb = da = db = R::zero();
        const uint16_t* row = x + head * set.x_head;
        if (in && p.has_a) xa = __ldcs(reinterpret_cast<const V*>(row + p.a));
        if (in && p.has_b) xb = __ldcs(reinterpret_cast<const V*>(row + p.b));
        if constexpr (kBwd) {
          const uint16_t* drow = dy + head * set.dy_head;
          if (in && p.has_a) da = __ldcs(reinterpret_cast<const V*>(drow + p.a));
          if (in && p.has_b) db = __ldcs(reinterpret_cast<const V*>(drow + p.b));
        }
      };
      load(from);
      for (int it = from; it < to; ++it) {
        const int head = it * groups + g;
        float a[VEC], b[VEC], na[VEC], nb[VEC];
        R::unpack(xa, a);
        R::unpack(xb, b);
        if constexpr (kBwd) {
          R::unpack(da, na);
          R::unpack(db, nb);
        }
        load(it + 1);
        if constexpr (MODE != kRope) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
          ss = head_sum(ss, lanes);
          const float rstd = rsqrtf(__fdiv_rn(ss, static_cast<float>(r.dim)) + r.eps);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            a[i] *= rstd;
            b[i] *= rstd;
          }
          if constexpr (kBwd) {
            turn<VEC, INTER>(p, c, s, true, na, nb);   // the gradient of the normed head
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float ta = na[i] * a[i], tb = nb[i] * b[i];
              dga[k][i] += ta;
              dgb[k][i] += tb;
              dot = fmaf(ta, ga[i], fmaf(tb, gb[i], dot));
            }
            dot = __fdiv_rn(head_sum(dot, lanes), static_cast<float>(r.dim));
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              a[i] = rstd * fmaf(-dot, a[i], na[i] * ga[i]);
              b[i] = rstd * fmaf(-dot, b[i], nb[i] * gb[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              a[i] *= ga[i];
              b[i] *= gb[i];
            }
          }
        }
        if constexpr (!kBwd) turn<VEC, INTER>(p, c, s, r.inverse, a, b);
        uint16_t* row = set.y + t * set.y_token + head * set.y_head;
        if (head < set.heads) {
          if (p.has_a) __stcs(reinterpret_cast<V*>(row + p.a), R::pack(a));
          if (p.has_b) __stcs(reinterpret_cast<V*>(row + p.b), R::pack(b));
        }
      }
    }
  }
  grid_dependency_trigger();
  if constexpr (kBwd) {
    // The gains' gradients: the head groups of a warp, then the block's warps, each in a
    // fixed order; the block leaves one partial row, or the result where it is alone.
    if (!r.set[0].dgain && !r.set[1].dgain) return;
    __shared__ float sum[8][512];   // [warp][set][element]
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        for (int o = 16; o >= lanes; o >>= 1) {
          dga[k][i] += __shfl_xor_sync(0xffffffffu, dga[k][i], o);
          dgb[k][i] += __shfl_xor_sync(0xffffffffu, dgb[k][i], o);
        }
        if (g == 0 && p.has_a) sum[warp][k * r.dim + p.a + i] = dga[k][i];
        if (g == 0 && p.has_b) sum[warp][k * r.dim + p.b + i] = dgb[k][i];
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * r.dim; e += 256) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += sum[w][e];
      const int k = e >= r.dim;
      if (gridDim.x > 1) r.part[static_cast<int64_t>(blockIdx.x) * 2 * r.dim + e] = v;
      else if (r.set[k].dgain) r.set[k].dgain[e - k * r.dim] = v;
    }
  }
}

// The partial rows of `blocks` blocks: 16 columns a block, 64 runs of rows side by side.
__global__ void __launch_bounds__(1024) qk_dgain_kernel(const float* part, int blocks, int dim,
                                                        float* dq_gain, float* dk_gain) {
  __shared__ float sum[64][17];
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + col;
  grid_dependency_wait();
  grid_dependency_trigger();
  float s = 0.0f;
  if (e < 2 * dim)
    for (int b = run; b < blocks; b += 64) s += __ldcg(part + static_cast<int64_t>(b) * 2 * dim + e);
  sum[run][col] = s;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp a column
  if (warp >= 16) return;
  s = sum[lane][warp] + sum[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int at = blockIdx.x * 16 + warp;
  if (lane != 0 || at >= 2 * dim) return;
  float* out = at < dim ? dq_gain : dk_gain;
  if (out) out[at < dim ? at : at - dim] = s;
}

struct RopePlan {
  int vec, lanes, chunks, grid;
};
int round_up_pow2(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}
// Vectors of eight, or of four where half the rotated part is no multiple of eight.
// Chunks: a warp a token where the tokens fill the GPU (16 warps an SM), else as many
// warps a token as there are head groups.
RopePlan rope_plan(int64_t tokens, int heads0, int heads1, int dim, int rot, bool interleaved,
                   bool backward, int num_sms) {
  RopePlan p;
  p.vec = interleaved || rot % 16 == 0 ? 8 : 4;
  const int turning = rot / (2 * p.vec), rest = dim - rot;
  const int need = interleaved ? (dim + 15) / 16
                               : turning + (rest + 2 * p.vec - 1) / (2 * p.vec);
  p.lanes = round_up_pow2(need);
  const int groups = 32 / p.lanes;
  const int its = (heads0 + groups - 1) / groups + (heads1 + groups - 1) / groups;
  const int64_t target = static_cast<int64_t>(num_sms) * 16;
  int64_t chunks = (target + tokens - 1) / tokens;
  p.chunks = static_cast<int>(chunks < its ? chunks : its);
  const int64_t blocks = (tokens * p.chunks + 7) / 8;
  const int64_t most = static_cast<int64_t>(num_sms) * (backward ? 2 : 4);
  p.grid = static_cast<int>(blocks < most ? blocks : most);
  return p;
}

template <int MODE>
cudaError_t launch_mode(const RopeArgs& a, const RopePlan& p, cudaStream_t stream) {
  auto go = [&](auto kern) {
    return launch_chained(kern, p.grid, 256, 0, 0, stream, a, p.lanes, p.chunks);
  };
  if (a.interleaved) return go(rope_kernel<8, true, MODE>);
  return p.vec == 8 ? go(rope_kernel<8, false, MODE>) : go(rope_kernel<4, false, MODE>);
}
RopePlan plan_of(const RopeArgs& a, bool backward, int num_sms) {
  return rope_plan(a.tokens, a.set[0].heads, a.sets > 1 ? a.set[1].heads : 0, a.dim, a.rot,
                   a.interleaved != 0, backward, num_sms);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  return launch_mode<kRope>(a, plan_of(a, false, num_sms), stream);
}
cudaError_t launch_qk_norm_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  return launch_mode<kQkNorm>(a, plan_of(a, false, num_sms), stream);
}

int qk_bwd_blocks(int num_sms) { return 2 * num_sms; }

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  const RopePlan p = plan_of(a, true, num_sms);
  const cudaError_t e = launch_mode<kQkNormBwd>(a, p, stream);
  float* k_gain = a.sets > 1 ? a.set[1].dgain : nullptr;
  if (e != cudaSuccess || p.grid == 1 || (!a.set[0].dgain && !k_gain)) return e;
  return launch_chained(qk_dgain_kernel, (2 * a.dim + 15) / 16, 1024, 0, 0, stream,
                        static_cast<const float*>(a.part), p.grid, a.dim, a.set[0].dgain, k_gain);
}

}  // namespace forge

// Rotary positions, and the norm of queries and keys with the rotation, forward and
// backward.
//
// The rotation.  Pair i of a head at position p turns by the angle 2 pi p f_i.  f_i, in
// turns per position, is a 64-bit fraction F_i / 2^64, so p F_i modulo 2^64 is the
// angle in fractions of a turn, exact for every position (one 64-bit integer product in
// place of a 64-bit floating one and a reduction by pi).  Its upper 32 bits give the
// quadrant and, within it, an angle of at most pi / 4, which is all that is rounded to
// fp32.
//
// The layout of the work.  A head's row is cut into vectors of VEC elements.  A lane
// holds two of them, VEC pairs: where pairs lie half the rotated part apart, the two
// vectors that turn into each other; where they lie side by side, two neighbouring ones,
// whose even elements are then one half of the pairs and whose odd ones the other.  P
// lanes (a power of two) hold a head, 32 / P heads a warp at a time: one step.
// A block keeps to one chunk of steps of the queries' or the keys' heads and walks the
// tokens with it, a warp a token: pointers only move on, gains and their gradients' sums
// stay in registers, and as soon as a step's values are unpacked those STEPS steps
// further (of this token or the next) are asked for in their place, so that loads stay
// in flight throughout.  The warp's sines and cosines are formed once a token, each lane
// some of them, and shared through memory of the warp's own.
//
// Bound by memory, and by how many loads 16 warps an SM keep in flight beside about 200
// instructions a step (the backward pass 350).  32 + 8 heads of 128 that turn whole, halves,
// with the time of the bytes at 6.79 TB/s: 8192 tokens rotated 28.4 to 29.1 us (24.7), with the
// norm 32.1 (24.7), its backward pass 48.3 to 49.2 (37.1; 2.2 of them the second launch); 1999
// tokens 9.3, 10.5 and 16.8 to 17.1 (6.0 and 9.0; the norm with half a head turning,
// neighbouring pairs, 9.8); one token 2 on the device.
// Measured and dropped: fp32 arithmetic one value at a time (it trades the packed forms'
// moves for twice the operations: backward pass 49.6 us), four elements a vector (62),
// a block a few tokens without a walk (31.0 rotated, 13.1 for the norm of 1999 tokens), and
// asking for the next token's rows in L2 ahead (rotated 29.0 to 29.4, norm 31.9 to 31.3 and
// of 1999 tokens 10.4 to 10.6, its backward pass 48.4 to 52.3).
#include <cuda_bf16.h>

#include "forge_e4m3.cuh"
#include "forge_internal.h"
#include "forge_launch.cuh"
#include "forge_layer.cuh"

namespace forge {
namespace {

enum RopeMode { kRope = 0, kQkNorm = 1, kQkNormBwd = 2 };
// By mode: the steps whose loads are in flight at once, and the most steps of a chunk
// (longer chunks form fewer sines and cosines, shorter ones leave more blocks and less to
// wait for: norm and rotation of 1999 tokens, whole heads, 10.5 us with chunks of two, 11.2 of
// four and 12.4 of eight; its backward pass 17.0, 18.0 and 20.4).
constexpr int kSteps[] = {4, 2, 1}, kChunk[] = {4, 2, 2};
// Two blocks of 256 threads an SM, with up to 128 registers a thread; three, with 80,
// spill (backward pass of 8192 tokens 82 us in place of 49).
constexpr int kBlocks = 2;

// Which blocks take what: the chunks of set k, `per` steps each (a multiple of the steps
// in flight), have `blocks` blocks each, one chunk's after the other's.
struct RopeGrid {
  int lanes;
  struct {
    int chunks, per, blocks;
  } set[2];
};

// VEC bf16 values as 32-bit words.
template <int VEC>
struct Words {
  using V = std::conditional_t<VEC == 8, uint4, uint2>;
  uint32_t w[VEC / 2];
  __device__ __forceinline__ Words() = default;
  __device__ __forceinline__ explicit Words(V v) {
    w[0] = v.x;
    w[1] = v.y;
    if constexpr (VEC == 8) {
      w[2] = v.z;
      w[3] = v.w;
    }
  }
  __device__ __forceinline__ V vec() const {
    if constexpr (VEC == 8) return make_uint4(w[0], w[1], w[2], w[3]);
    else return make_uint2(w[0], w[1]);
  }
  static __device__ __forceinline__ V all(uint32_t v) {
    if constexpr (VEC == 8) return make_uint4(v, v, v, v);
    else return make_uint2(v, v);
  }
  static __device__ __forceinline__ V zero() { return all(0u); }
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

// The two vectors as the first and second elements of VEC pairs, two pairs a float2.
template <int VEC, bool INTER>
__device__ __forceinline__ void to_pairs(typename Words<VEC>::V va, typename Words<VEC>::V vb,
                                         float2 (&a)[VEC / 2], float2 (&b)[VEC / 2]) {
  const Words<VEC> x(va), y(vb);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    if constexpr (INTER) {
      const uint32_t w0 = i < VEC / 4 ? x.w[2 * i] : y.w[2 * i - VEC / 2];
      const uint32_t w1 = i < VEC / 4 ? x.w[2 * i + 1] : y.w[2 * i + 1 - VEC / 2];
      a[i] = make_float2(bf16_lo(w0), bf16_lo(w1));
      b[i] = make_float2(bf16_hi(w0), bf16_hi(w1));
    } else {
      a[i] = make_float2(bf16_lo(x.w[i]), bf16_hi(x.w[i]));
      b[i] = make_float2(bf16_lo(y.w[i]), bf16_hi(y.w[i]));
    }
  }
}
template <int VEC, bool INTER>
__device__ __forceinline__ void from_pairs(const float2 (&a)[VEC / 2], const float2 (&b)[VEC / 2],
                                           typename Words<VEC>::V& va,
                                           typename Words<VEC>::V& vb) {
  Words<VEC> x, y;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    if constexpr (INTER) {
      uint32_t* w = i < VEC / 4 ? x.w + 2 * i : y.w + 2 * i - VEC / 2;
      w[0] = pack_bf16x2(a[i].x, b[i].x);
      w[1] = pack_bf16x2(a[i].y, b[i].y);
    } else {
      x.w[i] = pack_bf16x2(a[i].x, a[i].y);
      y.w[i] = pack_bf16x2(b[i].x, b[i].y);
    }
  }
  va = x.vec();
  vb = y.vec();
}
// The element of component j (0, 1) of the first (s = 0) or second elements a[i], b[i],
// and whether it exists.
template <int VEC, bool INTER>
__device__ __forceinline__ int element_of(const LanePart& p, int i, int j, int s) {
  if (INTER) return p.a + 2 * (2 * i + j) + s;
  return (s ? p.b : p.a) + 2 * i + j;
}
template <int VEC, bool INTER>
__device__ __forceinline__ bool exists(const LanePart& p, int i, int s) {
  return (INTER ? i < VEC / 4 : s == 0) ? p.has_a : p.has_b;
}

// Sine and cosine of 2 pi turn / 2^32.  The nearest quarter turn comes off exactly; for
// the rest, |x| <= pi / 4, the Taylor series to x^9 and x^10 leave less than 2^-28 and
// 2^-30; rounding the angle and the last operations of the series to fp32 costs more, about
// 2^-24 in all.  (sincospi does the same for any argument: the backward pass of 8192 tokens
// 53.9 us with it.)
__device__ __forceinline__ void sin_cos(uint32_t turn, float& s, float& c) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) *
                  1.4629180792671596e-9f;   // 2 pi / 2^32
  const float q = x * x;
  const float sx = fmaf(fmaf(fmaf(fmaf(1.0f / 362880.0f, q, -1.0f / 5040.0f), q, 1.0f / 120.0f), q,
                             -1.0f / 6.0f), q * x, x);
  const float cx = fmaf(fmaf(fmaf(fmaf(fmaf(-1.0f / 3628800.0f, q, 1.0f / 40320.0f), q,
                                       -1.0f / 720.0f), q, 1.0f / 24.0f), q, -0.5f), q, 1.0f);
  s = quarter & 1u ? cx : sx;
  c = quarter & 1u ? sx : cx;
  if (quarter & 2u) s = -s;
  if ((quarter + 1u) & 2u) c = -c;
}
// Those of all the head's pairs at a position, times the magnitude, into the warp's
// tables: cosines, sines (back = -1: of the opposite angle) and their negatives.
__device__ __forceinline__ void fill_turns(const RopeArgs& r, int64_t pos, int lane, float back,
                                           float (*table)[128]) {
  for (int i = lane; i < r.rot / 2; i += 32) {
    const uint64_t at = static_cast<uint64_t>(pos) * r.freqs[i];
    float s, c;
    sin_cos(static_cast<uint32_t>(at >> 32), s, c);
    s *= back * r.magnitude;
    table[0][i] = c * r.magnitude;
    table[1][i] = s;
    table[2][i] = -s;
  }
}
// Those of the lane's VEC pairs, which follow one another.
template <int VEC>
__device__ __forceinline__ void load_turns(const float* t, float2 (&v)[VEC / 2]) {
#pragma unroll
  for (int i = 0; i < VEC / 2; i += 2) {
    const float4 w = *reinterpret_cast<const float4*>(t + 2 * i);
    v[i] = make_float2(w.x, w.y);
    v[i + 1] = make_float2(w.z, w.w);
  }
}
// The pairs turned by the angle whose cosines, sines and their negatives are c, s and n.
template <int VEC>
__device__ __forceinline__ void turn(const LanePart& p, const float2 (&c)[VEC / 2],
                                     const float2 (&s)[VEC / 2], const float2 (&n)[VEC / 2],
                                     float2 (&a)[VEC / 2], float2 (&b)[VEC / 2]) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    if (i < VEC / 4 ? p.rot_a : p.rot_b) {
      const float2 x = a[i], y = b[i];
      a[i] = fma2(n[i], y, mul2(c[i], x));
      b[i] = fma2(s[i], x, mul2(c[i], y));
    }
  }
}

// Sum over the `lanes` lanes of a head (P of them where P is not 0).
template <int P>
__device__ __forceinline__ float head_sum(float v, int lanes) {
  if constexpr (P > 0) {
#pragma unroll
    for (int o = P >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  } else {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// P: lanes of a head, 0 where the launch says them.
template <int VEC, bool INTER, int MODE, int P>
__global__ void __launch_bounds__(256, kBlocks)
    rope_kernel(const RopeArgs r, const RopeGrid grid) {
  using V = typename Words<VEC>::V;
  constexpr bool kBwd = MODE == kQkNormBwd;
  constexpr int STEPS = kSteps[MODE];
  constexpr int N = VEC / 2;
  __shared__ __align__(16) float tables[8][3][128];   // [warp][table][pair]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = P > 0 ? P : grid.lanes, u = lane & (lanes - 1), g = lane / lanes, groups = 32 / lanes;
  const LanePart p = lane_part<VEC, INTER>(u, r.dim, r.rot);
  const int of0 = grid.set[0].chunks * grid.set[0].blocks;
  const int k = static_cast<int>(blockIdx.x) >= of0;
  const int rank = static_cast<int>(blockIdx.x) - (k ? of0 : 0);
  const int chunk = rank / grid.set[k].blocks, sub = rank - chunk * grid.set[k].blocks;
  const HeadSet& set = r.set[k];
  const int per = grid.set[k].per, first = chunk * per * groups, head0 = first + g;
  const int end = min(set.heads, first + per * groups);
  // a step whose heads all exist has nothing to ask where the lanes fill a head
  const bool whole = 2 * VEC * lanes == r.dim;
  auto all_of = [&](int step) { return whole && first + (step + 1) * groups <= end; };

  const int64_t walk = static_cast<int64_t>(grid.set[k].blocks) * 8;   // tokens from one to the next
  int64_t t = static_cast<int64_t>(sub) * 8 + warp;
  const int64_t x_step = groups * set.x_head, x_jump = walk * set.x_token - per * x_step;
  const int64_t y_step = groups * set.y_head, y_jump = walk * set.y_token - per * y_step;
  const int64_t dy_step = groups * set.dy_head, dy_jump = walk * set.dy_token - per * dy_step;
  const int ab = p.b - p.a;
  // the next load: its pointers, the token's and the lane's head
  const uint16_t* x = set.x + t * set.x_token + head0 * set.x_head + p.a;
  const uint16_t* dy = kBwd ? set.dy + t * set.dy_token + head0 * set.dy_head + p.a : nullptr;
  uint16_t* y = set.y + t * set.y_token + head0 * set.y_head + p.a;
  int64_t load_t = t;
  int load_step = 0;

  V xa[STEPS], xb[STEPS], da[kBwd ? STEPS : 1], db[kBwd ? STEPS : 1];
  auto load = [&](int j) {
    const bool more = load_t < r.tokens;
    if (more && all_of(load_step)) {
      xa[j] = __ldcs(reinterpret_cast<const V*>(x));
      xb[j] = __ldcs(reinterpret_cast<const V*>(x + ab));
      if constexpr (kBwd) {
        da[j] = __ldcs(reinterpret_cast<const V*>(dy));
        db[j] = __ldcs(reinterpret_cast<const V*>(dy + ab));
      }
    } else {
      const bool in = more && head0 + load_step * groups < end;
      // Backward, an absent head is of ones with gradients of zero: finite whatever eps is
      // (zeros with eps = 0 are not), so that it adds nothing to the gain's gradient.
      xa[j] = xb[j] = Words<VEC>::all(kBwd && !in ? 0x3F803F80u : 0u);
      if (in && p.has_a) xa[j] = __ldcs(reinterpret_cast<const V*>(x));
      if (in && p.has_b) xb[j] = __ldcs(reinterpret_cast<const V*>(x + ab));
      if constexpr (kBwd) {
        da[j] = db[j] = Words<VEC>::zero();
        if (in && p.has_a) da[j] = __ldcs(reinterpret_cast<const V*>(dy));
        if (in && p.has_b) db[j] = __ldcs(reinterpret_cast<const V*>(dy + ab));
      }
    }
    x += x_step;
    if constexpr (kBwd) dy += dy_step;
    if (++load_step == per) {
      load_step = 0;
      load_t += walk;
      x += x_jump;
      if constexpr (kBwd) dy += dy_jump;
    }
  };
  float2 ga[N], gb[N], dga[N], dgb[N];
#pragma unroll
  for (int i = 0; i < N; ++i) ga[i] = gb[i] = dga[i] = dgb[i] = make_float2(0.0f, 0.0f);
  grid_dependency_wait();
#pragma unroll
  for (int j = 0; j < STEPS; ++j) load(j);
  int64_t pos = t < r.tokens ? (r.positions ? r.positions[t] : t) : 0;
  if constexpr (MODE != kRope) {
    auto gain = [&](int i, int j, int s) {
      if (!exists<VEC, INTER>(p, i, s)) return 0.0f;
      const int e = element_of<VEC, INTER>(p, i, j, s);
      return r.gain_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(set.gain)[e])
                         : static_cast<const float*>(set.gain)[e];
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ga[i] = make_float2(gain(i, 0, 0), gain(i, 1, 0));
      gb[i] = make_float2(gain(i, 0, 1), gain(i, 1, 1));
    }
  }
  float(*table)[128] = tables[warp];
  const float back = kBwd || r.inverse ? -1.0f : 1.0f;
#pragma unroll 1
  for (; t < r.tokens; t += walk) {
    __syncwarp();
    fill_turns(r, pos, lane, back, table);
    __syncwarp();
    if (t + walk < r.tokens) pos = r.positions ? r.positions[t + walk] : t + walk;
    float2 c[N], s[N], n[N];
    auto turns = [&]() {   // the lane's pairs, VEC from VEC u on
      if (!p.rot_a) return;
      load_turns<VEC>(table[0] + VEC * u, c);
      load_turns<VEC>(table[1] + VEC * u, s);
      load_turns<VEC>(table[2] + VEC * u, n);
    };
    // (with the norm again at every step: registers are short)
    if constexpr (MODE == kRope) turns();
#pragma unroll 1
    for (int step = 0; step < per; step += STEPS) {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        float2 a[N], b[N], na[N], nb[N];
        to_pairs<VEC, INTER>(xa[j], xb[j], a, b);
        if constexpr (kBwd) to_pairs<VEC, INTER>(da[j], db[j], na, nb);
        load(j);
        if constexpr (MODE != kRope) {
          float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < N; ++i) sq = fma2(b[i], b[i], fma2(a[i], a[i], sq));
          const float rstd = rsqrtf(head_sum<P>(sq.x + sq.y, lanes) * r.inv_dim + r.eps);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            a[i] = mul2(a[i], dup2(rstd));
            b[i] = mul2(b[i], dup2(rstd));
          }
          if constexpr (kBwd) {
            turns();
            turn<VEC>(p, c, s, n, na, nb);   // the gradient of the normed head
            float2 dots = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dga[i] = fma2(na[i], a[i], dga[i]);
              dgb[i] = fma2(nb[i], b[i], dgb[i]);
              na[i] = mul2(na[i], ga[i]);
              nb[i] = mul2(nb[i], gb[i]);
              dots = fma2(nb[i], b[i], fma2(na[i], a[i], dots));
            }
            const float dot = head_sum<P>(dots.x + dots.y, lanes) * r.inv_dim;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              a[i] = mul2(dup2(rstd), fma2(dup2(-dot), a[i], na[i]));
              b[i] = mul2(dup2(rstd), fma2(dup2(-dot), b[i], nb[i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              a[i] = mul2(a[i], ga[i]);
              b[i] = mul2(b[i], gb[i]);
            }
          }
        }
        if constexpr (MODE == kQkNorm) turns();
        if constexpr (!kBwd) turn<VEC>(p, c, s, n, a, b);
        V va, vb;
        from_pairs<VEC, INTER>(a, b, va, vb);
        if (all_of(step + j)) {
          __stcs(reinterpret_cast<V*>(y), va);
          __stcs(reinterpret_cast<V*>(y + ab), vb);
        } else {
          const bool in = head0 + (step + j) * groups < end;
          if (in && p.has_a) __stcs(reinterpret_cast<V*>(y), va);
          if (in && p.has_b) __stcs(reinterpret_cast<V*>(y + ab), vb);
        }
        y += y_step;
      }
    }
    y += y_jump;
  }
  grid_dependency_trigger();
  if constexpr (kBwd) {
    // The gain's gradient: the head groups of a warp, then the block's warps, each in a
    // fixed order; the block leaves one partial row, or the result where it is alone.
    if (!set.dgain) return;
    __shared__ float sum[8][256];   // [warp][element]
#pragma unroll
    for (int i = 0; i < N; ++i) {
      for (int o = 16; o >= lanes; o >>= 1) {
        dga[i].x += __shfl_xor_sync(0xffffffffu, dga[i].x, o);
        dga[i].y += __shfl_xor_sync(0xffffffffu, dga[i].y, o);
        dgb[i].x += __shfl_xor_sync(0xffffffffu, dgb[i].x, o);
        dgb[i].y += __shfl_xor_sync(0xffffffffu, dgb[i].y, o);
      }
      if (g == 0 && exists<VEC, INTER>(p, i, 0)) {
        sum[warp][element_of<VEC, INTER>(p, i, 0, 0)] = dga[i].x;
        sum[warp][element_of<VEC, INTER>(p, i, 1, 0)] = dga[i].y;
      }
      if (g == 0 && exists<VEC, INTER>(p, i, 1)) {
        sum[warp][element_of<VEC, INTER>(p, i, 0, 1)] = dgb[i].x;
        sum[warp][element_of<VEC, INTER>(p, i, 1, 1)] = dgb[i].y;
      }
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < r.dim) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += sum[w][threadIdx.x];
      const bool alone = grid.set[k].chunks * grid.set[k].blocks == 1;
      (alone ? set.dgain : r.part + static_cast<int64_t>(blockIdx.x) * r.dim)[threadIdx.x] = v;
    }
  }
}

// The partial rows of each set: 16 columns a block, 64 runs of rows side by side.
__global__ void __launch_bounds__(1024) qk_dgain_kernel(const float* part, int rows0, int rows1,
                                                        int dim, float* dq_gain, float* dk_gain) {
  __shared__ float sum[64][17];
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col, k = blockIdx.y;
  const int first = k ? rows0 : 0, rows = k ? rows1 : rows0;
  float* out = k ? dk_gain : dq_gain;
  grid_dependency_wait();
  grid_dependency_trigger();
  if (!out || rows <= 1) return;   // (one row: written where it belongs)
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 4
    for (int b = run; b < rows; b += 64) s += __ldcg(part + static_cast<int64_t>(first + b) * dim + c);
  }
  sum[run][col] = s;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp a column
  if (warp >= 16) return;
  s = sum[lane][warp] + sum[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 16 + warp < dim) out[blockIdx.x * 16 + warp] = s;
}

struct RopePlan {
  int vec;
  RopeGrid grid;
  int blocks(int k) const { return grid.set[k].chunks * grid.set[k].blocks; }
};
int round_up_pow2(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}
// Vectors of eight, or of four where half the rotated part is no multiple of eight.
// As many blocks as are resident at once, shared among the chunks by their steps (and
// two for a token's sines and cosines), or one a chunk and eight tokens where there are
// fewer.
RopePlan rope_plan(const RopeArgs& a, RopeMode mode, int num_sms) {
  RopePlan p;
  p.vec = a.interleaved || a.rot % 16 == 0 ? 8 : 4;
  const int turning = a.rot / (2 * p.vec), rest = a.dim - a.rot;
  const int need = a.interleaved ? (a.dim + 15) / 16
                                 : turning + (rest + 2 * p.vec - 1) / (2 * p.vec);
  p.grid.lanes = round_up_pow2(need);
  const int groups = 32 / p.grid.lanes;
  const int flight = kSteps[mode];
  const int64_t cap = static_cast<int64_t>(num_sms) * kBlocks;
  const int64_t full = (a.tokens + 7) / 8;
  // few tokens: shorter chunks, for more blocks
  int most = kChunk[mode];
  auto chunks_of = [&](int k) {
    const int steps = (a.set[k].heads + groups - 1) / groups;
    return (steps + most - 1) / most;
  };
  while (most > flight && full * (chunks_of(0) + chunks_of(1)) * 2 <= cap) most /= 2;
  int64_t weight = 0;
  for (int k = 0; k < 2; ++k) {
    auto& s = p.grid.set[k];
    const int steps = (a.set[k].heads + groups - 1) / groups;
    s.chunks = chunks_of(k);
    s.per = s.chunks ? ((steps + s.chunks - 1) / s.chunks + flight - 1) / flight * flight : 0;
    if (s.per) s.chunks = (steps + s.per - 1) / s.per;
    weight += static_cast<int64_t>(s.chunks) * (s.per + 2);
  }
  for (int k = 0; k < 2; ++k) {
    auto& s = p.grid.set[k];
    int64_t n = s.chunks ? cap * (s.per + 2) / weight : 1;
    n = n < full ? n : full;
    s.blocks = static_cast<int>(n > 1 ? n : 1);
  }
  return p;
}

template <int MODE>
cudaError_t launch_mode(const RopeArgs& a, const RopePlan& p, cudaStream_t stream) {
  auto go = [&](auto kern) {
    return launch_chained(kern, p.blocks(0) + p.blocks(1), 256, 0, 0, stream, a, p.grid);
  };
  // Heads of 128 (down to 65) and of 64 know their lanes; not the backward pass of
  // neighbouring pairs, which spills more so (8192 tokens 54.5 us in place of 52).
  if (a.interleaved) {
    if constexpr (MODE != kQkNormBwd) {
      if (p.grid.lanes == 8) return go(rope_kernel<8, true, MODE, 8>);
      if (p.grid.lanes == 4) return go(rope_kernel<8, true, MODE, 4>);
    }
    return go(rope_kernel<8, true, MODE, 0>);
  }
  if (p.vec == 4) return go(rope_kernel<4, false, MODE, 0>);
  if (p.grid.lanes == 8) return go(rope_kernel<8, false, MODE, 8>);
  if (p.grid.lanes == 4) return go(rope_kernel<8, false, MODE, 4>);
  return go(rope_kernel<8, false, MODE, 0>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  return launch_mode<kRope>(a, rope_plan(a, kRope, num_sms), stream);
}
cudaError_t launch_qk_norm_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  return launch_mode<kQkNorm>(a, rope_plan(a, kQkNorm, num_sms), stream);
}

// A block a chunk at least: kMaxHeads heads of each kind, one a step where they are widest.
int qk_bwd_blocks(int num_sms) { return kBlocks * num_sms + 2 * (kMaxHeads / kSteps[kQkNormBwd]); }

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  const RopePlan p = rope_plan(a, kQkNormBwd, num_sms);
  const cudaError_t e = launch_mode<kQkNormBwd>(a, p, stream);
  if (e != cudaSuccess) return e;
  const bool join = (a.set[0].dgain && p.blocks(0) > 1) || (a.set[1].dgain && p.blocks(1) > 1);
  if (!join) return e;
  return launch_chained_2d(qk_dgain_kernel, dim3((a.dim + 15) / 16, 2, 1), 1024, 0, 0, stream,
                           static_cast<const float*>(a.part), p.blocks(0), p.blocks(1), a.dim,
                           a.set[0].dgain, a.set[1].dgain);
}

}  // namespace forge

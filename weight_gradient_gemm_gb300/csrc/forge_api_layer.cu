// Host side of the operators between a layer's 16-bit products: the product with its
// epilogue, the epilogue's gradient, dropout, rotary positions and the norm of queries
// and keys.  Arguments are checked before anything is enqueued; every entry point
// answers with a status and no C++ exception leaves it.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <numeric>

#include "forge.h"
#include "forge_internal.h"

using namespace forge;

namespace {

constexpr int64_t kMaxIndex = (1LL << 31) - 1;
constexpr int64_t kMaxValues = 1LL << 40;   // of one elementwise call

bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}
bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}

struct Span {
  const void* p;
  uint64_t n;
};
bool meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}
// Whether an output overlaps any of `others`.
bool meets_any(const Span& o, std::initializer_list<Span> others) {
  for (const Span& s : others)
    if (meet(o, s)) return true;
  return false;
}
// Whether an output overlaps an input other than by taking its place (the same buffer:
// each element is read before it is written, by the same thread).
bool meets_apart(const Span& o, std::initializer_list<Span> ins) {
  for (const Span& s : ins)
    if (o.p != s.p && meet(o, s)) return true;
  return false;
}

// The status of a call's launches; a failed one leaves no error behind.
forge_status status(cudaError_t e) {
  if (e == cudaSuccess) return FORGE_OK;
  (void)cudaGetLastError();
  return FORGE_ERR_LAUNCH;
}

bool is_dtype(forge_dtype t) { return t == FORGE_DT_FP32 || t == FORGE_DT_BF16; }
uint64_t size_of(forge_dtype t) { return t == FORGE_DT_FP32 ? 4 : 2; }
bool is_act(forge_activation a) { return a >= FORGE_ACT_NONE && a <= FORGE_ACT_SILU; }

// A call's dropout (null: none).
forge_status drop_args(const forge_drop* d, DropArgs* out) {
  *out = DropArgs{0u, 1.0f, 0, 0, nullptr};
  if (!d) return FORGE_OK;
  if (!(d->p >= 0.0f && d->p < 1.0f)) return FORGE_ERR_HYPER;
  if (!aligned(d->counter, 8)) return FORGE_ERR_ALIGN;
  // p 2^16 is exact; to the nearest whole number, ties to even, and never all
  const double t = std::nearbyint(static_cast<double>(d->p) * 65536.0);
  out->threshold = t > 65535.0 ? 65535u : static_cast<uint32_t>(t);
  out->scale = static_cast<float>(65536.0 / (65536.0 - out->threshold));
  out->seed = d->seed;
  out->offset = d->offset;
  out->counter = d->counter;
  return FORGE_OK;
}
Span counter_span(const DropArgs& d) { return Span{d.counter, 8}; }

// ---------------------------------------------------------------- the product
// The tile, by a count of cycles.
//   Single CTAs with 128 outputs along M and up to 128 tokens (forge_gemm_linear_few.cu):
//   a step of 64 of the reduction takes 512 cycles with 128 tokens, what its operands need
//   at the 64 bytes a cycle that an SM loads.  The reduction is split over a cluster as
//   long as its CTAs are all resident at once (`clusters`: [i] of 2^i, i from 1) and have two
//   steps each.  What follows takes 6000 cycles on one CTA, 5000 on two that share the
//   epilogue, 4000 on more.
//   Pairs with 256 tokens and bn outputs: 370 + 5 bn / 8 cycles a step (measured; 530 for
//   bn = 256, whose products take 512), tiles in waves, the last tile's epilogue after them.
// 333 tokens, 1032 -> 520, 7.3 us on single CTAs and 8.1 on pairs; 300, 4096 -> 1024, 9.7
// and 18.0; 512, 4096 -> 14336, 74 and 40; 150, 4096 -> 14336, 48.7 and 25.4.
// Up to 128 tokens the pairs' form leaves half of its rows empty (128 tokens, 4096 ->
// 14336, 23.1 us and 26.0), and the weight's bytes need every SM: the largest split there
// is.  Tiles of 128 tokens, one an SM, do not overlap one's end with the next's start:
// where there are more than SMs the persistent pairs take them (128 tokens, 4096 -> 20480,
// 38.6 us and 52.7, -> 57344 81.7 and 91.4, -> 131072 173 and 221); up to 64, two an SM do
// (64 tokens, -> 57344, 78.9 us and 80.7).
LinearConfig choose_linear(int64_t m, int64_t n, int64_t num_kb, const forge_tuning& tune,
                           int num_sms, const int (&clusters)[4], int most_bn = 256) {
  const int nt = m <= 16 ? 16 : (m <= 32 ? 32 : (m <= 64 ? 64 : 128));
  const int64_t tiles = (n + 127) / 128 * ((m + 127) / 128);
  LinearConfig best{nt, 128, 1};
  int64_t least = (tiles + num_sms - 1) / num_sms * num_kb * 512 + 6000;
  for (int i = 1; i <= 3; ++i) {
    const int splits = 1 << i;
    if (tune.splits ? splits > tune.splits : tiles > clusters[i] || num_kb < 2 * splits) continue;
    const int64_t cost = (num_kb + splits - 1) / splits * 512 + (splits > 2 ? 4000 : 5000);
    if (tune.splits || m <= 128 || cost < least) least = cost, best.splits = splits;
  }
  const bool waves_of_128 = m <= 128 && nt == 128 && tiles > num_sms;
  if (tune.cta_group == 1 || (m <= 128 && tune.cta_group == 0 && !waves_of_128)) return best;
  if (tune.cta_group == 2 || waves_of_128) least = INT64_MAX;
  const int64_t pairs = num_sms / 2, tiles_m = (m + 255) / 256;
  for (int bn = most_bn; bn >= 64; bn -= 32) {
    if (tune.bn && bn != (tune.bn < most_bn ? tune.bn : most_bn)) continue;
    // (a kernel counts columns in 32 bits: the last tile has to end there)
    if ((n + bn - 1) / bn * bn > kMaxIndex + 1) continue;
    const int64_t waves = (tiles_m * ((n + bn - 1) / bn) + pairs - 1) / pairs;
    const int64_t cost = waves * num_kb * (370 + 5 * bn / 8) + 24 * bn + 1500;
    if (cost < least) least = cost, best = LinearConfig{0, bn, 1};
  }
  return best;
}

}  // namespace

extern "C" {

forge_status forge_linear_bf16(const void* X, const void* W, void* Y, forge_dtype y_dtype,
                               const forge_epilogue* epilogue, int64_t bt, int64_t d_in,
                               int64_t d_out, forge_stream stream) {
  if (bt < 0 || bt > kMaxIndex || d_in <= 0 || d_in > kMaxIndex || d_out <= 0 || d_out > kMaxIndex)
    return FORGE_ERR_SHAPE;
  if (d_in % 8 != 0 || d_out % 8 != 0) return FORGE_ERR_SHAPE;
  if (!is_dtype(y_dtype)) return FORGE_ERR_FORMAT;
  forge_epilogue e;
  std::memset(&e, 0, sizeof(e));
  if (epilogue) e = *epilogue;
  if (!is_act(e.act) || (e.bias && !is_dtype(e.bias_dtype))) return FORGE_ERR_FORMAT;
  LinearArgs a;
  std::memset(&a, 0, sizeof(a));
  forge_status s = drop_args(&e.drop, &a.e.drop);
  if (s != FORGE_OK) return s;
  if (bt == 0) return FORGE_OK;
  if (!X || !W || !Y) return FORGE_ERR_NULL;
  if (!all_aligned16({X, W, Y, e.bias, e.mul, e.residual, e.z})) return FORGE_ERR_ALIGN;
  const uint64_t m = bt, k = d_in, n = d_out;
  const uint64_t es = size_of(y_dtype), bs = e.bias ? size_of(e.bias_dtype) : 0;
  const Span in_x{X, 2 * m * k}, in_w{W, 2 * n * k}, in_b{e.bias, bs * n};
  const Span in_m{e.mul, 2 * m * n}, in_r{e.residual, 2 * m * n}, in_c = counter_span(a.e.drop);
  const Span o_y{Y, es * m * n}, o_z{e.z, 2 * m * n};
  if (meets_any(o_y, {in_x, in_w, in_b, in_c, o_z}) ||
      meets_any(o_z, {in_x, in_w, in_b, in_c, in_m, in_r}))
    return FORGE_ERR_ALIAS;
  // Y may take the place of the residual or of mul, in the same type
  if (es == 2 ? meets_apart(o_y, {in_m, in_r}) : meets_any(o_y, {in_m, in_r}))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  forge_tuning tune;
  forge_get_tuning(&tune);
  const int64_t num_kb = (d_in + 63) / 64;
  int clusters[4] = {};
  const int nt = bt <= 16 ? 16 : (bt <= 32 ? 32 : (bt <= 64 ? 64 : 128));
  for (int i = 1; i < 4; ++i) {
    const cudaError_t r = linear_few_clusters(nt, 1 << i, d.num_sms, &clusters[i]);
    if (r != cudaSuccess) return status(r);
  }
  const LinearConfig cfg = choose_linear(bt, d_out, num_kb, tune, d.num_sms, clusters,
                                         es == 4 ? kMaxLinearF32 : 256);
  const int64_t rows = cfg.few ? cfg.few : 256, tiles_m = (bt + rows - 1) / rows;
  const int64_t tiles_n = (d_out + cfg.bn - 1) / cfg.bn;
  if (tiles_m * tiles_n > kMaxIndex / 8) return FORGE_ERR_SHAPE;
  const CUtensorMapDataType b16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint32_t rows_a = cfg.few ? cfg.few : 128, rows_b = cfg.few ? 128 : cfg.bn / 2;
  bool maps = host_map(&a.a, X, b16, k, m, k * 2, 64, rows_a, sw) &&
              host_map(&a.b, W, b16, k, n, k * 2, 64, rows_b, sw);
  if (!maps) return FORGE_ERR_LAUNCH;
  a.e.bias = e.bias;
  a.e.bias_bf16 = e.bias && e.bias_dtype == FORGE_DT_BF16;
  a.e.act = e.act;
  a.e.mul = static_cast<const uint16_t*>(e.mul);
  a.e.residual = static_cast<const uint16_t*>(e.residual);
  a.e.z = static_cast<uint16_t*>(e.z);
  a.e.y = Y;
  a.e.y_fp32 = es == 4;
  a.m = static_cast<int32_t>(bt);
  a.n = static_cast<int32_t>(d_out);
  a.num_kb = static_cast<int32_t>(num_kb);
  a.chunk = es == 4 ? kLinearChunk : a.num_kb;
  a.tiles_m = static_cast<int32_t>(tiles_m);
  a.tiles_n = static_cast<int32_t>(tiles_n);
  a.num_tiles = static_cast<int32_t>(tiles_m * tiles_n);
  a.group_m = tune.group_m >= 1 && tune.group_m <= 64 ? tune.group_m : 16;
  if (a.group_m > a.tiles_m) a.group_m = a.tiles_m;
  a.bn = cfg.bn;
  a.wide = d_out % 16 == 0 && aligned(Y, 32) && aligned(e.mul, 32) && aligned(e.residual, 32) &&
           aligned(e.z, 32);
  a.splits = cfg.splits;
  a.err = d.err;
  a.err_site = d.err_site;
  a.timeout_ns = d.timeout_ns;
  a.drop_first_arrival = host_drop_flag();
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return status(cfg.few ? launch_gemm_linear_few(cfg.few, a, d.num_sms, cs)
                        : launch_gemm_linear(a, d.num_sms, cs));
}

size_t forge_epilogue_backward_workspace_bytes(int64_t rows, int64_t cols) {
  HostDevice d;
  if (rows < 0 || rows > kMaxIndex || cols <= 0 || cols > kMaxIndex || cols % 8 != 0) return 0;
  if (host_device(&d) != FORGE_OK) return 0;
  return static_cast<size_t>(epilogue_bwd_rows(rows, cols, d.num_sms)) *
         static_cast<size_t>(cols) * 4;
}

forge_status forge_epilogue_backward(const void* dY, const void* Z, const void* mul,
                                     forge_activation act, const forge_drop* drop, void* dZ,
                                     void* dmul, float* dbias, int64_t rows, int64_t cols,
                                     void* workspace, size_t workspace_bytes,
                                     forge_stream stream) {
  if (rows < 0 || rows > kMaxIndex || cols <= 0 || cols > kMaxIndex || cols % 8 != 0)
    return FORGE_ERR_SHAPE;
  if (rows > kMaxValues / cols) return FORGE_ERR_SHAPE;
  if (!is_act(act)) return FORGE_ERR_FORMAT;
  EpiBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  forge_status s = drop_args(drop, &a.drop);
  if (s != FORGE_OK) return s;
  if (!dZ && !dmul && !dbias) return FORGE_ERR_NULL;
  if (dmul && !mul && rows > 0) return FORGE_ERR_NULL;
  if (rows > 0 && (!dY || (!Z && (act != FORGE_ACT_NONE || dmul)))) return FORGE_ERR_NULL;
  if (!all_aligned16({dY, Z, mul, dZ, dmul, dbias, workspace})) return FORGE_ERR_ALIGN;
  const uint64_t n = static_cast<uint64_t>(rows) * cols;
  const Span in_dy{dY, 2 * n}, in_z{Z, 2 * n}, in_m{mul, 2 * n}, in_c = counter_span(a.drop);
  const Span o_dz{dZ, 2 * n}, o_dm{dmul, 2 * n}, o_db{dbias, static_cast<uint64_t>(cols) * 4};
  const Span ws{dbias ? workspace : nullptr, workspace_bytes};
  if (meets_any(o_db, {in_dy, in_z, in_m, in_c, o_dz, o_dm, ws}) ||
      meets_any(ws, {in_dy, in_z, in_m, in_c, o_dz, o_dm}) || meets_any(o_dz, {o_dm, in_c}) ||
      meets_any(o_dm, {in_c}))
    return FORGE_ERR_ALIAS;
  if (meets_apart(o_dz, {in_dy, in_z, in_m}) || meets_apart(o_dm, {in_dy, in_z, in_m}))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (rows == 0)   // no rows: the sum over them is zero
    return dbias ? status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(cols) * 4, cs)) : FORGE_OK;
  if (dbias) {
    const size_t want = forge_epilogue_backward_workspace_bytes(rows, cols);
    if (want > 0 && !workspace) return FORGE_ERR_NULL;
    if (workspace_bytes < want) return FORGE_ERR_SHAPE;
  }
  a.dy = static_cast<const uint16_t*>(dY);
  a.z = static_cast<const uint16_t*>(Z);
  a.mul = static_cast<const uint16_t*>(mul);
  a.dz = static_cast<uint16_t*>(dZ);
  a.dmul = static_cast<uint16_t*>(dmul);
  a.dbias = dbias;
  a.part = static_cast<float*>(workspace);
  a.rows = rows;
  a.cols = cols;
  a.act = act;
  return status(launch_epilogue_bwd(a, d.num_sms, cs));
}

forge_status forge_dropout(const void* x, const void* residual, void* y, const forge_drop* drop,
                           int64_t rows, int64_t cols, forge_stream stream) {
  if (rows < 0 || rows > kMaxIndex || cols <= 0 || cols > kMaxIndex || cols % 8 != 0)
    return FORGE_ERR_SHAPE;
  if (rows > kMaxValues / cols) return FORGE_ERR_SHAPE;
  if (!drop) return FORGE_ERR_NULL;
  DropArgs dr;
  forge_status s = drop_args(drop, &dr);
  if (s != FORGE_OK) return s;
  if (rows == 0) return FORGE_OK;
  if (!x || !y) return FORGE_ERR_NULL;
  if (!all_aligned16({x, residual, y})) return FORGE_ERR_ALIGN;
  const uint64_t n = 2 * static_cast<uint64_t>(rows) * cols;
  if (meets_apart({y, n}, {{x, n}, {residual, n}}) || meet({y, n}, counter_span(dr)))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  return status(launch_dropout(static_cast<const uint16_t*>(x),
                               static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(y),
                               rows, cols, dr, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------- heads
namespace {

constexpr int kMaxHeadDim = 256;

// One view [tokens, heads, dim] of a call.
struct View {
  const void* p;
  int64_t token, head;   // strides in elements (0 where there is one token or head)
  int64_t tokens, heads, dim;

  View() = default;
  View(const void* ptr, int64_t token_stride, int64_t head_stride, int64_t t, int64_t h, int64_t d)
      : p(ptr), token(t > 1 ? token_stride : 0), head(h > 1 ? head_stride : 0), tokens(t),
        heads(h), dim(d) {}

  // elements from the first to behind the last
  uint64_t extent() const {
    return static_cast<uint64_t>((tokens - 1) * token + (heads - 1) * head + dim);
  }
  Span span() const { return Span{p, p ? 2 * extent() : 0}; }
};
bool same_place(const View& a, const View& b) {
  return a.p == b.p && a.token == b.token && a.head == b.head && a.heads == b.heads;
}
forge_status check_view(const View& v, bool output) {
  if (!v.p) return FORGE_ERR_NULL;
  if (!aligned(v.p, 16)) return FORGE_ERR_ALIGN;
  constexpr int64_t kMaxStride = 1LL << 40;
  if (v.token < 0 || v.head < 0 || v.token > kMaxStride || v.head > kMaxStride ||
      v.token % 8 != 0 || v.head % 8 != 0)
    return FORGE_ERR_SHAPE;
  if ((v.tokens > 1 && v.token > (1LL << 60) / v.tokens) ||
      (v.heads > 1 && v.head > (1LL << 60) / v.heads))
    return FORGE_ERR_SHAPE;
  if (output) {   // no element twice: one dimension lies within the other's steps
    const bool in_token = (v.heads == 1 || v.head >= v.dim) &&
                          (v.tokens == 1 || v.token >= (v.heads - 1) * v.head + v.dim);
    const bool in_head = (v.tokens == 1 || v.token >= v.dim) &&
                         (v.heads == 1 || v.head >= (v.tokens - 1) * v.token + v.dim);
    if (!in_token && !in_head) return FORGE_ERR_ALIAS;
  }
  return FORGE_OK;
}
// Whether two views share an element: their bounds meet, and they are not interleaved
// rows of one buffer (as queries and keys in the projections' fused output are), token by
// token, head by head or, where all strides are multiples of one step ([tokens, heads, 3,
// dim]), within that step.
bool views_meet(const View& a, const View& b) {
  if (!a.p || !b.p || !meet(a.span(), b.span())) return false;
  auto interleaved = [&](int64_t step_a, int64_t step_b, uint64_t row_a, uint64_t row_b) {
    if (step_a != step_b || step_a <= 0) return false;
    const uint64_t step = 2 * static_cast<uint64_t>(step_a);   // bytes
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uint64_t at = (pb >= pa ? (pb - pa) % step : (step - (pa - pb) % step) % step);
    return 2 * row_a <= at && at + 2 * row_b <= step;   // b's row behind a's, before a's next
  };
  const uint64_t ta = (a.heads - 1) * a.head + a.dim, tb = (b.heads - 1) * b.head + b.dim;
  const uint64_t ha = (a.tokens - 1) * a.token + a.dim, hb = (b.tokens - 1) * b.token + b.dim;
  const int64_t step = std::gcd(std::gcd(a.token, a.head), std::gcd(b.token, b.head));
  return !interleaved(a.token, b.token, ta, tb) && !interleaved(a.head, b.head, ha, hb) &&
         !interleaved(step, step, a.dim, b.dim);
}

struct HeadCall {
  View x[2], dy[2], y[2];
};

// Checks the parts that the three calls share and fills the kernel's arguments.
forge_status rope_args(const forge_heads* sets, int n, const forge_rotation* rot, int64_t tokens,
                       int64_t head_dim, bool norm, forge_dtype gain_dtype, float eps,
                       bool backward, RopeArgs* a, HostDevice* d) {
  std::memset(a, 0, sizeof(*a));
  if (!sets || !rot) return FORGE_ERR_NULL;
  if (n < 1 || n > 2 || tokens < 0 || tokens > kMaxIndex) return FORGE_ERR_SHAPE;
  if (head_dim <= 0 || head_dim > kMaxHeadDim || head_dim % 8 != 0) return FORGE_ERR_SHAPE;
  if (rot->dim <= 0 || rot->dim > head_dim || rot->dim % 8 != 0) return FORGE_ERR_SHAPE;
  if (rot->layout != FORGE_ROPE_HALF && rot->layout != FORGE_ROPE_INTERLEAVED)
    return FORGE_ERR_FORMAT;
  if (norm && !is_dtype(gain_dtype)) return FORGE_ERR_FORMAT;
  if (!std::isfinite(rot->magnitude)) return FORGE_ERR_HYPER;
  if (norm && (!(eps >= 0.0f) || !std::isfinite(eps))) return FORGE_ERR_HYPER;
  for (int i = 0; i < n; ++i)
    if (sets[i].heads < 0 || sets[i].heads > kMaxHeads) return FORGE_ERR_SHAPE;
  if (!rot->freqs && tokens > 0) return FORGE_ERR_NULL;
  if (!aligned(rot->freqs, 8) || !aligned(rot->positions, 8)) return FORGE_ERR_ALIGN;
  const Span small[2] = {{rot->freqs, static_cast<uint64_t>(rot->dim) * 4},
                         {rot->positions, static_cast<uint64_t>(tokens) * 8}};
  const uint64_t gain_bytes =
      norm ? static_cast<uint64_t>(head_dim) * size_of(gain_dtype) : 0;
  HeadCall c;
  int used = 0;
  for (int i = 0; i < n; ++i) {
    const forge_heads& s = sets[i];
    if (norm && (!s.gain && (tokens > 0 && s.heads > 0))) return FORGE_ERR_NULL;
    if (norm && !all_aligned16({s.gain, backward ? s.dgain : nullptr})) return FORGE_ERR_ALIGN;
    c.x[i] = View{s.x, s.x_token, s.x_head, tokens, s.heads, head_dim};
    c.dy[i] = View{backward ? s.dy : nullptr, s.dy_token, s.dy_head, tokens, s.heads, head_dim};
    c.y[i] = View{s.y, s.y_token, s.y_head, tokens, s.heads, head_dim};
    if (tokens > 0 && s.heads > 0) {
      ++used;
      forge_status st = check_view(c.x[i], false);
      if (st == FORGE_OK && backward) st = check_view(c.dy[i], false);
      if (st == FORGE_OK) st = check_view(c.y[i], true);
      if (st != FORGE_OK) return st;
    } else {
      c.x[i].p = c.dy[i].p = c.y[i].p = nullptr;   // nothing of it is touched
    }
  }
  for (int i = 0; i < n; ++i) {
    const Span dg{backward ? sets[i].dgain : nullptr, static_cast<uint64_t>(head_dim) * 4};
    for (int j = 0; j < n; ++j) {
      // an output may take the place of its own set's input
      for (const View* in : {&c.x[j], &c.dy[j]})
        if (!(i == j && c.y[i].p && in->p && same_place(c.y[i], *in)) && views_meet(c.y[i], *in))
          return FORGE_ERR_ALIAS;
      if (i < j && views_meet(c.y[i], c.y[j])) return FORGE_ERR_ALIAS;
      const Span gain{norm ? sets[j].gain : nullptr, gain_bytes};
      const Span dg_j{backward ? sets[j].dgain : nullptr, static_cast<uint64_t>(head_dim) * 4};
      if (c.y[i].p && meets_any(c.y[i].span(), {gain, dg_j})) return FORGE_ERR_ALIAS;
      if (meets_any(dg, {gain, c.x[j].p ? c.x[j].span() : Span{nullptr, 0},
                         c.dy[j].p ? c.dy[j].span() : Span{nullptr, 0}}) ||
          (i < j && meet(dg, dg_j)))
        return FORGE_ERR_ALIAS;
    }
    for (const Span& s : small)
      if ((c.y[i].p && meet(c.y[i].span(), s)) || meet(dg, s)) return FORGE_ERR_ALIAS;
  }
  const int st = host_device(d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  for (int i = 0; i < n; ++i) {
    const forge_heads& s = sets[i];
    HeadSet& h = a->set[i];
    h.x = static_cast<const uint16_t*>(s.x);
    h.dy = static_cast<const uint16_t*>(backward ? s.dy : nullptr);
    h.y = static_cast<uint16_t*>(s.y);
    h.gain = norm ? s.gain : nullptr;
    h.dgain = backward ? s.dgain : nullptr;
    h.x_token = c.x[i].token; h.x_head = c.x[i].head;
    h.dy_token = c.dy[i].token; h.dy_head = c.dy[i].head;
    h.y_token = c.y[i].token; h.y_head = c.y[i].head;
    h.heads = tokens > 0 ? static_cast<int32_t>(s.heads) : 0;
  }
  a->dim = static_cast<int32_t>(head_dim);
  a->rot = rot->dim;
  a->interleaved = rot->layout == FORGE_ROPE_INTERLEAVED;
  a->gain_bf16 = norm && gain_dtype == FORGE_DT_BF16;
  a->freqs = rot->freqs;
  a->positions = rot->positions;
  a->magnitude = rot->magnitude;
  a->eps = eps;
  a->inv_dim = 1.0f / static_cast<float>(head_dim);
  a->tokens = used ? tokens : 0;
  return FORGE_OK;
}

}  // namespace

extern "C" {

forge_status forge_rope(const forge_heads* sets, int n, const forge_rotation* rot, int inverse,
                        int64_t tokens, int64_t head_dim, forge_stream stream) {
  RopeArgs a;
  HostDevice d;
  const forge_status s = rope_args(sets, n, rot, tokens, head_dim, false, FORGE_DT_FP32, 0.0f,
                                   false, &a, &d);
  if (s != FORGE_OK || a.tokens == 0) return s;
  a.inverse = inverse != 0;
  return status(launch_rope(a, d.num_sms, static_cast<cudaStream_t>(stream)));
}

forge_status forge_qk_norm_rope(const forge_heads* sets, int n, forge_dtype gain_dtype, float eps,
                                const forge_rotation* rot, int64_t tokens, int64_t head_dim,
                                forge_stream stream) {
  RopeArgs a;
  HostDevice d;
  const forge_status s =
      rope_args(sets, n, rot, tokens, head_dim, true, gain_dtype, eps, false, &a, &d);
  if (s != FORGE_OK || a.tokens == 0) return s;
  return status(launch_qk_norm_rope(a, d.num_sms, static_cast<cudaStream_t>(stream)));
}

size_t forge_qk_norm_rope_backward_workspace_bytes(int64_t head_dim) {
  HostDevice d;
  if (head_dim <= 0 || head_dim > kMaxHeadDim || head_dim % 8 != 0) return 0;
  if (host_device(&d) != FORGE_OK) return 0;
  return static_cast<size_t>(qk_bwd_blocks(d.num_sms)) * static_cast<size_t>(head_dim) * 4;
}

forge_status forge_qk_norm_rope_backward(const forge_heads* sets, int n, forge_dtype gain_dtype,
                                         float eps, const forge_rotation* rot, int64_t tokens,
                                         int64_t head_dim, void* workspace, size_t workspace_bytes,
                                         forge_stream stream) {
  RopeArgs a;
  HostDevice d;
  const forge_status s =
      rope_args(sets, n, rot, tokens, head_dim, true, gain_dtype, eps, true, &a, &d);
  if (s != FORGE_OK) return s;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  bool gains = false;
  for (int i = 0; i < n; ++i) gains |= a.set[i].dgain != nullptr;
  if (gains) {
    if (!workspace) return FORGE_ERR_NULL;
    if (!aligned(workspace, 16)) return FORGE_ERR_ALIGN;
    if (workspace_bytes < forge_qk_norm_rope_backward_workspace_bytes(head_dim))
      return FORGE_ERR_SHAPE;
    const Span ws{workspace, workspace_bytes};
    for (int i = 0; i < n; ++i) {
      const forge_heads& h = sets[i];
      const bool any = tokens > 0 && h.heads > 0;
      auto span = [&](const void* p, int64_t token, int64_t head) {
        return any ? View{p, token, head, tokens, h.heads, head_dim}.span() : Span{nullptr, 0};
      };
      if (meets_any(ws, {span(h.x, h.x_token, h.x_head), span(h.dy, h.dy_token, h.dy_head),
                         span(h.y, h.y_token, h.y_head),
                         {h.gain, static_cast<uint64_t>(head_dim) * size_of(gain_dtype)},
                         {h.dgain, static_cast<uint64_t>(head_dim) * 4},
                         {rot->freqs, static_cast<uint64_t>(rot->dim) * 4},
                         {rot->positions, static_cast<uint64_t>(tokens) * 8}}))
        return FORGE_ERR_ALIAS;
    }
  }
  for (int i = 0; i < n; ++i)   // nothing to sum: the gain's gradient is zero
    if (a.set[i].dgain && a.set[i].heads == 0) {
      const cudaError_t e =
          cudaMemsetAsync(a.set[i].dgain, 0, static_cast<size_t>(head_dim) * 4, cs);
      if (e != cudaSuccess) return status(e);
    }
  if (a.tokens == 0) return FORGE_OK;
  a.part = static_cast<float*>(workspace);
  return status(launch_qk_norm_rope_bwd(a, d.num_sms, cs));
}

forge_status forge_rope_frequencies(int dim, double theta, const forge_rope_scaling* scaling,
                                    uint64_t* freqs, float* magnitude) {
  if (dim <= 0 || dim > kMaxHeadDim || dim % 8 != 0) return FORGE_ERR_SHAPE;
  if (!freqs || !magnitude) return FORGE_ERR_NULL;
  if (!(theta > 1.0) || !std::isfinite(theta)) return FORGE_ERR_HYPER;
  forge_rope_scaling s;
  std::memset(&s, 0, sizeof(s));
  if (scaling) s = *scaling;
  if (s.kind < FORGE_ROPE_SCALE_NONE || s.kind > FORGE_ROPE_SCALE_YARN) return FORGE_ERR_FORMAT;
  if (s.kind != FORGE_ROPE_SCALE_NONE && (!(s.factor >= 1.0) || !std::isfinite(s.factor)))
    return FORGE_ERR_HYPER;
  const bool by_turns = s.kind == FORGE_ROPE_SCALE_LLAMA3 || s.kind == FORGE_ROPE_SCALE_YARN;
  if (by_turns && !(s.context > 0.0 && std::isfinite(s.context) && s.low > 0.0 && s.high > s.low &&
                    std::isfinite(s.high)))
    return FORGE_ERR_HYPER;
  const double two_pi = 6.283185307179586476925286766559;
  double base = theta;
  if (s.kind == FORGE_ROPE_SCALE_NTK) base *= std::pow(s.factor, dim / (dim - 2.0));
  // YaRN: the pair that makes `turns` turns over the context, as a real number
  auto pair_of = [&](double turns) {
    return dim * std::log(s.context / (turns * two_pi)) / (2.0 * std::log(theta));
  };
  double low = 0.0, high = 0.0;
  if (s.kind == FORGE_ROPE_SCALE_YARN) {
    low = std::fmax(std::floor(pair_of(s.high)), 0.0);
    high = std::fmin(std::ceil(pair_of(s.low)), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (s.kind == FORGE_ROPE_SCALE_LINEAR) f /= s.factor;
    if (s.kind == FORGE_ROPE_SCALE_LLAMA3) {
      const double turns = s.context * f / two_pi;
      const double keep = std::fmin(std::fmax((turns - s.low) / (s.high - s.low), 0.0), 1.0);
      f = (1.0 - keep) * f / s.factor + keep * f;
    }
    if (s.kind == FORGE_ROPE_SCALE_YARN) {
      const double slow =
          std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = slow * f / s.factor + (1.0 - slow) * f;
    }
    freqs[i] = static_cast<uint64_t>(std::nearbyint(f / two_pi * 18446744073709551616.0));
  }
  *magnitude = s.kind == FORGE_ROPE_SCALE_YARN
                   ? static_cast<float>(0.1 * std::log(s.factor) + 1.0) : 1.0f;
  return FORGE_OK;
}

}  // extern "C"

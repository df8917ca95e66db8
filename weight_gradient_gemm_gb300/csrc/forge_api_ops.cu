// Host side of the operators around the weight gradient: the RMS norm and its
// backward pass, the 128-block quantiser, the 8-bit products and the global
// gradient norm.  Arguments are checked before anything is enqueued; every
// entry point answers with a status and no C++ exception leaves it.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "forge.h"
#include "forge_internal.h"

using namespace forge;

namespace {

struct Span {
  const void* p;
  uint64_t n;
};

bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

bool meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether an output overlaps an input or another output.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (meet(*o, *q)) return true;
  }
  return false;
}

bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}

uint64_t blocks128(int64_t n) { return static_cast<uint64_t>((n + 127) / 128); }

constexpr int64_t kMaxIndex = (1LL << 31) - 1;

// The status of a call's launches; a failed one leaves no error behind.
forge_status status(cudaError_t e) {
  if (e == cudaSuccess) return FORGE_OK;
  (void)cudaGetLastError();
  return FORGE_ERR_LAUNCH;
}

NormWait norm_wait(const HostDevice& d) {
  return NormWait{d.err, d.err_site, d.timeout_ns, host_drop_flag()};
}

forge_status check_rows(int64_t rows, int64_t cols, int64_t max_cols) {
  if (rows < 0 || rows > kMaxIndex || cols <= 0 || cols > max_cols || cols % 8 != 0)
    return FORGE_ERR_SHAPE;
  return FORGE_OK;
}

// The products' tile.
// Up to 128 tokens the outputs lie along M (forge_gemm_b128_few.cu) and the
// reduction is split over as many CTAs of a cluster as leave at most one CTA
// an SM, with two blocks each at least: one token, 4096 -> 4096 (32 tiles),
// takes 10.8 us unsplit, 8.8 on two CTAs, 6.7 on four and 13.5 on eight (two
// waves); 4096 -> 14336 (112 tiles) 13.0 unsplit, 18.1 on two and 25.4 on four.
// Beyond, 256 x 256 on CTA pairs or 128 x 128 on single CTAs, by the waves
// each takes and the measured cycles of a block (770 and 490): 512 tokens,
// 4096 -> 4096, take 17.8 us on pairs and 14.2 on single CTAs, 1024 tokens
// 19.2 and 23.2.  The tiles of the last waves stay whole: cut along the reduction
// and shared out evenly, with the parts joined through memory, 2000 tokens,
// 14336 -> 4096 (128 tiles on 76 pairs), took 98 us in place of 91, since pairs
// at different depths no longer read the operands together.
B128Config choose_b128(int64_t m, int64_t n, int64_t num_kb, const forge_tuning& tune,
                       int num_sms) {
  B128Config c{1, 128, 0, 1};
  if (m <= 128 && tune.cta_group == 0) {
    c.few = m <= 16 ? 16 : (m <= 32 ? 32 : (m <= 64 ? 64 : 128));
    const int64_t tiles = (n + 127) / 128;
    while (c.splits < 8 && tiles * c.splits * 2 <= num_sms && num_kb >= 4 * c.splits) c.splits *= 2;
    if (tune.splits)   // the cluster sizes there are: powers of two
      c.splits = tune.splits >= 8 ? 8 : (tune.splits >= 4 ? 4 : (tune.splits >= 2 ? 2 : 1));
    return c;
  }
  const int64_t pairs = num_sms / 2;
  const int64_t tiles1 = (m + 127) / 128 * ((n + 127) / 128);
  const int64_t tiles2 = (m + 255) / 256 * ((n + 255) / 256);
  const int64_t t1 = (tiles1 + num_sms - 1) / num_sms * 490;
  const int64_t t2 = (tiles2 + pairs - 1) / pairs * 770;
  if (tune.cta_group ? tune.cta_group == 2 : t2 < t1) c.cg = 2, c.bn = 256;
  return c;
}

// Y = A W^T (forward) or A W (input gradient), A's codes [m, k].
forge_status product_b128(const void* A, const float* sa, const void* W, const float* sw, void* out,
                          forge_dtype dtype, int64_t m, int64_t k, int64_t n, bool dgrad,
                          forge_stream stream) {
  if (m < 0 || m > kMaxIndex || k <= 0 || n <= 0 || k > kMaxIndex || n > kMaxIndex)
    return FORGE_ERR_SHAPE;
  if (k % 16 != 0 || n % 16 != 0) return FORGE_ERR_SHAPE;
  if (dtype != FORGE_DT_FP32 && dtype != FORGE_DT_BF16) return FORGE_ERR_FORMAT;
  if (m == 0) return FORGE_OK;
  if (!A || !sa || !W || !sw || !out) return FORGE_ERR_NULL;
  if (!all_aligned16({A, sa, W, sw, out})) return FORGE_ERR_ALIGN;
  const uint64_t um = m, uk = k, un = n, es = dtype == FORGE_DT_FP32 ? 4 : 2;
  if (clash({{out, um * un * es}}, {{A, um * uk},
                                    {sa, um * blocks128(k) * 4},
                                    {W, uk * un},
                                    {sw, blocks128(k) * blocks128(n) * 4}}))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  forge_tuning tune;
  forge_get_tuning(&tune);
  const B128Config cfg =
      choose_b128(m, n, static_cast<int64_t>(blocks128(k)), tune, d.num_sms);
  B128Args a;
  std::memset(&a, 0, sizeof(a));
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint32_t bnl = cfg.bn / cfg.cg;
  const bool maps =
      host_map(&a.a, A, u8, uk, um, uk, 128, cfg.few ? cfg.few : 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
      (dgrad ? host_map(&a.b, W, u8, un, uk, un, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B)
             : host_map(&a.b, W, u8, uk, un, uk, 128, bnl, CU_TENSOR_MAP_SWIZZLE_128B)) &&
      (cfg.few || host_map(&a.out, out,
               es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, un, um,
               un * es, static_cast<uint32_t>(128 / es), 32, CU_TENSOR_MAP_SWIZZLE_128B));
  if (!maps) return FORGE_ERR_LAUNCH;
  a.sa = sa;
  a.sw = sw;
  a.m = static_cast<int32_t>(m);
  a.n = static_cast<int32_t>(n);
  a.num_kb = static_cast<int32_t>(blocks128(k));
  a.sw_n = dgrad ? 1 : a.num_kb;                              // sw [d_out / 128][d_in / 128]
  a.sw_k = dgrad ? static_cast<int32_t>(blocks128(n)) : 1;
  const int64_t tm = 128 * cfg.cg, tiles_m = cfg.few ? 1 : (m + tm - 1) / tm;
  const int64_t tiles_n = (n + cfg.bn - 1) / cfg.bn;
  if (tiles_m * tiles_n > kMaxIndex / 2) return FORGE_ERR_SHAPE;
  a.tiles_m = static_cast<int32_t>(tiles_m);
  a.tiles_n = static_cast<int32_t>(tiles_n);
  a.num_tiles = static_cast<int32_t>(tiles_m * tiles_n);
  a.group_m = 8;
  a.out_fp32 = es == 4;
  a.out_ptr = out;
  a.splits = cfg.splits;
  a.err = d.err;
  a.err_site = d.err_site;
  a.timeout_ns = d.timeout_ns;
  a.drop_first_arrival = host_drop_flag();
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return status(cfg.few ? launch_gemm_b128_few(cfg.few, dgrad, a, d.num_sms, cs)
                        : launch_gemm_b128(cfg, dgrad, a, d.num_sms, cs));
}

}  // namespace

extern "C" {

forge_status forge_rmsnorm(const void* x, const void* residual, const void* gain,
                           forge_dtype gain_dtype, void* sum, void* y, void* codes, float* scales,
                           float* rstd, int64_t rows, int64_t cols, float eps,
                           forge_stream stream) {
  forge_status s = check_rows(rows, cols, kNormMaxCols);
  if (s != FORGE_OK) return s;
  if (gain_dtype != FORGE_DT_FP32 && gain_dtype != FORGE_DT_BF16) return FORGE_ERR_FORMAT;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return FORGE_ERR_HYPER;
  if (rows == 0) return FORGE_OK;
  if (!x || !gain || (!y && !codes) || (!codes != !scales)) return FORGE_ERR_NULL;
  if (!all_aligned16({x, residual, gain, sum, y, codes, scales, rstd})) return FORGE_ERR_ALIGN;
  const uint64_t n = static_cast<uint64_t>(rows) * cols;
  const Span in_x{x, 2 * n}, in_r{residual, 2 * n};
  const Span in_g{gain, static_cast<uint64_t>(cols) * (gain_dtype == FORGE_DT_FP32 ? 4 : 2)};
  const Span o_sum{sum, 2 * n}, o_y{y, 2 * n}, o_c{codes, n};
  const Span o_s{scales, static_cast<uint64_t>(rows) * blocks128(cols) * 4};
  const Span o_r{rstd, static_cast<uint64_t>(rows) * 4};
  if (clash({o_y, o_c, o_s, o_r}, {in_x, in_r, in_g, o_sum})) return FORGE_ERR_ALIAS;
  // the sum may replace x or the residual (each element is read before it is written)
  if (meet(o_sum, in_g) || (sum != x && meet(o_sum, in_x)) ||
      (sum != residual && meet(o_sum, in_r)))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.gain = gain;
  a.gain_bf16 = gain_dtype == FORGE_DT_BF16;
  a.sum = static_cast<uint16_t*>(sum);
  a.y = static_cast<uint16_t*>(y);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.eps = eps;
  a.wait = norm_wait(d);
  return status(launch_rmsnorm(a, d.num_sms, static_cast<cudaStream_t>(stream)));
}

size_t forge_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  HostDevice d;
  if (check_rows(rows, cols, kNormMaxCols) != FORGE_OK || host_device(&d) != FORGE_OK) return 0;
  const int blocks = rmsnorm_bwd_blocks(rows, static_cast<int>(cols), d.num_sms);
  return static_cast<size_t>(blocks) * static_cast<size_t>(cols) * 4;
}

forge_status forge_rmsnorm_backward(const void* dY, const void* h, const void* gain,
                                    forge_dtype gain_dtype, const float* rstd, const void* dsum,
                                    void* dX, float* dgain, int64_t rows, int64_t cols,
                                    void* workspace, size_t workspace_bytes, forge_stream stream) {
  forge_status s = check_rows(rows, cols, kNormMaxCols);
  if (s != FORGE_OK) return s;
  if (gain_dtype != FORGE_DT_FP32 && gain_dtype != FORGE_DT_BF16) return FORGE_ERR_FORMAT;
  if (!gain || (rows > 0 && (!dY || !h || !rstd || !dX))) return FORGE_ERR_NULL;
  if (!all_aligned16({dY, h, gain, rstd, dsum, dX, dgain, workspace})) return FORGE_ERR_ALIGN;
  const uint64_t n = static_cast<uint64_t>(rows) * cols;
  const Span in_dy{dY, 2 * n}, in_h{h, 2 * n}, in_ds{dsum, 2 * n};
  const Span in_g{gain, static_cast<uint64_t>(cols) * (gain_dtype == FORGE_DT_FP32 ? 4 : 2)};
  const Span in_r{rstd, static_cast<uint64_t>(rows) * 4};
  const Span o_dx{dX, 2 * n}, o_dg{dgain, static_cast<uint64_t>(cols) * 4};
  const Span ws{dgain ? workspace : nullptr, workspace_bytes};
  if (clash({o_dg, ws}, {in_dy, in_h, in_ds, in_g, in_r, o_dx})) return FORGE_ERR_ALIAS;
  // dX may replace dsum (each element is read before it is written)
  if (meet(o_dx, in_dy) || meet(o_dx, in_h) || meet(o_dx, in_g) || meet(o_dx, in_r) ||
      (dX != dsum && meet(o_dx, in_ds)))
    return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (rows == 0)   // no rows: the sum over them is zero
    return dgain ? status(cudaMemsetAsync(dgain, 0, static_cast<size_t>(cols) * 4, cs)) : FORGE_OK;
  if (dgain) {
    if (!workspace) return FORGE_ERR_NULL;
    if (workspace_bytes < forge_rmsnorm_backward_workspace_bytes(rows, cols))
      return FORGE_ERR_SHAPE;
  }
  NormBwdArgs a;
  a.dy = static_cast<const uint16_t*>(dY);
  a.h = static_cast<const uint16_t*>(h);
  a.gain = gain;
  a.gain_bf16 = gain_dtype == FORGE_DT_BF16;
  a.rstd = rstd;
  a.dsum = static_cast<const uint16_t*>(dsum);
  a.dx = static_cast<uint16_t*>(dX);
  a.dgain = dgain;
  a.part = static_cast<float*>(workspace);
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.wait = norm_wait(d);
  return status(launch_rmsnorm_bwd(a, d.num_sms, cs));
}

forge_status forge_quantize_b128(const void* x, void* codes, float* scales, int64_t rows,
                                 int64_t cols, int block_rows, forge_stream stream) {
  forge_status s = check_rows(rows, cols, kMaxIndex);
  if (s != FORGE_OK) return s;
  if (block_rows != 1 && block_rows != 128) return FORGE_ERR_FORMAT;
  if (rows == 0) return FORGE_OK;
  if (!x || !codes || !scales) return FORGE_ERR_NULL;
  if (!all_aligned16({x, codes, scales})) return FORGE_ERR_ALIGN;
  const uint64_t n = static_cast<uint64_t>(rows) * cols;
  const uint64_t nb =
      (block_rows == 1 ? static_cast<uint64_t>(rows) : blocks128(rows)) * blocks128(cols);
  if (block_rows == 128 && nb > static_cast<uint64_t>(kMaxIndex)) return FORGE_ERR_SHAPE;
  if (clash({{codes, n}, {scales, nb * 4}}, {{x, 2 * n}})) return FORGE_ERR_ALIAS;
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  return status(launch_quantize_b128(static_cast<const uint16_t*>(x), static_cast<uint8_t*>(codes),
                                     scales, rows, cols, block_rows, d.num_sms, norm_wait(d),
                                     static_cast<cudaStream_t>(stream)));
}

forge_status forge_linear_fp8(const void* X, const float* x_scales, const void* W,
                              const float* w_scales, void* Y, forge_dtype y_dtype, int64_t bt,
                              int64_t d_in, int64_t d_out, forge_stream stream) {
  return product_b128(X, x_scales, W, w_scales, Y, y_dtype, bt, d_in, d_out, false, stream);
}

forge_status forge_dgrad_fp8(const void* dY, const float* dy_scales, const void* W,
                             const float* w_scales, void* dX, forge_dtype dx_dtype, int64_t bt,
                             int64_t d_in, int64_t d_out, forge_stream stream) {
  return product_b128(dY, dy_scales, W, w_scales, dX, dx_dtype, bt, d_out, d_in, true, stream);
}

size_t forge_grad_norm_workspace_bytes(int n) {
  HostDevice d;
  if (n <= 0 || host_device(&d) != FORGE_OK) return 0;
  const size_t launches = (static_cast<size_t>(n) + kNormTensors - 1) / kNormTensors;
  return launches * static_cast<size_t>(grad_norm_blocks(kMaxIndex, d.num_sms)) * sizeof(double);
}

forge_status forge_grad_norm(const forge_grad* grads, int n, float max_norm, float* out,
                             void* workspace, size_t workspace_bytes, forge_stream stream) {
  if (n < 0) return FORGE_ERR_SHAPE;
  if (!out || (n > 0 && !grads)) return FORGE_ERR_NULL;
  if (!aligned(out, 4) || !aligned(workspace, 16)) return FORGE_ERR_ALIGN;
  if (!(max_norm > 0.0f)) return FORGE_ERR_HYPER;
  const Span o{out, 8}, ws{workspace, workspace_bytes};
  if (meet(o, ws)) return FORGE_ERR_ALIAS;
  int64_t launch_units = 0;   // of the launch that takes tensor i
  for (int i = 0; i < n; ++i) {
    const forge_grad& g = grads[i];
    if (i % kNormTensors == 0) launch_units = 0;
    if (g.dtype != FORGE_DT_FP32 && g.dtype != FORGE_DT_BF16) return FORGE_ERR_FORMAT;
    if (g.numel < 0 || g.numel > (1LL << 44)) return FORGE_ERR_SHAPE;
    launch_units += (g.numel + kNormUnit - 1) / kNormUnit;
    if (launch_units > kMaxIndex / 2) return FORGE_ERR_SHAPE;
    if (g.numel == 0) continue;
    if (!g.data) return FORGE_ERR_NULL;
    if (!aligned(g.data, 16)) return FORGE_ERR_ALIGN;
    const Span in{g.data, static_cast<uint64_t>(g.numel) * (g.dtype == FORGE_DT_FP32 ? 4 : 2)};
    if (meet(o, in) || meet(ws, in)) return FORGE_ERR_ALIAS;
  }
  HostDevice d;
  const int st = host_device(&d);
  if (st != FORGE_OK) return static_cast<forge_status>(st);
  if (n > 0) {
    if (!workspace) return FORGE_ERR_NULL;
    if (workspace_bytes < forge_grad_norm_workspace_bytes(n)) return FORGE_ERR_SHAPE;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int parts = 0;
  for (int first = 0; first < n; first += kNormTensors) {
    GradNormArgs a;
    std::memset(&a, 0, sizeof(a));
    int64_t units = 0;
    const int last = n - first < kNormTensors ? n : first + kNormTensors;
    for (int i = first; i < last; ++i) {
      const forge_grad& g = grads[i];
      if (g.numel == 0) continue;
      a.ptr[a.n] = g.data;
      a.numel[a.n] = g.numel;
      if (g.dtype == FORGE_DT_BF16) a.bf16[a.n >> 6] |= 1ull << (a.n & 63);
      a.unit0[a.n] = static_cast<int32_t>(units);
      units += (g.numel + kNormUnit - 1) / kNormUnit;
      a.unit0[++a.n] = static_cast<int32_t>(units);
    }
    if (units == 0) continue;
    const int blocks = grad_norm_blocks(units, d.num_sms);
    a.part = part + parts;
    parts += blocks;
    const cudaError_t e = launch_grad_norm(a, blocks, cs);
    if (e != cudaSuccess) return status(e);
  }
  return status(launch_grad_norm_final(part, parts, max_norm, out, cs));
}

}  // extern "C"

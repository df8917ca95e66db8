// The calls of forge.py's operators around the weight gradient, with their
// argument checks, as a CPython extension: through Python attributes and
// ctypes a call costs 5 to 8 us on the host, more than its kernel takes on few
// rows; here about 3 us, most of it the launch.
//
// Each function makes the checks of its Python counterpart.  Where one fails
// (or anything unusual is met: another device, a subclass without storage) it
// returns -1 and does nothing, and the Python function goes through its own
// checks, which say what is wrong.  Otherwise it returns the library's status.
// No C++ exception leaves a function.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <vector>

#include "forge.h"

namespace {

// The library's functions (it is loaded by forge.py, which hands over their
// addresses).
struct {
  decltype(&forge_rmsnorm) rmsnorm;
  decltype(&forge_rmsnorm_backward) rmsnorm_backward;
  decltype(&forge_quantize_b128) quantize;
  decltype(&forge_linear_fp8) linear;
  decltype(&forge_dgrad_fp8) dgrad;
  decltype(&forge_grad_norm) grad_norm;
  decltype(&forge_adamw_clip) adamw_clip;
  decltype(&forge_linear_bf16) linear_bf16;
  decltype(&forge_epilogue_backward) epilogue_backward;
  decltype(&forge_dropout) dropout;
  decltype(&forge_rope) rope;
  decltype(&forge_qk_norm_rope) qk_norm_rope;
  decltype(&forge_qk_norm_rope_backward) qk_norm_rope_backward;
} lib;

// One call's view of its arguments: `bad` once a check has failed.
struct Args {
  PyObject* const* a;
  Py_ssize_t n;
  bool bad = false;
  int dev = -1;

  const at::Tensor* tensor(int i) {
    const at::Tensor* t = strided(i);
    if (t && !t->is_contiguous()) bad = true;
    return bad ? nullptr : t;
  }
  // A tensor of any strides.
  const at::Tensor* strided(int i) {
    if (bad || !THPVariable_Check(a[i])) {
      bad = true;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.defined() || !t.is_cuda() || t.layout() != c10::kStrided) {
      bad = true;
      return nullptr;
    }
    if (dev < 0) {
      dev = t.get_device();
      if (dev != c10::cuda::current_device()) bad = true;
    } else if (t.get_device() != dev) {
      bad = true;
    }
    return bad ? nullptr : &t;
  }
  // The data of argument i after its checks: shape [d0] (d1 < 0) or [d0, d1].
  void* ptr(int i, int64_t d0, int64_t d1, c10::ScalarType s0, c10::ScalarType s1) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    const c10::ScalarType s = t->scalar_type();
    const bool shape = d1 < 0 ? t->dim() == 1 && t->size(0) == d0
                              : t->dim() == 2 && t->size(0) == d0 && t->size(1) == d1;
    if (!shape || (s != s0 && s != s1)) {
      bad = true;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* ptr(int i, int64_t d0, int64_t d1, c10::ScalarType s) { return ptr(i, d0, d1, s, s); }
  void* opt(int i, int64_t d0, int64_t d1, c10::ScalarType s) {
    return a[i] == Py_None ? nullptr : ptr(i, d0, d1, s);
  }
  // A workspace: its address and size (none: null and 0).
  void* bytes(int i, size_t* n_bytes) {
    *n_bytes = 0;
    if (a[i] == Py_None) return nullptr;
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    *n_bytes = t->nbytes();
    return t->data_ptr();
  }
  forge_dtype dtype(int i) {
    return !bad && THPVariable_Unpack(a[i]).scalar_type() == at::kFloat ? FORGE_DT_FP32
                                                                        : FORGE_DT_BF16;
  }
  double number(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      bad = true;
    }
    return v;
  }
  int64_t integer(int i) {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      bad = true;
    }
    return v;
  }
  // One of a few small numbers; -1 for anything far from them.
  int choice(int i) {
    const int64_t v = integer(i);
    return v >= 0 && v < 256 ? static_cast<int>(v) : -1;
  }
  // None: the device's current stream; else a stream's address.
  void* stream(int i) {
    if (bad) return nullptr;
    if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    const unsigned long long v = PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      bad = true;
    }
    return reinterpret_cast<void*>(static_cast<uintptr_t>(v));
  }
};

constexpr auto kBF = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kF8 = at::kFloat8_e4m3fn;
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Runs `f`, which returns a status or sets args.bad; -1 for bad arguments.
template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F f) {
  long st = -1;
  if (n == want) {
    try {
      Args args{a, n};
      const long got = f(args);
      if (!args.bad) st = got;
    } catch (...) {   // the Python path says what is wrong
      PyErr_Clear();
    }
  }
  return PyLong_FromLong(st);
}
// The interpreter is released while one of these lives, and taken again however
// its block is left.
class Released {
 public:
  Released() : state_(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state_); }
  Released(const Released&) = delete;

 private:
  PyThreadState* state_;
};
// The library call, with the interpreter released.
#define FORGE_CALL(expr)     \
  [&]() -> long {            \
    if (c.bad) return -1;    \
    const Released released; \
    return (expr);           \
  }()

// bind(addresses in the order of `lib`)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** fn[] = {reinterpret_cast<void**>(&lib.rmsnorm),
                 reinterpret_cast<void**>(&lib.rmsnorm_backward),
                 reinterpret_cast<void**>(&lib.quantize), reinterpret_cast<void**>(&lib.linear),
                 reinterpret_cast<void**>(&lib.dgrad), reinterpret_cast<void**>(&lib.grad_norm),
                 reinterpret_cast<void**>(&lib.adamw_clip),
                 reinterpret_cast<void**>(&lib.linear_bf16),
                 reinterpret_cast<void**>(&lib.epilogue_backward),
                 reinterpret_cast<void**>(&lib.dropout), reinterpret_cast<void**>(&lib.rope),
                 reinterpret_cast<void**>(&lib.qk_norm_rope),
                 reinterpret_cast<void**>(&lib.qk_norm_rope_backward)};
  constexpr int kFns = sizeof(fn) / sizeof(fn[0]);
  if (n != kFns) {
    PyErr_Format(PyExc_TypeError, "bind takes %d addresses", kFns);
    return nullptr;
  }
  for (int i = 0; i < kFns; ++i) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
    *fn[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(v));
  }
  Py_RETURN_NONE;
}

// x, gain, eps, residual, sum_out, y, codes, scales, rstd, stream
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 10, [](Args& c) -> long {
    const at::Tensor* x = c.tensor(0);
    if (!x || x->dim() != 2) return c.bad = true, -1;
    const int64_t rows = x->size(0), cols = x->size(1);
    void* xp = c.ptr(0, rows, cols, kBF);
    void* g = c.ptr(1, cols, -1, kF32, kBF);
    const forge_dtype gt = c.dtype(1);
    const float eps = static_cast<float>(c.number(2));
    void *r = c.opt(3, rows, cols, kBF), *s = c.opt(4, rows, cols, kBF);
    void *y = c.opt(5, rows, cols, kBF), *q = c.opt(6, rows, cols, kF8);
    float* sc = static_cast<float*>(c.opt(7, rows, blocks(cols), kF32));
    float* rs = static_cast<float*>(c.opt(8, rows, -1, kF32));
    void* st = c.stream(9);
    return FORGE_CALL(lib.rmsnorm(xp, r, g, gt, s, y, q, sc, rs, rows, cols, eps, st));
  });
}

// dY, h, gain, rstd, dX, dgain, dsum, workspace, stream
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 9, [](Args& c) -> long {
    const at::Tensor* h = c.tensor(1);
    if (!h || h->dim() != 2) return c.bad = true, -1;
    const int64_t rows = h->size(0), cols = h->size(1);
    void *dy = c.ptr(0, rows, cols, kBF), *hp = c.ptr(1, rows, cols, kBF);
    void* g = c.ptr(2, cols, -1, kF32, kBF);
    const forge_dtype gt = c.dtype(2);
    const float* rs = static_cast<float*>(c.ptr(3, rows, -1, kF32));
    void* dx = c.ptr(4, rows, cols, kBF);
    float* dg = static_cast<float*>(c.opt(5, cols, -1, kF32));
    void* ds = c.opt(6, rows, cols, kBF);
    size_t wb;
    void* ws = c.bytes(7, &wb);
    void* st = c.stream(8);
    return FORGE_CALL(
        lib.rmsnorm_backward(dy, hp, g, gt, rs, ds, dx, dg, rows, cols, ws, wb, st));
  });
}

// x, codes, scales, block_rows, stream
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 5, [](Args& c) -> long {
    const at::Tensor* x = c.tensor(0);
    if (!x || x->dim() != 2) return c.bad = true, -1;
    const int64_t rows = x->size(0), cols = x->size(1), br = c.integer(3);
    void *xp = c.ptr(0, rows, cols, kBF), *q = c.ptr(1, rows, cols, kF8);
    float* sc = static_cast<float*>(c.ptr(2, br == 1 ? rows : blocks(rows), blocks(cols), kF32));
    void* st = c.stream(4);
    if (br != 1 && br != 128) return c.bad = true, -1;
    return FORGE_CALL(lib.quantize(xp, q, sc, rows, cols, static_cast<int>(br), st));
  });
}

// tokens, their scales, W, w_scales, output, stream
template <bool DGRAD>
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 6, [](Args& c) -> long {
    const at::Tensor *x = c.tensor(0), *w = c.tensor(2);
    if (!x || !w || x->dim() != 2 || w->dim() != 2) return c.bad = true, -1;
    const int64_t bt = x->size(0), d_out = w->size(0), d_in = w->size(1);
    const int64_t k = DGRAD ? d_out : d_in, m = DGRAD ? d_in : d_out;
    void* xp = c.ptr(0, bt, k, kF8);
    const float* xs = static_cast<float*>(c.ptr(1, bt, blocks(k), kF32));
    void* wp = c.ptr(2, d_out, d_in, kF8);
    const float* ws = static_cast<float*>(c.ptr(3, blocks(d_out), blocks(d_in), kF32));
    void* o = c.ptr(4, bt, m, kF32, kBF);
    const forge_dtype ot = c.dtype(4);
    void* st = c.stream(5);
    return FORGE_CALL((DGRAD ? lib.dgrad : lib.linear)(xp, xs, wp, ws, o, ot, bt, d_in, d_out, st));
  });
}

// grads (a list or tuple), max_norm, out, workspace, stream
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 5, [](Args& c) -> long {
    if (!PyList_Check(c.a[0]) && !PyTuple_Check(c.a[0])) return c.bad = true, -1;
    float* out = static_cast<float*>(c.ptr(2, 2, -1, kF32));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(c.a[0]);
    PyObject** items = PySequence_Fast_ITEMS(c.a[0]);
    Args g{items, count};
    g.dev = c.dev;
    std::vector<forge_grad> grads(count);
    for (Py_ssize_t i = 0; i < count && !c.bad; ++i) {
      const at::Tensor* t = g.tensor(static_cast<int>(i));
      if (!t || (t->scalar_type() != kF32 && t->scalar_type() != kBF)) return c.bad = true, -1;
      grads[i] = {t->data_ptr(), t->numel(),
                  t->scalar_type() == kF32 ? FORGE_DT_FP32 : FORGE_DT_BF16};
    }
    const float max_norm = static_cast<float>(c.number(1));
    size_t wb;
    void* ws = c.bytes(3, &wb);
    void* st = c.stream(4);
    return FORGE_CALL(lib.grad_norm(count ? grads.data() : nullptr, static_cast<int>(count),
                                    max_norm, out, ws, wb, st));
  });
}

// dW, W, m, v, clip, lr, beta1, beta2, eps, weight_decay, step, stream
// (fp32 or bf16 moments; the formats with scales take the Python path)
PyObject* adamw_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 12, [](Args& c) -> long {
    const at::Tensor* w = c.tensor(1);
    if (!w || w->dim() != 2) return c.bad = true, -1;
    const int64_t d_out = w->size(0), d_in = w->size(1);
    void* g = c.ptr(0, d_out, d_in, kF32, kBF);
    const forge_dtype gt = c.dtype(0);
    void* wp = c.ptr(1, d_out, d_in, kBF);
    void* m = c.ptr(2, d_out, d_in, kF32, kBF);
    const forge_dtype mt = c.dtype(2);
    void* v = c.ptr(3, d_out, d_in, mt == FORGE_DT_FP32 ? kF32 : kBF);
    const float* coef = static_cast<float*>(c.ptr(4, 2, -1, kF32));
    float h[5];
    for (int i = 0; i < 5; ++i) h[i] = static_cast<float>(c.number(5 + i));
    const int64_t step = c.integer(10);
    void* st = c.stream(11);
    const forge_moment_fmt fmt = mt == FORGE_DT_FP32 ? FORGE_MOM_FP32 : FORGE_MOM_BF16;
    return FORGE_CALL(lib.adamw_clip(g, gt, coef + 1, wp, forge_moment{m, nullptr},
                                     forge_moment{v, nullptr}, d_in, d_out, h[0], h[1], h[2], h[3],
                                     h[4], step, fmt, st));
  });
}

// p, seed, offset, counter from argument i on (the words are taken modulo 2^64)
forge_drop drop_of(Args& c, int i) {
  forge_drop d{static_cast<float>(c.number(i)), 0, 0, nullptr};
  d.seed = PyLong_AsUnsignedLongLongMask(c.a[i + 1]);
  if (!PyErr_Occurred()) d.offset = PyLong_AsUnsignedLongLongMask(c.a[i + 2]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    c.bad = true;
  }
  d.counter = static_cast<const uint64_t*>(c.opt(i + 3, 1, -1, at::kLong));
  return d;
}

// X, W, Y, bias, act, mul, residual, Z, p, seed, offset, counter, stream
PyObject* linear_bf16(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 13, [](Args& c) -> long {
    const at::Tensor *x = c.tensor(0), *w = c.tensor(1);
    if (!x || !w || x->dim() != 2 || w->dim() != 2) return c.bad = true, -1;
    const int64_t bt = x->size(0), d_in = x->size(1), d_out = w->size(0);
    void *xp = c.ptr(0, bt, d_in, kBF), *wp = c.ptr(1, d_out, d_in, kBF);
    void* y = c.ptr(2, bt, d_out, kF32, kBF);
    const forge_dtype yt = c.dtype(2);
    forge_epilogue e{};
    if (c.a[3] != Py_None) {
      e.bias = c.ptr(3, d_out, -1, kF32, kBF);
      e.bias_dtype = c.dtype(3);
    }
    e.act = static_cast<forge_activation>(c.choice(4));
    e.mul = c.opt(5, bt, d_out, kBF);
    e.residual = c.opt(6, bt, d_out, kBF);
    e.z = c.opt(7, bt, d_out, kBF);
    e.drop = drop_of(c, 8);
    void* st = c.stream(12);
    return FORGE_CALL(lib.linear_bf16(xp, wp, y, yt, &e, bt, d_in, d_out, st));
  });
}

// dY, dZ, Z, act, mul, dmul, dbias, p, seed, offset, counter, workspace, stream
PyObject* epilogue_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 13, [](Args& c) -> long {
    const at::Tensor* t = c.tensor(0);
    if (!t || t->dim() != 2) return c.bad = true, -1;
    const int64_t rows = t->size(0), cols = t->size(1);
    void *dy = c.ptr(0, rows, cols, kBF), *dz = c.opt(1, rows, cols, kBF);
    void* z = c.opt(2, rows, cols, kBF);
    const auto act = static_cast<forge_activation>(c.choice(3));
    void *mul = c.opt(4, rows, cols, kBF), *dmul = c.opt(5, rows, cols, kBF);
    float* db = static_cast<float*>(c.opt(6, cols, -1, kF32));
    const forge_drop drop = drop_of(c, 7);
    size_t wb;
    void* ws = c.bytes(11, &wb);
    void* st = c.stream(12);
    return FORGE_CALL(
        lib.epilogue_backward(dy, z, mul, act, &drop, dz, dmul, db, rows, cols, ws, wb, st));
  });
}

// x, y, p, seed, offset, counter, residual, stream
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 8, [](Args& c) -> long {
    const at::Tensor* t = c.tensor(0);
    if (!t || t->dim() != 2) return c.bad = true, -1;
    const int64_t rows = t->size(0), cols = t->size(1);
    void *x = c.ptr(0, rows, cols, kBF), *y = c.ptr(1, rows, cols, kBF);
    const forge_drop drop = drop_of(c, 2);
    void* r = c.opt(6, rows, cols, kBF);
    void* st = c.stream(7);
    return FORGE_CALL(lib.dropout(x, r, y, &drop, rows, cols, st));
  });
}

// The queries (argument i) and keys (j) of a call, and where their parts are given.
struct Heads {
  forge_heads set[2] = {};
  int n = 1;
  int64_t tokens = 0, dim = 0;
};
// The pointer and strides of argument i, [tokens, heads, dim] with dense rows.
void view_of(Args& c, int i, const Heads& h, int64_t heads, void** p, int64_t* token,
             int64_t* head) {
  const at::Tensor* t = c.strided(i);
  if (!t) return;
  if (t->dim() != 3 || t->size(0) != h.tokens || t->size(1) != heads || t->size(2) != h.dim ||
      (h.dim > 1 && t->stride(2) != 1) || t->scalar_type() != kBF) {
    c.bad = true;
    return;
  }
  *p = t->data_ptr();
  *token = t->stride(0);
  *head = t->stride(1);
}
// x: the arguments of the inputs (queries, then keys), y: of the outputs.
Heads heads_of(Args& c, int x, int y) {
  Heads h;
  const at::Tensor* q = c.strided(x);
  if (!q || q->dim() != 3) {
    c.bad = true;
    return h;
  }
  h.tokens = q->size(0);
  h.dim = q->size(2);
  h.n = c.a[x + 1] == Py_None ? 1 : 2;
  for (int k = 0; k < h.n && !c.bad; ++k) {
    const at::Tensor* t = c.strided(x + k);
    if (!t || t->dim() != 3) {
      c.bad = true;
      return h;
    }
    forge_heads& s = h.set[k];
    s.heads = t->size(1);
    void* xp = nullptr;
    view_of(c, x + k, h, s.heads, &xp, &s.x_token, &s.x_head);
    view_of(c, y + k, h, s.heads, &s.y, &s.y_token, &s.y_head);
    s.x = xp;
  }
  return h;
}
// The gains, from argument i on, of one type.
forge_dtype gains_of(Args& c, int i, Heads& h) {
  h.set[0].gain = c.ptr(i, h.dim, -1, kF32, kBF);
  const forge_dtype t = c.dtype(i);
  const auto s = t == FORGE_DT_FP32 ? kF32 : kBF;
  if (h.n > 1) h.set[1].gain = c.ptr(i + 1, h.dim, -1, s);
  return t;
}
// freqs, positions, magnitude and layout at the arguments given.
forge_rotation rotation_of(Args& c, int freqs, int positions, const Heads& h) {
  forge_rotation r{};
  const at::Tensor* f = c.tensor(freqs);
  if (!f || f->dim() != 1 || f->size(0) > 1 << 20) {
    c.bad = true;
    return r;
  }
  r.dim = static_cast<int32_t>(2 * f->size(0));
  r.freqs = static_cast<const uint64_t*>(c.ptr(freqs, f->size(0), -1, at::kLong));
  r.positions = static_cast<const int64_t*>(c.opt(positions, h.tokens, -1, at::kLong));
  r.magnitude = static_cast<float>(c.number(positions + 1));
  r.layout = static_cast<forge_rope_layout>(c.choice(positions + 2));
  return r;
}

// q, k, freqs, q_out, k_out, positions, magnitude, layout, inverse, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 10, [](Args& c) -> long {
    const Heads h = heads_of(c, 0, 3);
    const forge_rotation r = rotation_of(c, 2, 5, h);
    const int inverse = PyObject_IsTrue(c.a[8]);
    void* st = c.stream(9);
    if (inverse < 0) return PyErr_Clear(), c.bad = true, -1;
    return FORGE_CALL(lib.rope(h.set, h.n, &r, inverse, h.tokens, h.dim, st));
  });
}

// q, k, q_gain, k_gain, freqs, eps, q_out, k_out, positions, magnitude, layout, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 12, [](Args& c) -> long {
    Heads h = heads_of(c, 0, 6);
    const forge_dtype gt = gains_of(c, 2, h);
    const float eps = static_cast<float>(c.number(5));
    const forge_rotation r = rotation_of(c, 4, 8, h);
    void* st = c.stream(11);
    return FORGE_CALL(lib.qk_norm_rope(h.set, h.n, gt, eps, &r, h.tokens, h.dim, st));
  });
}

// dq, dk, q, k, q_gain, k_gain, freqs, eps, dq_out, dk_out, dq_gain, dk_gain, positions,
// magnitude, layout, workspace, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 17, [](Args& c) -> long {
    Heads h = heads_of(c, 2, 8);
    const forge_dtype gt = gains_of(c, 4, h);
    for (int k = 0; k < h.n && !c.bad; ++k) {
      forge_heads& s = h.set[k];
      void* dy = nullptr;
      view_of(c, k, h, s.heads, &dy, &s.dy_token, &s.dy_head);
      s.dy = dy;
      s.dgain = static_cast<float*>(c.opt(10 + k, h.dim, -1, kF32));
    }
    const float eps = static_cast<float>(c.number(7));
    const forge_rotation r = rotation_of(c, 6, 12, h);
    size_t wb;
    void* ws = c.bytes(15, &wb);
    void* st = c.stream(16);
    return FORGE_CALL(
        lib.qk_norm_rope_backward(h.set, h.n, gt, eps, &r, h.tokens, h.dim, ws, wb, st));
  });
}

using FastFn = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(FastFn f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"rmsnorm", fast(rmsnorm), METH_FASTCALL, nullptr},
                         {"rmsnorm_backward", fast(rmsnorm_backward), METH_FASTCALL, nullptr},
                         {"quantize", fast(quantize), METH_FASTCALL, nullptr},
                         {"linear", fast(product<false>), METH_FASTCALL, nullptr},
                         {"dgrad", fast(product<true>), METH_FASTCALL, nullptr},
                         {"grad_norm", fast(grad_norm), METH_FASTCALL, nullptr},
                         {"adamw_clip", fast(adamw_clip), METH_FASTCALL, nullptr},
                         {"linear_bf16", fast(linear_bf16), METH_FASTCALL, nullptr},
                         {"epilogue_backward", fast(epilogue_backward), METH_FASTCALL, nullptr},
                         {"dropout", fast(dropout), METH_FASTCALL, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"qk_norm_rope_backward", fast(qk_norm_rope_backward), METH_FASTCALL,
                          nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_forge_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module says which torch it was compiled against; another one's tensors may
// be laid out differently, so forge.py leaves it alone then.
PyMODINIT_FUNC PyInit__forge_call() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}

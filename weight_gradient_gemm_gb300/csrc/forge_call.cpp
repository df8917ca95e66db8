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
} lib;

// One call's view of its arguments: `bad` once a check has failed.
struct Args {
  PyObject* const* a;
  Py_ssize_t n;
  bool bad = false;
  int dev = -1;

  const at::Tensor* tensor(int i) {
    if (bad || !THPVariable_Check(a[i])) {
      bad = true;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.defined() || !t.is_cuda() || t.layout() != c10::kStrided || !t.is_contiguous()) {
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
                 reinterpret_cast<void**>(&lib.adamw_clip)};
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
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

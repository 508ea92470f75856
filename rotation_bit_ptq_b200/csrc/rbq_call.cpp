// _rbq_call: the ordinary calls of the block-scaled FP8 layer, made natively.
//
// A call on a few tokens is bound by the host: qlinear_fp8 took 9.4 us through
// ctypes, of which 3 were its launch, and takes 3.6 here.  Each function here makes
// the checks of its namesake in _fp8.py on the tensors themselves, allocates the
// results and calls the C ABI on the current stream.  What is not an ordinary
// call -- plain contiguous CUDA tensors of the right types and shapes on the
// current device, results to be allocated -- returns None, as does a call that
// fails, and the binding then makes it in Python, where the errors are worded.
// No error is decided here and no exception leaves a function.
//
// The interpreter lock is released while results are allocated and kernels
// launched, as ctypes and torch's own operators do: a launch waits when the
// stream's queue is full, and an allocation may.  What is used meanwhile are
// tensors of the call's own, not the arguments' objects.
//
// The entry points of librbq.so are handed over by bind(), so that the two
// libraries do not depend on one another.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "rbq.h"

namespace {

decltype(&quantize_fp8) p_quantize = nullptr;
decltype(&quantize_weights_fp8) p_weights = nullptr;
decltype(&qlinear_fp8) p_linear = nullptr;
decltype(&qlinear_fp8_wgrad) p_wgrad = nullptr;
decltype(&gelu_backward_fp8) p_gelu = nullptr;

constexpr int64_t kBlock = 128, kMost = INT32_MAX;
int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Without the interpreter lock, to the end of the scope.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// A matrix as every function wants it, owned; undefined for anything else.
at::Tensor matrix(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return {};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.dim() != 2 || !t.is_contiguous()) return {};
  return t.size(0) <= kMost && t.size(1) <= kMost ? t : at::Tensor();
}
bool width(int64_t n, int64_t step = 16) { return n > 0 && n % step == 0; }

// Codes [n, d] and their scales, one for `rows` rows of 128 values.
struct Codes {
  at::Tensor codes, scale;
  int64_t n = 0, d = 0;
  bool read(PyObject* c, PyObject* s, int64_t rows) {
    codes = matrix(c);
    scale = matrix(s);
    if (!codes.defined() || !scale.defined() || codes.scalar_type() != at::kFloat8_e4m3fn ||
        scale.scalar_type() != at::kFloat8_e8m0fnu || codes.get_device() != scale.get_device())
      return false;
    n = codes.size(0);
    d = codes.size(1);
    return width(d) && scale.size(0) == (rows == 1 ? n : blocks(n)) && scale.size(1) == blocks(d);
  }
};

template <typename T = uint8_t>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
int dtype_code(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? RBQ_BF16 : t.scalar_type() == at::kFloat ? RBQ_F32 : -1;
}
// The caching allocator's tensor itself: through the dispatcher a result costs
// 0.4 us more.
at::Tensor make(int64_t n, int64_t d, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda({n, d}, type, like.device(), std::nullopt);
}
at::Tensor make_codes(int64_t n, int64_t d, const at::Tensor& like) { return make(n, d, at::kFloat8_e4m3fn, like); }
at::Tensor make_scale(int64_t n, int64_t d, const at::Tensor& like) { return make(n, d, at::kFloat8_e8m0fnu, like); }
// The current stream of the tensor's device if that device is current.
bool stream_of(const at::Tensor& t, void** stream) {
  if (c10::cuda::current_device() != t.get_device()) return false;
  *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.get_device())).stream();
  return true;
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// `body` returns the result or nullptr: not an ordinary call.
template <typename F>
PyObject* attempt(F body) {
  PyObject* r = nullptr;
  try {
    r = body();
  } catch (...) {
    r = nullptr;
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// quantize_fp8(X, act, checkpoint)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    if (n != 3 || !p_quantize) return nullptr;
    const at::Tensor x = matrix(a[0]);
    const long act = PyLong_AsLong(a[1]);
    const bool ck = a[2] == Py_True;
    if (!x.defined() || dtype_code(x) < 0 || !width(x.size(1)) || (ck && act == RBQ_ACT_NONE)) return nullptr;
    void* st;
    if (!stream_of(x, &st)) return nullptr;
    const int64_t T = x.size(0), d = x.size(1);
    at::Tensor codes, scale, xc, xs;
    int rc;
    {
      Unlocked unlocked;
      codes = make_codes(T, d, x);
      scale = make_scale(T, blocks(d), x);
      if (ck) {
        xc = make_codes(T, d, x);
        xs = make_scale(T, blocks(d), x);
      }
      rc = p_quantize(x.data_ptr(), dtype_code(x), static_cast<int>(T), static_cast<int>(d), static_cast<int>(act),
                      ptr(codes), ptr(scale), ck ? ptr(xc) : nullptr, ck ? ptr(xs) : nullptr, st);
    }
    if (rc != RBQ_OK) return nullptr;
    return ck ? tuple({codes, scale, xc, xs}) : tuple({codes, scale});
  });
}

// quantize_weights_fp8(W, transposed)
PyObject* weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    if (n != 2 || !p_weights) return nullptr;
    const at::Tensor w = matrix(a[0]);
    const bool tr = a[1] == Py_True;
    if (!w.defined() || dtype_code(w) < 0 || !width(w.size(1)) || (tr && !width(w.size(0)))) return nullptr;
    void* st;
    if (!stream_of(w, &st)) return nullptr;
    const int64_t N = w.size(0), K = w.size(1);
    at::Tensor codes, scale, ct, sct;
    int rc;
    {
      Unlocked unlocked;
      codes = make_codes(N, K, w);
      scale = make_scale(blocks(N), blocks(K), w);
      if (tr) {
        ct = make_codes(K, N, w);
        sct = make_scale(blocks(K), blocks(N), w);
      }
      rc = p_weights(w.data_ptr(), dtype_code(w), static_cast<int>(N), static_cast<int>(K), ptr(codes), ptr(scale),
                     tr ? ptr(ct) : nullptr, tr ? ptr(sct) : nullptr, st);
    }
    if (rc != RBQ_OK) return nullptr;
    return tr ? tuple({codes, scale, ct, sct}) : tuple({codes, scale});
  });
}

// qlinear_fp8(a_codes, a_scale, w_codes, w_scale)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    Codes x, w;
    if (n != 4 || !p_linear || !x.read(a[0], a[1], 1) || !w.read(a[2], a[3], kBlock) || x.d != w.d ||
        x.codes.get_device() != w.codes.get_device())
      return nullptr;
    void* st;
    if (!stream_of(x.codes, &st)) return nullptr;
    at::Tensor y;
    int rc;
    {
      Unlocked unlocked;
      y = make(x.n, w.n, at::kBFloat16, x.codes);
      rc = p_linear(ptr(x.codes), ptr(x.scale), ptr(w.codes), ptr(w.scale), static_cast<int>(x.n),
                    static_cast<int>(w.n), static_cast<int>(x.d), ptr<uint16_t>(y), st);
    }
    return rc == RBQ_OK ? THPVariable_Wrap(y) : nullptr;
  });
}

// qlinear_fp8_wgrad(dY, a_codes, a_scale, fp32)
PyObject* wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    if (n != 4 || !p_wgrad) return nullptr;
    const at::Tensor dy = matrix(a[0]);
    Codes x;
    if (!dy.defined() || dy.scalar_type() != at::kBFloat16 || !x.read(a[1], a[2], 1) || dy.size(0) != x.n ||
        !width(dy.size(1), 8) || dy.get_device() != x.codes.get_device())
      return nullptr;
    void* st;
    if (!stream_of(dy, &st)) return nullptr;
    const bool f32 = a[3] == Py_True;
    at::Tensor dw;
    int rc;
    {
      Unlocked unlocked;
      dw = make(dy.size(1), x.d, f32 ? at::kFloat : at::kBFloat16, dy);
      rc = p_wgrad(ptr<uint16_t>(dy), ptr(x.codes), ptr(x.scale), static_cast<int>(x.n),
                   static_cast<int>(dy.size(1)), static_cast<int>(x.d), dw.data_ptr(), f32 ? RBQ_F32 : RBQ_BF16, st);
    }
    return rc == RBQ_OK ? THPVariable_Wrap(dw) : nullptr;
  });
}

// gelu_backward_fp8(dH, x_codes, x_scale, quantize)
PyObject* gelu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    if (n != 4 || !p_gelu) return nullptr;
    const at::Tensor dh = matrix(a[0]);
    Codes x;
    if (!dh.defined() || dh.scalar_type() != at::kBFloat16 || !x.read(a[1], a[2], 1) || dh.size(0) != x.n ||
        dh.size(1) != x.d || dh.get_device() != x.codes.get_device())
      return nullptr;
    void* st;
    if (!stream_of(dh, &st)) return nullptr;
    const bool quant = a[3] == Py_True;
    at::Tensor dx, codes, scale;
    int rc;
    {
      Unlocked unlocked;
      dx = make(x.n, x.d, at::kBFloat16, dh);
      if (quant) {
        codes = make_codes(x.n, x.d, dh);
        scale = make_scale(x.n, blocks(x.d), dh);
      }
      rc = p_gelu(ptr<uint16_t>(dh), ptr(x.codes), ptr(x.scale), static_cast<int>(x.n), static_cast<int>(x.d),
                  ptr<uint16_t>(dx), quant ? ptr(codes) : nullptr, quant ? ptr(scale) : nullptr, st);
    }
    if (rc != RBQ_OK) return nullptr;
    return quant ? tuple({dx, codes, scale}) : THPVariable_Wrap(dx);
  });
}

// bind(quantize_fp8, quantize_weights_fp8, qlinear_fp8, qlinear_fp8_wgrad, gelu_backward_fp8): addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[0]);
  p_weights = reinterpret_cast<decltype(p_weights)>(p[1]);
  p_linear = reinterpret_cast<decltype(p_linear)>(p[2]);
  p_wgrad = reinterpret_cast<decltype(p_wgrad)>(p[3]);
  p_gelu = reinterpret_cast<decltype(p_gelu)>(p[4]);
  Py_RETURN_NONE;
}

#define RBQ_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RBQ_METHOD("bind", bind),
                         RBQ_METHOD("quantize_fp8", quantize),
                         RBQ_METHOD("quantize_weights_fp8", weights),
                         RBQ_METHOD("qlinear_fp8", linear),
                         RBQ_METHOD("qlinear_fp8_wgrad", wgrad),
                         RBQ_METHOD("gelu_backward_fp8", gelu_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rbq_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for`: the torch and the Python whose headers this was compiled against;
// the binding calls nothing here under any other.
PyMODINIT_FUNC PyInit__rbq_call() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", RBQ_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

// binding.cpp -- the allocating Python entry points of the layer operators: they
// check the tensors, allocate the results on the current stream of the tensors'
// device and call the library. A decoded token's norm takes 2 us on the GPU; the
// same steps in Python, with ctypes, took 21 us of host time, here 8.
//
// Nothing is computed here. The library's functions are handed over by address
// (bind), so this module links against torch only.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <stdexcept>
#include <string>
#include <type_traits>
#include <vector>

#include "../../../include/fp8bw_layer.h"

namespace {

using NsJob = fp8bw_ns_job;

constexpr int kFunctions = 10;
constexpr Py_ssize_t kNsJobs = FP8BW_NS_MAX_JOBS;

struct Library {               // the types are the header's
  decltype(&fp8bw_rmsnorm_quantize) rmsnorm[2];          // by pow2
  decltype(&fp8bw_rmsnorm_backward_workspace) rmsnorm_bwd_ws;
  decltype(&fp8bw_rmsnorm_backward) rmsnorm_bwd;
  decltype(&fp8bw_swiglu_quantize) swiglu[2];
  decltype(&fp8bw_swiglu_backward_quantize) swiglu_bwd[2];
  decltype(&fp8bw_newton_schulz_workspace) ns_ws;
  decltype(&fp8bw_newton_schulz) ns;
} lib;
static_assert(std::is_same<decltype(&fp8bw_rmsnorm_quantize),
                           decltype(&fp8bw_rmsnorm_quantize_pow2)>::value &&
              std::is_same<decltype(&fp8bw_swiglu_quantize),
                           decltype(&fp8bw_swiglu_quantize_pow2)>::value &&
              std::is_same<decltype(&fp8bw_swiglu_backward_quantize),
                           decltype(&fp8bw_swiglu_backward_quantize_pow2)>::value,
              "the two scale rules' functions are called through one type");

// What the module was compiled against, for the build to find in the file.
__attribute__((used)) const char kBuiltFor[] = "fp8bw binding for torch " FP8BW_TORCH_VERSION;

// A refused argument (ValueError in Python).
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// Python's error indicator is set.
struct PythonError {};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

// Data of a contiguous input of that type and shape on `dev`.
void* input(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* name,
            const at::Device& dev) {
  if (t.scalar_type() != type || t.sizes() != shape)
    throw Refused(std::string(name) + ": expected " + at::toString(type) + " " +
                  shape_text(shape) + ", got " + at::toString(t.scalar_type()) + " " +
                  shape_text(t.sizes()));
  if (t.device() != dev)
    throw Refused("expected tensors on one CUDA device, got " + dev.str() + " and " +
                  t.device().str());
  if (!t.is_contiguous()) throw Refused("expected a contiguous tensor");
  return t.data_ptr();
}

const uint16_t* bf16_input(const at::Tensor& t, at::IntArrayRef shape, const char* name,
                           const at::Device& dev) {
  return static_cast<const uint16_t*>(input(t, at::kBFloat16, shape, name, dev));
}

// rows, cols of a 2-D bf16 tensor.
at::IntArrayRef matrix(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2)
    throw Refused(std::string(name) + ": expected a 2-D BFloat16 tensor, got " +
                  at::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  return t.sizes();
}

void need_cuda(const at::Device& dev) {
  if (!dev.is_cuda()) throw Refused("expected a CUDA tensor");
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pad16(int64_t rows) { return cdiv(rows, 16) * 16; }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }
uint16_t* hptr(const at::Tensor& t) { return static_cast<uint16_t*>(ptr(t)); }   // bf16
uint8_t* bptr(const at::Tensor& t) { return static_cast<uint8_t*>(ptr(t)); }

void* stream_of(const at::Device& dev) {
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

struct Codes {
  at::Tensor q, s, q_t, s_t;
  Codes(int64_t rows, int64_t cols, const at::Device& dev, bool colwise) {
    const int64_t rp = pad16(rows);
    q = empty({rp, cols}, at::kByte, dev);
    s = empty({cdiv(cols, 128), rp}, at::kFloat, dev);
    if (colwise) {
      q_t = empty({cols, rp}, at::kByte, dev);
      s_t = empty({cdiv(rp, 128), cols}, at::kFloat, dev);
    }
  }
};

// (status, tensors...): Python turns a status other than 0 into the library's
// error. An undefined tensor becomes None.
PyObject* result(int status, std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()) + 1);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor& t : ts) {
    PyObject* o;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// The norm's inputs: x (or h), gamma, residual (or dres) or None.
struct NormInputs {
  at::Device dev;
  int64_t rows, cols;
  int gamma_f32;
  const uint16_t *x, *residual = nullptr;
  const void* gamma;
  NormInputs(PyObject* ox, PyObject* og, PyObject* orr, const char* nx, const char* nr)
      : dev(at::kCPU) {
    const at::Tensor& tx = tensor(ox, nx);
    const at::Tensor& tg = tensor(og, "gamma");
    const at::IntArrayRef shape = matrix(tx, nx);
    dev = tx.device();
    rows = shape[0];
    cols = shape[1];
    const at::ScalarType gt = tg.scalar_type();
    if ((gt != at::kBFloat16 && gt != at::kFloat) || tg.dim() != 1 || tg.size(0) != cols)
      throw Refused("gamma: expected bf16 or fp32 (" + std::to_string(cols) + ",), got " +
                    at::toString(gt) + " " + shape_text(tg.sizes()));
    gamma_f32 = gt == at::kFloat;
    x = bf16_input(tx, shape, nx, dev);
    gamma = input(tg, gt, tg.sizes(), "gamma", dev);
    if (orr != Py_None) residual = bf16_input(tensor(orr, nr), shape, nr, dev);
  }
};

template <typename Fn>
PyObject* guarded(Fn&& fn) {
  try {
    return fn();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch == nullptr ? nullptr : PyObject_GetAttrString(torch, "OutOfMemoryError");
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

bool truth(PyObject* o) {
  const int t = o == Py_True ? 1 : o == Py_False ? 0 : PyObject_IsTrue(o);
  if (t < 0) throw PythonError();
  return t != 0;
}

// (x, gamma, residual, eps, rowwise, colwise, pow2) -> q, s, q_t, s_t, h, rstd, y
// with codes if rowwise, else the bf16 y.
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 7)) return nullptr;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const NormInputs in(a[0], a[1], a[2], "x", "residual");
    need_cuda(in.dev);
    const c10::cuda::CUDAGuard guard(in.dev);
    at::Tensor h = in.residual == nullptr ? tensor(a[0], "x")
                                          : empty({in.rows, in.cols}, at::kBFloat16, in.dev);
    at::Tensor rstd = empty({in.rows}, at::kFloat, in.dev), y;
    uint16_t* ph = in.residual == nullptr ? nullptr : hptr(h);
    if (!truth(a[4])) {
      y = empty({in.rows, in.cols}, at::kBFloat16, in.dev);
      const int st = lib.rmsnorm[0](in.x, in.residual, in.gamma, in.gamma_f32, in.rows, in.cols,
                                    static_cast<float>(eps), ph, fptr(rstd), hptr(y), nullptr,
                                    nullptr, nullptr, nullptr, stream_of(in.dev));
      return result(st, {y, h, rstd});
    }
    const Codes c(in.rows, in.cols, in.dev, truth(a[5]));
    const int st = lib.rmsnorm[truth(a[6])](
        in.x, in.residual, in.gamma, in.gamma_f32, in.rows, in.cols, static_cast<float>(eps), ph,
        fptr(rstd), nullptr, bptr(c.q), fptr(c.s), bptr(c.q_t), fptr(c.s_t), stream_of(in.dev));
    return result(st, {c.q, c.s, c.q_t, c.s_t, h, rstd});
  });
}

// (dy, h, rstd, gamma, dres) -> dh, dgamma
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const NormInputs in(a[1], a[3], a[4], "h", "dres");
    const int64_t shape[2] = {in.rows, in.cols};
    const uint16_t* dy = bf16_input(tensor(a[0], "dy"), shape, "dy", in.dev);
    const void* rstd = input(tensor(a[2], "rstd"), at::kFloat, {in.rows}, "rstd", in.dev);
    need_cuda(in.dev);
    const int64_t size = lib.rmsnorm_bwd_ws(in.rows, in.cols);
    if (size < 0) return result(static_cast<int>(size), {});
    const c10::cuda::CUDAGuard guard(in.dev);
    const at::Tensor dh = empty(shape, at::kBFloat16, in.dev);
    const at::Tensor dgamma = empty({in.cols}, at::kFloat, in.dev);
    const at::Tensor ws = empty({size}, at::kByte, in.dev);
    const int st = lib.rmsnorm_bwd(dy, in.x, static_cast<const float*>(rstd), in.gamma,
                                   in.gamma_f32, in.residual, in.rows, in.cols, hptr(dh),
                                   fptr(dgamma), ptr(ws), size, stream_of(in.dev));
    return result(st, {dh, dgamma});
  });
}

int64_t half_of(const at::IntArrayRef& shape) {
  if (shape[1] % 2 != 0)
    throw Refused("gu: expected an even number of columns, got " + std::to_string(shape[1]));
  return shape[1] / 2;
}

// (gu, colwise, pow2) -> q, s, q_t, s_t
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& gu = tensor(a[0], "gu");
    const at::IntArrayRef shape = matrix(gu, "gu");
    const int64_t f = half_of(shape);
    const at::Device dev = gu.device();
    const uint16_t* p = bf16_input(gu, shape, "gu", dev);
    need_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    const Codes c(shape[0], f, dev, truth(a[1]));
    const int st = lib.swiglu[truth(a[2])](p, shape[0], f, bptr(c.q), fptr(c.s), bptr(c.q_t),
                                           fptr(c.s_t), stream_of(dev));
    return result(st, {c.q, c.s, c.q_t, c.s_t});
  });
}

// (da, gu, pow2) -> q, s, q_t, s_t
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& gu = tensor(a[1], "gu");
    const at::IntArrayRef shape = matrix(gu, "gu");
    const int64_t f = half_of(shape);
    const at::Device dev = gu.device();
    const uint16_t* pg = bf16_input(gu, shape, "gu", dev);
    const uint16_t* pd = bf16_input(tensor(a[0], "da"), {shape[0], f}, "da", dev);
    need_cuda(dev);
    const c10::cuda::CUDAGuard guard(dev);
    const Codes c(shape[0], 2 * f, dev, true);
    const int st = lib.swiglu_bwd[truth(a[2])](pd, pg, shape[0], f, bptr(c.q), fptr(c.s),
                                               bptr(c.q_t), fptr(c.s_t), stream_of(dev));
    return result(st, {c.q, c.s, c.q_t, c.s_t});
  });
}

// (list of matrices, steps, a, b, c, eps) -> one bf16 result per matrix; up to
// kNsJobs per call of the library, with one workspace for all of them.
PyObject* newton_schulz(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 6)) return nullptr;
  if (!PyList_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "expected a list of tensors");
    return nullptr;
  }
  long steps = PyLong_AsLong(a[1]);
  if (steps > INT_MAX) steps = INT_MAX;       // refused by the library
  if (steps < 0) steps = 0;
  double c[4];
  for (int i = 0; i < 4; ++i) c[i] = PyFloat_AsDouble(a[2 + i]);
  if (PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    std::vector<NsJob> jobs(static_cast<size_t>(count));
    std::vector<at::Tensor> outs(static_cast<size_t>(count));
    if (count == 0) return result(0, {});
    const at::Tensor& first = tensor(PyList_GET_ITEM(a[0], 0), "gs[0]");
    const at::ScalarType type = first.scalar_type();
    const at::Device dev = first.device();
    if (type != at::kBFloat16 && type != at::kFloat)
      throw Refused(std::string("gs: expected bf16 or fp32 tensors, got ") + at::toString(type));
    for (Py_ssize_t i = 0; i < count; ++i) {
      const std::string name = "gs[" + std::to_string(i) + "]";
      const at::Tensor& g = tensor(PyList_GET_ITEM(a[0], i), name.c_str());
      if (g.scalar_type() != type || g.dim() != 2)
        throw Refused(name + ": expected a 2-D " + at::toString(type) + " tensor, got " +
                      at::toString(g.scalar_type()) + " " + shape_text(g.sizes()));
      jobs[i] = NsJob{input(g, type, g.sizes(), name.c_str(), dev), g.size(0), g.size(1), nullptr};
    }
    need_cuda(dev);
    int64_t size = 0;
    for (Py_ssize_t i = 0; i < count; i += kNsJobs) {
      const int64_t need = lib.ns_ws(&jobs[i], static_cast<int>(std::min(kNsJobs, count - i)));
      if (need < 0) return result(static_cast<int>(need), {});
      size = std::max(size, need);
    }
    const c10::cuda::CUDAGuard guard(dev);
    for (Py_ssize_t i = 0; i < count; ++i) {
      outs[i] = empty({jobs[i].n, jobs[i].k}, at::kBFloat16, dev);
      jobs[i].out = hptr(outs[i]);
    }
    const at::Tensor ws = empty({size}, at::kByte, dev);
    int st = 0;
    for (Py_ssize_t i = 0; i < count && st == 0; i += kNsJobs)
      st = lib.ns(&jobs[i], static_cast<int>(std::min(kNsJobs, count - i)), type == at::kFloat,
                  static_cast<int>(steps), static_cast<float>(c[0]), static_cast<float>(c[1]),
                  static_cast<float>(c[2]), static_cast<float>(c[3]), ptr(ws), size,
                  stream_of(dev));
    PyObject* r = PyTuple_New(count + 1);
    if (r == nullptr) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    for (Py_ssize_t i = 0; i < count; ++i) PyTuple_SET_ITEM(r, i + 1, THPVariable_Wrap(outs[i]));
    return r;
  });
}

// (leaf) -> whether its gradient accumulator is alive, held by an earlier graph, and
// belongs to the device's default stream.
PyObject* accumulates_on_default_stream(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 1)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& t = tensor(a[0], "leaf");
    need_cuda(t.device());
    const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
    const auto stream = node == nullptr ? std::nullopt : node->stream();
    return PyBool_FromLong(stream.has_value() && stream->device_type() == at::kCUDA &&
                           c10::cuda::CUDAStream(*stream) ==
                               c10::cuda::getDefaultCUDAStream(t.device().index()));
  });
}

// Addresses of the library's functions, in the order of Library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, kFunctions)) return nullptr;
  void* p[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  auto set = [](auto& fn, void* at) { fn = reinterpret_cast<std::decay_t<decltype(fn)>>(at); };
  set(lib.rmsnorm[0], p[0]);
  set(lib.rmsnorm[1], p[1]);
  set(lib.rmsnorm_bwd_ws, p[2]);
  set(lib.rmsnorm_bwd, p[3]);
  set(lib.swiglu[0], p[4]);
  set(lib.swiglu[1], p[5]);
  set(lib.swiglu_bwd[0], p[6]);
  set(lib.swiglu_bwd[1], p[7]);
  set(lib.ns_ws, p[8]);
  set(lib.ns, p[9]);
  Py_RETURN_NONE;
}

#define FAST(name) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"rmsnorm", FAST(rmsnorm), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", FAST(rmsnorm_backward), METH_FASTCALL, nullptr},
    {"swiglu", FAST(swiglu), METH_FASTCALL, nullptr},
    {"swiglu_backward", FAST(swiglu_backward), METH_FASTCALL, nullptr},
    {"newton_schulz", FAST(newton_schulz), METH_FASTCALL, nullptr},
    {"accumulates_on_default_stream", FAST(accumulates_on_default_stream), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() { return PyModule_Create(&module); }

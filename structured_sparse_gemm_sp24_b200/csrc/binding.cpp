// Native half of the Python binding for the e4m3 and norm entry points: checks
// the tensors and calls the C function.  A call of these kernels takes the GPU
// two to nine microseconds at a few tokens, and the same checks written in Python
// took four (one token through the norm: 7.6 us of host time, 3.4 this way; a
// decode GEMM 8.0 and 3.9).
//
// Every function takes its arguments by position (None for an absent tensor, the
// last one a raw stream or None for torch's current stream) and returns the C
// function's status; a tensor of another type, size, layout or device raises
// ValueError.  bind() receives the addresses of the library's functions, so the
// library itself is loaded in one place.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/sp24.h"

namespace {

decltype(&sp24_quantize_fp8) f_quantize = nullptr;
decltype(&sp24_prune_compress_fp8) f_convert = nullptr;
decltype(&sp24_compress_fp8) f_compress = nullptr;
decltype(&sp24_gemm_fp8) f_gemm = nullptr;
decltype(&sp24_rmsnorm_quant) f_norm = nullptr;
decltype(&sp24_rmsnorm_backward) f_back = nullptr;
decltype(&sp24_meta_bytes) f_meta_bytes = nullptr;
decltype(&sp24_rmsnorm_backward_workspace_bytes) f_back_bytes = nullptr;

constexpr auto kBF16 = at::ScalarType::BFloat16;
constexpr auto kF32 = at::ScalarType::Float;
constexpr auto kF64 = at::ScalarType::Double;
constexpr auto kE4M3 = at::ScalarType::Float8_e4m3fn;
constexpr auto kE8M0 = at::ScalarType::Float8_e8m0fnu;
constexpr auto kU8 = at::ScalarType::Byte;
constexpr auto kI8 = at::ScalarType::Char;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument("sp24: " + what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor& matrix(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be a matrix");
  return t;
}

// The current device, on which the call's tensors have to lie (`t` is asked
// first: without a GPU there is no current device).
int device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor on the current device");
  return c10::cuda::current_device();
}

// Pointer of a dense CUDA tensor of type `a` or `b` with `numel` elements on
// device `dev`; None gives a null pointer.
void* arg(PyObject* o, const char* name, at::ScalarType a, at::ScalarType b, int64_t numel, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(std::string(name) + " must be a CUDA tensor on the current device (" + std::to_string(dev) + ")");
  if (t.scalar_type() != a && t.scalar_type() != b)
    refuse(std::string(name) + " has type " + at::toString(t.scalar_type()) + ", expected " +
           at::toString(a) + (a == b ? "" : std::string(" or ") + at::toString(b)));
  if (t.numel() != numel || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous with " + std::to_string(numel) + " elements");
  return t.data_ptr();
}

void* arg(PyObject* o, const char* name, at::ScalarType a, int64_t numel, int dev) {
  return arg(o, name, a, a, numel, dev);
}

// Metadata: at least the layout's bytes (an allocation may be larger).
void* meta_arg(PyObject* o, int64_t n, int64_t k, int dev) {
  const int64_t need = (n + 127) / 128 * ((k + 127) / 128) * 2048;
  const int64_t have = o == Py_None ? 0 : tensor(o, "meta").numel();
  return arg(o, "meta", kU8, have > need ? have : need, dev);
}

int64_t scale_cols(int64_t k) { return 4 * ((k + 511) / 512); }

// The library's code of a stream type; another type is refused by arg().
int type_code(const at::Tensor& t) {
  return t.scalar_type() == kF32 ? SP24_F32 : t.scalar_type() == kBF16 ? SP24_BF16 : -1;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::runtime_error("");   // the Python error stands
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
  return v;
}

void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw std::runtime_error("");
  return p;
}

// The Python error of the C++ exception being handled: ValueError for a refused
// tensor, torch's own for its errors (torch.OutOfMemoryError for an allocation
// that fails, as torch.empty raises it), RuntimeError otherwise.
void to_python() {
  try {
    throw;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error&) {
    torch::translate_exception_to_python(std::current_exception());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
}

// Runs `body`, which returns a status, with the argument count checked and C++
// exceptions turned into Python ones.
template <class Body>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, const void* bound, Body&& body) {
  try {
    if (have != want) throw std::runtime_error("sp24: wrong number of arguments");
    if (bound == nullptr) throw std::runtime_error("sp24: the library is not loaded");
    return PyLong_FromLong(body());
  } catch (...) {
    to_python();
  }
  return nullptr;
}

// Calls the C function without the interpreter lock (a launch may wait for room
// in the stream's queue).
template <class F, class... A>
long call(F f, A... a) {
  sp24_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f(a...);
  Py_END_ALLOW_THREADS
  return static_cast<long>(st);
}

// (X, Xq, e_x, stream)
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, reinterpret_cast<void*>(f_quantize), [&] {
    const at::Tensor& x = matrix(a[0], "X");
    const int dev = device(x, "X");
    const int64_t m = x.size(0), k = x.size(1), all = x.numel();
    const void* px = arg(a[0], "X", kBF16, kF32, all, dev);
    void* q = arg(a[1], "Xq", kE4M3, all, dev);
    void* e = arg(a[2], "e_x", kE8M0, kU8, m * scale_cols(k), dev);
    return call(f_quantize, px, m, k, type_code(x), q, static_cast<uint8_t*>(e), stream_of(a[3], dev));
  });
}

// (W, mode, norms, mask_in, mask_out, vals, meta, e_w, stream)
PyObject* prune_compress_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, reinterpret_cast<void*>(f_convert), [&] {
    const at::Tensor& w = matrix(a[0], "W");
    const int dev = device(w, "W");
    const int64_t rows = w.size(0), k = w.size(1);
    const void* pw = arg(a[0], "W", kBF16, w.numel(), dev);
    void* norms = arg(a[2], "norms", kF64, k, dev);
    void* in = arg(a[3], "mask_in", kU8, rows * (k / 8), dev);
    void* out = arg(a[4], "mask_out", kU8, rows * (k / 8), dev);
    void* vals = arg(a[5], "vals", kE4M3, rows * (k / 2), dev);
    void* meta = meta_arg(a[6], rows, k, dev);
    void* e = arg(a[7], "e_w", kE8M0, kU8, (rows + 127) / 128 * scale_cols(k), dev);
    return call(f_convert, pw, rows, k, static_cast<int>(integer(a[1])),
                static_cast<const double*>(norms), static_cast<const uint8_t*>(in),
                static_cast<uint8_t*>(out), vals, meta, static_cast<uint8_t*>(e),
                stream_of(a[8], dev));
  });
}

// (W, mask, vals, meta, e_w, stream)
PyObject* compress_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, reinterpret_cast<void*>(f_compress), [&] {
    const at::Tensor& w = matrix(a[0], "W");
    const int dev = device(w, "W");
    const int64_t rows = w.size(0), k = w.size(1);
    const void* pw = arg(a[0], "W", kBF16, w.numel(), dev);
    void* mask = arg(a[1], "mask", kU8, rows * (k / 8), dev);
    void* vals = arg(a[2], "vals", kE4M3, rows * (k / 2), dev);
    void* meta = meta_arg(a[3], rows, k, dev);
    void* e = arg(a[4], "e_w", kE8M0, kU8, (rows + 127) / 128 * scale_cols(k), dev);
    return call(f_compress, pw, static_cast<const uint8_t*>(mask), rows, k, vals, meta,
                static_cast<uint8_t*>(e), stream_of(a[5], dev));
  });
}

// (X, e_x, vals, meta, e_w, N, out_kind, Y, stream)
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, reinterpret_cast<void*>(f_gemm), [&] {
    const at::Tensor& x = matrix(a[0], "X");
    const int dev = device(x, "X");
    const int64_t m = x.size(0), k = x.size(1), rows = integer(a[5]);
    const int kind = static_cast<int>(integer(a[6]));
    const void* px = arg(a[0], "X", kE4M3, x.numel(), dev);
    void* ex = arg(a[1], "e_x", kE8M0, kU8, m * scale_cols(k), dev);
    void* vals = arg(a[2], "vals", kE4M3, rows * (k / 2), dev);
    void* meta = meta_arg(a[3], rows, k, dev);
    void* ew = arg(a[4], "e_w", kE8M0, kU8, (rows + 127) / 128 * scale_cols(k), dev);
    void* y = arg(a[7], "Y", kind == SP24_OUT_F32 ? kF32 : kBF16, m * rows, dev);
    return call(f_gemm, px, static_cast<const uint8_t*>(ex), m, k, static_cast<const void*>(vals),
                static_cast<const void*>(meta), static_cast<const uint8_t*>(ew), rows, kind, y,
                stream_of(a[8], dev));
  });
}

// (X, R, gamma, eps, out_dtype, s_x, H, Y, e_y, rstd, stream)
PyObject* rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, reinterpret_cast<void*>(f_norm), [&] {
    const at::Tensor& x = matrix(a[0], "X");
    const int dev = device(x, "X");
    const int64_t m = x.size(0), k = x.size(1), all = x.numel();
    const at::ScalarType t = x.scalar_type();
    const int out = static_cast<int>(integer(a[4]));
    if (out != SP24_FP8 && out != SP24_INT8 && out != SP24_BF16) refuse("unknown out_dtype");
    const void* px = arg(a[0], "X", kBF16, kF32, all, dev);
    void* r = arg(a[1], "R", t, all, dev);
    void* gamma = arg(a[2], "gamma", t, k, dev);
    void* sx = arg(a[5], "s_x", kF32, 1, dev);
    void* h = arg(a[6], "H", t, all, dev);
    void* y = arg(a[7], "Y", out == SP24_FP8 ? kE4M3 : out == SP24_INT8 ? kI8 : kBF16, all, dev);
    void* e = arg(a[8], "e_y", kE8M0, kU8, m * scale_cols(k), dev);
    void* rstd = arg(a[9], "rstd", kF32, m, dev);
    return call(f_norm, px, static_cast<const void*>(r), static_cast<const void*>(gamma), m, k,
                type_code(x), static_cast<float>(number(a[3])), out, static_cast<const float*>(sx), h,
                y, static_cast<uint8_t*>(e), static_cast<float*>(rstd), stream_of(a[10], dev));
  });
}

// (dY, dH, H, gamma, rstd, dX, dgamma, workspace, stream)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, reinterpret_cast<void*>(f_back), [&] {
    const at::Tensor& h = matrix(a[2], "H");
    const int dev = device(h, "H");
    const int64_t m = h.size(0), k = h.size(1), all = h.numel();
    const at::ScalarType t = h.scalar_type();
    const void* ph = arg(a[2], "H", kBF16, kF32, all, dev);
    void* dy = arg(a[0], "dY", t, all, dev);
    void* dh = arg(a[1], "dH", t, all, dev);
    void* gamma = arg(a[3], "gamma", t, k, dev);
    void* rstd = arg(a[4], "rstd", kF32, m, dev);
    void* dx = arg(a[5], "dX", t, all, dev);
    void* dg = arg(a[6], "dgamma", kF32, k, dev);
    const int64_t bytes = tensor(a[7], "workspace").numel();
    void* ws = arg(a[7], "workspace", kU8, bytes, dev);
    return call(f_back, static_cast<const void*>(dy), static_cast<const void*>(dh), ph,
                static_cast<const void*>(gamma), static_cast<const float*>(rstd), m, k, type_code(h),
                dx, static_cast<float*>(dg), ws, static_cast<size_t>(bytes), stream_of(a[8], dev));
  });
}

// An uninitialised tensor of `type` on like's device.
PyObject* new_tensor(const at::Tensor& like, at::ScalarType type, at::IntArrayRef size) {
  return THPVariable_Wrap(at::empty(size, like.options().dtype(type).requires_grad(false)));
}

// Runs `body`, which returns a tensor, like guarded().
template <class Body>
PyObject* guarded_new(Py_ssize_t have, Py_ssize_t least, Py_ssize_t most, Body&& body) {
  try {
    if (have < least || have > most) throw std::runtime_error("sp24: wrong number of arguments");
    return body();
  } catch (...) {
    to_python();
  }
  return nullptr;
}

// (like, type code, size...).  Codes: 0 like's own type, 1 int8, 2 bf16, 3 float32,
// 4 e4m3, 5 e8m0, 6 uint8.
PyObject* new_empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded_new(n, 3, 4, [&] {
    constexpr at::ScalarType types[] = {kU8, kI8, kBF16, kF32, kE4M3, kE8M0, kU8};
    const at::Tensor& like = tensor(a[0], "like");
    const int64_t code = integer(a[1]);
    if (code < 0 || code > 6) refuse("unknown type code");
    const int64_t size[2] = {integer(a[2]), n == 4 ? integer(a[3]) : 0};
    return new_tensor(like, code == 0 ? like.scalar_type() : types[code],
                      at::IntArrayRef(size, static_cast<size_t>(n - 2)));
  });
}

// (like, N, K): the metadata bytes of an N x K weight.
PyObject* new_meta(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded_new(n, 3, 3, [&] {
    if (f_meta_bytes == nullptr) throw std::runtime_error("sp24: the library is not loaded");
    return new_tensor(tensor(a[0], "like"), kU8,
                      {static_cast<int64_t>(f_meta_bytes(integer(a[1]), integer(a[2])))});
  });
}

// (like, M, K): the norm gradient's workspace.
PyObject* new_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded_new(n, 3, 3, [&] {
    if (f_back_bytes == nullptr) throw std::runtime_error("sp24: the library is not loaded");
    return new_tensor(tensor(a[0], "like"), kU8,
                      {static_cast<int64_t>(f_back_bytes(integer(a[1]), integer(a[2])))});
  });
}

// bind(quantize, prune_compress, compress, gemm, norm, backward, meta bytes,
// workspace bytes): addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, reinterpret_cast<void*>(&bind), [&]() -> long {
    f_quantize = reinterpret_cast<decltype(f_quantize)>(PyLong_AsVoidPtr(a[0]));
    f_convert = reinterpret_cast<decltype(f_convert)>(PyLong_AsVoidPtr(a[1]));
    f_compress = reinterpret_cast<decltype(f_compress)>(PyLong_AsVoidPtr(a[2]));
    f_gemm = reinterpret_cast<decltype(f_gemm)>(PyLong_AsVoidPtr(a[3]));
    f_norm = reinterpret_cast<decltype(f_norm)>(PyLong_AsVoidPtr(a[4]));
    f_back = reinterpret_cast<decltype(f_back)>(PyLong_AsVoidPtr(a[5]));
    f_meta_bytes = reinterpret_cast<decltype(f_meta_bytes)>(PyLong_AsVoidPtr(a[6]));
    f_back_bytes = reinterpret_cast<decltype(f_back_bytes)>(PyLong_AsVoidPtr(a[7]));
    if (PyErr_Occurred()) throw std::runtime_error("");
    return 0;
  });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef entry(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {entry("quantize_fp8", quantize_fp8),
                         entry("prune_compress_fp8", prune_compress_fp8),
                         entry("compress_fp8", compress_fp8),
                         entry("gemm_fp8", gemm_fp8),
                         entry("rmsnorm_quant", rmsnorm_quant),
                         entry("rmsnorm_backward", rmsnorm_backward),
                         entry("new_empty", new_empty),
                         entry("new_meta", new_meta),
                         entry("new_workspace", new_workspace),
                         entry("bind", bind),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the Python and torch this was compiled against (build.py).
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module_def);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", SP24_BINDING_TAG) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

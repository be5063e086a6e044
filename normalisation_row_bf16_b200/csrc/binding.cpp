// binding.cpp -- argument marshalling of the layer-norm and feed-forward
// operators: checks tensors, allocates outputs and workspaces with torch's
// allocator and calls the C ABI on the given stream.  The same work in Python
// took 10 to 16 us a call, more than the small calls' kernels.
//
// Plain CPython functions with positional arguments (normalisation_row_bf16_b200
// /ops.py holds the documented signatures).  The library's entry points are
// handed over as addresses by set_library, so one copy of it is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <stdexcept>
#include <string>

#include "mxnorm.h"

namespace {

struct Library {
  decltype(&layernorm_fwd) ln_fwd;
  decltype(&layernorm_bwd) ln_bwd;
  decltype(&layernorm_bwd_workspace_size) ln_bwd_ws;
  decltype(&gated_ffn_fwd) ffn_fwd;
  decltype(&gated_ffn_bwd) ffn_bwd;
  decltype(&gated_ffn_bwd_workspace_size) ffn_bwd_ws;
  decltype(&mxfp8_gated_ffn) mx_ffn;
  decltype(&mxnorm_scales_bytes) scales;
  decltype(&mxnorm_last_error) last_error;
} g_lib;
PyObject* g_error = nullptr;             // MXNormError(status, message)

struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct LibraryError {
  int status;
};

using Args = PyObject* const*;
using at::Tensor;

std::string describe(const Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw BadValue(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

// The device of the call: `t` lies on it and it is the current one (the
// library launches there).
int launch_device(const Tensor& t) {
  if (!t.is_cuda()) throw BadValue("tensors must be CUDA tensors");
  const int dev = t.get_device(), cur = c10::cuda::current_device();
  if (dev != cur)
    throw BadValue("tensors are on cuda:" + std::to_string(dev) + ", the current device is cuda:" + std::to_string(cur));
  return dev;
}

void same_device(const Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw BadValue(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev));
}

// An input of the given type and shape (cols < 0: one dimension).  dense: the
// whole tensor is contiguous; else its rows are.
void* input(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t rows, int64_t cols, bool dense = true) {
  const Tensor& t = tensor(o, name);
  same_device(t, name, dev);
  const bool shape = cols < 0 ? t.dim() == 1 && t.size(0) == rows : t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
  if (t.scalar_type() != type || !shape)
    throw BadValue(std::string(name) + " must be " + c10::toString(type) + " [" + std::to_string(rows) +
                   (cols < 0 ? "" : ", " + std::to_string(cols)) + "], got " + describe(t));
  if (!t.is_contiguous()) {
    if (dense) throw BadValue(std::string(name) + " must be contiguous");
    if (t.stride(1) != 1 && cols != 1) throw BadValue(std::string("rows of ") + name + " must be contiguous");
  }
  return t.data_ptr();
}

// Row stride of a 2-D tensor (its width where it has at most one row).
int64_t ld(PyObject* o) {
  const Tensor& t = THPVariable_Unpack(o);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// A contiguous buffer of the caller's that holds at least `bytes`.
void* buffer(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t bytes, bool any_type = false) {
  const Tensor& t = tensor(o, name);
  same_device(t, name, dev);
  if ((!any_type && t.scalar_type() != type) || !t.is_contiguous())
    throw BadValue(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor");
  if ((int64_t)t.nbytes() < bytes)
    throw BadValue(std::string(name) + " holds " + std::to_string(t.nbytes()) + " bytes, " + std::to_string(bytes) + " needed");
  return t.data_ptr();
}

// An output: the caller's buffer, or a new tensor.
struct Out {
  Tensor t;
  PyObject* o = nullptr;                 // the caller's, borrowed
  void* p = nullptr;
  // New reference (None when there is no such output).
  PyObject* object() {
    if (o) return Py_NewRef(o);
    if (!t.defined()) return Py_NewRef(Py_None);
    return THPVariable_Wrap(std::move(t));
  }
};
Out output(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape, const Tensor& like) {
  Out r;
  if (given(o)) {
    int64_t n = 1;
    for (int64_t s : shape) n *= s;
    r.p = buffer(o, name, dev, type, n * (int64_t)c10::elementSize(type));
    r.o = o;
  } else {
    r.t = at::empty(shape, like.options().dtype(type));
    r.p = r.t.data_ptr();
  }
  return r;
}

Out workspace(PyObject* o, int dev, int64_t bytes, const Tensor& like, size_t* have) {
  Out r;
  if (given(o)) {
    r.p = buffer(o, "workspace", dev, at::kByte, bytes, true);
    *have = THPVariable_Unpack(o).nbytes();
  } else {
    *have = (size_t)(bytes < 16 ? 16 : bytes);
    r.t = at::empty({(int64_t)*have}, like.options().dtype(at::kByte));
    r.p = r.t.data_ptr();
  }
  return r;
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadValue(std::string(name) + " must be an integer");
  }
  return v;
}
bool flag(PyObject* o) { return PyObject_IsTrue(o) > 0; }
void* stream_of(PyObject* o) { return reinterpret_cast<void*>((uintptr_t)PyLong_AsUnsignedLongLong(o)); }
double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadValue(std::string(name) + " must be a number");
  }
  return v;
}

void check(int rc) {
  if (rc != MXN_OK) throw LibraryError{rc};
}

PyObject* tuple(Out* outs, int n) {
  PyObject* r = PyTuple_New(n);
  if (r)
    for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, outs[i].object());
  return r;
}

int ln_dtype(const Tensor& x) {
  if (x.dim() == 2) switch (x.scalar_type()) {
      case at::kBFloat16: return MXN_BF16;
      case at::kHalf: return MXN_FP16;
      case at::kFloat: return MXN_FP32;
      default: break;
    }
  throw BadValue("x must be a 2-D bf16, fp16 or fp32 tensor");
}

// (x, gamma, beta, eps, y, mean, rstd, want_stats, stream)
PyObject* ln_fwd(Args a) {
  const Tensor& x = tensor(a[0], "x");
  const int dev = launch_device(x), dtype = ln_dtype(x);
  const auto type = x.scalar_type();
  const int64_t T = x.size(0), D = x.size(1);
  void* px = input(a[0], "x", dev, type, T, D, false);
  void* pg = given(a[1]) ? input(a[1], "gamma", dev, type, D, -1) : nullptr;
  void* pb = given(a[2]) ? input(a[2], "beta", dev, type, D, -1) : nullptr;
  const bool stats = flag(a[7]);
  Out r[3] = {output(a[4], "y", dev, type, {T, D}, x)};
  if (stats || given(a[5])) r[1] = output(a[5], "mean", dev, at::kFloat, {T}, x);
  if (stats || given(a[6])) r[2] = output(a[6], "rstd", dev, at::kFloat, {T}, x);
  check(g_lib.ln_fwd(px, pg, pb, r[0].p, (float*)r[1].p, (float*)r[2].p, T, D, ld(a[0]), (float)real(a[3], "eps"), dtype,
                     stream_of(a[8])));
  return tuple(r, 3);
}

// (x, dy, gamma, mean, rstd, dx, dgamma, dbeta, workspace, want_dgamma, want_dbeta, stream)
PyObject* ln_bwd(Args a) {
  const Tensor& x = tensor(a[0], "x");
  const int dev = launch_device(x), dtype = ln_dtype(x);
  const auto type = x.scalar_type();
  const int64_t T = x.size(0), D = x.size(1);
  void* px = input(a[0], "x", dev, type, T, D, false);
  void* py = input(a[1], "dy", dev, type, T, D, false);
  void* pg = given(a[2]) ? input(a[2], "gamma", dev, type, D, -1) : nullptr;
  void* pm = input(a[3], "mean", dev, at::kFloat, T, -1);
  void* pr = input(a[4], "rstd", dev, at::kFloat, T, -1);
  Out r[3] = {output(a[5], "dx", dev, type, {T, D}, x)}, ws;
  if (given(a[6]) || (flag(a[9]) && pg)) r[1] = output(a[6], "dgamma", dev, type, {D}, x);
  if (given(a[7]) || flag(a[10])) r[2] = output(a[7], "dbeta", dev, type, {D}, x);
  size_t bytes = 0;
  if (r[1].p || r[2].p) ws = workspace(a[8], dev, (int64_t)g_lib.ln_bwd_ws(T, D, dtype), x, &bytes);
  check(g_lib.ln_bwd(px, py, pg, (const float*)pm, (const float*)pr, r[0].p, r[1].p, r[2].p, T, D, ld(a[0]), ld(a[1]), dtype,
                     ws.p, bytes, stream_of(a[11])));
  return tuple(r, 3);
}

// Operands of the bf16 projections.
struct Ffn {
  void *x, *wg, *wu;
  int64_t T, D, F, ld_x, ld_w;
  int dev;
};
Ffn ffn_inputs(PyObject* ox, PyObject* og, PyObject* ou) {
  const Tensor &x = tensor(ox, "x"), &w = tensor(og, "w_gate");
  Ffn f;
  f.dev = launch_device(x);
  if (x.dim() != 2 || w.dim() != 2) throw BadValue("x must be [T, D] and the weights [F, D]");
  f.T = x.size(0);
  f.D = x.size(1);
  f.F = w.size(0);
  f.x = input(ox, "x", f.dev, at::kBFloat16, f.T, f.D, false);
  f.wg = input(og, "w_gate", f.dev, at::kBFloat16, f.F, f.D, false);
  f.wu = input(ou, "w_up", f.dev, at::kBFloat16, f.F, f.D, false);
  f.ld_x = ld(ox);
  f.ld_w = ld(og);
  if (f.ld_w != ld(ou)) throw BadValue("w_gate and w_up must have the same row stride");
  return f;
}

// (x, w_gate, w_up, act, save, h, gate, up, stream)
PyObject* ffn_fwd(Args a) {
  const Ffn f = ffn_inputs(a[0], a[1], a[2]);
  const Tensor& x = THPVariable_Unpack(a[0]);
  Out r[3] = {output(a[5], "h", f.dev, at::kBFloat16, {f.T, f.F}, x)};
  if (flag(a[4]) || given(a[6]) || given(a[7])) {
    r[1] = output(a[6], "gate", f.dev, at::kBFloat16, {f.T, f.F}, x);
    r[2] = output(a[7], "up", f.dev, at::kBFloat16, {f.T, f.F}, x);
  }
  check(g_lib.ffn_fwd(f.x, f.wg, f.wu, r[0].p, r[1].p, r[2].p, f.T, f.D, f.F, f.ld_x, f.ld_w, (int)integer(a[3], "act"),
                      stream_of(a[8])));
  return tuple(r, 3);
}

// (dh, x, w_gate, w_up, gate, up, act, dx, dw_gate, dw_up, workspace, want_dx, want_dw, stream)
PyObject* ffn_bwd(Args a) {
  const Ffn f = ffn_inputs(a[1], a[2], a[3]);
  const Tensor& x = THPVariable_Unpack(a[1]);
  void* ph = input(a[0], "dh", f.dev, at::kBFloat16, f.T, f.F);
  void* pg = input(a[4], "gate", f.dev, at::kBFloat16, f.T, f.F);
  void* pu = input(a[5], "up", f.dev, at::kBFloat16, f.T, f.F);
  Out r[3];
  if (flag(a[11]) || given(a[7])) r[0] = output(a[7], "dx", f.dev, at::kBFloat16, {f.T, f.D}, x);
  if (flag(a[12]) || given(a[8]) || given(a[9])) {
    r[1] = output(a[8], "dw_gate", f.dev, at::kBFloat16, {f.F, f.D}, x);
    r[2] = output(a[9], "dw_up", f.dev, at::kBFloat16, {f.F, f.D}, x);
  }
  size_t bytes = 0;
  const int64_t need = given(a[10]) ? 4 * f.T * f.F : (int64_t)g_lib.ffn_bwd_ws(f.T, f.D, f.F);
  const Out ws = workspace(a[10], f.dev, need, x, &bytes);
  check(g_lib.ffn_bwd(ph, f.x, f.wg, f.wu, pg, pu, r[0].p, r[1].p, r[2].p, f.T, f.D, f.F, f.ld_x, f.ld_w,
                      (int)integer(a[6], "act"), ws.p, bytes, stream_of(a[13])));
  return tuple(r, 3);
}

// (a_q, a_s, g_q, g_s, u_q, u_s, T, F, K, act, out, scale_layout, h, h_s, stream)
PyObject* mx_ffn(Args a) {
  const Tensor& q = tensor(a[0], "a_q");
  const int dev = launch_device(q);
  const int64_t T = integer(a[6], "T"), F = integer(a[7], "F"), K = integer(a[8], "K");
  const int act = (int)integer(a[9], "act"), out = (int)integer(a[10], "out"), layout = (int)integer(a[11], "scale_layout");
  if (T < 0 || F < 0 || K < 0) throw BadValue("T, F and K must not be negative");
  const int64_t st = (int64_t)g_lib.scales(T, K, MXN_SCALES_MMA), sf = (int64_t)g_lib.scales(F, K, MXN_SCALES_MMA);
  void* p[6] = {buffer(a[0], "a_q", dev, at::kByte, T * K), buffer(a[1], "a_s", dev, at::kByte, st),
                buffer(a[2], "g_q", dev, at::kByte, F * K), buffer(a[3], "g_s", dev, at::kByte, sf),
                buffer(a[4], "u_q", dev, at::kByte, F * K), buffer(a[5], "u_s", dev, at::kByte, sf)};
  Out r[2];
  if (out == MXN_FFN_BF16) {
    r[0] = output(a[12], "h", dev, at::kBFloat16, {T, F}, q);
    if (given(a[13])) throw BadValue("h_s is given for bf16 output");
  } else {
    r[0] = output(a[12], "h", dev, at::kByte, {T, F}, q);
    const int64_t n = (int64_t)g_lib.scales(T, F, layout);
    if (given(a[13])) {
      r[1].p = buffer(a[13], "h_s", dev, at::kByte, n);
      r[1].o = a[13];
    } else {
      r[1].t = layout == MXN_SCALES_ROWMAJOR ? at::empty({T, F / 32}, q.options()) : at::zeros({n < 1 ? 1 : n}, q.options());
      r[1].p = r[1].t.data_ptr();
    }
  }
  check(g_lib.mx_ffn(p[0], p[1], p[2], p[3], p[4], p[5], r[0].p, r[1].p, T, F, K, act, out, layout, stream_of(a[14])));
  return tuple(r, 2);
}

template <PyObject* (*FN)(Args), int N>
PyObject* entry(PyObject*, Args args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return FN(args);
  } catch (const LibraryError& e) {
    if (PyObject* v = PyObject_CallFunction(g_error, "is", e.status, g_lib.last_error())) {
      PyErr_SetObject(g_error, v);
      Py_DECREF(v);
    }
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());      // torch's own, out of memory among them
  }
  return nullptr;
}

// (MXNormError, address of each entry point in the order of Library)
PyObject* set_library(PyObject*, Args args, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Library) / sizeof(void*);
  if (n != 1 + kEntries) {
    PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  std::memcpy(&g_lib, p, sizeof g_lib);
  Py_INCREF(args[0]);
  Py_XSETREF(g_error, args[0]);
  Py_RETURN_NONE;
}

#define ENTRY(name, fn, n) {name, (PyCFunction)(void (*)(void))entry<fn, n>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    {"set_library", (PyCFunction)(void (*)(void))set_library, METH_FASTCALL, nullptr},
    ENTRY("layernorm_fwd", ln_fwd, 9),
    ENTRY("layernorm_bwd", ln_bwd, 12),
    ENTRY("gated_ffn_fwd", ffn_fwd, 9),
    ENTRY("gated_ffn_bwd", ffn_bwd, 14),
    ENTRY("mxfp8_gated_ffn", mx_ffn, 15),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }

// Marshalling of the calls around the layer and on 4-bit weights: torch tensors
// are checked against the call's shapes and become pointers and strides.  In
// native code because a small call's kernel takes 3 to 5 us, and the same checks
// in Python took 6 and the look-up of the current stream 3.
// Every function returns the library's status; tensors of another shape, element
// type, layout or device raise ValueError before anything is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/twell.h"

namespace {

struct PyError {};                       // a Python exception is set

[[noreturn]] void refuse(const char* name, const std::string& what) {
  throw std::invalid_argument(std::string(name) + ": expected " + what);
}

std::string describe(const at::Tensor& t) {
  std::string s = "; got (";
  for (auto n : t.sizes()) s += std::to_string(n) + ",";
  s += ") strides (";
  for (auto n : t.strides()) s += std::to_string(n) + ",";
  return s + ") of " + c10::toString(t.scalar_type()) + " elements on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

void* on_gpu(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() && t.numel() > 0) refuse(name, "a tensor on the GPU" + describe(t));
  return t.data_ptr();
}

// What an argument's elements may be: a type, or for some the raw bits of it.
struct Elem {
  const char* name;
  at::ScalarType type, raw;
  bool holds(const at::Tensor& t) const { return t.scalar_type() == type || t.scalar_type() == raw; }
};
constexpr Elem E_F32{"float32", at::kFloat, at::kFloat}, E_BF16{"bfloat16", at::kBFloat16, at::kBFloat16},
    E_E4M3{"float8_e4m3fn or uint8", at::kFloat8_e4m3fn, at::kByte},
    E_E2M1{"float4_e2m1fn_x2 or uint8", at::kFloat4_e2m1fn_x2, at::kByte},
    E_E8M0{"float8_e8m0fnu or uint8", at::kFloat8_e8m0fnu, at::kByte}, E_U64{"int64 or uint64", at::kLong, at::kUInt64};
const Elem& elem_of(int dt) { return dt == TWELL_F32 ? E_F32 : dt == TWELL_BF16 ? E_BF16 : E_E4M3; }

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};
// A [T][d] matrix of rows of elements side by side.
Mat mat(PyObject* o, int64_t T, int64_t d, const Elem& elem, const char* name) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != d || !elem.holds(t) || (d > 1 && t.stride(1) != 1))
    refuse(name, "[" + std::to_string(T) + "][" + std::to_string(d) + "] of " + elem.name +
                     " elements with contiguous rows" + describe(t));
  return {on_gpu(t, name), t.stride(0)};
}
// n elements side by side, of any shape.
void* vec(PyObject* o, int64_t n, const Elem& elem, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.numel() != n || !elem.holds(t) || !t.is_contiguous())
    refuse(name, std::to_string(n) + " contiguous " + elem.name + " elements" + describe(t));
  return on_gpu(t, name);
}
struct Space {
  void* p = nullptr;
  size_t bytes = 0;
};
Space space(PyObject* o) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_contiguous()) refuse("workspace", "contiguous memory" + describe(t));
  return {on_gpu(t, "workspace"), t.nbytes()};
}

// The shape struct behind a ctypes structure (copied: the buffer is released).
template <class S>
S shape_of(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PyError{};
  if (b.len != (Py_ssize_t)sizeof(S)) {
    PyBuffer_Release(&b);
    refuse("shape", "another shape struct");
  }
  S s = *(const S*)b.buf;
  PyBuffer_Release(&b);
  return s;
}

hipStream_t stream_of(PyObject* o) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
  PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
  if (!v) throw PyError{};
  void* s = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!s && PyErr_Occurred()) throw PyError{};
  return (hipStream_t)s;
}

// The 4-bit weights behind a TwellW4: its codes and scales.
struct Weights {
  at::Tensor codes, scales;
  twell_w4 w;
};
at::Tensor attribute(PyObject* o, const char* attr, const char* name) {
  PyObject* v = PyObject_GetAttrString(o, attr);
  if (!v) throw PyError{};
  if (!THPVariable_Check(v)) {
    Py_DECREF(v);
    throw std::invalid_argument(std::string(name) + ": " + attr + " is no tensor");
  }
  at::Tensor t = THPVariable_Unpack(v);
  Py_DECREF(v);
  return t;
}
Weights w4(PyObject* o, const char* name) {
  Weights r{attribute(o, "codes", name), attribute(o, "scales", name), {}};
  const at::Tensor &c = r.codes, &s = r.scales;
  if (c.dim() != 2 || s.dim() != 2 || c.size(0) != s.size(0) || c.size(1) != 16 * s.size(1) || !E_E2M1.holds(c) ||
      !E_E8M0.holds(s) || !c.is_contiguous() || !s.is_contiguous())
    refuse(name, std::string("contiguous matrices of ") + E_E2M1.name + " codes [N][K / 2] and " + E_E8M0.name +
                     " scales [N][K / 32] elements" + describe(c) + describe(s));
  if (c.size(0) > INT32_MAX || c.size(1) > INT32_MAX / 2) refuse(name, "N and K below 2^31");
  r.w = {(int32_t)c.size(0), (int32_t)(2 * c.size(1)), (const uint8_t*)on_gpu(c, name), (const uint8_t*)on_gpu(s, name)};
  return r;
}

// Runs f with the C++ exceptions of a call turned into Python's.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const PyError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* add_rmsnorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const auto sh = shape_of<twell_norm_shape>(a[0]);
    const int64_t T = sh.T, d = sh.d;
    const Elem& rs = elem_of(sh.res_dt);
    const Mat x = mat(a[1], T, d, elem_of(sh.x_dt), "x"), res = mat(a[2], T, d, rs, "residual");
    void* w = vec(a[3], d, elem_of(sh.w_dt), "w");
    void* rng = vec(a[4], 2, E_U64, "rng");
    const Mat sum = mat(a[5], T, d, rs, "sum"), y = mat(a[6], T, d, elem_of(sh.y_dt), "y");
    void* ys = vec(a[7], T * ((d + 31) / 32), E_E8M0, "y_scale");
    void* rstd = vec(a[8], T, E_F32, "rstd");
    return twell_add_rmsnorm_fwd(&sh, x.p, x.ld, res.p, res.ld, w, (const uint64_t*)rng, sum.p, sum.ld, y.p, y.ld,
                                 (uint8_t*)ys, (float*)rstd, stream_of(a[9]));
  });
}

PyObject* add_rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const auto sh = shape_of<twell_norm_shape>(a[0]);
    const int64_t T = sh.T, d = sh.d;
    const Elem& rs = elem_of(sh.res_dt);
    const Mat dy = mat(a[1], T, d, elem_of(sh.y_dt), "dy"), ds = mat(a[2], T, d, rs, "dsum"),
              sum = mat(a[3], T, d, rs, "sum");
    void* w = vec(a[4], d, elem_of(sh.w_dt), "w");
    void* rstd = vec(a[5], T, E_F32, "rstd");
    void* rng = vec(a[6], 2, E_U64, "rng");
    const Mat dres = mat(a[7], T, d, rs, "dres"), dx = mat(a[8], T, d, elem_of(sh.x_dt), "dx");
    void* dw = vec(a[9], d, E_F32, "dw");
    const Space ws = space(a[10]);
    return twell_add_rmsnorm_bwd(&sh, dy.p, dy.ld, ds.p, ds.ld, sum.p, sum.ld, w, (const float*)rstd,
                                 (const uint64_t*)rng, dres.p, dres.ld, dx.p, dx.ld, (float*)dw, ws.p, ws.bytes,
                                 stream_of(a[11]));
  });
}

PyObject* dropout_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> int {
    const auto sh = shape_of<twell_norm_shape>(a[0]);
    const Mat x = mat(a[1], sh.T, sh.d, elem_of(sh.x_dt), "x"), res = mat(a[2], sh.T, sh.d, elem_of(sh.res_dt), "residual");
    void* rng = vec(a[3], 2, E_U64, "rng");
    const Mat y = mat(a[4], sh.T, sh.d, elem_of(sh.y_dt), "y");
    return twell_dropout_add(&sh, x.p, x.ld, res.p, res.ld, (const uint64_t*)rng, y.p, y.ld, stream_of(a[5]));
  });
}

PyObject* w4_matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> int {
    const at::Tensor &xt = tensor(a[0], "x"), &yt = tensor(a[4], "y");
    const auto y_type = yt.scalar_type();
    if (y_type != at::kFloat && y_type != at::kBFloat16) {
      PyErr_SetString(PyExc_TypeError, "y: expected float32 or bfloat16");
      throw PyError{};
    }
    const Weights weights = w4(a[2], "W");
    const twell_w4& W = weights.w;
    if (xt.dim() != 2 || xt.size(0) > INT32_MAX) refuse("x", "a matrix" + describe(xt));
    const int64_t T = xt.size(0);
    const twell_dtype x_dt = a[1] == Py_None ? TWELL_BF16 : TWELL_MXFP8, y_dt = y_type == at::kFloat ? TWELL_F32 : TWELL_BF16;
    const Mat x = mat(a[0], T, W.K, elem_of(x_dt), "x"), y = mat(a[4], T, W.N, elem_of(y_dt), "y");
    void* xs = vec(a[1], T * (W.K / 32), E_E8M0, "x_scale");
    void* bias = vec(a[3], W.N, E_BF16, "bias");
    return twell_w4_matvec((int32_t)T, x.p, x_dt, x.ld, (const uint8_t*)xs, &W, bias, y.p, y_dt, y.ld, stream_of(a[5]));
  });
}

PyObject* ffn_fwd_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const auto sh = shape_of<twell_ffn_shape>(a[0]);
    const int64_t T = sh.T, d = sh.d, F = sh.F;
    void* x = vec(a[1], T * d, elem_of(sh.in_dt), "x");
    void* xs = vec(a[2], T * (d / 32), E_E8M0, "x_scale");
    const Weights Wg = w4(a[3], "Wg"), Wu = w4(a[5], "Wu"), Wd = w4(a[6], "Wd");
    void* bg = vec(a[4], F, E_BF16, "bg");
    void* y = vec(a[7], T * d, elem_of(sh.out_dt), "y");
    const Space ws = space(a[8]);
    return twell_ffn_fwd_w4(&sh, x, (const uint8_t*)xs, &Wg.w, bg, &Wu.w, &Wd.w, y, ws.p, ws.bytes, stream_of(a[9]));
  });
}

PyMethodDef methods[] = {
    {"add_rmsnorm_fwd", (PyCFunction)(void (*)(void))add_rmsnorm_fwd, METH_FASTCALL, nullptr},
    {"add_rmsnorm_bwd", (PyCFunction)(void (*)(void))add_rmsnorm_bwd, METH_FASTCALL, nullptr},
    {"dropout_add", (PyCFunction)(void (*)(void))dropout_add, METH_FASTCALL, nullptr},
    {"w4_matvec", (PyCFunction)(void (*)(void))w4_matvec, METH_FASTCALL, nullptr},
    {"ffn_fwd_w4", (PyCFunction)(void (*)(void))ffn_fwd_w4, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_twell_bind", "Marshalling of libtwell calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__twell_bind() { return PyModule_Create(&module); }

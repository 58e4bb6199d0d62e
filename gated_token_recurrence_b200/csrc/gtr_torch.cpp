// Argument marshalling of the state space and block norm calls for the Python binding.
//
// These calls take a few microseconds on the device and up to fourteen tensors; looking at
// shape, type, device, strides and address of each from Python costs more than the call.  This
// module does exactly that and nothing else, for torch tensors, and calls the C ABI of
// include/gtr.h through the addresses that the binding hands it (bind), so that there is one
// loaded libgtr.so.  No exception leaves a function: each becomes a Python exception.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>

#include "gtr.h"

namespace {

decltype(&gtr_ssm_conv) call_conv;
decltype(&gtr_ssm_scan) call_scan;
decltype(&gtr_ssm_step) call_step;
decltype(&gtr_block_norm) call_norm;

using Sizes = std::initializer_list<int64_t>;

[[noreturn]] void refuse(const char* name, const std::string& why) {
  throw std::invalid_argument(std::string(name) + ": " + why);
}

void print(std::ostringstream& s, const int64_t* v, size_t n) {
  s << "(";
  for (size_t i = 0; i < n; ++i) s << (i ? ", " : "") << v[i];
  s << ")";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  return THPVariable_Unpack(o);
}

// A tensor of these sizes and this type on device dev.
void expect(const char* name, const at::Tensor& t, Sizes sizes, at::ScalarType type, int dev) {
  if (t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == at::IntArrayRef(sizes)) return;
  std::ostringstream s;
  s << "expected a CUDA tensor of type " << type << " and shape ";
  print(s, sizes.begin(), sizes.size());
  s << " on the current device, got " << t.scalar_type() << " ";
  print(s, t.sizes().data(), t.sizes().size());
  s << " on " << t.device();
  refuse(name, s.str());
}

// The address of a contiguous one; None gives a null pointer.
void* whole(const char* name, PyObject* o, Sizes sizes, at::ScalarType type, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(name, o);
  expect(name, t, sizes, type, dev);
  if (!t.is_contiguous()) refuse(name, "must be contiguous");
  return t.data_ptr();
}

// The distance between the rows of consecutive tokens of a tensor whose first `tokens` (1 or 2)
// axes are batch and token axes; a row itself (the other 1 or 2 axes) is contiguous.
int64_t row_distance(const char* name, const at::Tensor& t, int tokens) {
  const auto size = t.sizes(), stride = t.strides();
  const int n = (int)size.size();
  int64_t width = 1;
  for (int i = n - 1; i >= tokens; --i) {
    if (size[i] != 1 && stride[i] != width) refuse(name, "the values of one token must be contiguous");
    width *= size[i];
  }
  if (size[tokens - 1] != 1) {
    const int64_t ld = stride[tokens - 1];
    if (tokens == 2 && size[0] != 1 && stride[0] != size[1] * ld) refuse(name, "consecutive tokens must be evenly spaced");
    return ld;
  }
  if (size[0] != 1) return stride[0];
  const int64_t unit = 16 / (int64_t)t.element_size();  // one token in all: any valid distance
  return (width + unit - 1) / unit * unit;
}

struct Rows {
  void* p;
  int64_t ld;
};

// A tensor that may be a column range of wider rows.
Rows rows(const char* name, PyObject* o, Sizes sizes, at::ScalarType type, int dev, int tokens) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(name, o);
  expect(name, t, sizes, type, dev);
  return {t.data_ptr(), row_distance(name, t, tokens)};
}

int type_code(const char* name, at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GTR_F32;
    case at::kHalf: return GTR_F16;
    case at::kBFloat16: return GTR_BF16;
    default: refuse(name, "must be float32, float16 or bfloat16");
  }
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::domain_error("");  // the Python error stands
  return v;
}
int as_int(PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int)v) throw std::invalid_argument("an integer argument is out of range");
  return (int)v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw std::domain_error("");
  return v;
}
gtr_stream_t stream_of(PyObject* o) { return reinterpret_cast<gtr_stream_t>((uintptr_t)PyLong_AsUnsignedLongLongMask(o)); }

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  try {
    if (given != wanted) throw std::invalid_argument("wrong number of arguments");
    return PyLong_FromLong((long)f());
  } catch (const std::domain_error&) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

void dims(const char* name, const at::Tensor& t, int n) {
  if (t.dim() != n) refuse(name, "expected " + std::to_string(n) + " axes, got " + std::to_string(t.dim()));
}

// conv(x, w, bias, H, W, direction, silu, state, state_out, lengths, out, device, stream)
PyObject* conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() {
    const at::Tensor &x = tensor("x", a[0]), &w = tensor("w", a[1]);
    dims("x", x, 3);
    dims("w", w, 2);
    const int64_t B = x.size(0), L = x.size(1), C = x.size(2), K = w.size(1);
    const auto ty = x.scalar_type();
    const int code = type_code("x", ty), dev = as_int(a[11]);
    const Rows r = rows("x", a[0], {B, L, C}, ty, dev, 2);
    return call_conv(r.p, r.ld, (const float*)whole("w", a[1], {C, K}, at::kFloat, dev),
                     (const float*)whole("bias", a[2], {C}, at::kFloat, dev), whole("state", a[7], {B, K - 1, C}, ty, dev),
                     whole("state_out", a[8], {B, K - 1, C}, ty, dev), (const int*)whole("lengths", a[9], {B}, at::kInt, dev),
                     whole("out", a[10], {B, L, C}, ty, dev), (int)B, as_int(a[3]), as_int(a[4]), (int)C, (int)K, as_int(a[5]),
                     truth(a[6]), code, stream_of(a[12]));
  });
}

struct Mixer {  // what a scan and a step share
  Rows u, dt, bm, cm, z;
  const float *A, *skip, *bias;
  int64_t D, N, G;
  at::ScalarType ty;
  int code;
};
// lead: (B, L) or (B); a: u, dt, A, Bm, Cm, skip, z, dt_bias
Mixer mixer(PyObject* const* a, int tokens, int64_t B, int64_t L, int dev) {
  const at::Tensor &u = tensor("u", a[0]), &A = tensor("A", a[2]), &bm = tensor("Bm", a[3]);
  dims("A", A, 2);
  dims("Bm", bm, tokens + 2);
  Mixer m;
  m.D = A.size(0), m.N = A.size(1), m.G = bm.size(tokens);
  m.ty = u.scalar_type();
  m.code = type_code("u", m.ty);
  const auto line = [&](const char* name, PyObject* o) {
    return tokens == 2 ? rows(name, o, {B, L, m.D}, m.ty, dev, 2) : rows(name, o, {B, m.D}, m.ty, dev, 1);
  };
  const auto group = [&](const char* name, PyObject* o) {
    return tokens == 2 ? rows(name, o, {B, L, m.G, m.N}, m.ty, dev, 2) : rows(name, o, {B, m.G, m.N}, m.ty, dev, 1);
  };
  m.u = line("u", a[0]);
  m.dt = line("dt", a[1]);
  m.A = (const float*)whole("A", a[2], {m.D, m.N}, at::kFloat, dev);
  m.bm = group("Bm", a[3]);
  m.cm = group("Cm", a[4]);
  m.skip = (const float*)whole("skip", a[5], {m.D}, at::kFloat, dev);
  m.z = line("z", a[6]);
  m.bias = (const float*)whole("dt_bias", a[7], {m.D}, at::kFloat, dev);
  return m;
}

// scan(u, dt, A, Bm, Cm, skip, z, dt_bias, softplus, state, state_out, lengths, out, H, W, direction, device, stream)
PyObject* scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() {
    const at::Tensor& u = tensor("u", a[0]);
    dims("u", u, 3);
    const int64_t B = u.size(0), L = u.size(1);
    const int dev = as_int(a[16]);
    const Mixer m = mixer(a, 2, B, L, dev);
    return call_scan(m.u.p, m.u.ld, m.dt.p, m.dt.ld, m.A, m.bm.p, m.bm.ld, m.cm.p, m.cm.ld, m.z.p, m.z.ld, m.skip, m.bias,
                     truth(a[8]), (const float*)whole("state", a[9], {B, m.D, m.N}, at::kFloat, dev),
                     (float*)whole("state_out", a[10], {B, m.D, m.N}, at::kFloat, dev),
                     (const int*)whole("lengths", a[11], {B}, at::kInt, dev), whole("out", a[12], {B, L, m.D}, m.ty, dev),
                     (int)B, as_int(a[13]), as_int(a[14]), (int)m.D, (int)m.N, (int)m.G, as_int(a[15]), m.code,
                     stream_of(a[17]));
  });
}

// step(u, dt, A, Bm, Cm, skip, z, dt_bias, softplus, state, state_out, out, device, stream)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() {
    const at::Tensor& u = tensor("u", a[0]);
    dims("u", u, 2);
    const int64_t B = u.size(0);
    const int dev = as_int(a[12]);
    const Mixer m = mixer(a, 1, B, 1, dev);
    return call_step(m.u.p, m.u.ld, m.dt.p, m.dt.ld, m.A, m.bm.p, m.bm.ld, m.cm.p, m.cm.ld, m.z.p, m.z.ld, m.skip, m.bias,
                     truth(a[8]), (const float*)whole("state", a[9], {B, m.D, m.N}, at::kFloat, dev),
                     (float*)whole("state_out", a[10], {B, m.D, m.N}, at::kFloat, dev),
                     whole("out", a[11], {B, m.D}, m.ty, dev), (int)B, (int)m.D, (int)m.N, (int)m.G, m.code, stream_of(a[13]));
  });
}

// norm(y, h, post_w, pre_w, gate, gate_silu, scale, eps, h_out, n_out, device, stream)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() {
    const at::Tensor &y = tensor("y", a[0]), &h = tensor("h", a[1]);
    dims("y", y, 3);
    const int64_t B = y.size(0), L = y.size(1), C = y.size(2);
    const auto ty = y.scalar_type(), th = h.scalar_type();
    const int code = type_code("y", ty), code_h = type_code("h", th), dev = as_int(a[10]);
    const bool per_token = a[4] != Py_None && tensor("gate", a[4]).dim() == 3;
    const double eps = PyFloat_AsDouble(a[7]);
    if (eps == -1.0 && PyErr_Occurred()) throw std::domain_error("");
    void* gate = per_token ? whole("gate", a[4], {B, L, C}, ty, dev) : whole("gate", a[4], {B, C}, ty, dev);
    return call_norm(whole("y", a[0], {B, L, C}, ty, dev), whole("h", a[1], {B, L, C}, th, dev),
                     (const float*)whole("post_w", a[2], {C}, at::kFloat, dev),
                     (const float*)whole("pre_w", a[3], {C}, at::kFloat, dev), gate, per_token, truth(a[5]),
                     (const float*)whole("scale", a[6], {C}, at::kFloat, dev), (float)eps,
                     whole("h_out", a[8], {B, L, C}, th, dev), whole("n_out", a[9], {B, L, C}, ty, dev), (int)B, L, (int)C,
                     code, code_h, stream_of(a[11]));
  });
}

// row_distance(tensor, tokens): what a strided input is passed with
PyObject* distance(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() { return row_distance("tensor", tensor("tensor", a[0]), as_int(a[1])); });
}

// bind(conv, scan, step, norm): addresses of the C ABI's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() {
    call_conv = reinterpret_cast<decltype(call_conv)>((uintptr_t)integer(a[0]));
    call_scan = reinterpret_cast<decltype(call_scan)>((uintptr_t)integer(a[1]));
    call_step = reinterpret_cast<decltype(call_step)>((uintptr_t)integer(a[2]));
    call_norm = reinterpret_cast<decltype(call_norm)>((uintptr_t)integer(a[3]));
    return 0;
  });
}

#define GTR_FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GTR_FAST(conv), GTR_FAST(scan), GTR_FAST(step),         GTR_FAST(norm),
                         GTR_FAST(bind), GTR_FAST(distance), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gtr_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gtr_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", GTR_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

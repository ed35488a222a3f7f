// binding.cpp -- the Python side of sa_append_kv and sa_attend_chunk: tensors are checked against
// the geometry and handed to the library as plain pointers.  The calls of a decode step are short
// (5 us on the device), and the same checks in Python with ctypes took 9 us of a call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sa.h"

namespace {

using Append = decltype(&sa_append_kv);
using Attend = decltype(&sa_attend_chunk);
Append append_fn = nullptr;
Attend attend_fn = nullptr;

struct Refused {};  // a Python error is set

bool is_bf16(at::ScalarType t) {  // bf16 values or their bit patterns
  return t == at::kBFloat16 || t == at::kShort || t == at::ScalarType::UInt16;
}
bool is_i32(at::ScalarType t) { return t == at::kInt; }
bool is_f32(at::ScalarType t) { return t == at::kFloat; }
bool is_u8(at::ScalarType t) { return t == at::kByte; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: need a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const at::Tensor& t, const char* name, const char* what, int dev) {
  std::ostringstream s;
  s << name << ": need " << what << " on cuda:" << dev << ", got shape " << t.sizes()
    << " strides " << t.strides() << " of " << t.scalar_type() << " on " << t.device();
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  throw Refused();
}

bool here(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// address of a dense tensor of this shape and type on CUDA device `dev`
void* need(PyObject* o, const char* name, at::IntArrayRef shape, bool (*type)(at::ScalarType),
           int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || !type(t.scalar_type()) || !here(t, dev) || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a dense "
      << (type == is_bf16 ? "bfloat16" : type == is_i32 ? "int32" : type == is_f32 ? "float32"
                                                                                   : "uint8")
      << " of shape " << shape;
    refuse(t, name, s.str().c_str(), dev);
  }
  return t.data_ptr();
}

// address of [n, heads, width] rows and elements per token; only tokens may be strided
void* rows(PyObject* o, const char* name, int64_t heads, int64_t width, int64_t n, int dev,
           int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  const int64_t shape[3] = {n, heads, width};
  if (t.sizes() != at::IntArrayRef(shape, 3) || !is_bf16(t.scalar_type()) || !here(t, dev)) {
    std::ostringstream s;
    s << "bfloat16 rows of shape " << at::IntArrayRef(shape, 3);
    refuse(t, name, s.str().c_str(), dev);
  }
  *stride = heads * width;
  if (n == 0) return t.data_ptr() ? t.data_ptr() : reinterpret_cast<void*>(16);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != width))
    refuse(t, name, "the heads of a token side by side", dev);
  if (n > 1) *stride = t.stride(0);  // (of one row torch keeps whatever stride it was sliced from)
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int narrow(PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int)v) {
    PyErr_SetString(PyExc_OverflowError, "integer does not fit 32 bits");
    throw Refused();
  }
  return (int)v;
}

sa_geom geometry(PyObject* o) {
  static PyObject* names[9] = {};
  if (!names[0]) {
    const char* f[9] = {"B", "Hq", "Hkv", "Dk", "Dv", "P", "max_pages", "n_pool", "v_aliases_k"};
    for (int i = 8; i >= 0; --i) names[i] = PyUnicode_InternFromString(f[i]);
  }
  int32_t v[9];
  for (int i = 0; i < 9; ++i) {
    PyObject* x = PyObject_GetAttr(o, names[i]);
    if (!x) throw Refused();
    const int64_t n = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (n == -1 && PyErr_Occurred()) throw Refused();
    if (n != (int32_t)n) {
      PyErr_SetString(PyExc_OverflowError, "geometry does not fit 32 bits");
      throw Refused();
    }
    v[i] = (int32_t)n;
  }
  return sa_geom{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8]};
}

struct Cache {
  const int32_t *cu, *table, *lens;
  void *k, *v;
  Cache(const sa_geom& g, PyObject* cu_, PyObject* table_, PyObject* lens_, PyObject* k_,
        PyObject* v_, int dev) {
    cu = (const int32_t*)need(cu_, "cu_new", {(int64_t)g.B + 1}, is_i32, dev);
    table = (const int32_t*)need(table_, "page_table", {g.B, g.max_pages}, is_i32, dev);
    lens = (const int32_t*)need(lens_, "seq_lens", {g.B}, is_i32, dev);
    k = need(k_, "k_cache", {g.n_pool, g.Hkv, g.P, g.Dk}, is_bf16, dev);
    v = nullptr;
    if (g.v_aliases_k) return;
    if (v_ == Py_None) {
      PyErr_SetString(PyExc_ValueError, "v_cache is needed (the geometry's V does not alias K)");
      throw Refused();
    }
    v = need(v_, "v_cache", {g.n_pool, g.Hkv, g.P, g.Dv}, is_bf16, dev);
  }
};

bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// (dev, geom, k, v, cu_new, page_table, seq_lens, k_cache, v_cache, q, q_out, inv_freq, rot_start,
//  interleaved, logical_lens, summ, summ8, ws, ws_bytes, stream) -> status
PyObject* py_append(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  if (!count(nx, 20)) return nullptr;
  try {
    const int dev = narrow(x[0]);
    const sa_geom g = geometry(x[1]);
    const at::Tensor& k = tensor(x[2], "k");
    const int64_t n = k.dim() ? k.size(0) : 0;
    const Cache c(g, x[4], x[5], x[6], x[7], x[8], dev);
    int64_t ks = 0, vs = 0, qs = 0;
    const void* kp = rows(x[2], "k", g.Hkv, g.Dk, n, dev, &ks);
    const void *vp = nullptr, *qp = nullptr, *fq = nullptr, *ll = nullptr;
    void *qo = nullptr, *s16 = nullptr, *s8 = nullptr;
    int rot = 0;
    if (!g.v_aliases_k) {
      if (x[3] == Py_None) {
        PyErr_SetString(PyExc_ValueError, "v is needed (the geometry's V does not alias K)");
        return nullptr;
      }
      vp = rows(x[3], "v", g.Hkv, g.Dv, n, dev, &vs);
    }
    if (x[9] != Py_None) {
      qp = rows(x[9], "q", g.Hq, g.Dk, n, dev, &qs);
      qo = n ? need(x[10], "q_out", {n, g.Hq, g.Dk}, is_bf16, dev) : const_cast<void*>(qp);
    }
    if (x[11] != Py_None) {
      const int64_t half = tensor(x[11], "inv_freq").numel();
      fq = need(x[11], "inv_freq", {half}, is_f32, dev);
      rot = (int)std::min<int64_t>(2 * half, 1 << 30);
    }
    if (x[14] != Py_None) ll = need(x[14], "logical_lens", {g.B}, is_i32, dev);
    if (x[15] != Py_None) s16 = need(x[15], "summ", {g.n_pool, g.Hkv, 2, g.Dk}, is_bf16, dev);
    if (x[16] != Py_None)
      s8 = need(x[16], "summ8", {g.n_pool, g.Hkv, 2 * (int64_t)g.Dk + 16}, is_u8, dev);
    const int start = narrow(x[12]), inter = PyObject_IsTrue(x[13]);
    if (inter < 0) return nullptr;
    void* ws = (void*)integer(x[17]);
    const size_t bytes = (size_t)integer(x[18]);
    void* stream = (void*)integer(x[19]);
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = append_fn(&g, qp, qs, kp, ks, vp, vs, (int)n, c.cu, c.table, c.lens, (const int32_t*)ll,
                   (const float*)fq, start, rot, inter, qo, c.k, c.v, s16, s8, ws, bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (dev, geom, q, cu_new, k_cache, v_cache, page_table, seq_lens, sink, window, scale, out, lse, ws,
//  ws_bytes, stream) -> status
PyObject* py_attend(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  if (!count(nx, 16)) return nullptr;
  try {
    const int dev = narrow(x[0]);
    const sa_geom g = geometry(x[1]);
    const at::Tensor& q = tensor(x[2], "q");
    const int64_t n = q.dim() ? q.size(0) : 0;
    const Cache c(g, x[3], x[6], x[7], x[4], x[5], dev);
    const void* qp = need(x[2], "q", {n, g.Hq, g.Dk}, is_bf16, dev);
    void* out = need(x[11], "out", {n, g.Hq, g.Dv}, is_bf16, dev);
    void* lse = need(x[12], "lse", {n, g.Hq}, is_f32, dev);
    const int sink = narrow(x[8]), window = narrow(x[9]);
    const double scale = PyFloat_AsDouble(x[10]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    void* ws = (void*)integer(x[13]);
    const size_t bytes = (size_t)integer(x[14]);
    void* stream = (void*)integer(x[15]);
    int st = 0;
    if (n) {
      Py_BEGIN_ALLOW_THREADS;
      st = attend_fn(&g, qp, (int)n, c.cu, c.k, c.v, c.table, c.lens, sink, window, (float)scale,
                     out, (float*)lse, ws, bytes, stream);
      Py_END_ALLOW_THREADS;
    }
    return PyLong_FromLong(st);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (address of sa_append_kv, address of sa_attend_chunk)
PyObject* py_bind(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  if (!count(nx, 2)) return nullptr;
  try {
    append_fn = (Append)integer(x[0]);
    attend_fn = (Attend)integer(x[1]);
  } catch (const Refused&) {
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append_kv", (PyCFunction)(void*)py_append, METH_FASTCALL, nullptr},
                         {"attend_chunk", (PyCFunction)(void*)py_attend, METH_FASTCALL, nullptr},
                         {"bind", (PyCFunction)(void*)py_bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }

// sv_bind.cpp -- Python binding of the paged cache calls (include/sv.h).
//
// Argument marshalling only, as the ctypes binding of the other calls, but in
// C++: these calls stand between the layers of a model, where looking at each
// tensor from Python (5 to 8 us a call) took longer than most of the kernels:
// plan 12.5 -> 4.6 us of host time, append 9.7 -> 4.1 us.  Each function checks
// its tensors, runs on their device and its current stream, and returns the
// status of the C call; `plan` and `attend` return the dict of outputs instead
// where the status is SV_OK.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/sv.h"

namespace {

struct Refusal {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refusal{PyExc_ValueError, s}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  return t;
}

// A dense device tensor of one type, on device `dev` (-1: any).
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
               c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (dev >= 0 && t.get_device() != dev)
    value_error(std::string(name) + " must be on cuda:" + std::to_string(dev));
  return t;
}

// Its data pointer; None is NULL.
template <class T>
T* data(PyObject* o, const char* name, at::ScalarType type, int dev, int64_t numel) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = dense(o, name, type, dev);
  if (t.numel() != numel)
    value_error(std::string(name) + " must have " + std::to_string(numel) + " entries, got " +
                std::to_string(t.numel()));
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(PyObject* o, const char* name, int dev, int64_t numel) {
  return data<int32_t>(o, name, at::kInt, dev, numel);
}

// An int32 matrix of B rows.
int32_t* matrix(PyObject* o, const char* name, int dev, int64_t B, int* width) {
  const at::Tensor& t = dense(o, name, at::kInt, dev);
  if (t.dim() != 2 || t.size(0) != B)
    value_error(std::string(name) + " must be a matrix of " + std::to_string(B) + " rows");
  if (t.size(1) > 0x7fffffffLL) value_error(std::string(name) + " is too wide");
  *width = (int)t.size(1);
  return static_cast<int32_t*>(t.data_ptr());
}

int to_int(int64_t x, const char* name) {
  if (x < -0x80000000LL || x > 0x7fffffffLL) value_error(std::string(name) + " is out of range");
  return (int)x;
}
int to_int(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refusal{nullptr, {}};
  return to_int((int64_t)x, name);
}

// The stride of a dimension that has one: with a single entry it is never
// taken, and torch lets it hold anything.
int64_t step(const at::Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }
bool same_steps(const at::Tensor& a, const at::Tensor& b) {
  for (int64_t i = 0; i < a.dim(); ++i)
    if (step(a, i) != step(b, i)) return false;
  return true;
}

// Caches [num_pages, page_size, heads, head_dim], or [layers, ...] of them.
struct Cache {
  sv_kv_cache c;
  at::ScalarType type;
  int dev;
  int64_t layers, layer_stride;
};
Cache cache(PyObject* ko, PyObject* vo, bool layered) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  const int64_t n = k.dim();
  if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() ||
      k.get_device() != v.get_device() || !(n == 4 || (layered && n == 5)))
    value_error("k_cache and v_cache must be [num_pages, page_size, heads, head_dim] of one "
                "shape, type and device");
  if (!same_steps(k, v) || (k.size(n - 1) > 1 && k.stride(n - 1) != 1))
    value_error("k_cache and v_cache must have the same strides and dense rows");
  Cache r = {};
  r.type = k.scalar_type();
  if (r.type != at::kFloat && r.type != at::kBFloat16)
    type_error(std::string("unsupported dtype ") + c10::toString(r.type));
  r.dev = k.get_device();
  r.layers = n == 5 ? k.size(0) : 1;
  r.layer_stride = n == 5 ? step(k, 0) : 0;
  r.c.k = k.data_ptr();
  r.c.v = v.data_ptr();
  r.c.dtype = r.type == at::kBFloat16 ? SV_BF16 : SV_F32;
  r.c.num_pages = to_int(k.size(n - 4), "num_pages");
  r.c.page_size = to_int(k.size(n - 3), "page_size");
  r.c.heads = to_int(k.size(n - 2), "heads");
  r.c.head_dim = to_int(k.size(n - 1), "head_dim");
  r.c.page_stride = step(k, n - 4);
  r.c.token_stride = step(k, n - 3);
  r.c.head_stride = step(k, n - 2);
  return r;
}

// [B, n, heads, head_dim] with the heads of a token dense.
const at::Tensor& token_rows(PyObject* o, const char* name, const Cache& c, int64_t heads) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 4 || t.size(3) != c.c.head_dim || (heads && t.size(2) != heads))
    value_error(std::string(name) + " must be [B, n, heads, head_dim] matching the cache");
  if (t.scalar_type() != c.type || t.get_device() != c.dev)
    value_error(std::string(name) + " must have the cache's type and device");
  if ((t.size(3) > 1 && t.stride(3) != 1) || (t.size(2) > 1 && t.stride(2) != t.size(3)))
    value_error(std::string("the heads of a token of ") + name + " must be dense");
  return t;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// The output `name` of a dict, allocated if it is not there.
PyObject* output(PyObject* dict, const char* name, at::IntArrayRef shape, at::ScalarType type,
                 int dev) {
  PyObject* o = PyDict_GetItemString(dict, name);  // borrowed
  if (o) return o;
  o = THPVariable_Wrap(
      at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev)));
  if (!o) throw Refusal{nullptr, {}};
  const int rc = PyDict_SetItemString(dict, name, o);
  Py_DECREF(o);  // the dict holds it
  if (rc) throw Refusal{nullptr, {}};
  return o;
}
struct Dict {  // a copy of the caller's, or a new one
  PyObject* d;
  explicit Dict(PyObject* out) : d(out == Py_None ? PyDict_New() : nullptr) {
    if (!d) {
      if (!PyDict_Check(out)) type_error("out must be a dict");
      d = PyDict_Copy(out);
    }
    if (!d) throw Refusal{nullptr, {}};
  }
  ~Dict() { Py_XDECREF(d); }
  PyObject* take(sv_status st) {
    if (st != SV_OK) return PyLong_FromLong(st);
    PyObject* r = d;
    d = nullptr;
    return r;
  }
};

PyObject* do_plan(PyObject* const* a) {
  enum { kLen, kTable, kPages, kFree, kCount, kNew, kMaxNew, kPage, kWritten, kAcc, kRel, kOut,
         kStatus };
  const at::Tensor& len = dense(a[kLen], "kv_len", at::kInt, -1);
  const int dev = len.get_device();
  const int64_t B = len.numel();
  const int max_new = to_int(a[kMaxNew], "max_new"), page = to_int(a[kPage], "page_size");
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  const at::Tensor& free_pages = dense(a[kFree], "free_pages", at::kInt, dev);
  int max_pages = 0;
  int32_t* table = matrix(a[kTable], "block_table", dev, B, &max_pages);
  Dict o(a[kOut]);
  const int64_t slots = B * (max_new < 0 ? 0 : max_new), wide[2] = {B, max_new < 0 ? 0 : max_new};
  const int64_t one = 1;
  const sv_status st = sv_kv_plan(
      static_cast<int32_t*>(len.data_ptr()), ints(a[kWritten], "written", dev, B),
      ints(a[kAcc], "accepted_len", dev, B), ints(a[kRel], "release", dev, B),
      ints(a[kNew], "new_len", dev, B), to_int(B, "B"), max_new, page,
      to_int(free_pages.numel(), "free_pages"), table, max_pages, ints(a[kPages], "pages", dev, B),
      static_cast<int32_t*>(free_pages.data_ptr()), ints(a[kCount], "free_count", dev, 1),
      ints(output(o.d, "kv_len", B, at::kInt, dev), "kv_len", dev, B),
      ints(output(o.d, "pages", B, at::kInt, dev), "pages", dev, B),
      ints(output(o.d, "free_count", one, at::kInt, dev), "free_count", dev, 1),
      ints(output(o.d, "q_len", B, at::kInt, dev), "q_len", dev, B),
      data<int64_t>(output(o.d, "slot_map", wide, at::kLong, dev), "slot_map", at::kLong, dev,
                    slots),
      ints(output(o.d, "positions", wide, at::kInt, dev), "positions", dev, slots),
      ints(a[kStatus], "device_status", dev, 1), stream_of(dev));
  return o.take(st);
}

PyObject* do_append(PyObject* const* a) {
  enum { kK, kV, kSlots, kKc, kVc, kStatus };
  const Cache c = cache(a[kKc], a[kVc], false);
  const at::Tensor& k = token_rows(a[kK], "k", c, c.c.heads);
  const at::Tensor& v = token_rows(a[kV], "v", c, c.c.heads);
  if (k.sizes() != v.sizes() || !same_steps(k, v))
    value_error("k and v must have the same shape and strides");
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
  return PyLong_FromLong(
      sv_kv_append(&c.c, k.data_ptr(), v.data_ptr(), to_int(k.size(0), "B"), to_int(k.size(1), "n"),
                   step(k, 0), step(k, 1),
                   data<int64_t>(a[kSlots], "slot_map", at::kLong, c.dev, k.size(0) * k.size(1)),
                   ints(a[kStatus], "device_status", c.dev, 1), stream_of(c.dev)));
}

PyObject* do_attend(PyObject* const* a) {
  enum { kQ, kKc, kVc, kTable, kLen, kQLen, kParents, kScale, kOut, kScratch, kStatus };
  const Cache c = cache(a[kKc], a[kVc], false);
  const at::Tensor& q = token_rows(a[kQ], "q", c, 0);
  const int64_t B = q.size(0), n = q.size(1), hq = q.size(2), d = q.size(3);
  int max_pages = 0;
  int32_t* table = matrix(a[kTable], "block_table", c.dev, B, &max_pages);
  double scale = 1.0 / std::sqrt((double)d);
  if (a[kScale] != Py_None) {
    scale = PyFloat_AsDouble(a[kScale]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, {}};
  }
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
  Dict o(a[kOut]);
  void* out = data<void>(output(o.d, "out", {B, n, hq, d}, c.type, c.dev), "out", c.type, c.dev,
                         q.numel());
  float* lse = data<float>(output(o.d, "lse", {B, n, hq}, at::kFloat, c.dev), "lse", at::kFloat,
                           c.dev, B * n * hq);
  at::Tensor own;  // the stream keeps what is freed here for its later calls
  if (a[kScratch] == Py_None)
    own = at::empty(
        (int64_t)sv_kv_attend_scratch_size(to_int(B, "B"), to_int(n, "n"), to_int(hq, "q_heads"),
                                           c.c.heads, c.c.head_dim, c.c.dtype),
        at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)c.dev));
  else
    own = dense(a[kScratch], "scratch", at::kByte, c.dev);
  const sv_status st = sv_kv_attend(
      &c.c, q.data_ptr(), step(q, 0), step(q, 1), to_int(B, "B"), to_int(n, "n"),
      to_int(hq, "q_heads"), table, max_pages, ints(a[kLen], "kv_len", c.dev, B),
      ints(a[kQLen], "q_len", c.dev, B), ints(a[kParents], "parents", c.dev, B * n), (float)scale,
      out, lse, own.data_ptr(), (size_t)own.numel(), ints(a[kStatus], "device_status", c.dev, 1),
      stream_of(c.dev));
  return o.take(st);
}

PyObject* do_commit(PyObject* const* a) {
  enum { kKc, kVc, kTable, kLen, kNodes, kAcc, kQLen, kStatus };
  const Cache c = cache(a[kKc], a[kVc], true);
  if (c.layers == 0) return PyLong_FromLong(SV_OK);
  const at::Tensor& len = dense(a[kLen], "kv_len", at::kInt, c.dev);
  const int64_t B = len.numel();
  int max_pages = 0, width = 0;
  int32_t* table = matrix(a[kTable], "block_table", c.dev, B, &max_pages);
  int32_t* nodes = matrix(a[kNodes], "accepted_nodes", c.dev, B, &width);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
  return PyLong_FromLong(sv_kv_commit_ragged(
      &c.c, to_int(c.layers, "layers"), c.layer_stride, to_int(B, "B"), table, max_pages,
      static_cast<int32_t*>(len.data_ptr()), ints(a[kQLen], "q_len", c.dev, B), nodes, width,
      ints(a[kAcc], "accepted_len", c.dev, B), ints(a[kStatus], "device_status", c.dev, 1),
      stream_of(c.dev)));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<do_plan, 13>("plan"), method<do_append, 6>("append"),
                           method<do_attend, 11>("attend"), method<do_commit, 8>("commit"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_svkv", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__svkv() { return PyModule_Create(&g_module); }

// paged_binding.cpp -- the Python side of the paged calls: reads the tensors'
// layouts, allocates outputs and workspace from torch's allocator on the current
// stream of the cache's device, and calls the C entry points of the same name.
//
// A decode step of a small batch takes the GPU a few microseconds, and the same
// checks written in Python took the host 7 (append) to 11 us (decode) a call.
// Like the rest of the binding this only marshals; the C entries validate sizes,
// strides, alignment and overlap.  A status other than ATTN_OK comes back as a
// Python int, and the caller raises it.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "attn.h"

namespace {

// The ctypes structure of PagedKV: the ABI's, and the device it lives on.
struct Cache {
  attn_paged_kv_t kv;
  int device;
};

const Cache* cache_of(PyObject* address) { return static_cast<const Cache*>(PyLong_AsVoidPtr(address)); }

bool is_none(PyObject* o) { return o == Py_None; }

// A strided tensor on the cache's device, or null with the error set.
const at::Tensor* tensor_of(const char* name, PyObject* o, const Cache& c) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.is_cuda() && t.layout() == c10::kStrided && t.get_device() == c.device) return &t;
  }
  PyErr_Format(PyExc_TypeError, "%s must be a tensor on the cache's device", name);
  return nullptr;
}

const char* type_name(c10::ScalarType t) {
  return t == c10::kBFloat16 ? "bf16" : t == c10::kHalf ? "fp16" : t == c10::kFloat ? "float32" : "int32";
}

bool check_type(const char* name, const at::Tensor& t, c10::ScalarType want) {
  if (t.scalar_type() == want) return true;
  PyErr_Format(PyExc_TypeError, "%s must be %s", name, type_name(want));
  return false;
}

// Element type code of new rows: the cache's own type, or either for e4m3; -1 with the error set.
int x_type_of(const Cache& c, const at::Tensor& t) {
  const int x = t.scalar_type() == c10::kBFloat16 ? ATTN_TYPE_BF16 : t.scalar_type() == c10::kHalf ? ATTN_TYPE_F16 : -1;
  if (x >= 0 && (c.kv.type == ATTN_TYPE_E4M3 || c.kv.type == x)) return x;
  PyErr_SetString(PyExc_TypeError, c.kv.type == ATTN_TYPE_E4M3 ? "an e4m3 cache takes bf16 or fp16 rows"
                                                               : "the cache takes rows of its own type");
  return -1;
}

// [rows, heads, d] with contiguous channels; rows or heads < 0: any.
bool rows_of(const char* name, const at::Tensor& t, const Cache& c, int64_t heads, int64_t rows, attn_rows_t* out) {
  if (t.dim() == 3 && t.size(2) == c.kv.head_dim && t.stride(2) == 1 && (rows < 0 || t.size(0) == rows) &&
      (heads < 0 || t.size(1) == heads) && t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX) {
    *out = {t.data_ptr(), t.stride(0), t.stride(1)};
    return true;
  }
  PyErr_Format(PyExc_ValueError, "%s must be [%s, %s, %d] with contiguous channels", name,
               rows < 0 ? "rows" : std::to_string(rows).c_str(), heads < 0 ? "heads" : std::to_string(heads).c_str(),
               c.kv.head_dim);
  return false;
}

at::Tensor empty(const Cache& c, c10::IntArrayRef size, c10::ScalarType type) {
  return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)), std::nullopt);
}

// Device memory for one call; it goes back to the pool of the call's stream.
c10::DataPtr scratch(int64_t bytes) {
  return bytes > 0 ? c10::cuda::CUDACachingAllocator::get()->allocate(static_cast<size_t>(bytes)) : c10::DataPtr();
}

bool args_are(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// (cache, k, v, q, q_out, token_start, cos, sin, interleaved) -> q_out
PyObject* paged_append(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!args_are(nargs, 9)) return nullptr;
  const Cache& c = *cache_of(arg[0]);
  const at::Tensor *k = tensor_of("k", arg[1], c), *v = k ? tensor_of("v", arg[2], c) : nullptr;
  if (!v) return nullptr;
  const int x = x_type_of(c, *k);
  attn_rows_t rk, rv, rq, ro;
  if (x < 0 || !check_type("v", *v, k->scalar_type()) || !rows_of("k", *k, c, c.kv.kv_heads, -1, &rk)) return nullptr;
  const int64_t rows = k->size(0);
  if (!rows_of("v", *v, c, c.kv.kv_heads, rows, &rv)) return nullptr;
  const int* start = nullptr;
  if (!is_none(arg[5])) {
    const at::Tensor* t = tensor_of("token_start", arg[5], c);
    if (!t) return nullptr;
    if (t->scalar_type() != c10::kInt || t->dim() != 1 || t->size(0) != c.kv.B + 1 || !t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "token_start must be a contiguous int32 [%d] on the cache's device", c.kv.B + 1);
      return nullptr;
    }
    start = static_cast<const int*>(t->data_ptr());
  } else if (rows != c.kv.B) {
    PyErr_Format(PyExc_ValueError, "without token_start k and v must have one row per sequence (%d)", c.kv.B);
    return nullptr;
  }
  const float *cos = nullptr, *sin = nullptr;
  int table_rows = 0, rot = 0;
  if (!is_none(arg[6]) || !is_none(arg[7])) {
    if (is_none(arg[6]) || is_none(arg[7])) {
      PyErr_SetString(PyExc_ValueError, "cos and sin come together");
      return nullptr;
    }
    const at::Tensor *a = tensor_of("cos", arg[6], c), *b = a ? tensor_of("sin", arg[7], c) : nullptr;
    if (!b || !check_type("cos", *a, c10::kFloat) || !check_type("sin", *b, c10::kFloat)) return nullptr;
    if (a->dim() != 2 || !a->is_contiguous() || !b->is_contiguous() || a->sizes() != b->sizes() ||
        a->size(0) > INT32_MAX || a->size(1) > INT32_MAX / 2) {
      PyErr_SetString(PyExc_ValueError, "cos and sin must be contiguous [positions, rot_dim / 2] of one shape");
      return nullptr;
    }
    cos = static_cast<const float*>(a->data_ptr()), sin = static_cast<const float*>(b->data_ptr());
    table_rows = static_cast<int>(a->size(0)), rot = static_cast<int>(2 * a->size(1));
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  const at::Tensor* q = nullptr;
  at::Tensor made;
  int heads = 0;
  if (!is_none(arg[3])) {
    if (!(q = tensor_of("q", arg[3], c)) || !check_type("q", *q, k->scalar_type()) || !rows_of("q", *q, c, -1, rows, &rq))
      return nullptr;
    heads = static_cast<int>(q->size(1));
    const at::Tensor* out = &made;
    if (is_none(arg[4])) made = empty(c, q->sizes(), q->scalar_type());
    else if (!(out = tensor_of("q_out", arg[4], c)) || !check_type("q_out", *out, k->scalar_type())) return nullptr;
    if (!rows_of("q_out", *out, c, heads, rows, &ro)) return nullptr;
  } else if (!is_none(arg[4])) {
    PyErr_SetString(PyExc_ValueError, "q_out without q");
    return nullptr;
  }
  const int interleaved = PyObject_IsTrue(arg[8]);
  if (interleaved < 0) return nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_paged_append(&c.kv, &rk, &rv, q ? &rq : nullptr, q ? &ro : nullptr, heads, static_cast<int>(rows), start, cos,
                         sin, table_rows, rot, interleaved, x, stream);
  Py_END_ALLOW_THREADS
  if (rc) return PyLong_FromLong(rc);
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(arg[4]);
  return arg[4];
  END_HANDLE_TH_ERRORS
}

// A contiguous int32 [B, kv_heads, n] list of pages; n or -1 with the error set.
int64_t pages_of(PyObject* o, const Cache& c, const int** p) {
  const at::Tensor* t = tensor_of("pages", o, c);
  if (!t) return -1;
  if (t->scalar_type() != c10::kInt || t->dim() != 3 || t->size(0) != c.kv.B || t->size(1) != c.kv.kv_heads ||
      t->size(2) < 1 || t->size(2) > INT32_MAX || !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "pages must be a contiguous int32 [%d, %d, n >= 1] on the cache's device", c.kv.B,
                 c.kv.kv_heads);
    return -1;
  }
  *p = static_cast<const int*>(t->data_ptr());
  return t->size(2);
}

// (cache, q, pages, scale, o, lse) -> (o, lse)
PyObject* paged_decode(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!args_are(nargs, 6)) return nullptr;
  const Cache& c = *cache_of(arg[0]);
  const at::Tensor* q = tensor_of("q", arg[1], c);
  if (!q) return nullptr;
  const int x = x_type_of(c, *q);
  attn_rows_t rq;
  if (x < 0 || !rows_of("q", *q, c, -1, c.kv.B, &rq)) return nullptr;
  const int heads = static_cast<int>(q->size(1));
  const int* pages = nullptr;
  int64_t n = 0;
  if (!is_none(arg[2]) && (n = pages_of(arg[2], c, &pages)) < 0) return nullptr;
  double scale = 1.0 / std::sqrt(static_cast<double>(c.kv.head_dim));
  if (!is_none(arg[3])) {
    scale = PyFloat_AsDouble(arg[3]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  at::Tensor o, lse;
  if (is_none(arg[4])) {
    o = empty(c, q->sizes(), q->scalar_type());
  } else {
    const at::Tensor* t = tensor_of("o", arg[4], c);
    if (!t || !check_type("o", *t, q->scalar_type())) return nullptr;
    if (t->sizes() != q->sizes() || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "o must be contiguous and have q's shape");
      return nullptr;
    }
    o = *t;
  }
  if (is_none(arg[5])) {
    lse = empty(c, {c.kv.B, heads}, c10::kFloat);
  } else {
    const at::Tensor* t = tensor_of("lse", arg[5], c);
    if (!t || !check_type("lse", *t, c10::kFloat)) return nullptr;
    if (t->dim() != 2 || t->size(0) != c.kv.B || t->size(1) != heads || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "lse must be a contiguous [B, q_heads]");
      return nullptr;
    }
    lse = *t;
  }
  const c10::DataPtr ws = scratch(attn_paged_decode_workspace(&c.kv, heads, static_cast<int>(n)));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  void *po = o.data_ptr(), *pl = lse.data_ptr();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_paged_decode(&c.kv, &rq, heads, po, static_cast<float*>(pl), pages, static_cast<int>(n),
                         static_cast<float>(scale), x, ws.get(), stream);
  Py_END_ALLOW_THREADS
  if (rc) return PyLong_FromLong(rc);
  PyObject* result = PyTuple_New(2);
  if (!result) return nullptr;
  for (int i = 0; i < 2; ++i) {
    PyObject* t = arg[4 + i];
    if (is_none(t)) t = THPVariable_Wrap(i ? lse : o);
    else Py_INCREF(t);
    if (!t) {
      Py_DECREF(result);
      return nullptr;
    }
    PyTuple_SET_ITEM(result, i, t);
  }
  return result;
  END_HANDLE_TH_ERRORS
}

// (cache, q, n_select, keep_first, keep_last, pages) -> pages
PyObject* paged_select(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!args_are(nargs, 6)) return nullptr;
  const Cache& c = *cache_of(arg[0]);
  const at::Tensor* q = tensor_of("q", arg[1], c);
  if (!q) return nullptr;
  const int x = x_type_of(c, *q);
  attn_rows_t rq;
  if (x < 0 || !rows_of("q", *q, c, -1, c.kv.B, &rq)) return nullptr;
  long want[3];  // n_select, keep_first, keep_last
  for (int i = 0; i < 3; ++i) {
    want[i] = PyLong_AsLong(arg[2 + i]);
    if (want[i] == -1 && PyErr_Occurred()) return nullptr;
  }
  if (want[0] < 1 || want[0] > INT32_MAX || want[1] < 0 || want[2] < 0 || want[1] > want[0] || want[2] > want[0] - want[1]) {
    PyErr_SetString(PyExc_ValueError, "n_select must be at least 1 and keep_first + keep_last, both at least 0");
    return nullptr;
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  at::Tensor made;
  const int* pages = nullptr;
  if (is_none(arg[5])) {
    made = empty(c, {c.kv.B, c.kv.kv_heads, want[0]}, c10::kInt);
    pages = static_cast<const int*>(made.data_ptr());
  } else {
    const int64_t n = pages_of(arg[5], c, &pages);
    if (n < 0) return nullptr;
    if (n != want[0]) {
      PyErr_SetString(PyExc_ValueError, "pages must be [B, kv_heads, n_select]");
      return nullptr;
    }
  }
  const c10::DataPtr ws = scratch(attn_paged_select_workspace(&c.kv));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_paged_select(&c.kv, &rq, static_cast<int>(q->size(1)), const_cast<int*>(pages), static_cast<int>(want[0]),
                         static_cast<int>(want[1]), static_cast<int>(want[2]), x, ws.get(), stream);
  Py_END_ALLOW_THREADS
  if (rc) return PyLong_FromLong(rc);
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(arg[5]);
  return arg[5];
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_decode)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_select)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", "Marshalling of the paged calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }

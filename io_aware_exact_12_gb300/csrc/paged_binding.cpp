// paged_binding.cpp -- the Python side of the paged and windowed calls: reads the
// tensors' layouts, allocates outputs and workspace from torch's allocator on the
// current stream of the cache's (windowed: q's) device, and calls the C entry
// points of the same name.
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

// A count of tokens, cut to what the sizes of the library can mean; -1 with the error set.
int64_t count_of(const char* name, PyObject* o, int64_t least) {
  int overflow = 0;
  const long long n = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (n == -1 && !overflow && PyErr_Occurred()) return -1;
  if (overflow < 0 || (!overflow && n < least)) {
    PyErr_Format(PyExc_ValueError, "%s must be at least %d", name, static_cast<int>(least));
    return -1;
  }
  return overflow || n > (1 << 30) ? 1 << 30 : n;
}

bool scale_of(PyObject* o, int64_t d, double* scale) {
  *scale = is_none(o) ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(o);
  return is_none(o) || *scale != -1.0 || !PyErr_Occurred();
}

PyObject* decode_any(PyObject* const* arg, Py_ssize_t at, bool windowed);

// (cache, q, pages, scale, o, lse) -> (o, lse)
PyObject* paged_decode(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return args_are(nargs, 6) ? decode_any(arg, 3, false) : nullptr;
}

// (cache, q, window, sinks, scale, o, lse) -> (o, lse)
PyObject* paged_decode_window(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  return args_are(nargs, 7) ? decode_any(arg, 4, true) : nullptr;
}

// scale, o and lse are the arguments from `at` on.
PyObject* decode_any(PyObject* const* arg, Py_ssize_t at, bool windowed) {
  HANDLE_TH_ERRORS
  const Cache& c = *cache_of(arg[0]);
  const at::Tensor* q = tensor_of("q", arg[1], c);
  if (!q) return nullptr;
  const int x = x_type_of(c, *q);
  attn_rows_t rq;
  if (x < 0 || !rows_of("q", *q, c, -1, c.kv.B, &rq)) return nullptr;
  const int heads = static_cast<int>(q->size(1));
  const int* pages = nullptr;
  int64_t n = 0;
  int64_t window = 0, sinks = 0;
  if (windowed) {
    if ((window = count_of("window", arg[2], 1)) < 0 || (sinks = count_of("sinks", arg[3], 0)) < 0) return nullptr;
  } else if (!is_none(arg[2]) && (n = pages_of(arg[2], c, &pages)) < 0) {
    return nullptr;
  }
  double scale;
  if (!scale_of(arg[at], c.kv.head_dim, &scale)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  at::Tensor o, lse;
  if (is_none(arg[at + 1])) {
    o = empty(c, q->sizes(), q->scalar_type());
  } else {
    const at::Tensor* t = tensor_of("o", arg[at + 1], c);
    if (!t || !check_type("o", *t, q->scalar_type())) return nullptr;
    if (t->sizes() != q->sizes() || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "o must be contiguous and have q's shape");
      return nullptr;
    }
    o = *t;
  }
  if (is_none(arg[at + 2])) {
    lse = empty(c, {c.kv.B, heads}, c10::kFloat);
  } else {
    const at::Tensor* t = tensor_of("lse", arg[at + 2], c);
    if (!t || !check_type("lse", *t, c10::kFloat)) return nullptr;
    if (t->dim() != 2 || t->size(0) != c.kv.B || t->size(1) != heads || !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "lse must be a contiguous [B, q_heads]");
      return nullptr;
    }
    lse = *t;
  }
  const c10::DataPtr ws = scratch(windowed ? attn_paged_decode_window_workspace(&c.kv, heads, static_cast<int>(window), static_cast<int>(sinks))
                                           : attn_paged_decode_workspace(&c.kv, heads, static_cast<int>(n)));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  void *po = o.data_ptr(), *pl = lse.data_ptr();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = windowed ? attn_paged_decode_window(&c.kv, &rq, heads, po, static_cast<float*>(pl), static_cast<int>(window),
                                           static_cast<int>(sinks), static_cast<float>(scale), x, ws.get(), stream)
                : attn_paged_decode(&c.kv, &rq, heads, po, static_cast<float*>(pl), pages, static_cast<int>(n),
                                    static_cast<float>(scale), x, ws.get(), stream);
  Py_END_ALLOW_THREADS
  if (rc) return PyLong_FromLong(rc);
  PyObject* result = PyTuple_New(2);
  if (!result) return nullptr;
  for (int i = 0; i < 2; ++i) {
    PyObject* t = arg[at + 1 + i];
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

// A contiguous tensor of integers [n], n < 0: of any size above 0; null with the error set.
const at::Tensor* ints_of(const char* name, PyObject* o, const Cache& c, int64_t n, c10::ScalarType type = c10::kInt) {
  const at::Tensor* t = tensor_of(name, o, c);
  if (!t) return nullptr;
  if (t->scalar_type() == type && t->dim() == 1 && t->is_contiguous() && (n < 0 ? t->size(0) > 0 && t->size(0) <= INT32_MAX : t->size(0) == n))
    return t;
  PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s [%s] on the cache's device", name, type == c10::kInt ? "int32" : "int64",
               n < 0 ? "n" : std::to_string(n).c_str());
  return nullptr;
}

// (cache, n_new, free_pages, free_state, lens, free_out, token_start, slots, rows, window, sinks) -> token_start
PyObject* paged_assign(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!args_are(nargs, 11)) return nullptr;
  const Cache& c = *cache_of(arg[0]);
  const at::Tensor *n_new = ints_of("n_new", arg[1], c, c.kv.B), *ring = n_new ? ints_of("free_pages", arg[2], c, -1) : nullptr;
  const at::Tensor* state = ring ? ints_of("free_state", arg[3], c, 2) : nullptr;
  if (!state) return nullptr;
  const at::Tensor *lens = nullptr, *out = nullptr, *slots = nullptr, *start = nullptr;
  if (!is_none(arg[4]) && !(lens = ints_of("lens", arg[4], c, c.kv.B))) return nullptr;
  if (!is_none(arg[5]) && !(out = ints_of("free_out", arg[5], c, 2))) return nullptr;
  if (!is_none(arg[6]) && !(start = ints_of("token_start", arg[6], c, static_cast<int64_t>(c.kv.B) + 1))) return nullptr;
  int64_t rows = c.kv.B;
  if (!is_none(arg[8]) && (rows = count_of("rows", arg[8], 0)) < 0) return nullptr;
  if (!is_none(arg[7])) {
    if (!THPVariable_Check(arg[7])) return tensor_of("slots", arg[7], c), nullptr;
    const int64_t n = THPVariable_Unpack(arg[7]).numel();
    if (!(slots = ints_of("slots", arg[7], c, n, c10::kLong))) return nullptr;
    if (!is_none(arg[8]) && rows != n) {
      PyErr_SetString(PyExc_ValueError, "rows must be the size of slots");
      return nullptr;
    }
    rows = std::min<int64_t>(n, INT32_MAX);  // the entry refuses what is too many
  }
  const int64_t window = count_of("window", arg[9], 0), sinks = window < 0 ? -1 : count_of("sinks", arg[10], 0);
  if (sinks < 0) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  at::Tensor made;
  if (!start) made = empty(c, {static_cast<int64_t>(c.kv.B) + 1}, c10::kInt), start = &made;
  const c10::DataPtr ws = scratch(attn_paged_assign_workspace(&c.kv));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  auto ptr = [](const at::Tensor* t) { return t ? static_cast<int*>(t->data_ptr()) : nullptr; };
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_paged_assign(&c.kv, ptr(n_new), ptr(lens), ptr(ring), static_cast<int>(ring->size(0)), ptr(state), ptr(out), ptr(start),
                         slots ? static_cast<long long*>(slots->data_ptr()) : nullptr, static_cast<int>(rows),
                         static_cast<int>(window), static_cast<int>(sinks), ws.get(), stream);
  Py_END_ALLOW_THREADS
  if (rc) return PyLong_FromLong(rc);
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(arg[6]);
  return arg[6];
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ sliding window

// A CUDA tensor [B, heads, N, d] with contiguous channels, of q's type and device (q itself: null `like`).
const at::Tensor* bhnd_of(const char* name, PyObject* o, const at::Tensor* like, attn_bhnd_t* out) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != c10::kStrided) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return nullptr;
  }
  if (!like && t.scalar_type() != c10::kBFloat16 && t.scalar_type() != c10::kHalf) {
    PyErr_Format(PyExc_TypeError, "%s must be bf16 or fp16", name);
    return nullptr;
  }
  if (like && t.scalar_type() != like->scalar_type()) return check_type(name, t, like->scalar_type()), nullptr;
  if (like && t.device() != like->device()) {
    PyErr_Format(PyExc_ValueError, "%s must be on q's device", name);
    return nullptr;
  }
  bool fits = t.dim() == 4 && (t.size(3) == 1 || t.stride(3) == 1);
  for (int i = 0; fits && i < 4; ++i) fits = t.size(i) >= 1 && t.size(i) <= INT32_MAX;
  if (!fits) {
    PyErr_Format(PyExc_ValueError, "%s must be [B, heads, N, d] with contiguous channels", name);
    return nullptr;
  }
  *out = {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
  return &t;
}

bool same_sizes(const char* name, const at::Tensor& t, const at::Tensor& want, const char* whose) {
  if (t.sizes() == want.sizes()) return true;
  PyErr_Format(PyExc_ValueError, "%s must have %s's shape", name, whose);
  return false;
}

// A tensor of t's shape and type, dense, in t's order of positions and heads.
at::Tensor like_of(const at::Tensor& t, attn_bhnd_t* out) {
  const c10::Device dev = t.device();
  at::Tensor r;
  if (t.stride(2) > t.stride(1) && t.size(1) > 1) {
    const int64_t row = t.size(1) * t.size(3);
    r = at::detail::empty_strided_cuda(t.sizes(), {t.size(2) * row, t.size(3), row, 1}, t.scalar_type(), dev);
  } else {
    r = at::detail::empty_cuda(t.sizes(), t.scalar_type(), dev, std::nullopt);
  }
  *out = {r.data_ptr(), r.stride(0), r.stride(1), r.stride(2)};
  return r;
}

// What both passes take: q, k, v, their sizes, the window.
struct Window {
  const at::Tensor *q, *k, *v;
  attn_bhnd_t rq, rk, rv;
  int B, Hq, Hk, Nq, Nk, d, window, sinks, type;
  double scale;
};

bool window_of(PyObject* q, PyObject* k, PyObject* v, PyObject* window, PyObject* sinks, PyObject* scale, Window* w) {
  if (!(w->q = bhnd_of("q", q, nullptr, &w->rq)) || !(w->k = bhnd_of("k", k, w->q, &w->rk)) || !(w->v = bhnd_of("v", v, w->q, &w->rv))) return false;
  auto at = [](const at::Tensor* t, int i) { return static_cast<int>(t->size(i)); };
  if (at(w->k, 0) != at(w->q, 0) || at(w->k, 3) != at(w->q, 3) || at(w->q, 1) % at(w->k, 1) || at(w->k, 2) < at(w->q, 2)) {
    PyErr_SetString(PyExc_ValueError, "k must be [B, kv_heads, Nk, d] with q's B and d, kv_heads a divisor of its heads and Nk >= its N");
    return false;
  }
  if (!same_sizes("v", *w->v, *w->k, "k")) return false;
  const int64_t n = count_of("window", window, 1), s = n < 0 ? -1 : count_of("sinks", sinks, 0);
  if (s < 0 || !scale_of(scale, at(w->q, 3), &w->scale)) return false;
  w->B = at(w->q, 0), w->Hq = at(w->q, 1), w->Hk = at(w->k, 1), w->Nq = at(w->q, 2), w->Nk = at(w->k, 2), w->d = at(w->q, 3);
  w->window = static_cast<int>(n), w->sinks = static_cast<int>(s);
  w->type = w->q->scalar_type() == c10::kBFloat16 ? ATTN_TYPE_BF16 : ATTN_TYPE_F16;
  return true;
}

const at::Tensor* row_stats(PyObject* o, const Window& w) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.device() == w.q->device() && t.scalar_type() == c10::kFloat && t.is_contiguous() && t.dim() == 3 && t.size(0) == w.B &&
        t.size(1) == w.Hq && t.size(2) == w.Nq)
      return &t;
  }
  PyErr_SetString(PyExc_ValueError, "lse must be a contiguous float32 [B, q_heads, Nq] on q's device");
  return nullptr;
}

// The call's outputs as a tuple: those that came in, and those that were made.
PyObject* outputs(PyObject* const* given, at::Tensor* made, int n) {
  PyObject* result = PyTuple_New(n);
  if (!result) return nullptr;
  for (int i = 0; i < n; ++i) {
    PyObject* t = given[i];
    if (is_none(t)) t = THPVariable_Wrap(made[i]);
    else Py_INCREF(t);
    if (!t) {
      Py_DECREF(result);
      return nullptr;
    }
    PyTuple_SET_ITEM(result, i, t);
  }
  return result;
}

// (q, k, v, window, sinks, scale, o, lse) -> (o, lse)
PyObject* fwd_window(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  Window w;
  if (!args_are(nargs, 8) || !window_of(arg[0], arg[1], arg[2], arg[3], arg[4], arg[5], &w)) return nullptr;
  const c10::cuda::CUDAGuard guard(w.q->device());
  at::Tensor made[2];
  attn_bhnd_t ro;
  const at::Tensor* lse = &made[1];
  if (is_none(arg[6])) {
    made[0] = like_of(*w.q, &ro);
  } else {
    const at::Tensor* t = bhnd_of("o", arg[6], w.q, &ro);
    if (!t || !same_sizes("o", *t, *w.q, "q")) return nullptr;
  }
  if (is_none(arg[7])) made[1] = at::detail::empty_cuda({w.B, w.Hq, w.Nq}, c10::kFloat, w.q->device(), std::nullopt);
  else if (!(lse = row_stats(arg[7], w))) return nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream(w.q->get_device()).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_fwd_window(&w.rq, &w.rk, &w.rv, &ro, static_cast<float*>(lse->data_ptr()), w.B, w.Hq, w.Hk, w.Nq, w.Nk, w.d, w.window,
                       w.sinks, static_cast<float>(w.scale), w.type, stream);
  Py_END_ALLOW_THREADS
  return rc ? PyLong_FromLong(rc) : outputs(arg + 6, made, 2);
  END_HANDLE_TH_ERRORS
}

// (q, k, v, o, do, lse, window, sinks, scale, dq, dk, dv) -> (dq, dk, dv)
PyObject* bwd_window(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  Window w;
  if (!args_are(nargs, 12) || !window_of(arg[0], arg[1], arg[2], arg[6], arg[7], arg[8], &w)) return nullptr;
  attn_bhnd_t ro, rdo, rd[3];
  const at::Tensor *o = bhnd_of("o", arg[3], w.q, &ro), *dO = o ? bhnd_of("do", arg[4], w.q, &rdo) : nullptr;
  if (!dO || !same_sizes("o", *o, *w.q, "q") || !same_sizes("do", *dO, *w.q, "q")) return nullptr;
  const at::Tensor* lse = row_stats(arg[5], w);
  if (!lse) return nullptr;
  const c10::cuda::CUDAGuard guard(w.q->device());
  at::Tensor made[3];
  const char* const names[3] = {"dq", "dk", "dv"};
  for (int i = 0; i < 3; ++i) {
    const at::Tensor& like = i == 0 ? *w.q : i == 1 ? *w.k : *w.v;
    if (is_none(arg[9 + i])) {
      made[i] = like_of(like, &rd[i]);
    } else {
      const at::Tensor* t = bhnd_of(names[i], arg[9 + i], w.q, &rd[i]);
      if (!t || !same_sizes(names[i], *t, like, i ? "k" : "q")) return nullptr;
    }
  }
  const c10::DataPtr ws = scratch(attn_bwd_window_workspace(w.B, w.Hq, w.Hk, w.Nq, w.Nk, w.d, w.window, w.sinks));
  void* stream = c10::cuda::getCurrentCUDAStream(w.q->get_device()).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attn_bwd_window(&w.rq, &w.rk, &w.rv, &ro, &rdo, static_cast<const float*>(lse->data_ptr()), &rd[0], &rd[1], &rd[2], w.B, w.Hq,
                       w.Hk, w.Nq, w.Nk, w.d, w.window, w.sinks, static_cast<float>(w.scale), w.type, ws.get(), stream);
  Py_END_ALLOW_THREADS
  return rc ? PyLong_FromLong(rc) : outputs(arg + 9, made, 3);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_decode)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_select)), METH_FASTCALL, nullptr},
    {"decode_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_decode_window)), METH_FASTCALL, nullptr},
    {"assign", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_assign)), METH_FASTCALL, nullptr},
    {"fwd_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fwd_window)), METH_FASTCALL, nullptr},
    {"bwd_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bwd_window)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", "Marshalling of the paged and windowed calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }

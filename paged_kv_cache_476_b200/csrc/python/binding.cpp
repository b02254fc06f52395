// The common case of the rotation and shared-prefix calls, straight from Python's
// arguments to the C ABI: a decode step's calls are a few microseconds on the GPU,
// and the checks and ctypes conversions in Python took 15 to 20.
//
// Each function takes what the wrapper of the same name has been given, for
// results that the call allocates, on the current stream and device.  It returns
// NotImplemented for everything it does not find in order (an argument to
// refuse, another device, a status of the host's checks), without having launched
// anything: the wrapper then goes the long way, which says what is wrong.  A CUDA
// error may come behind a launch, so it is raised here and nothing is done twice;
// for the same reason the results are whole Python objects before the call.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "paged_kv.h"

namespace {

decltype(&pkv_qk_norm_rope) c_norm_rope;
decltype(&paged_kv_append_rope) c_append_rope;
decltype(&paged_decode_attention_shared) c_shared;
PyObject* error_class;  // PagedKVError(what, status)

PyObject* not_handled() { Py_RETURN_NOTIMPLEMENTED; }

// The tensor behind `o` where it is a plain one of this kind on device `dev`.
const at::Tensor* tensor(PyObject* o, int dev, at::ScalarType type, int dims) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != dims)
    return nullptr;
  return &t;
}

const at::Tensor* ints(PyObject* o, int dev, int dims) {
  const at::Tensor* t = tensor(o, dev, at::kInt, dims);
  return t && t->is_contiguous() ? t : nullptr;
}

// Rows [tokens][heads][head_dim] whose tokens may lie apart.
struct Rows {
  const at::Tensor* t = nullptr;
  int64_t tokens = 0, heads = 0, dim = 0, stride = 0;
  bool from(PyObject* o, int dev) {
    t = tensor(o, dev, at::kBFloat16, 3);
    if (!t) return false;
    tokens = t->size(0), heads = t->size(1), dim = t->size(2);
    if ((dim > 1 && t->stride(2) != 1) || (heads > 1 && t->stride(1) != dim)) return false;
    stride = tokens > 1 ? t->stride(0) : heads * dim;
    return true;
  }
  void* data() const { return t ? t->data_ptr() : nullptr; }
};

// (address of the C struct, device, head_dim its weights want or 0, has a table)
struct RopeArgs {
  const pkv_rope* rope;
  int dev, dim, table;
  bool from(PyObject* o) {
    if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 4) return false;
    rope = static_cast<const pkv_rope*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
    dev = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 1));
    dim = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 2));
    table = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 3));
    return rope != nullptr;
  }
  bool fits(int device, int64_t head_dim) const {
    return (dev < 0 || dev == device) && (dim == 0 || dim == head_dim);
  }
};

// (address of the C struct, device)
struct CacheArgs {
  const pkv_cache* cache;
  int dev;
  bool from(PyObject* o) {
    if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 2) return false;
    cache = static_cast<const pkv_cache*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
    dev = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 1));
    return cache != nullptr && dev == c10::cuda::current_device();
  }
};

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

// An object that goes with its owner unless it is released as the result.
struct Result {
  PyObject* o = nullptr;
  explicit Result(PyObject* x) : o(x) {}
  ~Result() { Py_XDECREF(o); }
  PyObject* release() {
    PyObject* x = o;
    o = nullptr;
    return x;
  }
};

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

PyObject* wrap2(const at::Tensor& a, const at::Tensor& b) {
  Result x(wrap(a)), y(wrap(b));
  return x.o && y.o ? PyTuple_Pack(2, x.o, y.o) : nullptr;
}

// The call's answer, by its status.
PyObject* answer(const char* what, int status, Result& result) {
  if (status == PKV_OK) return result.release();
  if (status != PKV_ERR_CUDA) return not_handled();  // nothing was launched
  PyObject* e = PyObject_CallFunction(error_class, "si", what, status);
  if (e) PyErr_SetObject(error_class, e);
  Py_XDECREF(e);
  return nullptr;
}

at::Tensor like(const at::Tensor& t, at::IntArrayRef sizes) { return at::empty(sizes, t.options()); }

// rope, q, k, positions, error_flags
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  RopeArgs r;
  if (n != 5 || !r.from(a[0])) return not_handled();
  const int dev = c10::cuda::current_device();
  Rows q, k;
  if (a[1] != Py_None && !q.from(a[1], dev)) return not_handled();
  if (a[2] != Py_None && !k.from(a[2], dev)) return not_handled();
  const Rows& x = q.t ? q : k;
  if (!x.t || !r.fits(dev, x.dim)) return not_handled();
  if (q.t && k.t && (q.tokens != k.tokens || q.dim != k.dim)) return not_handled();
  if (x.tokens > INT32_MAX || q.heads > INT32_MAX || k.heads > INT32_MAX) return not_handled();
  const at::Tensor* pos = nullptr;
  if (a[3] != Py_None) {
    pos = ints(a[3], dev, 1);
    if (!pos || pos->size(0) != x.tokens) return not_handled();
  } else if (r.table) {
    return not_handled();
  }
  const at::Tensor* flags = nullptr;
  if (a[4] != Py_None) {
    if (!THPVariable_CheckExact(a[4])) return not_handled();
    flags = ints(a[4], dev, (int)THPVariable_Unpack(a[4]).dim());
    if (!flags) return not_handled();
  }
  at::Tensor qo, ko;
  if (q.t) qo = like(*q.t, q.t->sizes());
  if (k.t) ko = like(*k.t, k.t->sizes());
  Result out(wrap2(qo, ko));
  if (!out.o) return nullptr;
  const int st = c_norm_rope(
      r.rope, q.data(), q.stride, (int32_t)q.heads, k.data(), k.stride, (int32_t)k.heads,
      (int32_t)x.dim, pos ? pos->data_ptr<int32_t>() : nullptr, (int32_t)x.tokens,
      q.t ? qo.data_ptr() : nullptr, k.t ? ko.data_ptr() : nullptr,
      flags ? flags->data_ptr<int32_t>() : nullptr, stream_of(dev));
  return answer("pkv_qk_norm_rope", st, out);
}

// cache, rope, page_table, seq_lens_before, cu_new_tokens, k_new, v_new, q, positions,
// total_new_tokens
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CacheArgs c;
  RopeArgs r;
  if (n != 10 || !c.from(a[0]) || !r.from(a[1])) return not_handled();
  const int dev = c.dev;
  const at::Tensor *table = ints(a[2], dev, 2), *before = ints(a[3], dev, 1),
                   *cu = ints(a[4], dev, 1);
  Rows k, v, q;
  if (!table || !before || !cu || !k.from(a[5], dev) || !v.from(a[6], dev)) return not_handled();
  if (a[7] != Py_None && !q.from(a[7], dev)) return not_handled();
  const int64_t batch = before->size(0);
  int64_t total = k.tokens;
  if (a[9] != Py_None) {
    if (!PyLong_CheckExact(a[9])) return not_handled();
    total = PyLong_AsLongLong(a[9]);
    if (total == -1 && PyErr_Occurred()) PyErr_Clear();
  }
  if (k.tokens != v.tokens || k.heads != v.heads || k.dim != v.dim ||
      k.heads != c.cache->num_kv_heads || k.dim != c.cache->head_dim || !r.fits(dev, k.dim) ||
      table->size(0) != batch || cu->size(0) != batch + 1 || total < 0 || total > k.tokens ||
      total > INT32_MAX || (q.t && (q.tokens < total || q.dim != k.dim)))
    return not_handled();
  const at::Tensor* pos = nullptr;
  if (a[8] != Py_None) {
    pos = ints(a[8], dev, 1);
    if (!pos || pos->size(0) < total) return not_handled();
  }
  at::Tensor out;
  if (q.t) out = like(*q.t, q.t->sizes());
  Result result(wrap(out));
  if (!result.o) return nullptr;
  const int st = c_append_rope(
      c.cache, r.rope, table->data_ptr<int32_t>(), (int32_t)table->size(1),
      before->data_ptr<int32_t>(), cu->data_ptr<int32_t>(), (int32_t)batch, (int32_t)total,
      k.data(), k.stride, v.data(), v.stride, q.data(), q.stride, (int32_t)q.heads,
      q.t ? out.data_ptr() : nullptr, pos ? pos->data_ptr<int32_t>() : nullptr, stream_of(dev));
  return answer("paged_kv_append_rope", st, result);
}

// cache, q, page_table, seq_lens, max_seq_len, cu_groups, prefix_lens, softmax_scale,
// workspace, want_lse
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CacheArgs c;
  if (n != 10 || !c.from(a[0])) return not_handled();
  const int dev = c.dev;
  const at::Tensor* q = tensor(a[1], dev, at::kBFloat16, 3);
  const at::Tensor *table = ints(a[2], dev, 2), *lens = ints(a[3], dev, 1),
                   *cu = ints(a[5], dev, 1), *prefix = ints(a[6], dev, 1);
  if (!q || !q->is_contiguous() || !table || !lens || !cu || !prefix) return not_handled();
  if (!PyLong_CheckExact(a[4]) || !THPVariable_CheckExact(a[8])) return not_handled();
  const at::Tensor& work = THPVariable_Unpack(a[8]);
  if (!work.is_cuda() || work.get_device() != dev || !work.is_contiguous()) return not_handled();
  const int64_t batch = q->size(0), heads = q->size(1), dim = q->size(2);
  const int64_t groups = prefix->size(0);
  const long long max_len = PyLong_AsLongLong(a[4]);
  if (max_len == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return not_handled();
  }
  if (dim != c.cache->head_dim || table->size(0) != batch || lens->size(0) != batch ||
      cu->size(0) != groups + 1 || max_len < 0 || max_len > INT32_MAX || heads > INT32_MAX ||
      batch > INT32_MAX || c.cache->num_kv_heads < 1)
    return not_handled();
  double scale = 1.0 / std::sqrt((double)dim);
  if (a[7] != Py_None) {
    if (!PyFloat_CheckExact(a[7])) return not_handled();
    scale = PyFloat_AS_DOUBLE(a[7]);
  }
  const bool want_lse = PyObject_IsTrue(a[9]) == 1;
  at::Tensor out = like(*q, q->sizes()), lse;
  if (want_lse) lse = at::empty({batch, heads}, q->options().dtype(at::kFloat));
  Result result(wrap2(out, lse));
  if (!result.o) return nullptr;
  const int st = c_shared(
      c.cache, q->data_ptr(), (int32_t)heads, (int32_t)(heads / c.cache->num_kv_heads),
      table->data_ptr<int32_t>(), (int32_t)table->size(1), lens->data_ptr<int32_t>(),
      (int32_t)batch, (int32_t)max_len, cu->data_ptr<int32_t>(), prefix->data_ptr<int32_t>(),
      (int32_t)groups, (float)scale, out.data_ptr(), want_lse ? lse.data_ptr<float>() : nullptr,
      work.data_ptr(), work.nbytes(), stream_of(dev));
  return answer("paged_decode_attention_shared", st, result);
}

// C++ exceptions (an allocation that fails, before any launch): the wrapper meets
// the same in Python, and raises it there.
template <PyObject* (*kCall)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return kCall(self, a, n);
  } catch (...) {
    return not_handled();
  }
}

// Addresses of the three entry points in libpagedkv.so, as the package loaded it, and
// the class of its errors.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *x, *y, *z, *e;
  if (!PyArg_ParseTuple(args, "OOOO", &x, &y, &z, &e)) return nullptr;
  c_norm_rope = reinterpret_cast<decltype(c_norm_rope)>(PyLong_AsVoidPtr(x));
  c_append_rope = reinterpret_cast<decltype(c_append_rope)>(PyLong_AsVoidPtr(y));
  c_shared = reinterpret_cast<decltype(c_shared)>(PyLong_AsVoidPtr(z));
  if (PyErr_Occurred()) return nullptr;
  Py_XSETREF(error_class, Py_NewRef(e));
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"norm_rope", fast(&guarded<norm_rope>), METH_FASTCALL, nullptr},
    {"append_rope", fast(&guarded<append_rope>), METH_FASTCALL, nullptr},
    {"decode_shared", fast(&guarded<decode_shared>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// KEY: the torch and Python this was built against; the package binds no other.
PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "KEY", PKV_BINDING_KEY) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

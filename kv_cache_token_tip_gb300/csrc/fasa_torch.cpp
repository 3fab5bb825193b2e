// The paged cache's calls for torch tensors: argument marshalling in compiled
// code.  A call of one small batch is host time (2 us of kernel), and reading ten
// tensors' properties from Python takes twice as long as the launch.  Module
// _fasa_torch; fasa.py holds its public functions.
//
// Each function checks its tensors (type, number of elements, device, contiguous:
// ValueError), passes their addresses and the current stream to the C entry point
// that bind() was given, and returns its status.  Nothing here computes on the data.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "../../include/fasa.h"

namespace {

decltype(&fasa_paged_append) c_append = nullptr;
decltype(&fasa_paged_attention) c_attention = nullptr;
decltype(&fasa_paged_evict) c_evict = nullptr;

const char* type_name(at::ScalarType t) {
  return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : c10::toString(t);
}

// Address of a tensor that fits; sets ValueError and *ok = false for another.
void* address(PyObject* x, const char* name, int here, at::ScalarType type, int64_t count, bool* ok) {
  if (!*ok) return nullptr;
  *ok = false;
  if (!THPVariable_Check(x)) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(x);
  if (!t.is_cuda() || t.get_device() != here)
    PyErr_Format(PyExc_ValueError, "%s must be a tensor on the current CUDA device", name);
  else if (t.scalar_type() != type)
    PyErr_Format(PyExc_ValueError, "%s has dtype %s, expected %s", name, type_name(t.scalar_type()), type_name(type));
  else if (t.numel() != count)
    PyErr_Format(PyExc_ValueError, "%s has %lld elements, expected %lld", name, (long long)t.numel(), (long long)count);
  else if (!t.is_contiguous())
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  else
    *ok = true;
  return *ok ? t.data_ptr() : nullptr;
}

// The same, of a tensor that may be None.
void* optional(PyObject* x, const char* name, int here, at::ScalarType type, int64_t count, bool* ok) {
  return x == Py_None ? nullptr : address(x, name, here, type, count, ok);
}

// A workspace: any contiguous tensor on the device.
void* room(PyObject* x, int here, size_t* bytes, bool* ok) {
  if (!*ok) return nullptr;
  if (THPVariable_Check(x)) {
    const at::Tensor& t = THPVariable_Unpack(x);
    if (t.is_cuda() && t.get_device() == here && t.is_contiguous()) {
      *bytes = t.nbytes();
      return t.data_ptr();
    }
  }
  PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous tensor on the current CUDA device");
  *ok = false;
  return nullptr;
}

// What a call's shapes and placement are checked against.
struct Call {
  const fasa_paged_dims_t* d;
  int here;
  fasa_stream_t stream;
  at::ScalarType store;
  int64_t batch, row, pool, slots, entries, heads;
  bool sizes;  // dims that can be reckoned with (the C entry point says what is wrong with others)

  // dims: the structure's address; stream: a handle, or None for the current one.
  bool read(PyObject* dims, PyObject* stream_arg) {
    d = static_cast<const fasa_paged_dims_t*>(PyLong_AsVoidPtr(dims));
    if (!d) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "dims is missing");
      return false;
    }
    here = c10::cuda::current_device();
    if (stream_arg == Py_None) {
      stream = reinterpret_cast<fasa_stream_t>(c10::cuda::getCurrentCUDAStream(here).stream());
    } else {
      stream = static_cast<fasa_stream_t>(PyLong_AsVoidPtr(stream_arg));
      if (PyErr_Occurred()) return false;
    }
    store = d->dtype == FASA_F32 ? at::kFloat : at::kBFloat16;
    sizes = d->batch > 0 && d->n_q_heads > 0 && d->n_kv_heads > 0 && d->head_dim > 0 && d->page_size > 0 &&
            d->n_pages > 0 && d->max_pages > 0;
    batch = d->batch;
    row = (int64_t)d->n_kv_heads * d->head_dim;
    pool = (int64_t)d->n_pages * d->page_size * row;
    slots = batch * d->n_kv_heads * d->max_pages * d->page_size;
    entries = batch * d->max_pages;
    heads = batch * d->n_q_heads * d->head_dim;
    return true;
  }
};

bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return false;
}

// No C++ exception leaves a call.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "an unknown error");
  }
  return nullptr;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 3)) return nullptr;
  c_append = reinterpret_cast<decltype(c_append)>(PyLong_AsVoidPtr(a[0]));
  c_attention = reinterpret_cast<decltype(c_attention)>(PyLong_AsVoidPtr(a[1]));
  c_evict = reinterpret_cast<decltype(c_evict)>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// append(k_new, v_new, pos, k_pages, v_pages, page_table, seq_lens, cu_new, weight, token_pos, dims, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (!counted(n, 12) || !c.read(a[10], a[11])) return nullptr;
    if (!c.sizes) return PyLong_FromLong(FASA_ERR_INVALID_ARG);
    if (!THPVariable_Check(a[0])) {
      PyErr_SetString(PyExc_ValueError, "k_new must be a tensor");
      return nullptr;
    }
    const int64_t tokens = THPVariable_Unpack(a[0]).numel() / c.row, count = tokens * c.row;
    if (tokens > INT_MAX) return PyLong_FromLong(FASA_ERR_UNSUPPORTED);
    bool ok = true;
    void* k_new = address(a[0], "k_new", c.here, c.store, count, &ok);
    void* v_new = address(a[1], "v_new", c.here, c.store, count, &ok);
    void* pos = address(a[2], "pos", c.here, at::kInt, c.batch, &ok);
    void* k_pages = address(a[3], "k_pages", c.here, c.store, c.pool, &ok);
    void* v_pages = address(a[4], "v_pages", c.here, c.store, c.pool, &ok);
    void* table = address(a[5], "page_table", c.here, at::kInt, c.entries, &ok);
    void* lens = address(a[6], "seq_lens", c.here, at::kInt, c.batch, &ok);
    void* cu_new = optional(a[7], "cu_new", c.here, at::kInt, c.batch + 1, &ok);
    void* weight = optional(a[8], "weight", c.here, at::kFloat, c.slots, &ok);
    void* token_pos = optional(a[9], "token_pos", c.here, at::kInt, c.slots, &ok);
    if (!ok) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = c_append(k_new, v_new, (int32_t)tokens, (const int32_t*)cu_new, (const int32_t*)pos, (const int32_t*)table,
                  (const int32_t*)lens, k_pages, v_pages, (float*)weight, (int32_t*)token_pos, c.d, c.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// attention(q, pos, k_pages, v_pages, page_table, seq_lens, out, weight, workspace, dims, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (!counted(n, 11) || !c.read(a[9], a[10])) return nullptr;
    if (!c.sizes) return PyLong_FromLong(FASA_ERR_INVALID_ARG);
    bool ok = true;
    size_t bytes = 0;
    void* q = address(a[0], "q", c.here, c.store, c.heads, &ok);
    void* pos = address(a[1], "pos", c.here, at::kInt, c.batch, &ok);
    void* k_pages = address(a[2], "k_pages", c.here, c.store, c.pool, &ok);
    void* v_pages = address(a[3], "v_pages", c.here, c.store, c.pool, &ok);
    void* table = address(a[4], "page_table", c.here, at::kInt, c.entries, &ok);
    void* lens = address(a[5], "seq_lens", c.here, at::kInt, c.batch, &ok);
    void* out = address(a[6], "out", c.here, at::kFloat, c.heads, &ok);
    void* weight = optional(a[7], "weight", c.here, at::kFloat, c.slots, &ok);
    void* workspace = room(a[8], c.here, &bytes, &ok);
    if (!ok) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = c_attention(q, (const int32_t*)pos, k_pages, v_pages, (const int32_t*)table, (const int32_t*)lens,
                     (float*)out, (float*)weight, workspace, bytes, c.d, c.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// evict(weight, token_pos, pos, k_pages, v_pages, page_table, seq_lens, keep, new_lens, sinks, recent, weight_out,
//       token_pos_out, workspace, dims, stream)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (!counted(n, 16) || !c.read(a[14], a[15])) return nullptr;
    if (!c.sizes) return PyLong_FromLong(FASA_ERR_INVALID_ARG);
    long bound[3];
    for (int i = 0; i < 3; ++i) {
      bound[i] = PyLong_AsLong(a[i == 0 ? 7 : 8 + i]);
      if (bound[i] == -1 && PyErr_Occurred()) return nullptr;
      if (bound[i] < INT_MIN || bound[i] > INT_MAX) return PyLong_FromLong(FASA_ERR_INVALID_ARG);
    }
    bool ok = true;
    size_t bytes = 0;
    void* weight = address(a[0], "weight", c.here, at::kFloat, c.slots, &ok);
    void* token_pos = address(a[1], "token_pos", c.here, at::kInt, c.slots, &ok);
    void* pos = address(a[2], "pos", c.here, at::kInt, c.batch, &ok);
    void* k_pages = address(a[3], "k_pages", c.here, c.store, c.pool, &ok);
    void* v_pages = address(a[4], "v_pages", c.here, c.store, c.pool, &ok);
    void* table = address(a[5], "page_table", c.here, at::kInt, c.entries, &ok);
    void* lens = address(a[6], "seq_lens", c.here, at::kInt, c.batch, &ok);
    void* new_lens = address(a[8], "new_lens", c.here, at::kInt, c.batch, &ok);
    void* weight_out = optional(a[11], "weight_out", c.here, at::kFloat, c.slots, &ok);
    void* token_pos_out = optional(a[12], "token_pos_out", c.here, at::kInt, c.slots, &ok);
    void* workspace = room(a[13], c.here, &bytes, &ok);
    if (!ok) return nullptr;
    if (a[11] == Py_None) weight_out = weight;
    if (a[12] == Py_None) token_pos_out = token_pos;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = c_evict((const float*)weight, (const int32_t*)token_pos, (const int32_t*)pos, (const int32_t*)table,
                 (const int32_t*)lens, (int32_t)bound[0], (int32_t)bound[1], (int32_t)bound[2], k_pages, v_pages,
                 (float*)weight_out, (int32_t*)token_pos_out, (int32_t*)new_lens, workspace, bytes, c.d, c.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fasa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was compiled for, which has to be the one that runs.
PyMODINIT_FUNC PyInit__fasa_torch(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FASA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

// binding.cpp -- the calls of a decode step's small operators from Python without
// ctypes: rotary positions and the 4-bit KV cache.
//
// A step runs these between launches of a few microseconds, where a call's
// checks and argument conversion in Python (4.5 us of 7.0 us for a rotation;
// the launch itself is 2.5 us) would be what the step waits for.  Each function
// here checks its operands as the Python function of the same name does and
// calls the C entry point; where any of them is not as expected it launches
// nothing and returns None, and the Python function, which has the words for
// it, takes over.  Otherwise it returns the entry point's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp8q.h"

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor* t, at::ScalarType type, int dev) {
  return t && t->is_cuda() && t->layout() == at::kStrided && t->scalar_type() == type && t->get_device() == dev;
}

// A [T, H, D] bf16 operand with contiguous elements, and its strides (those of dimensions of size 1 as if contiguous).
struct Heads {
  void* data;
  int64_t T, H, D, token, head;
};
bool heads(PyObject* o, int dev, Heads* h) {
  const at::Tensor* t = tensor(o);
  if (!on(t, at::kBFloat16, dev) || t->dim() != 3) return false;
  h->T = t->size(0);
  h->H = t->size(1);
  h->D = t->size(2);
  if (t->stride(2) != 1 && h->D != 1) return false;
  h->token = h->T > 1 ? t->stride(0) : h->H * h->D;
  h->head = h->H > 1 ? t->stride(1) : h->D;
  h->data = t->data_ptr();
  return true;
}
bool same(const Heads& a, const Heads& b) { return a.T == b.T && a.H == b.H && a.D == b.D; }

// A contiguous 1-D operand of n elements (any number for n < 0).
bool list(PyObject* o, at::ScalarType type, int dev, int64_t n, const at::Tensor** out) {
  const at::Tensor* t = tensor(o);
  if (!on(t, type, dev) || t->dim() != 1 || !t->is_contiguous() || (n >= 0 && t->numel() != n)) return false;
  *out = t;
  return true;
}

bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;               // (bool counts)
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool real(PyObject* o, float* v) {
  if (!PyFloat_Check(o)) return false;
  *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}
const fp8q_kv4_cache* cache_at(PyObject* address) {
  int64_t a;
  return whole(address, &a) ? reinterpret_cast<const fp8q_kv4_cache*>(a) : nullptr;
}
bool of_cache(const Heads& h, const fp8q_kv4_cache* c, int64_t T) {
  return h.T == T && h.H == c->kv_heads && h.D == c->head_dim;
}
bool current(int dev) { return dev >= 0 && dev == c10::cuda::current_device(); }
void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

PyObject* ask_python() { Py_RETURN_NONE; }

// (x, positions, freq, flags, mscale, out)
PyObject* rope_checked(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return ask_python();
  const at::Tensor *x0 = tensor(a[0]), *pos, *freq;
  if (!x0 || !x0->is_cuda()) return ask_python();
  const int dev = x0->get_device();
  Heads x, y;
  int64_t flags;
  float m;
  if (!current(dev) || !heads(a[0], dev, &x) || !heads(a[5], dev, &y) || !same(x, y)) return ask_python();
  if (!list(a[1], at::kLong, dev, x.T, &pos) || !list(a[2], at::kDouble, dev, -1, &freq)) return ask_python();
  if (!whole(a[3], &flags) || !real(a[4], &m)) return ask_python();
  return PyLong_FromLong(fp8q_rope(x.data, x.T, x.H, x.D, x.token, x.head, pos->const_data_ptr<int64_t>(),
                                   freq->const_data_ptr<double>(), 2 * freq->numel(), static_cast<int>(flags), m, y.data,
                                   y.token, y.head, stream(dev)));
}

// (cache address, device, k, v, slots, positions or None, freq or None, flags, mscale)
PyObject* append_checked(PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return ask_python();
  const fp8q_kv4_cache* c = cache_at(a[0]);
  int64_t dev, flags;
  Heads k, v;
  float m;
  const at::Tensor *slots, *pos = nullptr, *freq = nullptr;
  if (!c || !whole(a[1], &dev) || !current(static_cast<int>(dev))) return ask_python();
  const int d = static_cast<int>(dev);
  if (!heads(a[2], d, &k) || !heads(a[3], d, &v) || !of_cache(k, c, k.T) || !of_cache(v, c, k.T)) return ask_python();
  if (!list(a[4], at::kLong, d, k.T, &slots) || !whole(a[7], &flags) || !real(a[8], &m)) return ask_python();
  if ((a[5] == Py_None) != (a[6] == Py_None)) return ask_python();
  if (a[5] != Py_None && (!list(a[5], at::kLong, d, k.T, &pos) || !list(a[6], at::kDouble, d, -1, &freq))) return ask_python();
  return PyLong_FromLong(fp8q_kv4_append(c, k.data, k.token, k.head, v.data, v.token, v.head,
                                         slots->const_data_ptr<int64_t>(), k.T, pos ? pos->const_data_ptr<int64_t>() : nullptr,
                                         freq ? freq->const_data_ptr<double>() : nullptr, freq ? 2 * freq->numel() : 0,
                                         static_cast<int>(flags), m, stream(d)));
}

// (cache address, device, slots, k, v)
PyObject* read_checked(PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return ask_python();
  const fp8q_kv4_cache* c = cache_at(a[0]);
  int64_t dev;
  Heads k, v;
  const at::Tensor* slots;
  if (!c || !whole(a[1], &dev) || !current(static_cast<int>(dev))) return ask_python();
  const int d = static_cast<int>(dev);
  if (!list(a[2], at::kLong, d, -1, &slots) || !heads(a[3], d, &k) || !heads(a[4], d, &v)) return ask_python();
  if (!of_cache(k, c, slots->numel()) || !of_cache(v, c, slots->numel())) return ask_python();
  return PyLong_FromLong(fp8q_kv4_read(c, slots->const_data_ptr<int64_t>(), k.T, k.data, k.token, k.head, v.data, v.token,
                                       v.head, stream(d)));
}

// (cache address, device, q, page_table, kv_len, q_start or None, max_q_len, sm_scale, causal, window, out, lse or None,
//  workspace)
PyObject* attention_checked(PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return ask_python();
  const fp8q_kv4_cache* c = cache_at(a[0]);
  int64_t dev, max_q, causal, window;
  Heads q, o;
  float scale;
  if (!c || !whole(a[1], &dev) || !current(static_cast<int>(dev))) return ask_python();
  const int d = static_cast<int>(dev);
  if (!heads(a[2], d, &q) || !heads(a[10], d, &o) || !same(q, o) || q.D != c->head_dim) return ask_python();
  const at::Tensor *table = tensor(a[3]), *lens, *starts = nullptr, *lse = nullptr, *ws = tensor(a[12]);
  if (!on(table, at::kInt, d) || table->dim() != 2) return ask_python();
  const int64_t B = table->size(0), pages = table->size(1);
  if (table->stride(1) != 1 && pages > 1) return ask_python();
  if (!list(a[4], at::kInt, d, B, &lens)) return ask_python();
  if (a[5] != Py_None && !list(a[5], at::kInt, d, B + 1, &starts)) return ask_python();
  if (!whole(a[6], &max_q) || !real(a[7], &scale) || !whole(a[8], &causal) || !whole(a[9], &window)) return ask_python();
  if (a[11] != Py_None) {
    lse = tensor(a[11]);
    if (!on(lse, at::kFloat, d) || lse->dim() != 2 || lse->size(0) != q.T || lse->size(1) != q.H || !lse->is_contiguous())
      return ask_python();
  }
  if (!on(ws, at::kByte, d) || !ws->is_contiguous()) return ask_python();
  return PyLong_FromLong(fp8q_kv4_attention(
      c, q.data, q.token, q.head, q.T, q.H, table->const_data_ptr<int32_t>(), B > 1 ? table->stride(0) : pages, pages,
      lens->const_data_ptr<int32_t>(), starts ? starts->const_data_ptr<int32_t>() : nullptr, B, max_q, scale,
      causal ? 1 : 0, window, o.data, o.token, o.head, lse ? lse->mutable_data_ptr<float>() : nullptr, ws->data_ptr(),
      static_cast<size_t>(ws->numel()), stream(d)));
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (...) {                                    // a kind of tensor that has no such property
    PyErr_Clear();
    return ask_python();
  }
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<rope_checked>)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<append_checked>)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<read_checked>)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<attention_checked>)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4_binding() { return PyModule_Create(&module); }

// The tensor-level calls of the window and paged-cache operators for Python: checks of the
// tensors, outputs from torch's allocator, and the C entry point on the current stream, in one
// native call. (The same steps in Python and ctypes cost more than the small calls' kernels:
// a decode step's append 7.8 us a call against 3.1 here, a single sequence's tree 17.6
// against 6.3, the forward 14.8 against 6.1, on the GB300's host.)
//
// Each function returns its outputs, or None when a tensor is not what the call needs (the
// Python caller then says which), or the entry point's status as a number. The entry points
// are those of the libxattn that the binding has loaded (bind).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "xattn.h"

namespace {

decltype(&xattn_window_fwd) g_window_fwd;
decltype(&xattn_window_fwd_f32) g_window_fwd_f32;
decltype(&xattn_window_bwd) g_window_bwd;
decltype(&xattn_window_bwd_f32) g_window_bwd_f32;
decltype(&xattn_tree_decode) g_tree_decode;
decltype(&xattn_cache_append) g_cache_append;
decltype(&xattn_cache_compact) g_cache_compact;

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// Argument i as a tensor, or null.
const Tensor *tensor(PyObject *const *args, int i) {
  return THPVariable_Check(args[i]) ? &THPVariable_Unpack(args[i]) : nullptr;
}

// A contiguous CUDA tensor of this type and shape, on this device.
bool fits(const Tensor *t, ScalarType type, IntArrayRef shape, int device) {
  return t && t->is_cuda() && t->scalar_type() == type && t->get_device() == device && t->sizes() == shape &&
         t->is_contiguous();
}

// An int argument, clamped to int32 (a window or sinks beyond it mean the same).
int clamped(PyObject *x) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(x, &over);
  if (over) return over > 0 ? XATTN_NO_WINDOW : -XATTN_NO_WINDOW;
  return v > XATTN_NO_WINDOW ? XATTN_NO_WINDOW : (v < -XATTN_NO_WINDOW ? -XATTN_NO_WINDOW : static_cast<int>(v));
}

float scale_of(PyObject *x, int64_t hd) {
  return static_cast<float>(x == Py_None ? 1.0 / std::sqrt(static_cast<double>(hd)) : PyFloat_AsDouble(x));
}

// The sizes fit the entry points' ints.
bool ints(IntArrayRef shape) {
  for (const int64_t x : shape)
    if (x > 0x7fffffff) return false;
  return true;
}

PyObject *result(int status, std::initializer_list<Tensor> outputs) {
  if (status != XATTN_OK) return PyLong_FromLong(status);
  if (outputs.size() == 0) Py_RETURN_TRUE;
  PyObject *tuple = PyTuple_New(static_cast<Py_ssize_t>(outputs.size()));
  if (!tuple) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor &t : outputs) PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(t));
  return tuple;
}

// The calls that write tensors in place say so to autograd, as torch's in-place operations do (a
// tensor that some backward saved is then refused there). Inference tensors have no version.
PyObject *written(int status, std::initializer_list<const Tensor *> tensors) {
  if (status == XATTN_OK)
    for (const Tensor *t : tensors)
      if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  return result(status, {});
}

// What every call begins with (the number of arguments), and what follows its checks: the
// tensors' device is the current one, and this is its stream.
#define XATTN_CALL(count)                                     \
  HANDLE_TH_ERRORS                                            \
  if (n != (count)) {                                         \
    PyErr_SetString(PyExc_TypeError, "wrong argument count"); \
    return nullptr;                                           \
  }
#define XATTN_HERE(device)                                    \
  if (c10::cuda::current_device() != (device)) Py_RETURN_NONE; \
  void *const stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream()

struct Window {
  const Tensor *q, *k, *v;
  ScalarType type;
  int64_t B, S, nh, nkv, hd;
  int device;
  bool ok;
  explicit Window(PyObject *const *args) : q(tensor(args, 0)), k(tensor(args, 1)), v(tensor(args, 2)), ok(false) {
    if (!q || !k || !q->is_cuda() || q->dim() != 4 || k->dim() != 4 || !ints(q->sizes()) || !ints(k->sizes())) return;
    type = q->scalar_type();
    device = q->get_device();
    B = q->size(0), S = q->size(1), nh = q->size(2), hd = q->size(3), nkv = k->size(2);
    ok = (type == at::kBFloat16 || type == at::kFloat) && fits(q, type, {B, S, nh, hd}, device) &&
         fits(k, type, {B, S, nkv, hd}, device) && fits(v, type, {B, S, nkv, hd}, device);
  }
};

// window_fwd(q, k, v, window, sinks, scale) -> (o, lse)
PyObject *window_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(6)
  const Window w(args);
  if (!w.ok) Py_RETURN_NONE;
  XATTN_HERE(w.device);
  const int window = clamped(args[3]), sinks = clamped(args[4]);
  const float scale = scale_of(args[5], w.hd);
  if (PyErr_Occurred()) return nullptr;
  const Tensor o = at::empty(w.q->sizes(), w.q->options());
  const Tensor lse = at::empty({w.B, w.S, w.nh}, w.q->options().dtype(at::kFloat));
  const void *q = w.q->data_ptr(), *k = w.k->data_ptr(), *v = w.v->data_ptr();
  float *l = lse.data_ptr<float>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  if (w.type == at::kBFloat16)
    status = g_window_fwd(q, k, v, w.B, w.S, w.nh, w.nkv, w.hd, window, sinks, scale, o.data_ptr(), l, stream);
  else
    status = g_window_fwd_f32(static_cast<const float *>(q), static_cast<const float *>(k),
                              static_cast<const float *>(v), w.B, w.S, w.nh, w.nkv, w.hd, window, sinks, scale,
                              o.data_ptr<float>(), l, stream);
  Py_END_ALLOW_THREADS
  return result(status, {o, lse});
  END_HANDLE_TH_ERRORS
}

// window_bwd(q, k, v, o, dO, lse, window, sinks, scale, deterministic) -> (dq, dk, dv)
PyObject *window_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(10)
  const Window w(args);
  const Tensor *o = tensor(args, 3), *dO = tensor(args, 4), *lse = tensor(args, 5);
  if (!w.ok || !fits(o, w.type, w.q->sizes(), w.device) || !fits(dO, w.type, w.q->sizes(), w.device) ||
      !fits(lse, at::kFloat, {w.B, w.S, w.nh}, w.device))
    Py_RETURN_NONE;
  XATTN_HERE(w.device);
  const int window = clamped(args[6]), sinks = clamped(args[7]);
  const float scale = scale_of(args[8], w.hd);
  const int deterministic = PyObject_IsTrue(args[9]);
  if (PyErr_Occurred()) return nullptr;
  const Tensor dq = at::empty(w.q->sizes(), w.q->options()), dk = at::empty(w.k->sizes(), w.k->options()),
               dv = at::empty(w.k->sizes(), w.k->options());
  const void *in[5] = {w.q->data_ptr(), w.k->data_ptr(), w.v->data_ptr(), o->data_ptr(), dO->data_ptr()};
  const float *l = lse->data_ptr<float>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  if (w.type == at::kBFloat16) {
    status = g_window_bwd(in[0], in[1], in[2], in[3], in[4], l, w.B, w.S, w.nh, w.nkv, w.hd, window, sinks, scale,
                          deterministic, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), stream);
  } else {
    auto f = [&](int i) { return static_cast<const float *>(in[i]); };
    status = g_window_bwd_f32(f(0), f(1), f(2), f(3), f(4), l, w.B, w.S, w.nh, w.nkv, w.hd, window, sinks, scale,
                              dq.data_ptr<float>(), dk.data_ptr<float>(), dv.data_ptr<float>(), stream);
  }
  Py_END_ALLOW_THREADS
  return result(status, {dq, dk, dv});
  END_HANDLE_TH_ERRORS
}

struct Pool {
  const Tensor *k, *v, *table, *lens;
  int64_t B, max_pages, num_pages, page_size, nkv, hd;
  int device;
  bool ok;
  Pool(PyObject *const *args, int at)
      : k(tensor(args, at)), v(tensor(args, at + 1)), table(tensor(args, at + 2)), lens(tensor(args, at + 3)), ok(false) {
    if (!k || !table || !k->is_cuda() || k->dim() != 4 || table->dim() != 2 || !ints(k->sizes()) || !ints(table->sizes())) return;
    device = k->get_device();
    B = table->size(0), max_pages = table->size(1);
    num_pages = k->size(0), page_size = k->size(1), nkv = k->size(2), hd = k->size(3);
    ok = fits(k, at::kBFloat16, k->sizes(), device) && fits(v, at::kBFloat16, k->sizes(), device) &&
         fits(table, at::kInt, table->sizes(), device) && fits(lens, at::kInt, {B}, device);
  }
};

// tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree or None, window or None, sinks,
//             scale) -> (o, lse)
PyObject *tree_decode(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(9)
  const Pool p(args, 1);
  const Tensor *q = tensor(args, 0), *tree = tensor(args, 5);
  if (!p.ok || !q || q->dim() != 4 || !ints(q->sizes())) Py_RETURN_NONE;
  const int64_t tokens = q->size(1), nh = q->size(2);
  if (!fits(q, at::kBFloat16, {p.B, tokens, nh, p.hd}, p.device) ||
      (args[5] != Py_None && !fits(tree, at::kLong, {p.B, tokens}, p.device)))
    Py_RETURN_NONE;
  XATTN_HERE(p.device);
  const int window = args[6] == Py_None ? XATTN_NO_WINDOW : clamped(args[6]), sinks = clamped(args[7]);
  const float scale = scale_of(args[8], p.hd);
  if (PyErr_Occurred()) return nullptr;
  const Tensor o = at::empty(q->sizes(), q->options());
  const Tensor lse = at::empty({p.B, tokens, nh}, q->options().dtype(at::kFloat));
  const auto *words =
      tree ? reinterpret_cast<const unsigned long long *>(tree->data_ptr<int64_t>()) : nullptr;
  const void *qp = q->data_ptr(), *kp = p.k->data_ptr(), *vp = p.v->data_ptr();
  const int *table = p.table->data_ptr<int>(), *lens = p.lens->data_ptr<int>();
  void *op = o.data_ptr();
  float *l = lse.data_ptr<float>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_tree_decode(qp, kp, vp, table, lens, words, p.B, tokens, nh, p.nkv, p.hd, p.num_pages, p.page_size,
                         p.max_pages, window, sinks, scale, op, l, stream);
  Py_END_ALLOW_THREADS
  return result(status, {o, lse});
  END_HANDLE_TH_ERRORS
}

// cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens) -> True
PyObject *cache_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(6)
  const Pool p(args, 2);
  const Tensor *k = tensor(args, 0), *v = tensor(args, 1);
  if (!p.ok || !k || k->dim() != 4 || !ints(k->sizes())) Py_RETURN_NONE;
  const int64_t rows = k->size(1);
  if (!fits(k, at::kBFloat16, {p.B, rows, p.nkv, p.hd}, p.device) ||
      !fits(v, at::kBFloat16, {p.B, rows, p.nkv, p.hd}, p.device))
    Py_RETURN_NONE;
  XATTN_HERE(p.device);
  const void *kn = k->data_ptr(), *vn = v->data_ptr();
  void *kp = p.k->data_ptr(), *vp = p.v->data_ptr();
  const int *table = p.table->data_ptr<int>(), *lens = p.lens->data_ptr<int>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_cache_append(kn, vn, kp, vp, table, lens, p.B, rows, p.nkv, p.hd, p.num_pages, p.page_size, p.max_pages,
                          stream);
  Py_END_ALLOW_THREADS
  return written(status, {p.k, p.v});
  END_HANDLE_TH_ERRORS
}

// cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted) -> True
PyObject *cache_compact(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(6)
  const Pool p(args, 0);
  const Tensor *path = tensor(args, 4), *accepted = tensor(args, 5);
  if (!p.ok || !path || path->dim() != 2 || !ints(path->sizes())) Py_RETURN_NONE;
  const int64_t rows = path->size(1);
  if (!fits(path, at::kInt, {p.B, rows}, p.device) || !fits(accepted, at::kInt, {p.B}, p.device)) Py_RETURN_NONE;
  XATTN_HERE(p.device);
  void *kp = p.k->data_ptr(), *vp = p.v->data_ptr();
  const int *table = p.table->data_ptr<int>(), *lens = p.lens->data_ptr<int>();
  const int *pp = path->data_ptr<int>(), *ap = accepted->data_ptr<int>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_cache_compact(kp, vp, table, lens, pp, ap, p.B, rows, p.nkv, p.hd, p.num_pages, p.page_size, p.max_pages,
                           stream);
  Py_END_ALLOW_THREADS
  return written(status, {p.k, p.v});
  END_HANDLE_TH_ERRORS
}

// bind(seven addresses): the entry points to call.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void **const targets[] = {reinterpret_cast<void **>(&g_window_fwd),  reinterpret_cast<void **>(&g_window_fwd_f32),
                            reinterpret_cast<void **>(&g_window_bwd),  reinterpret_cast<void **>(&g_window_bwd_f32),
                            reinterpret_cast<void **>(&g_tree_decode), reinterpret_cast<void **>(&g_cache_append),
                            reinterpret_cast<void **>(&g_cache_compact)};
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) *targets[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

#define XATTN_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {XATTN_METHOD(window_fwd),   XATTN_METHOD(window_bwd),    XATTN_METHOD(tree_decode),
                           XATTN_METHOD(cache_append), XATTN_METHOD(cache_compact), XATTN_METHOD(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "xattn_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_xattn_torch(void) { return PyModule_Create(&g_module); }

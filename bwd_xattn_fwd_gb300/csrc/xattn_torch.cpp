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

decltype(&xattn_latent_fwd) g_latent_fwd;
decltype(&xattn_latent_bwd) g_latent_bwd;
decltype(&xattn_latent_decode) g_latent_decode;
decltype(&xattn_cache_reserve) g_cache_reserve;
decltype(&xattn_cache_release) g_cache_release;
decltype(&xattn_cache_write) g_cache_write;
decltype(&xattn_latent_write) g_latent_write;

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

struct Latent {
  const Tensor *q, *kv, *rope;
  int64_t B, S, nh, dn, dr, dv;
  int device;
  bool ok;
  explicit Latent(PyObject *const *args) : q(tensor(args, 0)), kv(tensor(args, 1)), rope(tensor(args, 2)), ok(false) {
    if (!q || !kv || !rope || !q->is_cuda() || q->dim() != 4 || kv->dim() != 4 || rope->dim() != 3 || !ints(q->sizes()) ||
        !ints(kv->sizes()))
      return;
    device = q->get_device();
    B = q->size(0), S = q->size(1), nh = q->size(2), dr = rope->size(2), dn = q->size(3) - dr, dv = kv->size(3) - dn;
    ok = dn > 0 && dv > 0 && fits(q, at::kBFloat16, {B, S, nh, dn + dr}, device) &&
         fits(kv, at::kBFloat16, {B, S, nh, dn + dv}, device) && fits(rope, at::kBFloat16, {B, S, dr}, device);
  }
};

// latent_fwd(q, kv, k_rope, scale) -> (o, lse)
PyObject *latent_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(4)
  const Latent x(args);
  if (!x.ok) Py_RETURN_NONE;
  XATTN_HERE(x.device);
  const float scale = scale_of(args[3], x.dn + x.dr);
  if (PyErr_Occurred()) return nullptr;
  const Tensor o = at::empty({x.B, x.S, x.nh, x.dv}, x.q->options());
  const Tensor lse = at::empty({x.B, x.S, x.nh}, x.q->options().dtype(at::kFloat));
  const void *q = x.q->data_ptr(), *kv = x.kv->data_ptr(), *rope = x.rope->data_ptr();
  void *op = o.data_ptr();
  float *l = lse.data_ptr<float>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_latent_fwd(q, kv, rope, x.B, x.S, x.nh, x.dn, x.dr, x.dv, scale, op, l, stream);
  Py_END_ALLOW_THREADS
  return result(status, {o, lse});
  END_HANDLE_TH_ERRORS
}

// latent_bwd(q, kv, k_rope, o, dO, lse, scale) -> (dq, dkv, dk_rope)
PyObject *latent_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(7)
  const Latent x(args);
  const Tensor *o = tensor(args, 3), *dO = tensor(args, 4), *lse = tensor(args, 5);
  if (!x.ok || !fits(o, at::kBFloat16, {x.B, x.S, x.nh, x.dv}, x.device) ||
      !fits(dO, at::kBFloat16, {x.B, x.S, x.nh, x.dv}, x.device) || !fits(lse, at::kFloat, {x.B, x.S, x.nh}, x.device))
    Py_RETURN_NONE;
  XATTN_HERE(x.device);
  const float scale = scale_of(args[6], x.dn + x.dr);
  if (PyErr_Occurred()) return nullptr;
  const Tensor dq = at::empty(x.q->sizes(), x.q->options()), dkv = at::empty(x.kv->sizes(), x.kv->options()),
               drope = at::empty(x.rope->sizes(), x.rope->options());
  const void *in[5] = {x.q->data_ptr(), x.kv->data_ptr(), x.rope->data_ptr(), o->data_ptr(), dO->data_ptr()};
  const float *l = lse->data_ptr<float>();
  void *out[3] = {dq.data_ptr(), dkv.data_ptr(), drope.data_ptr()};
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_latent_bwd(in[0], in[1], in[2], in[3], in[4], l, x.B, x.S, x.nh, x.dn, x.dr, x.dv, scale, out[0], out[1],
                        out[2], stream);
  Py_END_ALLOW_THREADS
  return result(status, {dq, dkv, drope});
  END_HANDLE_TH_ERRORS
}

// latent_decode(q, pages, page_table, ctx_lens, dc, scale) -> (o, lse)
PyObject *latent_decode(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(6)
  const Tensor *q = tensor(args, 0), *pages = tensor(args, 1), *table = tensor(args, 2), *lens = tensor(args, 3);
  if (!q || !pages || !table || !q->is_cuda() || q->dim() != 4 || pages->dim() != 3 || table->dim() != 2 ||
      !ints(q->sizes()) || !ints(pages->sizes()) || !ints(table->sizes()))
    Py_RETURN_NONE;
  const int device = q->get_device();
  const int64_t B = table->size(0), tokens = q->size(1), nh = q->size(2), width = pages->size(2);
  const int64_t dc = PyLong_AsLongLong(args[4]);
  const float scale = static_cast<float>(PyFloat_AsDouble(args[5]));
  if (PyErr_Occurred()) return nullptr;
  if (dc <= 0 || dc >= width || !fits(q, at::kBFloat16, {B, tokens, nh, width}, device) ||
      !fits(pages, at::kBFloat16, pages->sizes(), device) || !fits(table, at::kInt, table->sizes(), device) ||
      !fits(lens, at::kInt, {B}, device))
    Py_RETURN_NONE;
  XATTN_HERE(device);
  const Tensor o = at::empty({B, tokens, nh, dc}, q->options());
  const Tensor lse = at::empty({B, tokens, nh}, q->options().dtype(at::kFloat));
  const void *qp = q->data_ptr(), *pp = pages->data_ptr();
  const int *tp = table->data_ptr<int>(), *lp = lens->data_ptr<int>();
  void *op = o.data_ptr();
  float *l = lse.data_ptr<float>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_latent_decode(qp, pp, tp, lp, B, tokens, nh, dc, width - dc, pages->size(0), pages->size(1), table->size(1),
                           scale, op, l, stream);
  Py_END_ALLOW_THREADS
  return result(status, {o, lse});
  END_HANDLE_TH_ERRORS
}

// A page table, two arrays of lengths, and the stack of free pages.
struct Tables {
  const Tensor *table, *from, *to, *pages, *count;
  int64_t B, max_pages, num_pages;
  int device;
  bool ok;
  explicit Tables(PyObject *const *args)
      : table(tensor(args, 0)), from(tensor(args, 1)), to(tensor(args, 2)), pages(tensor(args, 3)), count(tensor(args, 4)),
        ok(false) {
    if (!table || !pages || !table->is_cuda() || table->dim() != 2 || pages->dim() != 1 || !ints(table->sizes()) ||
        !ints(pages->sizes()))
      return;
    device = table->get_device();
    B = table->size(0), max_pages = table->size(1), num_pages = pages->size(0);
    ok = fits(table, at::kInt, table->sizes(), device) && fits(from, at::kInt, {B}, device) &&
         fits(to, at::kInt, {B}, device) && fits(pages, at::kInt, pages->sizes(), device) &&
         fits(count, at::kInt, {1}, device);
  }
};

// cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, page_size, tokens) -> (slots, offsets, granted)
PyObject *cache_reserve(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(7)
  const Tables x(args);
  const int page_size = clamped(args[5]), tokens = clamped(args[6]);
  if (PyErr_Occurred()) return nullptr;
  if (!x.ok) Py_RETURN_NONE;
  XATTN_HERE(x.device);
  if (tokens < 0) return PyLong_FromLong(XATTN_ERR_BAD_SHAPE);
  const Tensor slots = at::empty({tokens}, x.table->options().dtype(at::kLong)),
               offsets = at::empty({x.B + 1}, x.table->options()), granted = at::empty({x.B}, x.table->options());
  int *table = x.table->data_ptr<int>(), *count = x.count->data_ptr<int>(), *op = offsets.data_ptr<int>(),
      *gp = granted.data_ptr<int>();
  const int *ctx = x.from->data_ptr<int>(), *fresh = x.to->data_ptr<int>(), *pages = x.pages->data_ptr<int>();
  auto *sp = reinterpret_cast<long long *>(slots.data_ptr<int64_t>());
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_cache_reserve(table, ctx, fresh, pages, count, x.B, x.num_pages, page_size, x.max_pages, tokens, sp, op, gp,
                           stream);
  Py_END_ALLOW_THREADS
  if (status == XATTN_OK) {
    PyObject *done = written(status, {x.table, x.count});
    Py_XDECREF(done);
  }
  return result(status, {slots, offsets, granted});
  END_HANDLE_TH_ERRORS
}

// cache_release(page_table, held_lens, keep_lens, free_pages, free_count, page_size) -> True
PyObject *cache_release(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(6)
  const Tables x(args);
  const int page_size = clamped(args[5]);
  if (PyErr_Occurred()) return nullptr;
  if (!x.ok) Py_RETURN_NONE;
  XATTN_HERE(x.device);
  int *table = x.table->data_ptr<int>(), *pages = x.pages->data_ptr<int>(), *count = x.count->data_ptr<int>();
  const int *held = x.from->data_ptr<int>(), *keep = x.to->data_ptr<int>();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_cache_release(table, held, keep, pages, count, x.B, x.num_pages, page_size, x.max_pages, stream);
  Py_END_ALLOW_THREADS
  return written(status, {x.table, x.pages, x.count});
  END_HANDLE_TH_ERRORS
}

// cache_write(k_new, v_new, k_pages, v_pages, slots) -> True
PyObject *cache_write(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(5)
  const Tensor *k = tensor(args, 0), *v = tensor(args, 1), *kp = tensor(args, 2), *vp = tensor(args, 3), *slots = tensor(args, 4);
  if (!kp || !slots || !kp->is_cuda() || kp->dim() != 4 || slots->dim() != 1 || !ints(kp->sizes()) || !ints(slots->sizes()))
    Py_RETURN_NONE;
  const int device = kp->get_device();
  const int64_t rows = slots->size(0), nkv = kp->size(2), hd = kp->size(3);
  if (!fits(kp, at::kBFloat16, kp->sizes(), device) || !fits(vp, at::kBFloat16, kp->sizes(), device) ||
      !fits(slots, at::kLong, {rows}, device) || !fits(k, at::kBFloat16, {rows, nkv, hd}, device) ||
      !fits(v, at::kBFloat16, {rows, nkv, hd}, device))
    Py_RETURN_NONE;
  XATTN_HERE(device);
  const void *kn = k->data_ptr(), *vn = v->data_ptr();
  void *kd = kp->data_ptr(), *vd = vp->data_ptr();
  const auto *sp = reinterpret_cast<const long long *>(slots->data_ptr<int64_t>());
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_cache_write(kn, vn, kd, vd, sp, rows, nkv, hd, kp->size(0), kp->size(1), stream);
  Py_END_ALLOW_THREADS
  return written(status, {kp, vp});
  END_HANDLE_TH_ERRORS
}

// latent_write(c, k_rope, pages, slots) -> True
PyObject *latent_write(PyObject *, PyObject *const *args, Py_ssize_t n) {
  XATTN_CALL(4)
  const Tensor *c = tensor(args, 0), *rope = tensor(args, 1), *pages = tensor(args, 2), *slots = tensor(args, 3);
  if (!c || !rope || !pages || !slots || !pages->is_cuda() || c->dim() != 2 || rope->dim() != 2 || pages->dim() != 3 ||
      slots->dim() != 1 || !ints(pages->sizes()) || !ints(slots->sizes()))
    Py_RETURN_NONE;
  const int device = pages->get_device();
  const int64_t rows = slots->size(0), dc = c->size(1), dr = rope->size(1);
  if (!fits(pages, at::kBFloat16, {pages->size(0), pages->size(1), dc + dr}, device) || !fits(slots, at::kLong, {rows}, device) ||
      !fits(c, at::kBFloat16, {rows, dc}, device) || !fits(rope, at::kBFloat16, {rows, dr}, device))
    Py_RETURN_NONE;
  XATTN_HERE(device);
  const void *cp = c->data_ptr(), *rp = rope->data_ptr();
  void *pp = pages->data_ptr();
  const auto *sp = reinterpret_cast<const long long *>(slots->data_ptr<int64_t>());
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = g_latent_write(cp, rp, pp, sp, rows, dc, dr, pages->size(0), pages->size(1), stream);
  Py_END_ALLOW_THREADS
  return written(status, {pages});
  END_HANDLE_TH_ERRORS
}

// bind(fourteen addresses): the entry points to call.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void **const targets[] = {reinterpret_cast<void **>(&g_window_fwd),  reinterpret_cast<void **>(&g_window_fwd_f32),
                            reinterpret_cast<void **>(&g_window_bwd),  reinterpret_cast<void **>(&g_window_bwd_f32),
                            reinterpret_cast<void **>(&g_tree_decode), reinterpret_cast<void **>(&g_cache_append),
                            reinterpret_cast<void **>(&g_cache_compact), reinterpret_cast<void **>(&g_latent_fwd),
                            reinterpret_cast<void **>(&g_latent_bwd),  reinterpret_cast<void **>(&g_latent_decode),
                            reinterpret_cast<void **>(&g_cache_reserve), reinterpret_cast<void **>(&g_cache_release),
                            reinterpret_cast<void **>(&g_cache_write), reinterpret_cast<void **>(&g_latent_write)};
  constexpr int kTargets = sizeof(targets) / sizeof(targets[0]);
  if (n != kTargets) {
    PyErr_SetString(PyExc_TypeError, "bind takes fourteen addresses");
    return nullptr;
  }
  for (int i = 0; i < kTargets; ++i) *targets[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

#define XATTN_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {XATTN_METHOD(window_fwd),   XATTN_METHOD(window_bwd),    XATTN_METHOD(tree_decode),
                           XATTN_METHOD(cache_append), XATTN_METHOD(cache_compact), XATTN_METHOD(latent_fwd),
                           XATTN_METHOD(latent_bwd),   XATTN_METHOD(latent_decode), XATTN_METHOD(cache_reserve),
                           XATTN_METHOD(cache_release), XATTN_METHOD(cache_write),  XATTN_METHOD(latent_write),
                           XATTN_METHOD(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "xattn_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_xattn_torch(void) { return PyModule_Create(&g_module); }

// paged_call.cpp -- the short way from torch tensors to the C ABI of the paged cache and of draft
// verification, for the calls that a decoding loop makes.
//
// A decoding step's kernels take a few microseconds, and reading a tensor's shape, strides, type and
// address from Python takes as long.  Each function here checks what the C ABI cannot see (types,
// devices, shapes, strides), allocates the outputs and makes the call.  It returns None, with nothing
// enqueued, for whatever is not plain and right: a wrong argument, another device than the current one,
// a status that the C ABI decides before its first launch.  paged.py then takes the call through its own
// checks, which name what is wrong, or through a graph's workspace.  A HIP error may come after a launch:
// its status is returned, and the call is not made again.  Enqueueing one conversation's step took 15.3 us
// by way of Python alone.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "keops_mi355x.h"

#ifndef PAGED_CALL_DEVICE      // the tests' build takes host tensors, over a stand-in for the library
#define PAGED_CALL_DEVICE c10::DeviceType::CUDA
#endif

namespace {

PyObject *g_raw_stream = nullptr;     // torch's current raw stream of a device

// A tensor as Python handed it over; null for None, and `bad` for what is no plain tensor.
struct Arg {
  const at::Tensor *t = nullptr;
  bool bad = false;
};
Arg arg(PyObject *o) {
  if (o == Py_None) return {};
  if (!THPVariable_CheckExact(o)) return {nullptr, true};
  return {&THPVariable_Unpack(o), false};
}

// What every tensor of a call has to share.
struct Call {
  int64_t dev = -1;
  bool ok = true;

  const at::Tensor *need(PyObject *o) {
    const Arg a = arg(o);
    if (!a.t) ok = false;
    return a.t;
  }
  const at::Tensor *maybe(PyObject *o) {
    const Arg a = arg(o);
    if (a.bad) ok = false;
    return a.t;
  }
  bool on_device(const at::Tensor &t) const {
    const c10::Device d = t.device();
    return d.type() == PAGED_CALL_DEVICE && d.index() == dev;
  }
  // the address of a dense tensor of this type and shape, null where it is another
  void *dense(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || !on_device(*t) || t->sizes() != shape || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  bool begin(const at::Tensor &t) {
    if (t.device().type() != PAGED_CALL_DEVICE) return false;
    dev = t.device().index();
    const c10::impl::VirtualGuardImpl guard(PAGED_CALL_DEVICE);
    return guard.getDevice().index() == dev;
  }
};

int type_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return KEOPS_TYPE_BF16;
    case at::kHalf: return KEOPS_TYPE_F16;
    case at::kFloat8_e4m3fn: return KEOPS_TYPE_E4M3;
    default: return -1;
  }
}

bool table_of(Call &c, const at::Tensor *t, int64_t seqs, const int32_t **at, int64_t *stride, int32_t *width) {
  if (!t || t->dim() != 2 || t->scalar_type() != at::kInt || !c.on_device(*t) || t->size(0) != seqs || t->size(1) > INT32_MAX ||
      (t->stride(1) != 1 && t->size(1) > 1))
    return false;
  *at = (const int32_t *)t->data_ptr();
  *stride = t->stride(0);
  *width = (int32_t)t->size(1);
  return true;
}

// k_pages, v_pages, weights, page_table, lens, k_scale, v_scale into the C ABI's structure.
bool cache_of(Call &c, PyObject *const *o, keops_cache_t *out) {
  const at::Tensor *k = c.need(o[0]), *v = c.need(o[1]), *w = c.maybe(o[2]), *table = c.need(o[3]), *lens = c.need(o[4]);
  const at::Tensor *ks = c.maybe(o[5]), *vs = c.maybe(o[6]);
  if (!c.ok || !c.begin(*k)) return false;
  const int type = type_of(k->scalar_type());
  if (type < 0 || k->dim() != 4 || k->stride(3) != 1 || v->scalar_type() != k->scalar_type() || !c.on_device(*v) ||
      v->sizes() != k->sizes() || v->strides() != k->strides())
    return false;
  if (lens->dim() != 1 || lens->scalar_type() != at::kInt || !c.on_device(*lens) || !lens->is_contiguous()) return false;
  const int64_t P = k->size(0), ps = k->size(1), H = k->size(2), D = k->size(3), S = lens->size(0);
  if (ps > INT32_MAX || H > INT32_MAX || D > INT32_MAX || S > INT32_MAX) return false;
  if ((type == KEOPS_TYPE_E4M3) != (ks != nullptr) || (ks != nullptr) != (vs != nullptr)) return false;
  *out = keops_cache_t{};
  out->k_pages = k->data_ptr();
  out->v_pages = v->data_ptr();
  out->weights = (float *)c.dense(w, at::kFloat, {P, H, ps});
  out->k_scale = (const float *)c.dense(ks, at::kFloat, {H});
  out->v_scale = (const float *)c.dense(vs, at::kFloat, {H});
  // the stride of a dimension of one is never used
  out->page_stride = P > 1 ? k->stride(0) : 0;
  out->slot_stride = ps > 1 ? k->stride(1) : 0;
  out->head_stride = H > 1 ? k->stride(2) : 0;
  out->pages = P;
  out->lens = (const int32_t *)lens->data_ptr();
  out->page_size = (int32_t)ps;
  out->heads = (int32_t)H;
  out->dim = (int32_t)D;
  out->type = type;
  out->seqs = (int32_t)S;
  return table_of(c, table, S, &out->page_table, &out->table_stride, &out->table_width) && c.ok;
}

// Token rows [tokens, heads, dim] of a 16-bit type, heads dense.
bool rows_of(const Call &c, const at::Tensor &t, const keops_cache_t &cache, int64_t *stride) {
  const int type = type_of(t.scalar_type());
  if ((type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16) || (cache.type != KEOPS_TYPE_E4M3 && cache.type != type)) return false;
  if (t.dim() != 3 || !c.on_device(t) || t.size(2) != cache.dim || t.size(1) > INT32_MAX) return false;
  const int64_t T = t.size(0), h = t.size(1);
  if (T && (t.stride(2) != 1 || (h > 1 && t.stride(1) != cache.dim))) return false;
  *stride = T > 1 ? t.stride(0) : h * cache.dim;
  return true;
}

bool number(PyObject *o, int32_t *v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  if (over || x < 0 || x > INT32_MAX) return false;
  *v = (int32_t)x;
  return true;
}

bool stream_of(const Call &c, void **stream) {
  PyObject *dev = PyLong_FromLongLong(c.dev);
  PyObject *s = dev ? PyObject_CallOneArg(g_raw_stream, dev) : nullptr;
  Py_XDECREF(dev);
  if (!s) return false;
  *stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

// Runs f without the interpreter's lock, which is back also where f throws.  No tensor is asked for
// anything in there: one without memory of its own (torch.vmap's, torch.func's) throws at its address.
template <class F>
int unlocked(F f) {
  struct Lock {
    PyThreadState *state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

// Runs f; anything thrown, and any Python error, is a call for the long way.
template <class F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  PyObject *r = nullptr;
  if (given == wanted && g_raw_stream) {
    try {
      r = f();
    } catch (...) {
      r = nullptr;
    }
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject *pair(const at::Tensor &a, PyObject *a_given, const at::Tensor &b, PyObject *b_given) {
  PyObject *x = a_given == Py_None ? THPVariable_Wrap(a) : Py_NewRef(a_given);
  PyObject *y = b_given == Py_None ? THPVariable_Wrap(b) : Py_NewRef(b_given);
  PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// What a call ends with.  `result` was made before it, so that nothing can fail once work is enqueued.
PyObject *ended(int rc, PyObject *result) {
  if (rc == KEOPS_OK) return result;
  Py_DECREF(result);
  return rc == KEOPS_ERR_HIP ? PyLong_FromLong(rc) : nullptr;
}

// An output: the caller's dense tensor, or a new one.
bool output(Call &c, PyObject *given, at::ScalarType type, at::IntArrayRef shape, const at::Tensor &like, at::Tensor *out) {
  if (given != Py_None) {
    const at::Tensor *t = c.need(given);
    if (!t) return false;
    c.dense(t, type, shape);
    *out = *t;
    return c.ok;
  }
  *out = at::empty(shape, like.options().dtype(type).requires_grad(false));
  return true;
}

// (k, v, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts) -> True; here and below a status, or None
PyObject *append(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    if (!cache_of(c, o + 2, &cache)) return nullptr;
    const at::Tensor *k = c.need(o[0]), *v = c.need(o[1]), *starts = c.need(o[9]);
    int64_t ks, vs;
    void *st;
    if (!c.ok || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || !rows_of(c, *k, cache, &ks) ||
        !rows_of(c, *v, cache, &vs) || k->size(1) != cache.heads)
      return nullptr;
    const int32_t *at = (const int32_t *)c.dense(starts, at::kInt, {(int64_t)cache.seqs + 1});
    if (!c.ok || !stream_of(c, &st)) return nullptr;
    const void *kp = k->data_ptr(), *vp = v->data_ptr();
    const int type = type_of(k->scalar_type());
    const int64_t T = k->size(0);
    const int rc = unlocked([&] { return keops_cache_append(&cache, kp, vp, ks, vs, type, at, T, st); });
    return ended(rc, Py_NewRef(Py_True));
  });
}

// (q, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts, max_q, max_len, scale, window, decay, out, lse)
PyObject *attention(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    if (!cache_of(c, o + 1, &cache)) return nullptr;
    const at::Tensor *q = c.need(o[0]), *starts = c.need(o[8]);
    int64_t stride;
    int32_t max_q, max_len, window;
    void *st;
    if (!c.ok || !rows_of(c, *q, cache, &stride) || !number(o[9], &max_q) || !number(o[10], &max_len) || !number(o[12], &window) ||
        (o[11] != Py_None && !PyFloat_CheckExact(o[11])) || !PyFloat_CheckExact(o[13]))
      return nullptr;
    const double scale = o[11] == Py_None ? 1.0 / std::sqrt((double)cache.dim) : PyFloat_AS_DOUBLE(o[11]);
    const double decay = PyFloat_AS_DOUBLE(o[13]);
    const int64_t T = q->size(0), heads = q->size(1);
    const void *qp = q->data_ptr();
    if (cache.heads < 1 || heads < 1 || heads % cache.heads) return nullptr;
    const int32_t *at = (const int32_t *)c.dense(starts, at::kInt, {(int64_t)cache.seqs + 1});
    at::Tensor out, lse;
    if (!c.ok || !output(c, o[14], q->scalar_type(), {T, heads, cache.dim}, *q, &out) ||
        !output(c, o[15], at::kFloat, {T, heads}, *q, &lse) || !stream_of(c, &st))
      return nullptr;
    const int type = type_of(q->scalar_type());
    void *op = out.data_ptr();
    float *lp = (float *)lse.data_ptr();
    PyObject *result = pair(out, o[14], lse, o[15]);
    if (!result) return nullptr;
    const int rc = unlocked([&] {
      return keops_paged_attention(&cache, qp, stride, type, (int32_t)heads, at, T, max_q, max_len, (float)scale, window,
                                   (float)decay, op, lp, nullptr, 0, st);
    });
    return ended(rc, result);
  });
}

// (k_pages, v_pages, weights, page_table, lens, None, None, new_table, budget, sink, recent, kept, new_lens)
PyObject *evict(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    // an 8-bit cache comes without its scales here: the long way
    if (!cache_of(c, o, &cache) || !cache.weights) return nullptr;
    int32_t budget, sink, recent, width;
    int64_t stride;
    const int32_t *table;
    void *st;
    if (!number(o[8], &budget) || !number(o[9], &sink) || !number(o[10], &recent)) return nullptr;
    const at::Tensor *nt = c.need(o[7]);
    if (!c.ok || !table_of(c, nt, cache.seqs, &table, &stride, &width)) return nullptr;
    // a budget without pages is refused before its output is allocated
    if (budget < 1 || width < std::min<int64_t>(((int64_t)budget + cache.page_size - 1) / std::max(cache.page_size, 1), cache.table_width))
      return nullptr;
    at::Tensor kept, lens;
    if (!output(c, o[11], at::kInt, {cache.seqs, cache.heads, budget}, *nt, &kept) ||
        !output(c, o[12], at::kInt, {cache.seqs}, *nt, &lens) || !stream_of(c, &st))
      return nullptr;
    int32_t *kp = (int32_t *)kept.data_ptr(), *lp = (int32_t *)lens.data_ptr();
    PyObject *result = pair(kept, o[11], lens, o[12]);
    if (!result) return nullptr;
    const int rc = unlocked([&] { return keops_cache_evict(&cache, table, stride, width, budget, sink, recent, kp, lp, st); });
    return ended(rc, result);
  });
}

// (target, draft, tokens, counts, u_accept, u_sample, out, accepted)
PyObject *verify(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    Call c;
    const at::Tensor *target = c.need(o[0]), *draft = c.maybe(o[1]), *tokens = c.need(o[2]), *counts = c.need(o[3]);
    const at::Tensor *ua = c.need(o[4]), *us = c.need(o[5]);
    if (!c.ok || !c.begin(*target) || target->dim() != 3 || tokens->dim() != 2) return nullptr;
    const int64_t S = tokens->size(0), K = tokens->size(1), V = target->size(2);
    if (S > INT32_MAX || K > INT32_MAX - 1 || V > INT32_MAX) return nullptr;
    const float *tp = (const float *)c.dense(target, at::kFloat, {S, K + 1, V});
    const float *dp = (const float *)c.dense(draft, at::kFloat, {S, K, V});
    const int32_t *xp = (const int32_t *)c.dense(tokens, at::kInt, {S, K}), *cp = (const int32_t *)c.dense(counts, at::kInt, {S});
    const float *ap = (const float *)c.dense(ua, at::kFloat, {S, K}), *sp = (const float *)c.dense(us, at::kFloat, {S});
    at::Tensor out, accepted;
    void *st;
    if (!c.ok || !output(c, o[6], at::kInt, {S, K + 1}, *target, &out) || !output(c, o[7], at::kInt, {S}, *target, &accepted) ||
        !stream_of(c, &st))
      return nullptr;
    int32_t *op = (int32_t *)out.data_ptr(), *np = (int32_t *)accepted.data_ptr();
    PyObject *result = pair(out, o[6], accepted, o[7]);
    if (!result) return nullptr;
    const int rc = unlocked([&] {
      return keops_verify_draft(tp, K ? dp : nullptr, xp, cp, ap, sp, (int32_t)S, (int32_t)K, (int32_t)V, op, np, nullptr, 0, st);
    });
    return ended(rc, result);
  });
}

// bind(raw_stream): the function that gives a device's current raw stream
PyObject *bind(PyObject *, PyObject *f) {
  Py_XDECREF(g_raw_stream);
  g_raw_stream = PyCallable_Check(f) ? Py_NewRef(f) : nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void *)append, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void *)attention, METH_FASTCALL, nullptr},
                         {"evict", (PyCFunction)(void *)evict, METH_FASTCALL, nullptr},
                         {"verify", (PyCFunction)(void *)verify, METH_FASTCALL, nullptr},
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call() { return PyModule_Create(&module); }

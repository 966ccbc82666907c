// call.h -- what the modules of the short way share: reading torch tensors, the cache's description, the
// current stream, outputs and what a call ends with.
#pragma once

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

namespace {      // each module that includes this has its own

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
    case at::ScalarType::Float4_e2m1fn_x2: return KEOPS_TYPE_E2M1;
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
  // a 4-bit element of torch holds two values
  const int64_t two = type == KEOPS_TYPE_E2M1 ? 2 : 1;
  const int64_t P = k->size(0), ps = k->size(1), H = k->size(2), D = k->size(3) * two, S = lens->size(0);
  if (ps > INT32_MAX || H > INT32_MAX || D > INT32_MAX || S > INT32_MAX) return false;
  if ((type == KEOPS_TYPE_E4M3 || type == KEOPS_TYPE_E2M1) != (ks != nullptr) || (ks != nullptr) != (vs != nullptr)) return false;
  *out = keops_cache_t{};
  out->k_pages = k->data_ptr();
  out->v_pages = v->data_ptr();
  out->weights = (float *)c.dense(w, at::kFloat, {P, H, ps});
  if (type == KEOPS_TYPE_E2M1) {
    out->k_powers = (uint8_t *)c.dense(ks, at::ScalarType::Float8_e8m0fnu, {P, H, ps, D / 32});
    out->v_powers = (uint8_t *)c.dense(vs, at::ScalarType::Float8_e8m0fnu, {P, H, ps, D / 32});
  } else {
    out->k_scale = (const float *)c.dense(ks, at::kFloat, {H});
    out->v_scale = (const float *)c.dense(vs, at::kFloat, {H});
  }
  // the stride of a dimension of one is never used
  out->page_stride = P > 1 ? k->stride(0) * two : 0;
  out->slot_stride = ps > 1 ? k->stride(1) * two : 0;
  out->head_stride = H > 1 ? k->stride(2) * two : 0;
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
  if (type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16) return false;
  if (cache.type != KEOPS_TYPE_E4M3 && cache.type != KEOPS_TYPE_E2M1 && cache.type != type) return false;
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

// bind(raw_stream): the function that gives a device's current raw stream
PyObject *bind(PyObject *, PyObject *f) {
  Py_XDECREF(g_raw_stream);
  g_raw_stream = PyCallable_Check(f) ? Py_NewRef(f) : nullptr;
  Py_RETURN_NONE;
}

}  // namespace

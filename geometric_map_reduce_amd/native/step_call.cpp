// step_call.cpp -- the short way from torch tensors to the C ABI of the operators around the paged cache:
// rotary positions, the append that rotates, reading slots back, and the adjustment of logits.  As in
// paged_call.cpp, None stands for a call that the long way takes or refuses by name.
#include "call.h"

#include <c10/core/GradMode.h>

namespace {

// A C double from a Python float or int.
bool real(PyObject *o, double *v) {
  if (PyFloat_CheckExact(o)) *v = PyFloat_AS_DOUBLE(o);
  else if (PyLong_CheckExact(o)) *v = PyLong_AsDouble(o);
  else return false;
  return !PyErr_Occurred();
}

// freqs [pairs] float64, interleaved, factor.
bool rotary_of(Call &c, PyObject *freqs, PyObject *interleaved, PyObject *factor, keops_rotary_t *r) {
  const at::Tensor *f = c.need(freqs);
  if (!f || f->dim() != 1 || f->size(0) > INT32_MAX || !PyBool_Check(interleaved) || !real(factor, &r->factor)) return false;
  r->freqs = (const double *)c.dense(f, at::kDouble, {f->size(0)});
  r->pairs = (int32_t)f->size(0);
  r->interleaved = interleaved == Py_True;
  return c.ok;
}

// An output that the call returns alone: the caller's tensor, whatever its rows' distance, or a new dense one.
bool rows_output(Call &c, PyObject *given, const at::Tensor &like, at::IntArrayRef shape, at::Tensor *out) {
  if (given == Py_None) {
    *out = at::empty(shape, like.options().requires_grad(false));
    return true;
  }
  const at::Tensor *t = c.need(given);
  if (!t || t->scalar_type() != like.scalar_type() || !c.on_device(*t) || t->sizes() != shape) return false;
  if (t->requires_grad() && c10::GradMode::is_enabled()) return false;
  *out = *t;
  return true;
}
PyObject *single(const at::Tensor &t, PyObject *given) { return given == Py_None ? THPVariable_Wrap(t) : Py_NewRef(given); }
// What such a call ends with: autograd is told that the caller's tensor has changed.
PyObject *ended(int rc, PyObject *result, const at::Tensor &out, PyObject *given) {
  if (rc == KEOPS_OK && given != Py_None && !out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
  return ended(rc, result);
}

// Rows [tokens, heads, dim] with dense heads: the distance of rows.
bool dense_heads(const at::Tensor &t, int64_t *stride) {
  const int64_t T = t.size(0), h = t.size(1), d = t.size(2);
  if (T && h && d && ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d))) return false;
  *stride = T > 1 ? t.stride(0) : h * d;
  return true;
}

// (x, positions, freqs, interleaved, factor, inverse, out)
PyObject *rotary(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    Call c;
    const at::Tensor *x = c.need(o[0]), *positions = c.need(o[1]);
    if (!c.ok || !c.begin(*x) || x->dim() != 3 || !PyBool_Check(o[5])) return nullptr;
    const int type = x->scalar_type() == at::kFloat ? KEOPS_TYPE_F32 : type_of(x->scalar_type());
    const int64_t T = x->size(0), H = x->size(1), D = x->size(2);
    if (H > INT32_MAX || D > INT32_MAX) return nullptr;
    keops_rotary_t r{};
    int64_t xs, os;
    at::Tensor out;
    void *st;
    const int32_t *at = (const int32_t *)c.dense(positions, at::kInt, {T});
    if (!rotary_of(c, o[2], o[3], o[4], &r) || !dense_heads(*x, &xs) || !rows_output(c, o[6], *x, {T, H, D}, &out) ||
        !dense_heads(out, &os) || !stream_of(c, &st))
      return nullptr;
    const void *xp = x->data_ptr();
    void *op = out.data_ptr();
    PyObject *result = single(out, o[6]);
    if (!result) return nullptr;
    const int inverse = o[5] == Py_True;
    const int rc = unlocked([&] { return keops_rotary(xp, xs, type, T, (int32_t)H, (int32_t)D, at, &r, inverse, op, os, st); });
    return ended(rc, result, out, o[6]);
  });
}

// (q, k, v, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts, freqs, positions, interleaved, factor, out)
PyObject *append_rotary(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    if (!cache_of(c, o + 3, &cache)) return nullptr;
    const at::Tensor *q = c.need(o[0]), *k = c.need(o[1]), *v = c.need(o[2]), *starts = c.need(o[10]), *positions = c.maybe(o[12]);
    keops_rotary_t r{};
    int64_t qs, ks, vs, os;
    at::Tensor out;
    void *st;
    if (!c.ok || !rows_of(c, *q, cache, &qs) || !rows_of(c, *k, cache, &ks) || !rows_of(c, *v, cache, &vs) ||
        k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || q->scalar_type() != k->scalar_type() ||
        k->size(1) != cache.heads || q->size(0) != k->size(0))
      return nullptr;
    const int64_t T = k->size(0), heads = q->size(1);
    const int32_t *at = (const int32_t *)c.dense(starts, at::kInt, {(int64_t)cache.seqs + 1});
    const int32_t *pos = (const int32_t *)c.dense(positions, at::kInt, {T});
    if (!rotary_of(c, o[11], o[13], o[14], &r) || !rows_output(c, o[15], *q, q->sizes(), &out) || !dense_heads(out, &os) ||
        !stream_of(c, &st))
      return nullptr;
    const void *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr();
    void *op = out.data_ptr();
    const int type = type_of(k->scalar_type());
    PyObject *result = single(out, o[15]);
    if (!result) return nullptr;
    const int rc = unlocked([&] {
      return keops_cache_append_rotary(&cache, qp, kp, vp, qs, ks, vs, type, (int32_t)heads, at, T, pos, &r, op, os, st);
    });
    return ended(rc, result, out, o[15]);
  });
}

// (k_pages, v_pages, None, page_table, lens, k_scale, v_scale, starts, tokens, type of the rows, k, v); the type as a
// tensor's: any of it
PyObject *read(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    if (!cache_of(c, o, &cache)) return nullptr;
    const at::Tensor *starts = c.need(o[7]), *pages = c.need(o[0]);
    int32_t T, half;
    if (!c.ok || !number(o[8], &T) || !number(o[9], &half) || half > 1) return nullptr;
    if (cache.type != KEOPS_TYPE_E4M3 && cache.type != KEOPS_TYPE_E2M1 && cache.type != half) return nullptr;
    const int32_t *at = (const int32_t *)c.dense(starts, at::kInt, {(int64_t)cache.seqs + 1});
    void *st;
    if (!c.ok || o[10] != Py_None || !stream_of(c, &st)) return nullptr;
    const auto options = pages->options().dtype(half == KEOPS_TYPE_F16 ? at::kHalf : at::kBFloat16).requires_grad(false);
    const at::Tensor k = at::empty({T, cache.heads, cache.dim}, options), v = at::empty({T, cache.heads, cache.dim}, options);
    void *kp = k.data_ptr(), *vp = v.data_ptr();
    PyObject *result = pair(k, Py_None, v, Py_None);
    if (!result) return nullptr;
    const int64_t row = (int64_t)cache.heads * cache.dim;
    const int rc = unlocked([&] { return keops_cache_read(&cache, kp, vp, row, row, half, at, T, st); });
    return ended(rc, result);
  });
}

// (logits, starts, text, lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias, mask, out)
PyObject *adjust(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    Call c;
    const at::Tensor *logits = c.need(o[0]), *starts = c.need(o[1]), *text = c.maybe(o[2]), *lens = c.maybe(o[3]), *prompt = c.maybe(o[4]);
    const at::Tensor *rep = c.maybe(o[5]), *pres = c.maybe(o[6]), *freq = c.maybe(o[7]), *ids = c.maybe(o[8]), *bias = c.maybe(o[9]);
    const at::Tensor *mask = c.maybe(o[10]);
    if (!c.ok || !c.begin(*logits) || logits->dim() != 2 || starts->dim() != 1 || starts->size(0) < 1) return nullptr;
    const int type = logits->scalar_type() == at::kFloat ? KEOPS_TYPE_F32 : type_of(logits->scalar_type());
    const int64_t T = logits->size(0), V = logits->size(1), S = starts->size(0) - 1;
    if (V < 1 || V > INT32_MAX || S > INT32_MAX || (V > 1 && logits->stride(1) != 1)) return nullptr;
    keops_logit_rules_t r{};
    r.seqs = (int32_t)S;
    r.starts = (const int32_t *)c.dense(starts, at::kInt, {S + 1});
    if (text && (!lens || !table_of(c, text, S, &r.text, &r.text_stride, &r.text_width))) return nullptr;
    if (!text && (rep || pres || freq || prompt)) return nullptr;
    r.lens = (const int32_t *)c.dense(lens, at::kInt, {S});
    r.prompt_lens = (const int32_t *)c.dense(prompt, at::kInt, {S});
    r.repetition = (const float *)c.dense(rep, at::kFloat, {S});
    r.presence = (const float *)c.dense(pres, at::kFloat, {S});
    r.frequency = (const float *)c.dense(freq, at::kFloat, {S});
    if ((ids != nullptr) != (bias != nullptr) || (ids && (ids->dim() != 2 || ids->size(1) > INT32_MAX))) return nullptr;
    if (ids) {
      r.bias_tokens = (const int32_t *)c.dense(ids, at::kInt, {S, ids->size(1)});
      r.bias = (const float *)c.dense(bias, at::kFloat, {S, ids->size(1)});
      r.biases = (int32_t)ids->size(1);
    }
    int32_t words = 0;
    if (mask && (!table_of(c, mask, T, &r.mask, &r.mask_stride, &words) || words != (V + 31) / 32)) return nullptr;
    at::Tensor out;
    void *st;
    if (!c.ok || !rows_output(c, o[11], *logits, {T, V}, &out) || (V > 1 && out.stride(1) != 1) || !stream_of(c, &st)) return nullptr;
    const void *lp = logits->data_ptr();
    void *op = out.data_ptr();
    const int64_t stride = T > 1 ? logits->stride(0) : V, os = T > 1 ? out.stride(0) : V;
    PyObject *result = single(out, o[11]);
    if (!result) return nullptr;
    const int rc = unlocked([&] { return keops_adjust_logits(lp, stride, type, T, (int32_t)V, &r, op, os, st); });
    return ended(rc, result, out, o[11]);
  });
}

PyMethodDef methods[] = {{"rotary", (PyCFunction)(void *)rotary, METH_FASTCALL, nullptr},
                         {"append_rotary", (PyCFunction)(void *)append_rotary, METH_FASTCALL, nullptr},
                         {"read", (PyCFunction)(void *)read, METH_FASTCALL, nullptr},
                         {"adjust", (PyCFunction)(void *)adjust, METH_FASTCALL, nullptr},
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_call", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__step_call() { return PyModule_Create(&module); }

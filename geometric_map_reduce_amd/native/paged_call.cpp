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
#include "call.h"

namespace {

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

// (k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, new_table, budget, sink, recent, kept, new_lens)
PyObject *evict(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    Call c;
    keops_cache_t cache;
    // an 8-bit cache may come without its scales: the long way
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

PyMethodDef methods[] = {{"append", (PyCFunction)(void *)append, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void *)attention, METH_FASTCALL, nullptr},
                         {"evict", (PyCFunction)(void *)evict, METH_FASTCALL, nullptr},
                         {"verify", (PyCFunction)(void *)verify, METH_FASTCALL, nullptr},
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call() { return PyModule_Create(&module); }
